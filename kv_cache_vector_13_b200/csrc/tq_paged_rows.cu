// Attention of a few query rows a request over a paged 4-bit cache (sm_100a):
// decode, and the verification of a few draft tokens.
//
// Work: a unit is (request, KV head, tile of query rows), a step 16 cached
// tokens.  All units' steps form one line, cut into equal ranges, one a CTA
// (one persistent CTA an SM), so requests of any lengths balance; a CTA's
// part of a unit is a piece, whose steps its warps take in turn.  Units cut by
// a range's end leave partial sums that a second kernel merges, in the order
// of the tokens, so the result does not depend on timing.
//
// A step of a warp: S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16 (fp16,
// fp32 sums), the tokens (then the coordinates) being the 16 rows and the
// query rows the 8 columns, and the running softmax in between.  Query rows
// and weights are carried as fp16 pairs hi + lo: up to 4 rows a tile put both
// into one product, as columns g and g + 4 (S and O are the sums of the two);
// up to 8 take two products into the same sums.  Codes become operand words
// without arithmetic: a code byte (two codes) indexes a 256-entry table of
// fp16 centroid pairs, one copy per lane, placed so that one byte permute
// forms the shared address.  For K the pair is two coordinates of a token; for
// V the codes of two tokens are first interleaved, so the pair is two tokens
// at one coordinate.  The order of coordinates within the products is free, so
// every lane loads whole 16-byte (K) and 8-byte (V) runs of a record.  Norms
// enter behind the products: ||k|| scales the logit, ||v|| the weight.

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"
#include "tq_paged_dev.cuh"

#include <float.h>

#include <type_traits>

namespace tq {
namespace {

using namespace paged;

constexpr int kStep = 16;                // tokens per step
constexpr uint32_t kTabAddr = 0x10000u;  // the pair tables: 64 KiB at this shared address
constexpr uint32_t kPartAddr = 0x20000u; // the warps' partial sums
constexpr int kMaxRows = 8;

template <int D>
struct Cfg {
  static constexpr int kWarps = 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPitch = D + 4;  // floats of a partial row (no bank clash between rows)
};

// Shared memory below the tables.
template <int D>
struct Low {
  int64_t base[Cfg<D>::kThreads];  // the line at each thread's first request
  int64_t warp[Cfg<D>::kWarps];
  __half q[2][8][D + 8];           // operand columns: hi of each row, lo of each row
  float f[kMaxRows];               // logit factor of each row
  float m[Cfg<D>::kWarps][kMaxRows], l[Cfg<D>::kWarps][kMaxRows];
  float scale[2];                  // the tables' scales
};

template <int D>
__host__ __device__ constexpr uint32_t smem_end() {
  return kPartAddr + Cfg<D>::kWarps * kMaxRows * Cfg<D>::kPitch * 4;
}

struct RowsParams {
  PagedAttentionArgs a;
  float *slots;     // [2 * ctas][kMaxRows][D + 2]: sums, then M and L
  int4 *desc;       // [ctas]: {pieces, request, tile, head} of the unit that starts last in the CTA's range
  unsigned *faults;
};

// One request: its rows, and the steps that any of its rows sees.
struct Req {
  int q0, n;        // query rows
  int kv;
  int lo, hi;       // steps [lo, hi)
  int tiles;
};

__device__ __forceinline__ Req load_req(const PagedAttentionArgs &a, int r, int rows_per_tile, unsigned *faults) {
  Req q;
  q.q0 = a.cu_q ? __ldg(a.cu_q + r) : r;
  const int q1 = a.cu_q ? __ldg(a.cu_q + r + 1) : r + 1;
  q.q0 = max(q.q0, 0);
  q.n = max(min(q1, (int)a.T) - q.q0, 0);
  q.kv = max(__ldg(a.kv_lens + r), 0);
  const int cap = a.max_pages * a.page_size;
  if (q.kv > cap) {
    atomicOr(faults, kFaultIndex);
    q.kv = cap;
  }
  q.tiles = (q.n * (a.Hq / a.Hkv) + rows_per_tile - 1) / rows_per_tile;
  q.lo = a.window > 0 ? max(q.kv - q.n + 1 - a.window, 0) / kStep : 0;
  // a request that sees nothing still has one (empty) step, which writes its zeros
  q.hi = max((q.kv + kStep - 1) / kStep, q.lo + 1);
  return q;
}

__device__ __forceinline__ int64_t weight(const Req &q, int Hkv) { return (int64_t)q.tiles * Hkv * (q.hi - q.lo); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// Table read of byte k of w: shared address {lane, byte k, table}.
template <int K>
__device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t base) {
  return lds32(__byte_perm(w, base, 0x7604 | (K << 4)));
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values, two of row lane / 4 a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes and norms of one step as a lane needs them.
template <int D>
struct Codes {
  uint32_t k[2][D / 32];  // tokens g and 8 + g, coordinates [q D/4, (q + 1) D/4)
  uint32_t v[4][D / 64];  // tokens 2q, 2q+1, 8+2q, 9+2q, coordinates [g D/8, (g + 1) D/8)
  float kn[2], vn[2];     // tokens g and 8 + g
};

template <int N>
__device__ __forceinline__ void ldg_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p));
    w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
  } else if constexpr (N == 2) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    w[0] = t.x; w[1] = t.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
  }
}

// P4: up to 4 query rows a tile, hi and lo in one product; else up to 8.
// UNIT: the tokens of a page lie side by side.
template <int D, bool P4, bool UNIT>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) paged_rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = Cfg<D>::kWarps, NT = Cfg<D>::kThreads, PITCH = Cfg<D>::kPitch;
  constexpr int RT = P4 ? 4 : 8;  // query rows per tile
  constexpr int KS = D / 16;      // k steps of the scores
  constexpr int MV = D / 16;      // m tiles of the values
  constexpr int QS = P4 ? 1 : 2;  // products per step
  extern __shared__ __align__(16) unsigned char s_raw[];
  Low<D> &sm = *reinterpret_cast<Low<D> *>(s_raw);
  auto &s_base = sm.base;
  auto &s_warp = sm.warp;
  auto &s_q = sm.q;
  auto &s_f = sm.f;
  auto &s_m = sm.m;
  auto &s_l = sm.l;
  auto &s_scale = sm.scale;

  const PagedAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int G = a.Hq / a.Hkv, c = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const uint32_t dyn = (uint32_t)__cvta_generic_to_shared(s_raw);
  uint32_t dyn_bytes;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn_bytes));
  if (dyn + sizeof(Low<D>) > kTabAddr || dyn + dyn_bytes < smem_end<D>()) {
    if (tid == 0) {
      atomicOr(p.faults, kFaultSmemLayout);
      p.desc[c] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  float *parts = reinterpret_cast<float *>(s_raw + (kPartAddr - dyn));  // [W][RT][PITCH]

  // ---- the tables: entry e, lane l at 256 e + 4 l (keys) and + 128 (values)
  if (warp < 2) {
    const float *cent = warp == 0 ? a.kq.centroids : a.vq.centroids;
    const float s = table_scale(cent, lane);
    if (lane == 0) s_scale[warp] = s;
    for (int e = lane; e < 256; e += 32) {
      const __half2 h = __floats2half2_rn(s * __ldg(cent + (e & 15)), s * __ldg(cent + (e >> 4)));
      reinterpret_cast<uint32_t *>(parts)[warp * 256 + e] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  // ---- the line of steps: a run of requests a thread
  const int per = (a.R + NT - 1) / NT;
  int64_t mine = 0;
  for (int r = tid * per; r < min((tid + 1) * per, a.R); ++r)
    mine += weight(load_req(a, r, RT, p.faults), a.Hkv);
  int64_t total;
  {
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(dev::kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int64_t base = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int64_t y = s_warp[i];
      if (i < warp) base += y;
      total += y;
    }
    s_base[tid] = base + x - mine;
  }
  {
    const uint32_t *pairs = reinterpret_cast<const uint32_t *>(parts);
    uint4 *tab = reinterpret_cast<uint4 *>(s_raw + (kTabAddr - dyn));
    for (int i = tid; i < 256 * 16; i += NT) {
      const uint32_t w = pairs[((i >> 3) & 1) * 256 + (i >> 4)];
      tab[i] = make_uint4(w, w, w, w);
    }
  }
  __syncthreads();

  // every range has a step at least, so no piece of a unit is missing
  const int ctas = (int)min((int64_t)gridDim.x, total);
  int64_t at = c < ctas ? total * c / ctas : 0;
  const int64_t end = c < ctas ? total * (c + 1) / ctas : 0;
  int4 desc = make_int4(0, 0, 0, 0);
  // the request of the range's start
  int r = 0;
  int64_t r_base = 0;
  Req req;
  if (at < end) {
    int i = 0, j = NT;
    while (j - i > 1) {
      const int m = (i + j) >> 1;
      if (s_base[m] <= at) i = m; else j = m;
    }
    r = i * per;
    r_base = s_base[i];
    for (; r < a.R; ++r) {
      req = load_req(a, r, RT, p.faults);
      const int64_t w = weight(req, a.Hkv);
      if (at < r_base + w) break;
      r_base += w;
    }
  }
  const uint32_t ktab = kTabAddr + 4 * lane, vtab = ktab + 128;
  const float kscale = a.scale * 1.4426950408889634f / (a.kq.sqrt_d * s_scale[0]);
  const float vscale = 1.0f / (a.vq.sqrt_d * s_scale[1]);

  while (at < end && r < a.R) {
    // ---- the piece: steps [s0, s1) of unit (r, h, tile)
    const int len = req.hi - req.lo;
    const int64_t x = at - r_base;
    const int unit = (int)(x / len);
    const int s0 = req.lo + (int)(x - (int64_t)unit * len);
    const int s1 = (int)min((int64_t)req.hi, s0 + (end - at));
    const int h = unit / req.tiles, tile = unit - h * req.tiles;
    const int row0 = tile * RT;
    const int nrows = min(RT, req.n * G - row0);

    // ---- query rows: sign flips, FWHT, a power of two that brings the largest into [1, 2)
    for (int i = warp; i < RT; i += W) {
      float v[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
      if (i < nrows) {
        const int qi = (row0 + i) / G, hq = h * G + (row0 + i) - qi * G;
        load_row<D>(a.q, a.dtype, (int64_t)(req.q0 + qi) * a.q_st + hq * a.q_sh, lane, v);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] *= (float)__ldg(a.kq.signs + lane * (D / 32) + e);
      }
      dev::fwht<32, D / 32>(v, lane);
      const float f = row_scale<D / 32>(v);
      if (lane == 0) s_f[i] = kscale / f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const float y = v[e] * f;
        const __half hi = __float2half_rn(y);
        s_q[0][i][lane * (D / 32) + e] = hi;
        s_q[P4 ? 0 : 1][P4 ? i + 4 : i][lane * (D / 32) + e] = __float2half_rn(y - __half2float(hi));
      }
    }
    __syncthreads();
    uint32_t qb[QS][KS][2];
#pragma unroll
    for (int o = 0; o < QS; ++o)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint2 t = *reinterpret_cast<const uint2 *>(&s_q[o][g][q4 * (D / 4) + 4 * s]);
        qb[o][s][0] = t.x;
        qb[o][s][1] = t.y;
      }
    // the lane's two rows; one that is not there sees everything (and goes nowhere)
    int see_lo[2], see_hi[2];
    float f[2], M[2], l[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int i = (2 * q4 + o) & (RT - 1);
      see_lo[o] = 0;
      see_hi[o] = INT_MAX;
      if (i < nrows) {
        const int pos = req.kv - req.n + (row0 + i) / G;
        see_hi[o] = a.causal ? max(pos + 1, 0) : req.kv;
        see_lo[o] = a.window > 0 ? max(pos + 1 - a.window, 0) : 0;
      }
      f[o] = s_f[i];
      M[o] = -FLT_MAX;
      l[o] = 0.f;
    }
    // steps that every row of the tile sees whole
    const int first_pos = req.kv - req.n + row0 / G, last_pos = req.kv - req.n + (row0 + nrows - 1) / G;
    const int full_hi = a.causal ? max(first_pos + 1, 0) : req.kv;
    const int full_lo = a.window > 0 ? max(last_pos + 1 - a.window, 0) : 0;

    float acc[MV][4];
#pragma unroll
    for (int j = 0; j < MV; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

    const int32_t *row = a.table + (int64_t)r * a.table_stride;
    const int n_steps = s1 - s0 > warp ? (s1 - s0 - warp + W - 1) / W : 0;
    // The records of 8 of the warp's steps, step it + lane % 8 a lane; -1 without a page.  They are found a
    // batch ahead and brought into L2 (lane / 8: codes and norms of K and of V).
    int64_t krec, vrec, krec2, vrec2;
    auto find = [&](int it, int64_t &kr, int64_t &vr) {
      const int s = s0 + warp + (it + (lane & 7)) * W;
      kr = vr = -1;
      const int t0 = s * kStep;
      if (s < s1 && t0 < req.kv) {
        const int page = t0 / a.page_size, off = t0 - page * a.page_size;
        const int id = __ldg(row + page);
        if ((unsigned)id < (unsigned)a.n_pages) {
          kr = id * a.k.sb + h * a.k.sh + off * a.k.sn;
          vr = id * a.v.sb + h * a.v.sh + off * a.v.sn;
        } else {
          atomicOr(p.faults, kFaultIndex);
        }
      }
    };
    auto warm = [&](int64_t kr, int64_t vr) {
      if (!UNIT || kr < 0) return;
      const int what = lane >> 3;
      const bool norm = what & 1;
      const char *at = norm ? reinterpret_cast<const char *>((what & 2 ? a.v.norms : a.k.norms) + (what & 2 ? vr : kr))
                            : reinterpret_cast<const char *>((what & 2 ? a.v.codes : a.k.codes) + (what & 2 ? vr : kr) * (D / 2));
      // a run of norms may begin inside a 16-byte word: the words that hold it
      const uintptr_t lo = (uintptr_t)at & ~(uintptr_t)15;
      const uint32_t n = norm ? (uint32_t)(((uintptr_t)at + 4 * kStep + 15 - lo) & ~(uintptr_t)15) : kStep * (D / 2);
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"(n) : "memory");
    };
    auto load_k = [&](int64_t kr, Codes<D> &cd) {
      if constexpr (UNIT) {
        const uint8_t *c = a.k.codes + kr * (D / 2) + (g * (D / 2) + q4 * (D / 8));
        ldg_words(c, cd.k[0]);
        ldg_words(c + 8 * (D / 2), cd.k[1]);
        const float *n = a.k.norms + kr + g;
        cd.kn[0] = __ldg(n);
        cd.kn[1] = __ldg(n + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ldg_words(a.k.codes + (kr + (8 * i + g) * a.k.sn) * (D / 2) + q4 * (D / 8), cd.k[i]);
          cd.kn[i] = __ldg(a.k.norms + kr + (8 * i + g) * a.k.sn);
        }
      }
    };
    auto load_v = [&](int64_t vr, Codes<D> &cd) {
      if constexpr (UNIT) {
        const uint8_t *c = a.v.codes + vr * (D / 2) + (q4 * D + g * (D / 16));
        ldg_words(c, cd.v[0]);
        ldg_words(c + D / 2, cd.v[1]);
        ldg_words(c + 8 * (D / 2), cd.v[2]);
        ldg_words(c + 9 * (D / 2), cd.v[3]);
        const float *n = a.v.norms + vr + g;
        cd.vn[0] = __ldg(n);
        cd.vn[1] = __ldg(n + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ldg_words(a.v.codes + (vr + (8 * (i >> 1) + 2 * q4 + (i & 1)) * a.v.sn) * (D / 2) + g * (D / 16), cd.v[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) cd.vn[i] = __ldg(a.v.norms + vr + (8 * i + g) * a.v.sn);
      }
    };
    // The running softmax of the lane's rows over its tokens g and 8 + g (value 2 i + o: token 8 i + g, row o):
    // scores in, weights times value norms out.  M is a reference that moves only when one of them would pass 2^8.
    auto soft = [&](auto edge, int t0, float (&t)[4], const Codes<D> &cd) {
      constexpr bool EDGE = decltype(edge)::value;
      float lv[2], mx[2], s[4];
      bool seen[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = t0 + 8 * i + g;
        lv[i] = fmaxf(log2_approx(cd.vn[i]), -64.f);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int e = 2 * i + o;
          seen[e] = !EDGE || (j >= see_lo[o] && j < see_hi[o] && j < req.kv);
          s[e] = t[e] * (f[o] * cd.kn[i]);
          t[e] = s[e] - M[o];
          if (EDGE && !seen[e]) t[e] = -INFINITY;
        }
      }
      if (__any_sync(dev::kFull, fmaxf(fmaxf(t[0], t[1]) + lv[0], fmaxf(t[2], t[3]) + lv[1]) > 8.f)) {
        float r2[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          mx[o] = fmaxf(seen[o] ? s[o] + lv[0] : -INFINITY, seen[2 + o] ? s[2 + o] + lv[1] : -INFINITY);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx[o] = fmaxf(mx[o], __shfl_xor_sync(dev::kFull, mx[o], x));
          const float m2 = fmaxf(M[o], mx[o]);
          r2[o] = exp2f(M[o] - m2);
          M[o] = m2;
          l[o] *= r2[o];
#pragma unroll
          for (int i = 0; i < 2; ++i) t[2 * i + o] = seen[2 * i + o] ? s[2 * i + o] - m2 : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < MV; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] *= r2[e & 1];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] = exp2_approx(t[e]);
        l[e & 1] += t[e];
        t[e] *= cd.vn[e >> 1];
        if (EDGE && !seen[e]) t[e] = 0.f;
      }
    };

    Codes<D> cd;
    bool have = false;  // the step has a page
    if (n_steps > 0) {
      find(0, krec, vrec);
      warm(krec, vrec);
      find(8, krec2, vrec2);
      const int64_t kr = __shfl_sync(dev::kFull, krec, 0), vr = __shfl_sync(dev::kFull, vrec, 0);
      have = kr >= 0;
      if (have) {
        load_k(kr, cd);
        load_v(vr, cd);
      }
    }
    for (int it = 0; it < n_steps; ++it) {
      const int t0 = (s0 + warp + it * W) * kStep;
      if ((it & 7) == 3) warm(krec2, vrec2);
      if ((it & 7) == 7) {
        krec = krec2;
        vrec = vrec2;
        find(it + 9, krec2, vrec2);
      }
      // find() gives -1 behind the piece's last step
      if (!have) {
        const int64_t kr = __shfl_sync(dev::kFull, krec, (it + 1) & 7);
        const int64_t vr = __shfl_sync(dev::kFull, vrec, (it + 1) & 7);
        have = kr >= 0;
        if (have) {
          load_k(kr, cd);
          load_v(vr, cd);
        }
        continue;
      }
      // ---- scores: value 2 i + o is token 8 i + g, column 2 q4 + o
      float sc[2][4];
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[c2][e] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t x = cd.k[0][w], y = cd.k[1][w];
        const uint32_t a0 = pair<0>(x, ktab), a1 = pair<0>(y, ktab), a2 = pair<1>(x, ktab), a3 = pair<1>(y, ktab);
        const uint32_t b0 = pair<2>(x, ktab), b1 = pair<2>(y, ktab), b2 = pair<3>(x, ktab), b3 = pair<3>(y, ktab);
#pragma unroll
        for (int o = 0; o < QS; ++o) {
          // two chains of sums
          mma(sc[0], a0, a1, a2, a3, qb[o][2 * w][0], qb[o][2 * w][1]);
          mma(sc[1], b0, b1, b2, b3, qb[o][2 * w + 1][0], qb[o][2 * w + 1][1]);
        }
      }
      float t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] = sc[0][e] + sc[1][e];
        if (P4) t[e] += __shfl_xor_sync(dev::kFull, t[e], 2);  // the hi and lo columns
      }
      if (t0 + kStep > full_hi || t0 < full_lo)
        soft(std::true_type{}, t0, t, cd);
      else
        soft(std::false_type{}, t0, t, cd);
      // weights to operand words: fp16 pairs of two rows at a token, transposed to two tokens of a row
      uint32_t pb[QS][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 hi = __floats2half2_rn(t[2 * i], t[2 * i + 1]);
        const float2 back = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(t[2 * i] - back.x, t[2 * i + 1] - back.y);
        const uint32_t wh = *reinterpret_cast<const uint32_t *>(&hi), wl = *reinterpret_cast<const uint32_t *>(&lo);
        if (P4) {
          pb[0][i] = transpose8(q4 < 2 ? wh : wl);
        } else {
          pb[0][i] = transpose8(wh);
          pb[QS - 1][i] = transpose8(wl);
        }
      }
      {
        const int64_t kr = __shfl_sync(dev::kFull, krec, (it + 1) & 7);
        have = kr >= 0;
        if (have) load_k(kr, cd);
      }
      // ---- values: tokens 2 q4 and 2 q4 + 1 interleaved (even and odd coordinates apart)
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        const uint32_t x0 = cd.v[0][w], x1 = cd.v[1][w], x2 = cd.v[2][w], x3 = cd.v[3][w];
        const uint32_t e0 = (x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u);
        const uint32_t o0 = ((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
        const uint32_t e1 = (x2 & 0x0f0f0f0fu) | ((x3 << 4) & 0xf0f0f0f0u);
        const uint32_t o1 = ((x2 >> 4) & 0x0f0f0f0fu) | (x3 & 0xf0f0f0f0u);
        auto tile = [&](auto k) {
          constexpr int K = decltype(k)::value;
          const uint32_t a0 = pair<K>(e0, vtab), a1 = pair<K>(o0, vtab), a2 = pair<K>(e1, vtab), a3 = pair<K>(o1, vtab);
#pragma unroll
          for (int o = 0; o < QS; ++o) mma(acc[4 * w + K], a0, a1, a2, a3, pb[o][0], pb[o][1]);
        };
        tile(std::integral_constant<int, 0>{});
        tile(std::integral_constant<int, 1>{});
        tile(std::integral_constant<int, 2>{});
        tile(std::integral_constant<int, 3>{});
      }
      const int64_t vr = __shfl_sync(dev::kFull, vrec, (it + 1) & 7);
      if (have) load_v(vr, cd);
    }

    // ---- the warps' sums: coordinate g (D/8) + 2 j + b of a row at 16 j + 2 g + b
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      float t = l[o];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(dev::kFull, t, x);
      if (g == 0 && 2 * q4 < RT) {
        s_m[warp][2 * q4 + o] = M[o];
        s_l[warp][2 * q4 + o] = t;
      }
    }
#pragma unroll
    for (int j = 0; j < MV; ++j)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        float x = acc[j][o], y = acc[j][2 + o];
        if (P4) {
          x += __shfl_xor_sync(dev::kFull, x, 2);
          y += __shfl_xor_sync(dev::kFull, y, 2);
        }
        if (2 * q4 < RT)
          *reinterpret_cast<float2 *>(parts + ((size_t)warp * kMaxRows + 2 * q4 + o) * PITCH + 16 * j + 2 * g) =
              make_float2(x, y);
      }
    __syncthreads();
    const bool starts = s0 == req.lo, ends = s1 == req.hi;
    for (int i = warp; i < nrows; i += W) {
      float m = s_m[0][i];
#pragma unroll
      for (int w = 1; w < W; ++w) m = fmaxf(m, s_m[w][i]);
      float L = 0.f, y[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) y[e] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float s = exp2f(s_m[w][i] - m);
        L += s * s_l[w][i];
        const float *src = parts + ((size_t)w * kMaxRows + i) * PITCH;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const int k = lane * (D / 32) + e, u = k % (D / 8);
          y[e] = fmaf(s, src[16 * (u / 2) + 2 * (k / (D / 8)) + (u & 1)], y[e]);
        }
      }
      if (starts && ends) {
        const int qi = (row0 + i) / G;
        store_out<D>(a, (int64_t)req.q0 + qi, h * G + (row0 + i) - qi * G, lane, y, m, L, vscale);
      } else {
        float *slot = p.slots + ((size_t)(2 * c + (starts ? 1 : 0)) * kMaxRows + i) * (D + 2);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) slot[lane * (D / 32) + e] = y[e];
        if (lane == 0) {
          slot[D] = m;
          slot[D + 1] = L;
        }
      }
    }
    if (starts && !ends) {
      // CTAs whose ranges the unit reaches: the last holds its last step
      const int64_t last = at + len - 1;
      int64_t e = last * ctas / total;  // a first guess, put right below
      while (e < ctas - 1 && total * (e + 1) / ctas <= last) ++e;
      while (e > c && total * e / ctas > last) --e;
      desc = make_int4((int)e - c + 1, r, tile, h);
    }
    __syncthreads();
    at += s1 - s0;
    if (at < end && at - r_base == weight(req, a.Hkv)) {
      r_base = at;
      while (++r < a.R) {
        req = load_req(a, r, RT, p.faults);
        if (weight(req, a.Hkv) > 0) break;
      }
    }
  }
  if (tid == 0) p.desc[c] = desc;
}

// Merges the pieces of the unit that starts last in CTA c's range and goes on
// behind it, a warp a row, in the order of the tokens.
template <int D, bool P4>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ RowsParams p) {
  constexpr int RT = P4 ? 4 : 8;
  const PagedAttentionArgs &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  const float vs = table_scale(a.vq.centroids, lane);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 desc = __ldcg(p.desc + c);
  if (desc.x == 0) return;
  const int G = a.Hq / a.Hkv;
  const Req req = load_req(a, desc.y, RT, p.faults);
  const int row0 = desc.z * RT, nrows = min(RT, req.n * G - row0);
  const float vscale = 1.0f / (a.vq.sqrt_d * vs);
  for (int i = warp; i < nrows; i += 8) {
    auto slot = [&](int k) {
      return p.slots + ((size_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * kMaxRows + i) * (D + 2);
    };
    float m = -FLT_MAX;
    for (int k = lane; k < desc.x; k += 32) m = fmaxf(m, __ldcg(slot(k) + D));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(dev::kFull, m, x));
    float L = 0.f, y[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) y[e] = 0.f;
#pragma unroll 4
    for (int k = 0; k < desc.x; ++k) {
      const float *s = slot(k);
      const float f = exp2f(__ldcg(s + D) - m);
      L = fmaf(f, __ldcg(s + D + 1), L);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) y[e] = fmaf(f, __ldcg(s + lane * (D / 32) + e), y[e]);
    }
    const int qi = (row0 + i) / G;
    store_out<D>(a, (int64_t)req.q0 + qi, desc.w * G + (row0 + i) - qi * G, lane, y, m, L, vscale);
  }
}

template <int D, bool P4, bool UNIT>
cudaError_t run_rows(const RowsParams &p, cudaStream_t s) {
  // dynamic shared memory starts behind the 1 KiB that the system keeps
  const int dyn = (int)smem_end<D>() - 1024;
  auto kern = paged_rows_kernel<D, P4, UNIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  const int ctas = decode_ctas();
  kern<<<ctas, Cfg<D>::kThreads, dyn, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, P4>, p);
}

template <int D>
cudaError_t run_d(const RowsParams &p, bool p4, cudaStream_t s) {
  const bool unit = p.a.k.sn == 1 && p.a.v.sn == 1;
  if (p4) return unit ? run_rows<D, true, true>(p, s) : run_rows<D, true, false>(p, s);
  return unit ? run_rows<D, false, true>(p, s) : run_rows<D, false, false>(p, s);
}

}  // namespace

size_t paged_rows_workspace(int d) {
  const size_t ctas = decode_ctas();
  return ctas * sizeof(int4) + 2 * ctas * kMaxRows * (d + 2) * sizeof(float);
}

cudaError_t launch_paged_rows(const PagedAttentionArgs &a, cudaStream_t s) {
  RowsParams p{a, nullptr, nullptr, nullptr};
  const cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  p.desc = static_cast<int4 *>(a.ws);
  p.slots = reinterpret_cast<float *>(p.desc + decode_ctas());
  const bool p4 = (int64_t)a.max_q * (a.Hq / a.Hkv) <= 4;
  return a.kq.d == 64 ? run_d<64>(p, p4, s) : run_d<128>(p, p4, s);
}

}  // namespace tq
