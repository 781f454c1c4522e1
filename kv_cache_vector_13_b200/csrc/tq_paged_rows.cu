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
// A step of a warp: S = Q K^T with mma.m16n8k16 (fp16, fp32 sums), the
// running softmax, O += P V.  A tile has 8 query rows, each as the fp16 pair
// hi + lo in rows g and g + 8 of the 16-row operand (S and O are the sums of
// the two), or 16 rows rounded once.  Codes become operand words without
// arithmetic: a code byte (two codes) indexes a 256-entry table of fp16
// centroid pairs, one copy per lane, placed so that one byte permute forms
// the shared address.  For K the pair is two coordinates of a token; for V
// the codes of two tokens are first interleaved, so the pair is two tokens at
// one coordinate.  The order of coordinates within the products is free, so
// every lane loads whole 16-byte (K) and 8-byte (V) runs of a record.
// Norms enter behind the products: ||k|| scales the logit, ||v|| the weight.
//
// What bounds it: table reads, 64 a lane per step (a 128-byte read per clock
// and SM), about 16 warp instructions per token and KV head.

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"
#include "tq_paged_dev.cuh"

#include <float.h>

namespace tq {
namespace {

using namespace paged;

constexpr int kStep = 16;                // tokens per step
constexpr uint32_t kTabAddr = 0x10000u;  // the pair tables: 64 KiB at this shared address
constexpr uint32_t kPartAddr = 0x20000u; // the warps' partial sums
constexpr int kMaxRows = 16;

template <int D>
struct Cfg {
  static constexpr int kWarps = D == 128 ? 12 : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPitch = D + 4;  // floats of a partial row (no bank clash between rows)
};

// Shared memory below the tables.
template <int D>
struct Low {
  int64_t base[Cfg<D>::kThreads];  // the line at each thread's first request
  int64_t warp[Cfg<D>::kWarps];
  __half q[2][8][D + 8];           // operand rows g and g + 8
  float f[kMaxRows];               // logit factor of each row
  float m[Cfg<D>::kWarps][kMaxRows], l[Cfg<D>::kWarps][kMaxRows];
  float scale[2];                  // the tables' scales
};

template <int D, bool HILO>
__host__ __device__ constexpr uint32_t smem_end() {
  return kPartAddr + Cfg<D>::kWarps * (HILO ? 8 : 16) * Cfg<D>::kPitch * 4;
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

// Codes and norms of one step as a lane needs them.
template <int D>
struct Codes {
  uint32_t k[2][D / 32];  // tokens g and 8 + g, coordinates [q D/4, (q + 1) D/4)
  uint32_t v[4][D / 64];  // tokens 2q, 2q+1, 8+2q, 9+2q, coordinates [g D/8, (g + 1) D/8)
  float kn[4], vn[4];     // tokens 2q, 2q+1, 8+2q, 9+2q
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

template <int D, bool HILO>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) paged_rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = Cfg<D>::kWarps, NT = Cfg<D>::kThreads, PITCH = Cfg<D>::kPitch;
  constexpr int RT = HILO ? 8 : 16;  // query rows per tile
  constexpr int KS = D / 16;         // k steps of the scores
  constexpr int NV = D / 8;          // n tiles of the values
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
  if (dyn + sizeof(Low<D>) > kTabAddr || dyn + dyn_bytes < smem_end<D, HILO>()) {
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
  const bool pairs_ok = a.k.sn == 1 && a.v.sn == 1 && ((a.k.sb | a.k.sh | a.v.sb | a.v.sh) & 1) == 0 &&
                        (((uintptr_t)a.k.norms | (uintptr_t)a.v.norms) & 7) == 0;

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
        s_q[HILO ? 0 : i >> 3][i & 7][lane * (D / 32) + e] = hi;
        if (HILO) s_q[1][i][lane * (D / 32) + e] = __float2half_rn(y - __half2float(hi));
      }
    }
    __syncthreads();
    uint32_t qa[KS][4];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const uint2 t = *reinterpret_cast<const uint2 *>(&s_q[o][g][q4 * (D / 4) + 4 * s]);
        qa[s][o] = t.x;
        qa[s][2 + o] = t.y;
      }
    // what each of the lane's rows sees; rows that are not there see everything (and go nowhere)
    constexpr int LR = HILO ? 1 : 2;
    int see_lo[LR], see_hi[LR];
    float f[LR], M[LR], l[LR];
#pragma unroll
    for (int o = 0; o < LR; ++o) {
      const int i = g + 8 * o;
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

    float acc[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

    const int32_t *row = a.table + (int64_t)r * a.table_stride;
    // records of the warp's next 32 steps, one a lane: -1 without a page
    int64_t krec = -1, vrec = -1;
    const int n_steps = s1 - s0 > warp ? (s1 - s0 - warp + W - 1) / W : 0;
    auto fetch_pages = [&](int it) {
      const int s = s0 + warp + (it + lane) * W;
      krec = vrec = -1;
      const int t0 = s * kStep;
      if (s < s1 && t0 < req.kv) {
        const int page = t0 / a.page_size, off = t0 - page * a.page_size;
        const int id = __ldg(row + page);
        if ((unsigned)id < (unsigned)a.n_pages) {
          krec = id * a.k.sb + h * a.k.sh + off * a.k.sn;
          vrec = id * a.v.sb + h * a.v.sh + off * a.v.sn;
        } else {
          atomicOr(p.faults, kFaultIndex);
        }
      }
    };
    auto load_k = [&](int64_t kr, Codes<D> &cd) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        ldg_words(a.k.codes + (kr + (8 * i + g) * a.k.sn) * (D / 2) + q4 * (D / 8), cd.k[i]);
      if (pairs_ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 t = __ldg(reinterpret_cast<const float2 *>(a.k.norms + kr + 8 * i + 2 * q4));
          cd.kn[2 * i] = t.x;
          cd.kn[2 * i + 1] = t.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cd.kn[i] = __ldg(a.k.norms + kr + (8 * (i >> 1) + 2 * q4 + (i & 1)) * a.k.sn);
      }
    };
    auto load_v = [&](int64_t vr, Codes<D> &cd) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ldg_words(a.v.codes + (vr + (8 * (i >> 1) + 2 * q4 + (i & 1)) * a.v.sn) * (D / 2) + g * (D / 16), cd.v[i]);
      if (pairs_ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 t = __ldg(reinterpret_cast<const float2 *>(a.v.norms + vr + 8 * i + 2 * q4));
          cd.vn[2 * i] = t.x;
          cd.vn[2 * i + 1] = t.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cd.vn[i] = __ldg(a.v.norms + vr + (8 * (i >> 1) + 2 * q4 + (i & 1)) * a.v.sn);
      }
    };

    Codes<D> cd;
    int64_t kr = -1, vr = -1;
    if (n_steps > 0) {
      fetch_pages(0);
      kr = __shfl_sync(dev::kFull, krec, 0);
      vr = __shfl_sync(dev::kFull, vrec, 0);
      if (kr >= 0) {
        load_k(kr, cd);
        load_v(vr, cd);
      }
    }
    for (int it = 0; it < n_steps; ++it) {
      const bool have = kr >= 0;
      const int t0 = (s0 + warp + it * W) * kStep;
      // the next step's records
      int64_t nkr = -1, nvr = -1;
      if (it + 1 < n_steps) {
        if (((it + 1) & 31) == 0) fetch_pages(it + 1);
        nkr = __shfl_sync(dev::kFull, krec, (it + 1) & 31);
        nvr = __shfl_sync(dev::kFull, vrec, (it + 1) & 31);
      }
      if (!have) {
        kr = nkr;
        vr = nvr;
        if (kr >= 0) {
          load_k(kr, cd);
          load_v(vr, cd);
        }
        continue;
      }
      // ---- scores of tokens 8 i + 2 q4 + {0, 1}
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t u = cd.k[i][w];
          mma(sc[i], qa[2 * w][0], qa[2 * w][1], qa[2 * w][2], qa[2 * w][3], pair<0>(u, ktab), pair<1>(u, ktab));
          mma(sc[i], qa[2 * w + 1][0], qa[2 * w + 1][1], qa[2 * w + 1][2], qa[2 * w + 1][3], pair<2>(u, ktab),
              pair<3>(u, ktab));
        }
      }
      float kn[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) kn[e] = cd.kn[e];
      if (nkr >= 0) load_k(nkr, cd);
      // ---- softmax; M is a reference that moves only when a weight times its norm would pass 2^8
      const bool edge = t0 + kStep > full_hi || t0 < full_lo;
      float lv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) lv[e] = fmaxf(__log2f(cd.vn[e]), -64.f);
      uint32_t pa[4];
#pragma unroll
      for (int o = 0; o < LR; ++o) {
        float z[4], t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[e] = HILO ? sc[e >> 1][e & 1] + sc[e >> 1][2 + (e & 1)] : sc[e >> 1][2 * o + (e & 1)];
          z[e] *= f[o] * kn[e];
        }
        bool seen[4] = {true, true, true, true};
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = t0 + 8 * (e >> 1) + 2 * q4 + (e & 1);
            seen[e] = j >= see_lo[o] && j < see_hi[o] && j < req.kv;
            if (!seen[e]) z[e] = -INFINITY;
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, seen[e] ? z[e] + lv[e] : -INFINITY);
        if (__any_sync(dev::kFull, mx > M[o] + 8.f)) {
          mx = fmaxf(mx, __shfl_xor_sync(dev::kFull, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(dev::kFull, mx, 2));
          const float m2 = fmaxf(M[o], mx), s = exp2f(M[o] - m2);
          M[o] = m2;
          l[o] *= s;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            acc[j][2 * o] *= s;
            acc[j][2 * o + 1] *= s;
            if (HILO) {
              acc[j][2] *= s;
              acc[j][3] *= s;
            }
          }
        }
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          t[e] = exp2_approx(z[e] - M[o]);
          l[o] += t[e];
          w[e] = seen[e] ? t[e] * cd.vn[e] : 0.f;
        }
        const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
        pa[o] = *reinterpret_cast<const uint32_t *>(&h0);
        pa[2 + o] = *reinterpret_cast<const uint32_t *>(&h1);
        if (HILO) {
          const float2 b0 = __half22float2(h0), b1 = __half22float2(h1);
          const __half2 l0 = __floats2half2_rn(w[0] - b0.x, w[1] - b0.y);
          const __half2 l1 = __floats2half2_rn(w[2] - b1.x, w[3] - b1.y);
          pa[1] = *reinterpret_cast<const uint32_t *>(&l0);
          pa[3] = *reinterpret_cast<const uint32_t *>(&l1);
        }
      }
      // ---- values: tokens 2 q4 and 2 q4 + 1 interleaved (even and odd coordinates apart)
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        const uint32_t x0 = cd.v[0][w], x1 = cd.v[1][w], x2 = cd.v[2][w], x3 = cd.v[3][w];
        const uint32_t e0 = (x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u);
        const uint32_t o0 = ((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
        const uint32_t e1 = (x2 & 0x0f0f0f0fu) | ((x3 << 4) & 0xf0f0f0f0u);
        const uint32_t o1 = ((x2 >> 4) & 0x0f0f0f0fu) | (x3 & 0xf0f0f0f0u);
        mma(acc[8 * w + 0], pa[0], pa[1], pa[2], pa[3], pair<0>(e0, vtab), pair<0>(e1, vtab));
        mma(acc[8 * w + 1], pa[0], pa[1], pa[2], pa[3], pair<0>(o0, vtab), pair<0>(o1, vtab));
        mma(acc[8 * w + 2], pa[0], pa[1], pa[2], pa[3], pair<1>(e0, vtab), pair<1>(e1, vtab));
        mma(acc[8 * w + 3], pa[0], pa[1], pa[2], pa[3], pair<1>(o0, vtab), pair<1>(o1, vtab));
        mma(acc[8 * w + 4], pa[0], pa[1], pa[2], pa[3], pair<2>(e0, vtab), pair<2>(e1, vtab));
        mma(acc[8 * w + 5], pa[0], pa[1], pa[2], pa[3], pair<2>(o0, vtab), pair<2>(o1, vtab));
        mma(acc[8 * w + 6], pa[0], pa[1], pa[2], pa[3], pair<3>(e0, vtab), pair<3>(e1, vtab));
        mma(acc[8 * w + 7], pa[0], pa[1], pa[2], pa[3], pair<3>(o0, vtab), pair<3>(o1, vtab));
      }
      if (nvr >= 0) load_v(nvr, cd);
      kr = nkr;
      vr = nvr;
    }

    // ---- the warps' sums: coordinate n (D/8) + j of a row at 8 j + n
#pragma unroll
    for (int o = 0; o < LR; ++o) {
      float t = l[o];
      t += __shfl_xor_sync(dev::kFull, t, 1);
      t += __shfl_xor_sync(dev::kFull, t, 2);
      if (q4 == 0) {
        s_m[warp][g + 8 * o] = M[o];
        s_l[warp][g + 8 * o] = t;
      }
      float *dst = parts + ((size_t)warp * RT + g + 8 * o) * PITCH + 2 * q4;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        *reinterpret_cast<float2 *>(dst + 8 * j) =
            HILO ? make_float2(acc[j][0] + acc[j][2], acc[j][1] + acc[j][3])
                 : make_float2(acc[j][2 * o], acc[j][2 * o + 1]);
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
        const float *src = parts + ((size_t)w * RT + i) * PITCH;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const int k = lane * (D / 32) + e;
          y[e] = fmaf(s, src[8 * (k % NV) + k / NV], y[e]);
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
template <int D, bool HILO>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ RowsParams p) {
  constexpr int RT = HILO ? 8 : 16;
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

template <int D, bool HILO>
cudaError_t run_rows(const RowsParams &p, cudaStream_t s) {
  // dynamic shared memory starts behind the 1 KiB that the system keeps
  const int dyn = (int)smem_end<D, HILO>() - 1024;
  auto kern = paged_rows_kernel<D, HILO>;
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
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, HILO>, p);
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
  const bool hilo = (int64_t)a.max_q * (a.Hq / a.Hkv) <= 8;
  if (a.kq.d == 64) return hilo ? run_rows<64, true>(p, s) : run_rows<64, false>(p, s);
  return hilo ? run_rows<128, true>(p, s) : run_rows<128, false>(p, s);
}

}  // namespace tq
