// Attention of a few query rows a request over a paged 4-bit cache (sm_100a):
// decode, and the verification of a few draft tokens; for d = 256 any number
// of rows.
//
// Work: a unit is (request, KV head, tile of query rows), a step 32 cached
// tokens.  All units' steps, and a fixed cost of each unit, form one line, cut
// into equal ranges, one a CTA (one persistent CTA an SM), so requests of any
// lengths balance; a CTA's part of a unit is a piece, whose steps its warps
// take in turn.  Units cut by a range's end leave partial sums that a second
// kernel merges, in the order of the tokens, so the result does not depend on
// timing.
//
// A step of a warp: S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16 (fp16,
// fp32 sums), the tokens (then the coordinates) being the 16 rows and the
// query rows the 8 columns, and the running softmax in between.  Query rows
// and weights are fp16 pairs hi + lo: up to 4 rows a tile put both into one
// product, as columns g and g + 4 (S and O are the sums of the two); more take
// two products into the same sums.  For bf16 outputs more than 4 rows are
// rounded once, 2^-11 against the output's 2^-8 (8 rows on 4 requests of up to
// 65536 tokens: 61 us, with pairs 68).  Codes become operand words without
// arithmetic: a code byte (two codes) indexes a 256-entry table of fp16
// centroid pairs, one copy per lane, placed so that one byte permute forms the
// shared address.  For K the pair is two coordinates of a token; for V the
// codes of two tokens are first interleaved, so the pair is two tokens at one
// coordinate.  The order of coordinates within the products is free, so every
// lane loads whole runs of a record.  Norms enter behind the products: ||k||
// scales the logit, ||v|| the weight.
//
// Beyond 8 rows a warp takes 16, two column tiles, and reads the tables once
// for both; beyond 16 two groups of warps, each with 16 of a unit's rows, go
// through the same steps together, so a record comes from memory once.  64
// requests of up to 4001 tokens, 16 and 32 rows, us, and with groups of 8 rows
// instead: bf16 91 and 149 (113 and 187), fp16 109 and 181 (121 and 203).  For
// d = 256 the registers hold one column tile, so a group is of 8 rows.
//
// A step's records come through a ring of two stages in shared memory a warp
// (cp.async): the next step's are on their way while one is worked on (4
// requests of up to 262144 tokens 206 us, against 265 with a single and 296
// with a double buffer in registers).
//
// Bound by the instruction stream, about 330 warp instructions per 16 tokens
// of a KV head (128 of them the byte permutes and table reads) at half of the
// issue slots, and by what a piece costs besides its steps, about 5 us.
// Measured on a B200: d = 128, 32 / 8 heads, bf16, 4 requests of up to 262144
// tokens (731 MB) 188 us, 3.9 TB/s; 16 of up to 65536 (551 MB) 148 us, 3.7
// TB/s; 1 x 32768 tokens 23.5 us, of which 11.5 are left with a single step; 128
// requests of 4 rows and up to 4001 tokens, 64 / 8 heads, fp16, 330 us; d =
// 256, 16 requests of up to 4001 tokens, 32 / 8 heads, bf16, 40 us.

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"
#include "tq_paged_dev.cuh"

#include <float.h>

#include <type_traits>

namespace tq {
namespace {

using namespace paged;

constexpr int kStep = 32;                // tokens per step, in two halves of 16 that may lie in two pages
constexpr uint32_t kTabAddr = 0x10000u;  // the pair tables: 64 KiB at this shared address
constexpr uint32_t kPartAddr = 0x20000u; // the warps' partial sums
constexpr int64_t kSteps = ((int64_t)1 << 42) - 1;
constexpr int kStages = 2;               // a warp's steps in shared memory: one worked on, one on its way

template <int D>
struct Cfg {
  // 168 registers a thread; 16 warps of 128 took 207 us where 12 take 198 (d = 128).  For d = 256 the sums, the query
  // operands and the ring are twice as large: 8 warps of 255 registers
  static constexpr int kWarps = D == 256 ? 8 : 12;
  static constexpr int kMaxRows = D == 256 ? 8 : 16;    // query rows of a group of warps
  static constexpr int kUnitRows = D == 256 ? 16 : 32;  // of a unit
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPitch = D + 4;  // floats of a partial row (no bank clash between rows)
  // a step: K codes, V codes, norms of each
  static constexpr int kStepBytes = kStep * D + 2 * kStep * 4;
  static constexpr int kRing = kStages * kStepBytes;
  // rings above the tables (the partial sums reuse the space), the rest below
  static constexpr int kFit = (227 * 1024 - (int)kPartAddr) / kRing;
  static constexpr int kHigh = kFit < kWarps ? kFit : kWarps;
};

// Shared memory below the tables.
template <int D>
struct Low {
  int64_t base[Cfg<D>::kThreads];  // the line at each thread's first request
  int64_t warp[Cfg<D>::kWarps];
  alignas(16) __half q[2][Cfg<D>::kUnitRows][D + 32];  // operand columns: hi of each row, lo of each row (q_place)
  float f[Cfg<D>::kUnitRows];                          // logit factor of each row
  int see_lo[Cfg<D>::kUnitRows], see_hi[Cfg<D>::kUnitRows];  // the tokens that each row sees
  float m[Cfg<D>::kWarps][Cfg<D>::kMaxRows], l[Cfg<D>::kWarps][Cfg<D>::kMaxRows];
  float scale[2];                  // what the tables' values are to be divided by
  unsigned key[2];
  __half level[2][16];             // the scaled levels
  float e[Cfg<D>::kWarps][Cfg<D>::kMaxRows], top[Cfg<D>::kUnitRows], sum[Cfg<D>::kUnitRows];  // merge of the warps
};

template <int D>
__host__ __device__ constexpr uint32_t smem_end() {
  constexpr uint32_t parts = Cfg<D>::kWarps * Cfg<D>::kMaxRows * Cfg<D>::kPitch * 4;
  constexpr uint32_t rings = Cfg<D>::kHigh * Cfg<D>::kRing;
  static_assert(kPartAddr + (parts > rings ? parts : rings) <= 227 * 1024, "");
  return kPartAddr + (parts > rings ? parts : rings);
}

struct RowsParams {
  PagedAttentionArgs a;
  int groups;       // warps are in so many groups of 4, 8 or 16 query rows, which go through the same steps
  float *slots;     // [2 * ctas][kUnitRows][D + 2]: sums, then M and L
  int4 *desc;       // [2 * ctas]: {pieces, rows, first row, head}, {first query row, what the values' table is to be
                    // divided by} of the unit that starts last in a range
  unsigned *faults;
};

// One request: its rows, and the steps that any of its rows sees.
struct Req {
  int q0, n;        // query rows
  int kv;
  int first;        // the first token that any of its rows sees
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
  q.first = window_start(q.kv - q.n, a.window);
  q.lo = q.first / kStep;
  // a request that sees nothing still has one (empty) step, which writes its zeros
  q.hi = max(runs(q.kv, kStep), q.lo + 1);
  return q;
}

// Places of a unit in the line: its steps, and before them `cost` for what it costs besides (the first copies' way, the
// merge of the warps), so that ranges of many short units do not end late: 16 requests of up to 65536 tokens 148 us,
// without it 188; 64 of up to 4001 with 16 rows 89 us, without it 155.  Flat between 30 and 50 steps of all 12 warps.
constexpr int kUnitCost = 36;
__device__ __forceinline__ int64_t weight(const Req &q, int Hkv, int cost) {
  return (int64_t)q.tiles * Hkv * (q.hi - q.lo + cost);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// Table read of byte k of w: shared address {lane, byte k, table}.
template <int K>
__device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t base) {
  uint32_t a;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(a) : "r"(w), "r"(base), "n"(0x7604 | (K << 4)));
  return lds32(a);
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

// Coordinate g (D/8) + 2 j + b of an unfinished row is kept at place 16 j + 2 g + b.
template <int D>
__device__ __forceinline__ int place(int k) {
  const int u = k % (D / 8);
  return 16 * (u / 2) + 2 * (k / (D / 8)) + (u & 1);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(a));
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// Where the staged V codes of token t, 16-byte word c, lie, so that a
// half-warp's reads (8 bytes of tokens 0, 2, 4, 6; a quarter-warp's 16 for d =
// 256) fall into different banks: two tokens swap places in every other group
// of four, and word pairs in every other pair of tokens; for d = 256, word
// pairs are exchanged by the pair of tokens.
template <int D>
__device__ __forceinline__ uint32_t v_place(int t, int c) {
  if constexpr (D == 256) return (uint32_t)(t * (D / 2) + (c ^ (((t >> 1) & 3) << 1)) * 16);
  return (uint32_t)((t ^ ((t >> 2) & 1)) * (D / 2) + (D == 128 ? (c ^ (((t >> 1) & 1) << 1)) * 16 : c * 16));
}
// And those of K: for d = 256, whose records are as long as all banks, words
// are exchanged by the token.
template <int D>
__device__ __forceinline__ uint32_t k_place(int t, int c) {
  return (uint32_t)(t * (D / 2) + (D == 256 ? c ^ (t & 7) : c) * 16);
}

// Where coordinate k of a query row lies: a lane's words of two k steps are 16
// bytes, and a quarter-warp's fall into different banks.
template <int D>
__device__ __forceinline__ int q_place(int k) {
  const int u = k % (D / 4);
  return 8 * (4 * (u / 8) + k / (D / 4)) + u % 8;
}

// RG: query rows of a group of warps.  Up to 4: hi and lo are columns of one
// product; 8: one column tile; 16: two, for which a warp reads the tables once.
// MULTI: several groups of warps.  UNIT: the tokens of a page lie side by side, and K and V records alike.
template <int D, int RG, bool MULTI, bool UNIT, bool HL>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) paged_rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = Cfg<D>::kWarps, NT = Cfg<D>::kThreads, PITCH = Cfg<D>::kPitch;
  constexpr int kMaxRows = Cfg<D>::kMaxRows, kUnitRows = Cfg<D>::kUnitRows;
  constexpr bool P4 = RG == 4;
  constexpr int NC = RG == 16 ? 2 : 1;  // column tiles
  constexpr int KS = D / 16;      // k steps of the scores
  constexpr int MV = D / 16;      // m tiles of the values
  constexpr int QS = HL && !P4 ? 2 : 1;  // products per step
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
  const int groups = MULTI ? p.groups : 1;
  const int RT = RG * groups, WG = W / groups;         // rows of a unit, warps of a group
  // the warp's group, its place there, the group's first row
  const int group = MULTI ? warp / WG : 0, wg = warp - group * WG, gr = RG * group;
  const int cost = kUnitCost / groups;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const uint32_t dyn = (uint32_t)__cvta_generic_to_shared(s_raw);
  uint32_t dyn_bytes;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn_bytes));
  if (dyn + sizeof(Low<D>) + (W - Cfg<D>::kHigh) * Cfg<D>::kRing > kTabAddr || dyn + dyn_bytes < smem_end<D>()) {
    if (tid == 0) {
      atomicOr(p.faults, kFaultSmemLayout);
      p.desc[2 * c] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  float *parts = reinterpret_cast<float *>(s_raw + (kPartAddr - dyn));  // [W][kMaxRows][PITCH]

  // ---- the tables' scales, and the line of steps: a run of requests a thread
  if (tid < 2) sm.key[tid] = 0xffffffffu;
  const int per = (a.R + NT - 1) / NT;
  int64_t mine = 0;  // steps, and units from bit 42 on
  for (int r = tid * per; r < min((tid + 1) * per, a.R); ++r) {
    const Req q = load_req(a, r, RT, p.faults);
    mine += weight(q, a.Hkv, cost) + (int64_t)((uint64_t)q.tiles * (uint64_t)a.Hkv << 42);
  }
  __syncthreads();
  find_scales(a.kq.centroids, a.vq.centroids, tid, NT, sm.key);
  int64_t total;
  int units;
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
    units = (int)(total >> 42);
    total &= kSteps;
    s_base[tid] = (base + x - mine) & kSteps;
  }
  __syncthreads();

  // Ranges.  Where the units are fewer than the CTAs, a multiple of them that idles at most a twentieth of the SMs:
  // equally long units are then cut evenly and no CTA has parts of two (1 x 32768 tokens, 8 KV heads: 144 CTAs).
  // Every range has a step at least, so no piece of a unit is missing.
  int ctas = (int)gridDim.x;
  if (units > 0 && units <= ctas && 20 * (ctas % units) <= ctas) ctas -= ctas % units;
  ctas = (int)min((int64_t)ctas, total);
  auto cut = [&](int i) {
    return total < (1 << 21) ? (int64_t)((uint32_t)total * (uint32_t)i / (uint32_t)ctas) : total * i / ctas;
  };
  int64_t at = c < ctas ? cut(c) : 0;
  const int64_t end = c < ctas ? cut(c + 1) : 0;
  int4 desc = make_int4(0, 0, 0, 0), where = desc;
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
      const int64_t w = weight(req, a.Hkv, cost);
      if (at < r_base + w) break;
      r_base += w;
    }
  }
  uint32_t ktab, vtab;  // opaque, so that a table address stays one byte permute
  asm("mov.b32 %0, %1;" : "=r"(ktab) : "r"(kTabAddr + 4 * lane));
  asm("mov.b32 %0, %1;" : "=r"(vtab) : "r"(kTabAddr + 4 * lane + 128));

  // the lane's 16 bytes of a half's records (of its first 8 tokens for d = 128) and its norm, and where they go
  const int64_t k_tok = a.k.sn * (D / 2), v_tok = a.v.sn * (D / 2);
  const uint8_t *kc_lane = a.k.codes + (lane / (D / 32)) * k_tok + (lane % (D / 32)) * 16;
  const uint8_t *vc_lane = a.v.codes + (lane / (D / 32)) * v_tok + (lane % (D / 32)) * 16;
  const float *n_lane = lane < 16 ? a.k.norms + lane * a.k.sn : a.v.norms + (lane - 16) * a.v.sn;
  const uint32_t k_to = k_place<D>(lane / (D / 32), lane % (D / 32));
  const uint32_t v_to = v_place<D>(lane / (D / 32), lane % (D / 32)), n_to = 4 * (lane & 15) + (lane < 16 ? 0 : 128);
  // and the lane's reads: V of tokens 2 q4 and 2 q4 + 1
  const uint32_t v_at0 = v_place<D>(2 * q4, g * (D / 16) / 16) + (g * (D / 16)) % 16;
  const uint32_t v_at1 = v_place<D>(2 * q4 + 1, g * (D / 16) / 16) + (g * (D / 16)) % 16;
  const uint32_t ring = warp < Cfg<D>::kHigh ? kPartAddr + warp * Cfg<D>::kRing
                                             : kTabAddr - (warp - Cfg<D>::kHigh + 1) * Cfg<D>::kRing;

  for (bool tables = false; at < end && r < a.R; tables = true) {
    // ---- the piece: steps [s0, s1) of unit (r, h, tile)
    const int len = req.hi - req.lo + cost;
    const int64_t x = at - r_base;
    const int unit = x < INT_MAX ? (int)((uint32_t)x / (uint32_t)len) : (int)(x / len);
    const int x0 = (int)(x - (int64_t)unit * len), x1 = (int)min((int64_t)len, x0 + (end - at));
    if (x1 <= cost) break;  // the range ends before the unit's first step
    const int s0 = req.lo + max(x0 - cost, 0), s1 = req.lo + x1 - cost;
    const int h = unit / req.tiles, tile = unit - h * req.tiles;
    const int row0 = tile * RT;
    const int nrows = min(RT, req.n * G - row0);

    const int32_t *row = a.table + (int64_t)r * a.table_stride;
    const int mine_rows = min(RG, nrows - gr);  // of the warp's group
    const int n_steps = mine_rows > 0 && s1 - s0 > wg ? (s1 - s0 - wg + WG - 1) / WG : 0;
    // The records of 4 of the warp's steps, half lane % 2 of step it + lane / 2 % 4 a lane, found a batch ahead;
    // -1 without a page and behind the piece's last step.
    int64_t krec, vrec, krec2, vrec2;
    auto find = [&](int it, int64_t &kr, int64_t &vr) {
      const int s = s0 + wg + (it + ((lane >> 1) & 3)) * WG;
      kr = vr = -1;
      const int t0 = s * kStep + 16 * (lane & 1);
      if (s < s1 && t0 < req.kv && t0 + 16 > req.first) {
        const int page = t0 / a.page_size, off = t0 - page * a.page_size;
        const int id = __ldg(row + page);
        if ((unsigned)id < (unsigned)a.n_pages) {
          kr = id * a.k.sb + h * a.k.sh + off * a.k.sn;
          vr = UNIT ? kr : id * a.v.sb + h * a.v.sh + off * a.v.sn;
        } else {
          atomicOr(p.faults, kFaultIndex);
        }
      }
    };
    // Step it's records into its stage, asynchronously; bits 2 stage + half of `ok` say whether there are any.
    uint32_t ok = 0;
    auto issue = [&](int it) {
      const int stage = it & 1;
      const uint32_t to = ring + stage * Cfg<D>::kStepBytes;
      ok &= ~(3u << (2 * stage));
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int64_t kr = __shfl_sync(dev::kFull, krec, 2 * (it & 3) + hf);
        const int64_t vr = UNIT ? kr : __shfl_sync(dev::kFull, vrec, 2 * (it & 3) + hf);
        if (kr >= 0) {
          ok |= 1u << (2 * stage + hf);
          const uint8_t *ks = kc_lane + kr * (D / 2), *vs = vc_lane + vr * (D / 2);
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            constexpr int TI = 1024 / D;                    // tokens of 32 lanes
            const uint32_t turn = D == 256 ? 64 * (i & 1) : 0;  // of k_place and v_place, TI i tokens on
            cp_async16(to + (k_to ^ turn) + hf * (8 * D) + 512 * i, ks + (UNIT ? 512 * i : TI * i * k_tok));
            cp_async16(to + kStep * (D / 2) + (v_to ^ turn) + hf * (8 * D) + 512 * i,
                       vs + (UNIT ? 512 * i : TI * i * v_tok));
          }
          // lanes 0..15 the norms of K, the others those of V
          cp_async4(to + kStep * D + n_to + 64 * hf, n_lane + (UNIT || lane < 16 ? kr : vr));
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (n_steps > 0) {
      find(0, krec, vrec);
      find(4, krec2, vrec2);
      issue(0);
    }

    if (!tables) {
      // ---- the tables, while the first records are on their way: entry e, lane l at 256 e + 4 l (keys) and + 128
      if (warp < 2) {
        const float *cent = warp == 0 ? a.kq.centroids : a.vq.centroids;
        float unit;
        const float s = scale_of(sm.key[warp], NT, cent, unit);
        if (lane < 16) sm.level[warp][lane] = __float2half_rn(s * __ldg(cent + lane));
        if (lane == 0) s_scale[warp] = unit;
      }
      __syncthreads();
      uint4 *tab = reinterpret_cast<uint4 *>(s_raw + (kTabAddr - dyn));
      for (int i = tid; i < 256 * 16; i += NT) {
        const __half *lv = sm.level[(i >> 3) & 1];
        const __half2 h = __halves2half2(lv[(i >> 4) & 15], lv[i >> 8]);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&h);
        tab[i] = make_uint4(w, w, w, w);
      }
    }
    const float kscale = a.scale * 1.4426950408889634f / (a.kq.sqrt_d * s_scale[0]);
    const float vscale = 1.0f / (a.vq.sqrt_d * s_scale[1]);

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
      if (lane == 0) {
        // a row that is not there sees everything (and goes nowhere)
        int lo = 0, hi = INT_MAX;
        if (i < nrows) {
          const int pos = req.kv - req.n + (row0 + i) / G;
          hi = a.causal ? max(pos + 1, 0) : req.kv;
          lo = window_start(pos, a.window);
        }
        s_f[i] = kscale / f;
        sm.see_lo[i] = lo;
        sm.see_hi[i] = hi;
      }
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const float y = v[e] * f;
        const __half hi = __float2half_rn(y);
        const int k = q_place<D>(lane * (D / 32) + e);
        s_q[0][i][k] = hi;
        if (HL) s_q[P4 ? 0 : 1][P4 ? i + 4 : i][k] = __float2half_rn(y - __half2float(hi));
      }
    }
    __syncthreads();
    // the query operands of k steps 2 w and 2 w + 1: kept in registers for one column tile
    uint4 qb[NC == 1 ? QS : 1][NC == 1 ? KS / 2 : 1];
    auto load_q = [&](int o, int ct, int w) {
      return *reinterpret_cast<const uint4 *>(&s_q[o][gr + 8 * ct + g][8 * (4 * w + q4)]);
    };
    if constexpr (NC == 1) {
#pragma unroll
      for (int o = 0; o < QS; ++o)
#pragma unroll
        for (int w = 0; w < KS / 2; ++w) qb[o][w] = load_q(o, 0, w);
    }
    // the lane's rows, two a column tile
    auto row_of = [&](int ct, int o) { return gr + 8 * ct + ((2 * q4 + o) & (RG < 8 ? RG - 1 : 7)); };
    float f[NC][2], M[NC][2], l[NC][2];
#pragma unroll
    for (int ct = 0; ct < NC; ++ct)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        f[ct][o] = s_f[row_of(ct, o)];
        M[ct][o] = -FLT_MAX;
        l[ct][o] = 0.f;
      }
    // steps that every row of the group sees whole
    const int first_pos = req.kv - req.n + (row0 + gr) / G,
              last_pos = req.kv - req.n + (row0 + gr + mine_rows - 1) / G;
    const int full_hi = a.causal ? max(first_pos + 1, 0) : req.kv;
    const int full_lo = window_start(last_pos, a.window);

    float acc[NC][MV][4];
#pragma unroll
    for (int ct = 0; ct < NC; ++ct)
#pragma unroll
      for (int j = 0; j < MV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[ct][j][e] = 0.f;

    // The running softmax of the lane's rows over its tokens 8 i + g (value [i][o]: row o): scores in, weights
    // times value norms out.  M is a reference that moves only when one of them would pass 2^15 (fp16 ends at 2^16),
    // and then to kRoom below the largest.
    auto soft = [&](auto edge, auto tile, int t0, uint32_t halves, float (&t)[4][2], const float (&kn)[4],
                    const float (&vn)[4], const float (&lv)[4]) {
      constexpr bool EDGE = decltype(edge)::value;
      constexpr int CT = decltype(tile)::value;
      float s[4][2], mx = -INFINITY;
      bool seen[4][2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int lo = EDGE ? sm.see_lo[row_of(CT, o)] : 0, hi = EDGE ? min(sm.see_hi[row_of(CT, o)], req.kv) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = t0 + 8 * i + g;
          seen[i][o] = !EDGE || (j >= lo && j < hi && (halves >> (i >> 1) & 1));
          s[i][o] = t[i][o] * (f[CT][o] * kn[i]);
          t[i][o] = s[i][o] - M[CT][o];
          if (EDGE && !seen[i][o]) t[i][o] = -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(t[i][0], t[i][1]) + lv[i]);
      if (__any_sync(dev::kFull, mx > kMost)) {
        float r2[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i)  // an infinite value norm brings every step here, and does not count (value_log2)
            m = fmaxf(m, seen[i][o] ? s[i][o] + (lv[i] < INFINITY ? lv[i] : -64.f) : -INFINITY);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(dev::kFull, m, x));
          m = fmaxf(M[CT][o], m - kRoom);
          r2[o] = exp2f(M[CT][o] - m);
          M[CT][o] = m;
          l[CT][o] *= r2[o];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i][o] = seen[i][o] ? s[i][o] - m : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < MV; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[CT][j][e] *= r2[e & 1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          t[i][o] = exp2_approx(t[i][o]);
          l[CT][o] += t[i][o];
          t[i][o] *= vn[i];
          if (EDGE && !seen[i][o]) t[i][o] = 0.f;
        }
    };

    for (int it = 0; it < n_steps; ++it) {
      const int t0 = (s0 + wg + it * WG) * kStep;
      const uint32_t halves = ok >> (2 * (it & 1)) & 3;
      const uint32_t from = ring + (it & 1) * Cfg<D>::kStepBytes;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      if (((it + 1) & 3) == 0) {
        krec = krec2;
        vrec = vrec2;
        find(it + 5, krec2, vrec2);
      }
      issue(it + 1);  // into the stage of step it - 1
      if (!halves) continue;
      // ---- scores: value 2 x + o of half i is token 16 i + 8 x + g, column 2 q4 + o
      float sc[NC][2][4];
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[ct][i][e] = 0.f;
      // a query operand that is not kept is read once for both halves, so their codes come in runs of two words
      constexpr int CW = 2, HV = 2;  // code words, halves a run
#pragma unroll
      for (int r0 = 0; r0 < D / 32 / CW; ++r0) {
        uint32_t c0[HV][CW], c1[HV][CW];  // codes of tokens 16 i + g and 16 i + 8 + g
#pragma unroll
        for (int x = 0; x < HV; ++x) {
          const int i = x, at_word = 4 * CW * r0;
          const uint32_t k_at = k_place<D>(g, (q4 * (D / 8) + at_word) / 16) + (q4 * (D / 8) + at_word) % 16;
          lds_words(from + 16 * i * (D / 2) + k_at, c0[x]);
          lds_words(from + (16 * i + 8) * (D / 2) + k_at, c1[x]);
        }
#pragma unroll
        for (int w = 0; w < CW; ++w) {
          uint4 qv[NC][QS];
#pragma unroll
          for (int ct = 0; ct < NC; ++ct)
#pragma unroll
            for (int o = 0; o < QS; ++o) {
              if constexpr (NC == 1) qv[ct][o] = qb[o][CW * r0 + w];
              else qv[ct][o] = load_q(o, ct, CW * r0 + w);
            }
#pragma unroll
          for (int x = 0; x < HV; ++x) {
            const int i = x;
            const uint32_t u = c0[x][w], v = c1[x][w];
            const uint32_t a0 = pair<0>(u, ktab), a1 = pair<0>(v, ktab), a2 = pair<1>(u, ktab), a3 = pair<1>(v, ktab);
            const uint32_t b0 = pair<2>(u, ktab), b1 = pair<2>(v, ktab), b2 = pair<3>(u, ktab), b3 = pair<3>(v, ktab);
#pragma unroll
            for (int o = 0; o < QS; ++o)
#pragma unroll
              for (int ct = 0; ct < NC; ++ct) mma(sc[ct][i], a0, a1, a2, a3, qv[ct][o].x, qv[ct][o].y);
#pragma unroll
            for (int o = 0; o < QS; ++o)
#pragma unroll
              for (int ct = 0; ct < NC; ++ct) mma(sc[ct][i], b0, b1, b2, b3, qv[ct][o].z, qv[ct][o].w);
          }
        }
      }
      float kn[4], vn[4], lv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kn[i] = lds_f32(from + kStep * D + 4 * (8 * i + g));
        vn[i] = lds_f32(from + kStep * D + 128 + 4 * (8 * i + g));
        lv[i] = fmaxf(log2_approx(vn[i]), -64.f);
      }
      const bool edge = (unsigned)t0 + kStep > (unsigned)full_hi || t0 < full_lo || halves != 3;
      uint32_t pb[NC][QS][4];
      auto weights = [&](auto tile) {
        constexpr int CT = decltype(tile)::value;
        float t[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            t[i][o] = sc[CT][i >> 1][2 * (i & 1) + o];
            if (P4) t[i][o] += __shfl_xor_sync(dev::kFull, t[i][o], 2);  // the hi and lo columns
          }
        if (edge)
          soft(std::true_type{}, tile, t0, halves, t, kn, vn, lv);
        else
          soft(std::false_type{}, tile, t0, halves, t, kn, vn, lv);
        // weights to operand words: fp16 pairs of two rows at a token, transposed to two tokens of a row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 hi = __floats2half2_rn(t[i][0], t[i][1]);
          const float2 back = __half22float2(hi);
          const __half2 lo = __floats2half2_rn(t[i][0] - back.x, t[i][1] - back.y);
          const uint32_t wh = *reinterpret_cast<const uint32_t *>(&hi), wl = *reinterpret_cast<const uint32_t *>(&lo);
          if (P4) {
            pb[CT][0][i] = transpose8(q4 < 2 ? wh : wl);
          } else {
            pb[CT][0][i] = transpose8(wh);
            if (HL) pb[CT][QS - 1][i] = transpose8(wl);
          }
        }
      };
      weights(std::integral_constant<int, 0>{});
      if constexpr (NC == 2) weights(std::integral_constant<int, 1>{});
      // ---- values: tokens 2 q4 and 2 q4 + 1 interleaved (even and odd coordinates apart)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t vf = from + kStep * (D / 2) + 16 * i * (D / 2);
        uint32_t c0[D / 64], c1[D / 64], c2[D / 64], c3[D / 64];
        lds_words(vf + v_at0, c0);
        lds_words(vf + v_at1, c1);
        lds_words(vf + 8 * (D / 2) + v_at0, c2);
        lds_words(vf + 8 * (D / 2) + v_at1, c3);
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          const uint32_t e0 = (c0[w] & 0x0f0f0f0fu) | ((c1[w] << 4) & 0xf0f0f0f0u);
          const uint32_t o0 = ((c0[w] >> 4) & 0x0f0f0f0fu) | (c1[w] & 0xf0f0f0f0u);
          const uint32_t e1 = (c2[w] & 0x0f0f0f0fu) | ((c3[w] << 4) & 0xf0f0f0f0u);
          const uint32_t o1 = ((c2[w] >> 4) & 0x0f0f0f0fu) | (c3[w] & 0xf0f0f0f0u);
          auto tile = [&](auto k) {
            constexpr int K = decltype(k)::value;
            const uint32_t a0 = pair<K>(e0, vtab), a1 = pair<K>(o0, vtab);
            const uint32_t a2 = pair<K>(e1, vtab), a3 = pair<K>(o1, vtab);
#pragma unroll
            for (int o = 0; o < QS; ++o)
#pragma unroll
              for (int ct = 0; ct < NC; ++ct)
                mma(acc[ct][4 * w + K], a0, a1, a2, a3, pb[ct][o][2 * i], pb[ct][o][2 * i + 1]);
          };
          tile(std::integral_constant<int, 0>{});
          tile(std::integral_constant<int, 1>{});
          tile(std::integral_constant<int, 2>{});
          tile(std::integral_constant<int, 3>{});
        }
      }
    }
    // all copies of this warp are in, and every warp is through with its ring before the sums go there
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    // ---- the warps' sums
#pragma unroll
    for (int ct = 0; ct < NC; ++ct) {
      const int i0 = 8 * ct + 2 * q4;
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        float t = l[ct][o];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(dev::kFull, t, x);
        if (g == 0 && i0 < RG) {
          s_m[warp][i0 + o] = M[ct][o];
          s_l[warp][i0 + o] = t;
        }
      }
#pragma unroll
      for (int j = 0; j < MV; ++j)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          float x = acc[ct][j][o], y = acc[ct][j][2 + o];
          if (P4) {
            x += __shfl_xor_sync(dev::kFull, x, 2);
            y += __shfl_xor_sync(dev::kFull, y, 2);
          }
          if (i0 < RG)
            *reinterpret_cast<float2 *>(parts + ((size_t)warp * kMaxRows + i0 + o) * PITCH + 16 * j + 2 * g) =
                make_float2(x, y);
        }
    }
    __syncthreads();
    const bool starts = s0 == req.lo, ends = s1 == req.hi;
    // each warp's factor for each row of its group
    if (tid < W * RG) {
      const int w = tid / RG, i = tid % RG, w0 = MULTI ? w - w % WG : 0;
      float m = s_m[w0][i];
      for (int x = w0 + 1; x < w0 + WG; ++x) m = fmaxf(m, s_m[x][i]);
      sm.e[w][i] = exp2f(s_m[w][i] - m);
      if (w == w0) sm.top[RG * (w / WG) + i] = m;
    }
    __syncthreads();
    float *slot = p.slots + (size_t)(2 * c + (starts ? 1 : 0)) * kUnitRows * (D + 2);
    for (int u = tid; u < nrows * D; u += NT) {
      const int i = u / D, k = u % D, w0 = MULTI ? i / RG * WG : 0, ri = i % RG;  // place k of the row
      float y = 0.f;
#pragma unroll
      for (int w = w0; w < w0 + WG; ++w) y = fmaf(sm.e[w][ri], parts[(w * kMaxRows + ri) * PITCH + k], y);
      if (starts && ends)
        parts[(w0 * kMaxRows + ri) * PITCH + k] = y;  // only this thread has read it
      else
        slot[i * (D + 2) + k] = y;
    }
    if (tid < nrows) {
      const int w0 = MULTI ? tid / RG * WG : 0, ri = tid % RG;
      float L = 0.f;
      for (int w = w0; w < w0 + WG; ++w) L = fmaf(sm.e[w][ri], s_l[w][ri], L);
      sm.sum[tid] = L;
      if (!(starts && ends)) {
        slot[tid * (D + 2) + D] = sm.top[tid];
        slot[tid * (D + 2) + D + 1] = L;
      }
    }
    if (starts && ends) {
      __syncthreads();
      for (int i = warp; i < nrows; i += W) {
        const float *src = parts + (size_t)(i / RG * WG * kMaxRows + i % RG) * PITCH;
        float y[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) y[e] = src[place<D>(lane * (D / 32) + e)];
        const int qi = (row0 + i) / G;
        store_out<D>(a, (int64_t)req.q0 + qi, h * G + (row0 + i) - qi * G, lane, y, sm.top[i], sm.sum[i], vscale);
      }
    }
    if (starts && !ends) {
      // CTAs whose ranges the unit reaches: the last holds its last step
      const int64_t last = at + (len - x0) - 1;
      int e = c;
      if (last >= end) {
        e = (int)(last * ctas / total);  // a first guess
        while (e < ctas - 1 && cut(e + 1) <= last) ++e;
        while (e > c && cut(e) > last) --e;
      }
      desc = make_int4(e - c + 1, nrows, row0, h);
      where = make_int4(req.q0, __float_as_int(s_scale[1]), 0, 0);
    }
    __syncthreads();
    at += x1 - x0;
    if (at < end && at - r_base == weight(req, a.Hkv, cost)) {
      r_base = at;
      while (++r < a.R) {
        req = load_req(a, r, RT, p.faults);
        if (weight(req, a.Hkv, cost) > 0) break;
      }
    }
  }
  if (tid == 0) {
    p.desc[2 * c] = desc;
    p.desc[2 * c + 1] = where;
  }
}

// Merges the pieces of the unit that starts last in CTA c's range and goes on
// behind it, in the order of the tokens: a block a unit and group of rows, a
// coordinate of a row a thread.
template <int D, int RT>
__global__ void __launch_bounds__(D * RT) paged_merge_kernel(const __grid_constant__ RowsParams p) {
  __shared__ float s_y[RT][D], s_top[RT];
  __shared__ float s_e[RT][32], s_l[RT];
  const PagedAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 desc = __ldcg(p.desc + 2 * c), where = __ldcg(p.desc + 2 * c + 1);
  const int r8 = RT * blockIdx.y;  // the block's first row of the unit
  const int n = desc.x, nrows = min(RT, desc.y - r8), row0 = desc.z + r8;
  if (n == 0 || nrows <= 0) return;
  const float vs = __int_as_float(where.y);
  const int G = a.Hq / a.Hkv;
  // piece k's slot
  auto slot = [&](int k) {
    return p.slots + ((size_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * Cfg<D>::kUnitRows + r8) * (D + 2);
  };
  const int i = tid / D, k = tid % D;
  // the first pieces' sums are on their way while their factors are made
  constexpr int N = 20;
  float first[N];
#pragma unroll
  for (int x = 0; x < N; ++x) first[x] = x < n && i < nrows ? __ldcg(slot(x) + i * (D + 2) + k) : 0.f;
  if (warp < nrows) {
    float m = -FLT_MAX, mk = -FLT_MAX, lk = 0.f;
    if (lane < n) {
      mk = __ldcg(slot(lane) + warp * (D + 2) + D);
      lk = __ldcg(slot(lane) + warp * (D + 2) + D + 1);
    }
    m = mk;
    for (int x = lane + 32; x < n; x += 32) m = fmaxf(m, __ldcg(slot(x) + warp * (D + 2) + D));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(dev::kFull, m, x));
    const float e = exp2f(mk - m);
    s_e[warp][lane] = e;
    float l = e * lk;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(dev::kFull, l, x);
    if (lane == 0) {
      s_top[warp] = m;
      s_l[warp] = l;
    }
  }
  __syncthreads();
  float y = 0.f;
  if (i < nrows) {
#pragma unroll
    for (int x = 0; x < N; ++x) y = x < n ? fmaf(s_e[i][x], first[x], y) : y;
    for (int x = N; x < min(n, 32); ++x) y = fmaf(s_e[i][x], __ldcg(slot(x) + i * (D + 2) + k), y);
  }
  for (int k0 = 32; k0 < n; k0 += 32) {  // only a grid of more SMs, or a unit of its own, has that many
    __syncthreads();
    if (warp < nrows) {
      float e = 0.f, l = 0.f;
      if (k0 + lane < n) {
        const float *s = slot(k0 + lane) + warp * (D + 2);
        e = exp2f(__ldcg(s + D) - s_top[warp]);
        l = e * __ldcg(s + D + 1);
      }
      s_e[warp][lane] = e;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(dev::kFull, l, x);
      if (lane == 0) s_l[warp] += l;
    }
    __syncthreads();
    if (i < nrows) {
      const int end = min(32, n - k0);
#pragma unroll 8
      for (int x = 0; x < end; ++x) y = fmaf(s_e[i][x], __ldcg(slot(k0 + x) + i * (D + 2) + k), y);
    }
  }
  s_y[i][k] = y;
  __syncthreads();
  if (warp < nrows) {
    float v[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = s_y[warp][place<D>(lane * (D / 32) + e)];
    const int qi = (row0 + warp) / G;
    store_out<D>(a, (int64_t)where.x + qi, desc.w * G + (row0 + warp) - qi * G, lane, v, s_top[warp], s_l[warp],
                 1.0f / (a.vq.sqrt_d * vs));
  }
}

template <int D, int RG, bool MULTI, bool UNIT, bool HL>
cudaError_t run_rows(const RowsParams &p, cudaStream_t s) {
  // dynamic shared memory starts behind the 1 KiB that the system keeps
  const int dyn = (int)smem_end<D>() - 1024;
  auto kern = paged_rows_kernel<D, RG, MULTI, UNIT, HL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  const int ctas = decode_ctas();
  kern<<<ctas, Cfg<D>::kThreads, dyn, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  constexpr int RT = D == 256 || RG == 4 ? 4 : 8;  // rows of a block
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)(p.groups * RG / RT));
  cfg.blockDim = dim3(D * RT);
  cfg.stream = s;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, RT>, p);
}

template <int D>
cudaError_t run_d(const RowsParams &p, int rg, cudaStream_t s) {
  const CacheView &k = p.a.k, &v = p.a.v;
  const bool unit = k.sn == 1 && v.sn == 1 && k.sb == v.sb && k.sh == v.sh;
  auto run = [&](auto rg_, auto multi, auto hl) {
    constexpr int RG = decltype(rg_)::value;
    constexpr bool M = decltype(multi)::value, HL = decltype(hl)::value;
    return unit ? run_rows<D, RG, M, true, HL>(p, s) : run_rows<D, RG, M, false, HL>(p, s);
  };
  using R4 = std::integral_constant<int, 4>;
  using R8 = std::integral_constant<int, 8>;
  using R16 = std::integral_constant<int, 16>;
  const std::true_type yes{};
  const std::false_type no{};
  if (rg == 4) return run(R4{}, no, yes);
  const bool hl = p.a.dtype != TQ_BF16, one = p.groups == 1;
  if (rg == 8 && one) return hl ? run(R8{}, no, yes) : run(R8{}, no, no);
  if constexpr (D == 256) {
    return hl ? run(R8{}, yes, yes) : run(R8{}, yes, no);
  } else {
    if (one) return hl ? run(R16{}, no, yes) : run(R16{}, no, no);
    return hl ? run(R16{}, yes, yes) : run(R16{}, yes, no);
  }
}

}  // namespace

size_t paged_rows_workspace(int d) {
  const size_t ctas = decode_ctas();
  const int rows = d == 256 ? Cfg<256>::kUnitRows : Cfg<128>::kUnitRows;
  return 2 * ctas * (sizeof(int4) + (size_t)rows * (d + 2) * sizeof(float));
}

cudaError_t launch_paged_rows(const PagedAttentionArgs &a, cudaStream_t s) {
  RowsParams p{};
  p.a = a;
  const cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  p.desc = static_cast<int4 *>(a.ws);
  p.slots = reinterpret_cast<float *>(p.desc + 2 * decode_ctas());
  // rows of a request and KV head that go through its tokens together; more of them are further units
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv);
  const int rg = rows <= 4 ? 4 : rows <= 8 || a.kq.d == 256 ? 8 : 16;
  const int unit_rows = a.kq.d == 256 ? Cfg<256>::kUnitRows : Cfg<128>::kUnitRows;
  p.groups = (int)((rows < unit_rows ? rows + rg - 1 : unit_rows) / rg);
  return a.kq.d == 64 ? run_d<64>(p, rg, s) : a.kq.d == 128 ? run_d<128>(p, rg, s) : run_d<256>(p, rg, s);
}

}  // namespace tq
