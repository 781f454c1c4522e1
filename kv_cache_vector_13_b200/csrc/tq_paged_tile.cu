// Attention of many query rows a request over a paged 4-bit cache (sm_100a):
// prefill, and decode with more rows a KV head than the small tiles take.
//
// A unit is (request, KV head, tile of query rows), a block 128 cached tokens.
// All units' blocks, and a fixed cost of each unit, form one line cut evenly
// over one persistent CTA an SM;
// units cut by a range's end leave partial sums that a last kernel merges in
// the order of the tokens.
//
// Per block, on the fifth-generation tensor cores: S = Q K^T and O += P V with
// fp16 operands and fp32 sums in tensor memory.  Roles of a CTA's 16 warps:
//   * 4 warps decode K and 4 V: a token's 64 code bytes become 128 fp16
//     centroids in the operand tile, a code byte (two codes) being one read of
//     a table of centroid pairs, one copy per lane, whose address is one byte
//     permute.  Both tiles have the same layout, a token's 8 coordinates a
//     16-byte row: K-major for the scores, and for the values, whose sum runs
//     over tokens, the transposed operand form.  No V transpose is ever made.
//   * 2 x 4 warps softmax, a query row a thread: scores from tensor memory
//     times ||k||, the running reference and sum, weights times ||v|| back
//     into tensor memory as the next product's operand.  One thread of each
//     set issues the set's products: the values' of a block, then the scores
//     of its next one, which take the weights' place behind them.
// Two sets of rows (or of blocks) alternate, so that one's products run while
// the other's softmax does:
//   wide:  256 rows a tile, both halves against every block (bf16 outputs;
//          operands rounded once, 2^-11 against the output's 2^-8);
//   split: 128 rows a tile, even blocks to one set, odd ones to the other,
//          which are merged at the end (few rows a unit); with HL the rows and
//          weights are fp16 pairs hi + lo, two products each (fp16 outputs).
//
// Bound by the chain from a block's scores through the softmax and the weights
// to its values' product, two sets deep: a softmax takes 2.4 to 3.5 thousand
// cycles, the products about 2 thousand.  Measured on a B200, bf16, 32 / 8
// heads, d = 128: 3 requests of 2048 rows on up to 16384 tokens, causal (920
// GFLOP), 1386 us, 664 TFLOP/s; 2048 rows on 8192 tokens, codes drawn evenly, 439 us.

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"
#include "tq_paged_dev.cuh"
#include "tq_umma.cuh"

#include <float.h>
#include <type_traits>

namespace tq {
namespace {

using namespace paged;

constexpr int kBlk = 128;                 // tokens per block
// What a unit costs in the line besides its blocks, in blocks (its rows' way to the operand tiles, the first block's way
// through the pipeline, the outputs), so that ranges of many short units do not end late: 8 requests of 512 rows and up to
// 4001 tokens 232 us, without it 547; 3 of 2048 rows and up to 16384 tokens 1376, without it 1496.  9 is slower again.
constexpr int kUnitCost = 5;
constexpr int kThreads = 512;             // 2 x 4 softmax warps, 4 warps decode K and 4 V
constexpr uint32_t kTabAddr = 0x10000u;   // the pair tables: 64 KiB at this shared address
constexpr uint32_t kHighAddr = 0x20000u;  // V, K and the second query tile

template <int D>
struct Tile {
  static constexpr int kGroup = (D / 8) * 128;         // bytes of 8 rows: D / 8 core matrices
  static constexpr int kBytes = (kBlk / 8) * kGroup;   // an operand tile of 128 rows
};

struct TileParams {
  PagedAttentionArgs a;
  int rt;                  // rows per tile: 256 wide, 128 split
  uint32_t page_mul;       // token / page_size = (token * page_mul) >> page_shift, below 2^31 tokens
  int page_shift;
  const __half *qhi, *qlo; // [T * Hq][D] turned rows
  const float *qf;         // [T * Hq] the factor their scores still need (softmax scale, log2 e, row scale)
  int64_t max_tiles;       // that `line` has room for
  int32_t *first;          // [R + 1] first tile of each request
  int64_t *line;           // [tiles + 1] places (of one KV head) before each tile: kUnitCost and its blocks
  float *slots;            // [2 * ctas][rt][D + 4]: a row's sums, then M and L
  int4 *desc;              // [ctas]
  float *v_unit;           // what the values' table is to be divided by
  unsigned *faults;
};

struct Req {
  int q0, n, kv;
};

__device__ __forceinline__ Req load_req(const PagedAttentionArgs &a, int r, unsigned *faults) {
  Req q;
  q.q0 = max(a.cu_q ? __ldg(a.cu_q + r) : r, 0);
  const int q1 = a.cu_q ? __ldg(a.cu_q + r + 1) : r + 1;
  q.n = max(min(q1, (int)a.T) - q.q0, 0);
  q.kv = max(__ldg(a.kv_lens + r), 0);
  const int cap = a.max_pages * a.page_size;
  if (q.kv > cap) {
    atomicOr(faults, kFaultIndex);
    q.kv = cap;
  }
  return q;
}

// Blocks [b0, b1) that any row of tile i of a request sees; one (empty) block
// for rows that see nothing, which writes their zeros.
__device__ __forceinline__ void tile_blocks(const PagedAttentionArgs &a, const Req &q, int rt, int i, int &b0, int &b1,
                                            int &first) {
  const int G = a.Hq / a.Hkv;
  const int p0 = q.kv - q.n + i * rt / G, p1 = q.kv - q.n + (min((i + 1) * rt, q.n * G) - 1) / G;
  const int hi = a.causal ? max(p1 + 1, 0) : q.kv;
  first = window_start(p0, a.window);
  b0 = first / kBlk;
  b1 = max(runs(hi, kBlk), b0 + 1);
}

// ------------------------------------------------- query rows and schedule

template <int N>
__device__ __forceinline__ int64_t scan(int64_t v, int64_t *s_warp, int64_t *total) {  // exclusive, N threads
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(dev::kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[w] = x;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < N / 32; ++i) {
    if (i < w) base += s_warp[i];
    all += s_warp[i];
  }
  __syncthreads();
  *total = all;
  return base + x - v;
}

// Block 0 lays out the line; the others turn the query rows: sign flips, FWHT
// (16 coordinates a lane), a power of two that brings the largest into [1, 2).
template <int D, bool HL>
__global__ void __launch_bounds__(256) paged_tile_prep_kernel(const __grid_constant__ TileParams p) {
  const PagedAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (blockIdx.x == 0) {
    __shared__ int64_t s_warp[8];
    const int G = a.Hq / a.Hkv;
    int64_t tiles = 0;
    for (int r0 = 0; r0 < a.R; r0 += 256) {
      const int r = r0 + tid;
      int64_t mine = 0, all;
      if (r < a.R) {
        const Req q = load_req(a, r, p.faults);
        mine = ((int64_t)q.n * G + p.rt - 1) / p.rt;
      }
      const int64_t before = tiles + scan<256>(mine, s_warp, &all);
      if (r < a.R) p.first[r] = (int32_t)before;
      tiles += all;
    }
    if (tiles > p.max_tiles) {  // rows named twice by cu_q: more tiles than T rows have, and none is worked on
      if (tid == 0) atomicOr(p.faults, kFaultIndex);
      __syncthreads();
      for (int r = tid; r < a.R; r += 256) p.first[r] = 0;
      tiles = 0;
    }
    if (tid == 0) p.first[a.R] = (int32_t)tiles;
    __syncthreads();  // the block reads what it wrote
    int64_t blocks = 0;
    for (int64_t t0 = 0; t0 < tiles; t0 += 256) {
      const int64_t t = t0 + tid;
      int64_t mine = 0, all;
      if (t < tiles) {
        int i = 0, j = a.R;  // the last request i with first[i] <= t
        while (j - i > 1) {
          const int m = (i + j) >> 1;
          if (p.first[m] <= t) i = m; else j = m;
        }
        int b0, b1, first;
        tile_blocks(a, load_req(a, i, p.faults), p.rt, (int)t - p.first[i], b0, b1, first);
        mine = b1 - b0 + kUnitCost;
      }
      const int64_t before = blocks + scan<256>(mine, s_warp, &all);
      if (t < tiles) p.line[t] = before;
      blocks += all;
    }
    if (tid == 0) p.line[tiles] = blocks;
    return;
  }
  constexpr int E = 16, T = D / E, RPW = 32 / T;
  const int t = lane % T;
  const int64_t rows = a.T * a.Hq;
  const float scale = a.scale * 1.4426950408889634f / a.kq.sqrt_d;
  uint32_t sg = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) sg |= (a.kq.signs[t * E + e] < 0 ? 1u : 0u) << e;
  for (int64_t r0 = ((int64_t)(blockIdx.x - 1) * 8 + warp) * RPW; r0 < rows; r0 += (int64_t)(gridDim.x - 1) * 8 * RPW) {
    int64_t row = r0 + lane / T;
    const bool active = row < rows;
    if (!active) row = r0;
    const int64_t tok = row / a.Hq;
    const int hq = (int)(row - tok * a.Hq);
    const uint16_t *src = static_cast<const uint16_t *>(a.q) + tok * a.q_st + hq * a.q_sh + t * E;
    float x[E];
    if (a.dtype == TQ_BF16) dev::load_block<TQ_BF16, E>(src, x);
    else dev::load_block<TQ_F16, E>(src, x);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __uint_as_float(__float_as_uint(x[e]) ^ ((sg >> e & 1u) << 31));
    dev::fwht<T, E>(x, t);
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
    for (int o = T / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(dev::kFull, m, o));
    const unsigned ex = m >> 23;
    const float f = ex == 255u || m == 0 ? 1.0f : __uint_as_float(min(max(254u - ex, 1u), 252u) << 23);
    uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float u = x[2 * e] * f, v = x[2 * e + 1] * f;
      const __half2 h = __floats2half2_rn(u, v);
      hi[e] = *reinterpret_cast<const uint32_t *>(&h);
      if (HL) {
        const float2 b = __half22float2(h);
        const __half2 l = __floats2half2_rn(u - b.x, v - b.y);
        lo[e] = *reinterpret_cast<const uint32_t *>(&l);
      }
    }
    if (active) {
      uint4 *o = reinterpret_cast<uint4 *>(const_cast<__half *>(p.qhi) + row * D + t * E);
      o[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      o[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      if (HL) {
        o = reinterpret_cast<uint4 *>(const_cast<__half *>(p.qlo) + row * D + t * E);
        o[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        o[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      }
      if (t == 0) const_cast<float *>(p.qf)[row] = scale / f;
    }
  }
}

// ------------------------------------------------------------ main kernel

struct Piece {
  int r, h, row0, nrows, q0, n, kv, first;
  int b0, b1;        // blocks
  int places;        // of the line
  int starts, ends;  // whether they hold the unit's first and last block
};

constexpr int kNormBufs = 8;

struct Low {
  // A tile's blocks alternate between two barriers: with split blocks a set waits for every other one only.
  uint64_t k_full[2], v_full[2], k_free, v_free, n_full[kNormBufs], s_full[2], o_fin[2];
  uint32_t tmem, pad;
  Piece piece;
  // of a block's tokens: ||k||, ||v||, value_log2 of it, and whether they have a record
  alignas(16) float kn[kNormBufs][kBlk], vn[kNormBufs][kBlk], lv[kNormBufs][kBlk];
  alignas(16) uint32_t valid[kNormBufs][kBlk / 32];
  float f[256];          // score factors of the rows
  float m[128], l[128];  // the odd set's references and sums (split)
  float scale[2];        // what the tables' values are to be divided by
  unsigned key[2];
  uint32_t sign[4];      // the value rotation's sign flips
};

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
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// D[tmem] (+)= A B for one K = 16 step, A in shared memory, and in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t at, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(at), "l"(bdesc), "r"(idesc), "r"(accum));
}

#define TQ_LIST16(v, b) "r"(v[b]), "r"(v[b + 1]), "r"(v[b + 2]), "r"(v[b + 3]), "r"(v[b + 4]), "r"(v[b + 5]), \
    "r"(v[b + 6]), "r"(v[b + 7]), "r"(v[b + 8]), "r"(v[b + 9]), "r"(v[b + 10]), "r"(v[b + 11]), "r"(v[b + 12]), \
    "r"(v[b + 13]), "r"(v[b + 14]), "r"(v[b + 15])
__device__ __forceinline__ void st16(uint32_t t, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
               "%13, %14, %15};" ::TQ_LIST16(v, 0), "r"(t) : "memory");
}
__device__ __forceinline__ void st32(uint32_t t, const uint32_t (&v)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
               "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
                   TQ_LIST16(v, 0), TQ_LIST16(v, 16), "r"(t) : "memory");
}
// 16 columns on their way; their values are there behind wait16.
__device__ __forceinline__ void ld16(uint32_t t, uint32_t (&v)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15}, [%16];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
               : "r"(t));
}
__device__ __forceinline__ void wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :: "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

template <int D, bool SPLIT, bool HL>
__global__ void __launch_bounds__(kThreads, 1) paged_tile_kernel(const __grid_constant__ TileParams p) {
  static_assert(SPLIT || !HL, "pairs of operands only with split blocks");
  constexpr int RT = SPLIT ? 128 : 256;
  constexpr int GB = Tile<D>::kGroup, TB = Tile<D>::kBytes;
  constexpr uint32_t kV = kHighAddr, kK = kHighAddr + TB, kQ1 = kHighAddr + 2 * TB, kQ0 = kTabAddr - TB;
  constexpr uint32_t kIdS = umma::idesc_f16(128, kBlk), kIdO = umma::idesc_f16(128, D) | (1u << 16);
  constexpr int NC = D / 32;  // 32-column runs of O
  extern __shared__ __align__(16) unsigned char s_raw[];
  Low &sm = *reinterpret_cast<Low *>(s_raw);
  const PagedAttentionArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  const int G = a.Hq / a.Hkv;
  const uint32_t dyn = (uint32_t)__cvta_generic_to_shared(s_raw);
  uint32_t dyn_bytes;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn_bytes));
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (dyn + sizeof(Low) > kQ0 || dyn + dyn_bytes < kQ1 + TB) {
    if (tid == 0) {
      atomicOr(p.faults, kFaultSmemLayout);
      p.desc[c] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  auto bar = [&](const uint64_t &b) { return (uint32_t)__cvta_generic_to_shared(&b); };

  // ---- the tables (see the rows kernel), barriers, tensor memory
  uint32_t *pairs = reinterpret_cast<uint32_t *>(s_raw + (kHighAddr - dyn));
  if (tid < 2) sm.key[tid] = 0xffffffffu;
  __syncthreads();
  find_scales(a.kq.centroids, a.vq.centroids, tid, kThreads, sm.key);
  __syncthreads();
  if (warp < 2) {
    const float *cent = warp == 0 ? a.kq.centroids : a.vq.centroids;
    float unit;
    const float s = scale_of(sm.key[warp], kThreads, cent, unit);
    if (lane == 0) {
      sm.scale[warp] = unit;
      if (warp == 1 && c == 0) *p.v_unit = unit;  // for the merge
    }
    for (int e = lane; e < 256; e += 32) {
      const __half2 h = __floats2half2_rn(s * __ldg(cent + (e & 15)), s * __ldg(cent + (e >> 4)));
      pairs[warp * 256 + e] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  if (warp == 2) {
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const unsigned m = __ballot_sync(dev::kFull, a.vq.signs[32 * w + lane] < 0);
      if (lane == 0) sm.sign[w] = m;
    }
  }
  if (warp == 15) umma::alloc(&sm.tmem, 512);
  if (tid == 0) {
    umma::mbar_init(bar(sm.k_free), 2);
    umma::mbar_init(bar(sm.v_free), 2);
    for (int x = 0; x < kNormBufs; ++x) umma::mbar_init(bar(sm.n_full[x]), 256);
    for (int x = 0; x < 2; ++x) {
      umma::mbar_init(bar(sm.k_full[x]), 128);
      umma::mbar_init(bar(sm.v_full[x]), 128);
      umma::mbar_init(bar(sm.s_full[x]), 1);
      umma::mbar_init(bar(sm.o_fin[x]), 1);
    }
  }
  __syncthreads();
  {
    uint4 *tab = reinterpret_cast<uint4 *>(s_raw + (kTabAddr - dyn));
    for (int i = tid; i < 256 * 16; i += kThreads) {
      const uint32_t w = pairs[((i >> 3) & 1) * 256 + (i >> 4)];
      tab[i] = make_uint4(w, w, w, w);
    }
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = sm.tmem;
  // columns: scores (and weights) of set 0 and 1, outputs of set 0 and 1
  auto s_col = [&](int x) { return tmem + 128 * x; };
  auto o_col = [&](int x) { return tmem + 256 + 128 * x; };

  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the line and the turned rows
  const int tiles = __ldcg(p.first + a.R);
  const int64_t total = tiles > 0 ? __ldcg(p.line + tiles) * a.Hkv : 0;
  const int ctas = (int)min((int64_t)gridDim.x, total);
  int64_t at = c < ctas ? total * c / ctas : 0;
  const int64_t end = c < ctas ? total * (c + 1) / ctas : 0;
  int4 desc = make_int4(0, 0, 0, 0);

  // blocks and items (a block for a set) that were done before, for the barriers' phases
  uint32_t blocks_done = 0, items_done[2] = {0, 0}, pieces_done[2] = {0, 0};
  bool dead = false;
  auto wait = [&](const uint64_t &b, uint32_t phase) {
    if (!dead) dead = !umma::mbar_wait_bounded(bar(b), phase & 1, p.faults, kFaultTimeout);
  };

  int r = -1, h = 0, tile = 0, ta = 0, tb = 0;  // the unit (thread 0)
  Req req{};
  Piece q;
  int nblk = 0;
  bool both = false;  // whether both sets have work
  // The next piece of the range, its query rows in the operand tiles: all threads together.
  auto next_piece = [&]() -> bool {
    if (nblk > 0) {
      blocks_done += nblk;
      items_done[0] += SPLIT && both ? (nblk + 1) / 2 : nblk;
      items_done[1] += !both ? 0 : SPLIT ? nblk / 2 : nblk;
      ++pieces_done[0];
      pieces_done[1] += both;
      at += q.places;
      umma::fence_before();
      __syncthreads();
      umma::fence_after();
    }
    if (at >= end) return false;
    // ---- the piece: one thread finds the first and walks on from unit to unit
    if (tid == 0) {
      int skip = 0;  // places of the unit in front of the range
      if (r < 0) {
        int i = 0, j = a.R;  // the last request whose line starts at or before `at`
        while (j - i > 1) {
          const int m = (i + j) >> 1;
          if (__ldcg(p.line + __ldcg(p.first + m)) * a.Hkv <= at) i = m; else j = m;
        }
        r = i;
        ta = __ldcg(p.first + r);
        tb = __ldcg(p.first + r + 1);
        const int64_t la = __ldcg(p.line + ta), per = __ldcg(p.line + tb) - la, x = at - la * a.Hkv;
        h = (int)(x / per);
        const int64_t y = la + (x - (int64_t)h * per);
        i = ta, j = tb;  // the last tile that starts at or before y
        while (j - i > 1) {
          const int m = (i + j) >> 1;
          if (__ldcg(p.line + m) <= y) i = m; else j = m;
        }
        tile = i;
        skip = (int)(y - __ldcg(p.line + i));
        req = load_req(a, r, p.faults);
      } else if (++tile == tb) {
        tile = ta;
        if (++h == a.Hkv) {
          h = 0;
          do {
            ++r;
            ta = tb;
            tb = __ldcg(p.first + r + 1);
          } while (tb == ta && r + 1 < a.R);
          tile = ta;
          req = load_req(a, r, p.faults);
        }
      }
      Piece q;
      int b0, b1;
      tile_blocks(a, req, RT, tile - ta, b0, b1, q.first);
      q.r = r;
      q.h = h;
      q.q0 = req.q0;
      q.n = req.n;
      q.kv = req.kv;
      q.row0 = (tile - ta) * RT;
      q.nrows = min(RT, req.n * G - q.row0);
      const int len = b1 - b0 + kUnitCost, to = (int)min((int64_t)len, skip + (end - at));
      q.places = to - skip;
      q.b0 = b0 + max(skip - kUnitCost, 0);
      q.b1 = max(b0 + to - kUnitCost, q.b0);  // none where the range ends before the unit's first block
      q.starts = skip <= kUnitCost;
      q.ends = to == len;
      sm.piece = q;
      if (q.starts && !q.ends && q.b1 > q.b0) {
        const int64_t last = at + (len - skip) - 1;
        int64_t e = last * ctas / total;
        while (e < ctas - 1 && total * (e + 1) / ctas <= last) ++e;
        while (e > c && total * e / ctas > last) --e;
        desc = make_int4((int)e - c + 1, r, tile - ta, h);
      }
    }
    __syncthreads();
    q = sm.piece;
    nblk = q.b1 - q.b0;
    if (nblk == 0) return false;
    both = SPLIT ? nblk > 1 : q.nrows > 128;
    // ---- query rows into the operand tiles: 16-byte words of 8 coordinates
    constexpr int QB = RT * (D / 8) / kThreads;  // a thread's words, their loads in flight together
    uint4 qx[QB], qy[HL ? QB : 1];
#pragma unroll
    for (int n = 0; n < QB; ++n) {
      const int i = n * kThreads + tid, row = i / D * 8 + (i & 7), w = (i >> 3) % (D / 8);
      qx[n] = make_uint4(0, 0, 0, 0);
      if (HL) qy[HL ? n : 0] = qx[n];
      if (row < q.nrows) {
        const int qi = (q.row0 + row) / G;
        const int64_t src = (int64_t)(q.q0 + qi) * a.Hq + q.h * G + (q.row0 + row - qi * G);
        qx[n] = __ldcg(reinterpret_cast<const uint4 *>(p.qhi + src * D) + w);
        if (HL) qy[HL ? n : 0] = __ldcg(reinterpret_cast<const uint4 *>(p.qlo + src * D) + w);
      }
    }
    if (tid < RT) {
      float f = 0.f;
      if (tid < q.nrows) {
        const int qi = (q.row0 + tid) / G;
        f = __ldcg(p.qf + (int64_t)(q.q0 + qi) * a.Hq + q.h * G + (q.row0 + tid - qi * G));
      }
      sm.f[tid] = f / sm.scale[0];
    }
#pragma unroll
    for (int n = 0; n < QB; ++n) {
      const int i = n * kThreads + tid, row = i / D * 8 + (i & 7), w = (i >> 3) % (D / 8);
      const uint32_t o = ((row & 127) >> 3) * GB + w * 128 + (row & 7) * 16;
      sts128((row < 128 ? kQ0 : kQ1) + o, qx[n].x, qx[n].y, qx[n].z, qx[n].w);
      if (HL) sts128(kQ1 + o, qy[HL ? n : 0].x, qy[HL ? n : 0].y, qy[HL ? n : 0].z, qy[HL ? n : 0].w);
    }
    umma::fence_async_smem();
    __syncthreads();

    return true;
  };

  if (warp >= 8) {
    // ================= codes to operands: K by warps 8..11, V by 12..15, 32 tokens of a block a warp, a 16-byte
    // word of each a lane
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const bool is_k = warp < 12;
    constexpr int TPI = D == 128 ? 8 : 16;  // tokens per pass
    constexpr int IT = 32 / TPI;
    const int wq = warp & 3, tk = lane % TPI, ch = lane / TPI;
    uint32_t tab;
    asm("mov.b32 %0, %1;" : "=r"(tab) : "r"(kTabAddr + 4 * lane + (is_k ? 0 : 128)));
    const uint32_t tile_at = is_k ? kK : kV;
    const CacheView cv = is_k ? a.k : a.v;
    while (next_piece()) {
      const int32_t *row = a.table + (int64_t)q.r * a.table_stride;
      // page of token 32 wq + lane of block b (none is needed: -1), and its record
      auto token = [&](int b) { return b * kBlk + 32 * wq + lane; };
      auto page = [&](int j) { return (int)(((uint64_t)(uint32_t)j * p.page_mul) >> p.page_shift); };
      auto wanted = [&](int b) { return b < q.b1 && token(b) >= q.first && token(b) < q.kv; };
      auto page_id = [&](int b) { return wanted(b) ? __ldg(row + page(token(b))) : -1; };
      auto record = [&](int b, int id) -> int64_t {
        if (!wanted(b)) return -1;
        if ((unsigned)id >= (unsigned)a.n_pages) {
          atomicOr(p.faults, kFaultIndex);
          return -1;
        }
        const int j = token(b), off = j - page(j) * a.page_size;
        return id * cv.sb + q.h * cv.sh + off * cv.sn;
      };
      uint4 x[IT];
      // 16 code bytes of the lane's token of each pass; the record comes from the lane that has it
      auto load = [&](int64_t rec) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int64_t r1 = __shfl_sync(dev::kFull, rec, TPI * i + tk);
          x[i] = r1 >= 0 ? __ldg(reinterpret_cast<const uint4 *>(cv.codes + r1 * (D / 2)) + ch) : make_uint4(0, 0, 0, 0);
        }
      };
      auto load_norm = [&](int64_t rec) { return rec >= 0 ? __ldg(cv.norms + rec) : 0.f; };
      // Block u's norms of token 32 wq + lane.  They go out a block ahead of the codes; the buffer was block
      // u - 8's, whose weights are long in a product that this thread has seen done.
      auto publish = [&](uint32_t u, float norm, bool have) {
        const int nb = u % kNormBufs;
        if (is_k) {
          sm.kn[nb][32 * wq + lane] = norm;
          const unsigned ok = __ballot_sync(dev::kFull, have);
          if (lane == 0) sm.valid[nb][wq] = ok;
        } else {
          sm.vn[nb][32 * wq + lane] = norm;
          sm.lv[nb][32 * wq + lane] = value_log2(norm);
        }
        arrive(bar(sm.n_full[nb]));
      };
      // Page numbers are read three blocks ahead, norms two, codes one.  A block's loads leave together at its end and
      // are used from the next one's start on: a load in between would be waited for with them.
      int id1 = page_id(q.b0 + 1), id2 = page_id(q.b0 + 2);
      const int64_t rec0 = record(q.b0, page_id(q.b0));
      load(rec0);
      publish(blocks_done, load_norm(rec0), rec0 >= 0);
      int64_t rec = record(q.b0 + 1, id1);
      float norm = load_norm(rec);
      for (int b = 0; b < nblk; ++b) {
        const uint32_t u = blocks_done + b;
        if (b + 1 < nblk) publish(u + 1, norm, rec >= 0);
        const int64_t rec2 = record(q.b0 + b + 2, id2);
        if (u > 0) wait(is_k ? sm.k_free : sm.v_free, u - 1);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int t = 32 * wq + TPI * i + tk;
          const uint32_t to = tile_at + (t >> 3) * GB + ch * 4 * 128 + (t & 7) * 16;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t v[4][4];  // all reads first: a write in between would hold the next ones back
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j][0] = pair<0>(w[j], tab);
            v[j][1] = pair<1>(w[j], tab);
            v[j][2] = pair<2>(w[j], tab);
            v[j][3] = pair<3>(w[j], tab);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) sts128(to + 128 * j, v[j][0], v[j][1], v[j][2], v[j][3]);
        }
        umma::fence_async_smem();
        arrive(bar(is_k ? sm.k_full[u & 1] : sm.v_full[u & 1]));
        load(rec);
        norm = load_norm(rec2);
        id2 = page_id(q.b0 + b + 3);
        rec = rec2;
      }
    }
  } else {
    // ================= softmax: set x, a row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    while (next_piece()) {
      const int x = warp >> 2, row = (warp & 3) * 32 + lane;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const int i = SPLIT ? row : 128 * x + row;  // row of the tile
      const bool live = i < q.nrows;
      int see_lo = 0, see_hi = INT_MAX;  // a lane without a row sees everything (and goes nowhere)
      if (live) {
        const int pos = q.kv - q.n + (q.row0 + i) / G;
        see_hi = a.causal ? max(pos + 1, 0) : q.kv;
        see_lo = window_start(pos, a.window);
      }
      const float f = sm.f[i];
      float M = -FLT_MAX, l = 0.f;
      // One thread issues the set's products.  The barriers that free a block's tiles take two arrivals: one a set,
      // or two of the only one that has the block.
      const bool issuer = (warp & 3) == 0 && lane == 0;
      auto free_tile = [&](const uint64_t &b) {
        umma::commit(bar(b));
        if (SPLIT || !both) umma::commit(bar(b));
      };
      auto block = [&](int k) { return SPLIT && both ? 2 * k + x : k; };  // of the set's item k
      auto scores = [&](int b) {
        const uint32_t u = blocks_done + b;
        wait(sm.k_full[u & 1], u >> 1);
        umma::fence_after();
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint64_t kd = umma::desc(kK + s * 256, 128, GB);
          if (HL) {
            mma_ss(s_col(x), umma::desc(kQ0 + s * 256, 128, GB), kd, kIdS, s > 0);
            mma_ss(s_col(x), umma::desc(kQ1 + s * 256, 128, GB), kd, kIdS, 1);
          } else {
            mma_ss(s_col(x), umma::desc((SPLIT || x == 0 ? kQ0 : kQ1) + s * 256, 128, GB), kd, kIdS, s > 0);
          }
        }
        umma::commit(bar(sm.s_full[x]));
        free_tile(sm.k_free);
      };
      auto values = [&](int b, bool first, bool last) {
        const uint32_t u = blocks_done + b;
        wait(sm.v_full[u & 1], u >> 1);
        umma::fence_after();
#pragma unroll
        for (int s = 0; s < kBlk / 16; ++s) {
          const uint64_t vd = umma::desc(kV + s * 2 * GB, GB, 128);
          const uint32_t pc = s_col(x) + 32 * (s >> 1) + 8 * (s & 1);
          mma_ts(o_col(x), pc, vd, kIdO, !first || s > 0);
          if (HL) mma_ts(o_col(x), pc + 16, vd, kIdO, 1);
        }
        free_tile(sm.v_free);
        if (last) umma::commit(bar(sm.o_fin[x]));
      };
      const int mine = x < (both ? 2 : 1) ? (SPLIT ? (both ? (nblk + 1 - x) / 2 : nblk) : nblk) : 0;
      if (mine > 0 && issuer) scores(block(0));
      __syncwarp();
      for (int k = 0; k < mine; ++k) {
        const int b = block(k);
        const uint32_t u = blocks_done + b;
        const int nb = u % kNormBufs, j0 = (q.b0 + b) * kBlk;
        wait(sm.n_full[nb], u / kNormBufs);
        wait(sm.s_full[x], items_done[x] + k);
        umma::fence_after();
        const uint4 vm = *reinterpret_cast<const uint4 *>(sm.valid[nb]);
        const uint32_t valid[4] = {vm.x, vm.y, vm.z, vm.w};
        const bool whole = see_lo <= j0 && (unsigned)see_hi >= (unsigned)j0 + kBlk && (vm.x & vm.y & vm.z & vm.w) == ~0u;
        const float *kns = sm.kn[nb], *vns = sm.vn[nb], *lvs = sm.lv[nb];
        auto mask = [&](int r) {  // tokens of run r (32 columns) that the row sees
          const int lo = max(see_lo - j0 - 32 * r, 0), hi = min(see_hi - j0 - 32 * r, 32);
          const uint32_t m = hi <= 0 || lo >= 32 ? 0u : (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
          return m & valid[r];
        };
        // fn(c, columns 16 c .. 16 c + 15) over the row's scores, the next 16 on their way meanwhile
        auto runs = [&](auto &&fn) {
          uint32_t s[2][16];
          ld16(s_col(x) + lanes, s[0]);
#pragma unroll
          for (int c8 = 0; c8 < 8; ++c8) {
            wait16(s[c8 & 1]);
            if (c8 < 7) ld16(s_col(x) + lanes + 16 * (c8 + 1), s[(c8 + 1) & 1]);
            fn(c8, s[c8 & 1]);
          }
        };
        // the largest logit + log2 ||v|| of the row
        auto top = [&](auto edge) {
          constexpr bool EDGE = decltype(edge)::value;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          runs([&](int c8, const uint32_t (&s)[16]) {
            const uint32_t m = EDGE ? mask(c8 >> 1) >> (16 * (c8 & 1)) : ~0u;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 kn = *reinterpret_cast<const float4 *>(kns + 16 * c8 + e);
              const float4 lv = *reinterpret_cast<const float4 *>(lvs + 16 * c8 + e);
              float k0, k1, k2, k3, t[4];
              dev::mul_x2(k0, k1, kn.x, kn.y, f, f);
              dev::mul_x2(k2, k3, kn.z, kn.w, f, f);
              dev::fma_x2(t[0], t[1], __uint_as_float(s[e]), __uint_as_float(s[e + 1]), k0, k1, lv.x, lv.y);
              dev::fma_x2(t[2], t[3], __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]), k2, k3, lv.z, lv.w);
#pragma unroll
              for (int o = 0; o < 4; ++o)
                if (!EDGE || (m >> (e + o) & 1)) mx[o] = fmaxf(mx[o], t[o]);
            }
          });
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        // Weights relative to M of 16 columns: their sums, and times ||v|| as operand words (hi, and with HL lo).
        auto weights = [&](auto edge, int c8, const uint32_t (&s)[16], float (&sum)[2], uint32_t *w, uint32_t *wl) {
          constexpr bool EDGE = decltype(edge)::value;
          const uint32_t m = EDGE ? mask(c8 >> 1) >> (16 * (c8 & 1)) : ~0u;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 kn = *reinterpret_cast<const float4 *>(kns + 16 * c8 + e);
            const float4 vn = *reinterpret_cast<const float4 *>(vns + 16 * c8 + e);
            float k0, k1, k2, k3, t[4];
            dev::mul_x2(k0, k1, kn.x, kn.y, f, f);
            dev::mul_x2(k2, k3, kn.z, kn.w, f, f);
            dev::fma_x2(t[0], t[1], __uint_as_float(s[e]), __uint_as_float(s[e + 1]), k0, k1, -M, -M);
            dev::fma_x2(t[2], t[3], __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]), k2, k3, -M, -M);
#pragma unroll
            for (int o = 0; o < 4; ++o) {
              t[o] = exp2_approx(t[o]);
              if (EDGE) t[o] = m >> (e + o) & 1 ? t[o] : 0.f;
            }
            dev::add_x2(sum[0], sum[1], sum[0], sum[1], t[0], t[1]);
            dev::add_x2(sum[0], sum[1], sum[0], sum[1], t[2], t[3]);
            dev::mul_x2(t[0], t[1], t[0], t[1], vn.x, vn.y);
            dev::mul_x2(t[2], t[3], t[2], t[3], vn.z, vn.w);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              if (EDGE) {  // a masked token's norm may be anything
                t[2 * o] = m >> (e + 2 * o) & 1 ? t[2 * o] : 0.f;
                t[2 * o + 1] = m >> (e + 2 * o + 1) & 1 ? t[2 * o + 1] : 0.f;
              }
              const __half2 h = __floats2half2_rn(t[2 * o], t[2 * o + 1]);
              w[e / 2 + o] = *reinterpret_cast<const uint32_t *>(&h);
              if (HL) {
                const float2 back = __half22float2(h);
                const __half2 lo = __floats2half2_rn(t[2 * o] - back.x, t[2 * o + 1] - back.y);
                wl[e / 2 + o] = *reinterpret_cast<const uint32_t *>(&lo);
              }
            }
          }
        };
        // moves the reference M to that room below the block's largest value if that is above it
        auto move = [&](float mx) {
          const float m2 = fmaxf(M, mx - (HL ? kRoom : kRoomOnce)), r2 = exp2f(M - m2);
          M = m2;
          l *= r2;
          if (k > 0) {  // the scores' barrier says that the products before them are done, those into O too
#pragma unroll
            for (int r = 0; r < NC; ++r) {
              uint32_t o[32];
              umma::ld32(o_col(x) + lanes + 32 * r, o);
              umma::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r2);
              st32(o_col(x) + lanes + 32 * r, o);
            }
          }
        };
        // M moves only when a weight times its norm would pass 2^15 (fp16 ends at 2^16): with HL that is looked for before the
        // weights, which take the scores' place at once; else the weights are kept in registers, and where one
        // is too large they are made again
        auto item = [&](auto edge) {
          float sum[2] = {0.f, 0.f};
          if constexpr (HL) {
            const float mx = top(edge);
            if (__any_sync(dev::kFull, mx > M + kMost)) move(mx);
            uint32_t w[16], wl[16];
            runs([&](int c8, const uint32_t (&s)[16]) {
              weights(edge, c8, s, sum, w + 8 * (c8 & 1), wl + 8 * (c8 & 1));
              if (c8 & 1) {
                st16(s_col(x) + lanes + 16 * (c8 - 1), w);
                st16(s_col(x) + lanes + 16 * c8, wl);
              }
            });
          } else {
            uint32_t w[4][16];
            bool again = k == 0;
            for (;;) {
              if (again) move(top(edge));
              sum[0] = sum[1] = 0.f;
              __half2 most = __float2half2_rn(0.f);
              runs([&](int c8, const uint32_t (&s)[16]) {
                uint32_t *to = w[c8 >> 1] + 8 * (c8 & 1);
                weights(edge, c8, s, sum, to, nullptr);
#pragma unroll
                for (int e = 0; e < 8; ++e) most = __hmax2(most, *reinterpret_cast<const __half2 *>(to + e));
              });
              // A reference that has just moved bounds the weights by 2 (and rounding).  A weight beyond fp32 whose value has
              // no norm is inf * 0 here, which the maximum drops, so the sum is looked at too: behind a move it is at most
              // 128 * 2^65, a value without a norm counting as one of 2^-64.
              const __half2 wide = __half2half2(__float2half(1 << (int)kMost));
              if (again || !__any_sync(dev::kFull, !__hbgt2(wide, most) || sum[0] + sum[1] > 0x1p80f)) break;
              again = true;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) st16(s_col(x) + lanes + 32 * r, w[r]);
          }
          l += sum[0] + sum[1];
        };
        // a warp without a row leaves its weights as they are: nothing reads what comes of them
        if (__any_sync(dev::kFull, live)) {
          if (__all_sync(dev::kFull, whole || !live)) item(std::false_type{});
          else item(std::true_type{});
        }
        wait_st();
        umma::fence_before();
        // every row's weights are in place: the products with them, and the set's next scores behind those
        if (x == 0) asm volatile("bar.sync 2, 128;" ::: "memory");
        else asm volatile("bar.sync 3, 128;" ::: "memory");
        if (issuer) {
          umma::fence_after();
          values(b, k == 0, k + 1 == mine);
          if (k + 1 < mine) scores(block(k + 1));
        }
        __syncwarp();
      }

      // ---- the piece's rows
      if (mine > 0) wait(sm.o_fin[x], pieces_done[x]);
      umma::fence_after();
      float f0 = 1.f, f1 = 0.f;
      if (SPLIT && both) {  // the even set's threads merge the odd one's
        if (x == 1) {
          sm.m[row] = M;
          sm.l[row] = l;
        }
        umma::fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        umma::fence_after();
        if (x == 0) {
          const float m1 = sm.m[row], m = fmaxf(M, m1);
          f0 = exp2f(M - m);
          f1 = exp2f(m1 - m);
          l = f0 * l + f1 * sm.l[row];
          M = m;
        }
      }
      if (x == 0 || (!SPLIT && both)) {
        const bool done = q.starts && q.ends;
        float *slot = p.slots + (size_t)(2 * c + (q.starts ? 1 : 0)) * RT * (D + 4) + (size_t)i * (D + 4);
        const float inv = 1.0f / (l * a.vq.sqrt_d * sm.scale[1]);
        float y[D];
#pragma unroll
        for (int r = 0; r < NC; ++r) {
          uint32_t o[32];
          umma::ld32(o_col(x) + lanes + 32 * r, o);
          umma::wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) y[32 * r + e] = __uint_as_float(o[e]);
          if (SPLIT && both) {
            umma::ld32(o_col(1) + lanes + 32 * r, o);
            umma::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) y[32 * r + e] = y[32 * r + e] * f0 + __uint_as_float(o[e]) * f1;
          }
        }
        if (!done && live) {
#pragma unroll
          for (int e = 0; e < D; e += 4)
            *reinterpret_cast<float4 *>(slot + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          *reinterpret_cast<float2 *>(slot + D) = make_float2(M, l);
        }
        if (done && live) {  // inverse rotation of the thread's row
          dev::fwht_local<D>(y);
          const bool none = l == 0.f;  // no token seen
          const int qi = (q.row0 + i) / G;
          const int64_t orow = (int64_t)(q.q0 + qi) * a.Hq + q.h * G + (q.row0 + i - qi * G);
          uint16_t *out = static_cast<uint16_t *>(a.out) + orow * D;
#pragma unroll
          for (int j = 0; j < D; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // bit j + 2 e of the sign masks: -1
              const uint32_t sg = sm.sign[j / 32] >> (j % 32 + 2 * e);
              const float u = none ? 0.f : __uint_as_float(__float_as_uint(y[j + 2 * e] * inv) ^ (sg << 31));
              const float t = none ? 0.f : __uint_as_float(__float_as_uint(y[j + 2 * e + 1] * inv) ^ ((sg >> 1) << 31));
              if (a.dtype == TQ_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(u, t);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
              } else {
                const __half2 h = __floats2half2_rn(u, t);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
              }
            }
            *reinterpret_cast<uint4 *>(out + j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (a.lse) a.lse[orow] = none ? -INFINITY : (M + __log2f(l)) * 0.6931471805599453f;
        }
      }
    }
  }
  if (tid == 0) p.desc[c] = desc;
  __syncthreads();
  if (warp == 15) umma::dealloc(tmem, 512);
}

// Merges the pieces of the unit that starts last in CTA c's range and goes on
// behind it, in the order of the tokens: a warp a row.
template <int D>
__global__ void __launch_bounds__(256) paged_tile_merge_kernel(const __grid_constant__ TileParams p) {
  const PagedAttentionArgs &a = p.a;
  const int lane = threadIdx.x & 31, i = 8 * blockIdx.y + (threadIdx.x >> 5), c = blockIdx.x, RT = p.rt;
  constexpr int C = D / 32;  // coordinates a lane
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 desc = __ldcg(p.desc + c);
  const int n = desc.x;
  if (n == 0) return;
  const float vs = __ldcg(p.v_unit);
  const int G = a.Hq / a.Hkv;
  const Req req = load_req(a, desc.y, p.faults);
  const int row0 = desc.z * RT;
  if (i >= min(RT, req.n * G - row0)) return;
  auto slot = [&](int k) { return p.slots + ((size_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * RT + i) * (D + 4); };
  float m = -FLT_MAX;
  for (int k = lane; k < n; k += 32) m = fmaxf(m, __ldcg(slot(k) + D));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(dev::kFull, m, x));
  float L = 0.f, y[C];
#pragma unroll
  for (int e = 0; e < C; ++e) y[e] = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    float f = 0.f;
    if (k0 + lane < n) {
      const float2 ml = __ldcg(reinterpret_cast<const float2 *>(slot(k0 + lane) + D));
      f = exp2f(ml.x - m);
      L = fmaf(f, ml.y, L);
    }
    const int end = min(32, n - k0);
#pragma unroll 8
    for (int k = 0; k < end; ++k) {
      const float fk = __shfl_sync(dev::kFull, f, k), *s = slot(k0 + k) + lane * C;
#pragma unroll
      for (int e = 0; e < C; e += 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(s + e));
        y[e] = fmaf(fk, v.x, y[e]);
        y[e + 1] = fmaf(fk, v.y, y[e + 1]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(dev::kFull, L, x);
  const int qi = (row0 + i) / G;
  store_out<D>(a, (int64_t)req.q0 + qi, desc.w * G + (row0 + i) - qi * G, lane, y, m, L, 1.0f / (a.vq.sqrt_d * vs));
}

// Workspace: descriptors, slots, the line, turned rows and their factors.
struct Layout {
  size_t slots, first, line, tiles, qhi, qlo, qf, end;
};

Layout layout(int R, int64_t T, int Hq, int Hkv, int d) {
  const size_t ctas = decode_ctas();
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Layout l;
  l.slots = up(ctas * sizeof(int4) + sizeof(float));
  l.first = up(l.slots + 2 * ctas * 256 * (d + 4) * sizeof(float));
  l.line = up(l.first + ((size_t)R + 1) * 4);
  l.tiles = (size_t)T * (Hq / Hkv) / 128 + R;  // at most, in tiles of 128 rows
  l.qhi = up(l.line + (l.tiles + 1) * 8);
  l.qlo = up(l.qhi + (size_t)T * Hq * d * 2);
  l.qf = up(l.qlo + (size_t)T * Hq * d * 2);
  l.end = up(l.qf + (size_t)T * Hq * 4);
  return l;
}

template <int D, bool SPLIT, bool HL>
cudaError_t run_tile(const TileParams &p, cudaStream_t s) {
  const int ctas = decode_ctas();
  const int64_t rows = p.a.T * p.a.Hq, rpb = 8 * (512 / D);
  const int prep = 1 + (int)min((rows + rpb - 1) / rpb, (int64_t)ctas * 8);
  paged_tile_prep_kernel<D, HL><<<prep, 256, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int dyn = (int)(kHighAddr + 3 * Tile<D>::kBytes) - 1024;
  e = cudaFuncSetAttribute(paged_tile_kernel<D, SPLIT, HL>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)dyn;
  e = cudaLaunchKernelEx(&cfg, paged_tile_kernel<D, SPLIT, HL>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)(p.rt / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_tile_merge_kernel<D>, p);
}

template <int D>
cudaError_t run_d(const TileParams &p, cudaStream_t s) {
  if (p.a.dtype == TQ_F16) return run_tile<D, true, true>(p, s);
  return p.rt == 128 ? run_tile<D, true, false>(p, s) : run_tile<D, false, false>(p, s);
}

}  // namespace

size_t paged_tile_workspace(int R, int64_t T, int Hq, int Hkv, int d) { return layout(R, T, Hq, Hkv, d).end; }

cudaError_t launch_paged_tile(const PagedAttentionArgs &a, cudaStream_t s) {
  TileParams p{};
  p.a = a;
  const cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  // few rows a unit, or fp16 outputs: the blocks are split over the two sets instead of the rows
  dev::magic31_div(a.page_size, p.page_mul, p.page_shift);
  p.rt = a.dtype == TQ_F16 || (int64_t)a.max_q * (a.Hq / a.Hkv) <= 128 ? 128 : 256;
  const Layout l = layout(a.R, a.T, a.Hq, a.Hkv, a.kq.d);
  char *w = static_cast<char *>(a.ws);
  p.desc = reinterpret_cast<int4 *>(w);
  p.v_unit = reinterpret_cast<float *>(p.desc + decode_ctas());
  p.slots = reinterpret_cast<float *>(w + l.slots);
  p.first = reinterpret_cast<int32_t *>(w + l.first);
  p.max_tiles = (int64_t)l.tiles;
  p.line = reinterpret_cast<int64_t *>(w + l.line);
  p.qhi = reinterpret_cast<const __half *>(w + l.qhi);
  p.qlo = reinterpret_cast<const __half *>(w + l.qlo);
  p.qf = reinterpret_cast<const float *>(w + l.qf);
  return a.kq.d == 64 ? run_d<64>(p, s) : run_d<128>(p, s);
}

}  // namespace tq
