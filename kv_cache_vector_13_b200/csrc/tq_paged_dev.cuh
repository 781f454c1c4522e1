// Device helpers of the paged attention kernels (sm_100a).
#pragma once

#include <float.h>

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"

namespace tq {
namespace paged {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The softmax reference: it moves when a weight times its value norm would pass 2^kMost (fp16 ends at 2^16), and is then
// put 2^kRoom below the largest.  As fp16 operands these end at 2^-25, half the smallest step, so what a token may lose is
// 2^-33 of the largest: 333000 tokens of 2^-25.2 beside 12 large ones lost all of the 1.8% of the output that they carry
// with no room, 0.03% with it, and draft verification (128 requests of 4 rows) takes 333 us in place of 331.
// Where rows and weights are rounded once, on the large tiles, a move costs the block's weights a second time: 3 x 2048
// rows take 1509 us with room 8, 1381 with 1 as without.  There it is 1, next to what the tensor cores' sums cut (2^-24).
constexpr float kMost = 15.f, kRoom = 8.f, kRoomOnce = 1.f;

// Runs of n tokens that hold the first `tokens` (which may be next to 2^31).
__device__ __forceinline__ int runs(int tokens, int n) { return (int)(((unsigned)tokens + n - 1) / n); }

// The first token that position p sees: p may be far below 0 and the window as large as an int.
__device__ __forceinline__ int window_start(int p, int window) {
  return window > 0 ? max(max(p + 1, 0) - window, 0) : 0;
}

// log2 of a value norm as it counts where the softmax reference is chosen: at least -64; an infinite one, whose
// product is infinite whatever the weight, does not count, so the other weights and their sum stay what they are.
__device__ __forceinline__ float value_log2(float norm) {
  const float x = log2_approx(norm);
  return x < INFINITY ? fmaxf(x, -64.f) : -64.f;
}

// Scale of a table of fp16 levels.  The 16 levels c_k, rounded to fp16 once,
// would be a fixed error of up to 2^-11 in every score and value; a factor s in
// [1, 2) moves them to where fp16 holds them best.  What counts is the error
// of a Gaussian coordinate's square, weighted by how often each level comes
// up, apart from a gain common to all levels, which the kernels divide out:
// over 192 candidates, one for every two threads of the block (256 on the large
// tiles, 128 for d = 256), it falls from 2e-4 to 8e-5 of a coordinate (d = 128;
// 4e-5 with 1024, for 5 us more a call).

// P(|N(0,1)| in the level's cell) times the level squared, over their sum, for
// the positive levels of the 16-level Lloyd-Max quantizer.
__device__ constexpr float kLevelWeight[8] = {0.0033913f, 0.0296217f, 0.0772600f, 0.1365659f,
                                               0.1927278f, 0.2258000f, 0.2113073f, 0.1233260f};

// Gain sum w e and variance sum w e^2 - gain^2 of the relative errors e of the
// levels c (rc = 1 / c); the difference of a value and its rounding is exact.
__device__ __forceinline__ float level_error(const float (&c)[8], const float (&rc)[8], float s, float &gain) {
  const float rs = __frcp_rn(s);
  float m = 0.f, v = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = s * c[k], e = (__half2float(__float2half_rn(x)) - x) * (rc[k] * rs), we = kLevelWeight[k] * e;
    m += we;
    v = fmaf(we, e, v);
  }
  gain = m;
  return fmaxf(v - m * m, 0.f);
}

__device__ __forceinline__ void load_levels(const float *cent, float (&c)[8], float (&rc)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c[k] = __ldg(cent + 8 + k);
    rc[k] = __frcp_rn(c[k]);
  }
}

// The best candidate into key[0] (the keys' table) and key[1] (the values'),
// ties to the smaller; keys must be 0xffffffff before, with a barrier on both
// sides.  All threads of the block call it, at most 512.
__device__ __forceinline__ float candidate(int i, int n) { return 1.0f + (float)i / (float)n; }

__device__ __forceinline__ void find_scales(const float *ck, const float *cv, int tid, int threads, unsigned *key) {
  const int half = threads / 2, side = tid >= half;
  const float *cent = side ? cv : ck;
  float c[8], rc[8];
  load_levels(cent, c, rc);
  const int i = side ? tid - half : tid;
  float gain;
  const float v = level_error(c, rc, candidate(i, half), gain);
  unsigned best = (__float_as_uint(v) & ~255u) | (unsigned)i;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) best = min(best, __shfl_xor_sync(dev::kFull, best, x));
  if ((tid & 31) == 0) atomicMin(key + side, best);
}

// The factor of a key, and in `unit` what table values are to be divided by.
__device__ __forceinline__ float scale_of(unsigned key, int threads, const float *cent, float &unit) {
  float c[8], rc[8], gain;
  load_levels(cent, c, rc);
  const float s = candidate((int)(key & 255u), threads / 2);
  level_error(c, rc, s, gain);
  unit = s * (1.0f + gain);
  return s;
}

// D / 32 consecutive elements of a bf16 or fp16 row from element `at`.
template <int D>
__device__ __forceinline__ void load_row(const void *p, int dt, int64_t at, int lane, float (&v)[D / 32]) {
  const uint32_t *s = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + at + lane * (D / 32));
  uint32_t w[D / 64];
  if constexpr (D / 64 == 4) {
    const uint4 t = __ldg(reinterpret_cast<const uint4 *>(s));
    w[0] = t.x;
    w[1] = t.y;
    w[2] = t.z;
    w[3] = t.w;
  } else if constexpr (D / 64 == 2) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(s));
    w[0] = t.x;
    w[1] = t.y;
  } else {
    w[0] = __ldg(s);
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    v[2 * i] = dt == TQ_BF16 ? dev::bf16lo(w[i]) : dev::f16lo(w[i]);
    v[2 * i + 1] = dt == TQ_BF16 ? dev::bf16hi(w[i]) : dev::f16hi(w[i]);
  }
}

// A power of two that brings the row's largest magnitude into [1, 2), so that
// rows of any size round to fp16 alike; 1 for rows of zeros, and for rows
// with an infinity or NaN, which keep it.
template <int C>
__device__ __forceinline__ float row_scale(const float (&v)[C]) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < C; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = max(m, __shfl_xor_sync(dev::kFull, m, x));
  const unsigned e = m >> 23;
  if (e == 255u || m == 0) return 1.0f;
  return __uint_as_float(min(max(254u - e, 1u), 252u) << 23);
}

// One finished row: y = sum w v in the rotated basis (coordinate lane * D/32 +
// e), its sum L and reference m.  Inverse rotation, normalisation, rounding.
// A row that saw no token (L == 0) gets zeros.
template <int D>
__device__ __forceinline__ void store_out(const PagedAttentionArgs &a, int64_t t, int hq, int lane, float (&y)[D / 32],
                                          float m, float L, float vscale) {
  dev::fwht<32, D / 32>(y, lane);
  const bool none = L == 0.f;
  const float inv = vscale / L;
  uint32_t w[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int k = lane * (D / 32) + 2 * i;
    const float y0 = none ? 0.f : y[2 * i] * inv * (float)__ldg(a.vq.signs + k);
    const float y1 = none ? 0.f : y[2 * i + 1] * inv * (float)__ldg(a.vq.signs + k + 1);
    if (a.dtype == TQ_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(y0, y1);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
      const __half2 b = __floats2half2_rn(y0, y1);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
  }
  uint16_t *o = static_cast<uint16_t *>(a.out) + (t * a.Hq + hq) * D + lane * (D / 32);
  if constexpr (D / 64 == 4)
    *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (D / 64 == 2)
    *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t *>(o) = w[0];
  if (a.lse && lane == 0) a.lse[t * a.Hq + hq] = none ? -INFINITY : (m + __log2f(L)) * 0.6931471805599453f;
}

}  // namespace paged
}  // namespace tq
