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

// A factor s in [1, 2) whose products s c_k round to fp16 with the smallest
// worst relative error over the 16 levels, out of 32 candidates (ties to the
// smaller one).  The whole warp calls it; every lane gets s.  A single
// rounding of the levels is a fixed error in every score and value, up to
// 2^-11; the factor takes it to about a quarter of that.
__device__ __forceinline__ float table_scale(const float *cent, int lane) {
  const float s = 1.0f + (float)lane * (1.0f / 32.0f);
  float worst = 0.f;
#pragma unroll
  for (int k = 8; k < 16; ++k) {
    const float v = s * __ldg(cent + k);
    worst = fmaxf(worst, fabsf(__half2float(__float2half_rn(v)) - v) / v);
  }
  // order by (error, lane)
  unsigned key = (__float_as_uint(worst) & ~31u) | (unsigned)lane;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) key = min(key, __shfl_xor_sync(dev::kFull, key, x));
  return 1.0f + (float)(key & 31u) * (1.0f / 32.0f);
}

// D / 32 consecutive elements of a bf16 or fp16 row from element `at`.
template <int D>
__device__ __forceinline__ void load_row(const void *p, int dt, int64_t at, int lane, float (&v)[D / 32]) {
  const uint32_t *s = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + at + lane * (D / 32));
  uint32_t w[D / 64];
  if constexpr (D / 64 == 2) {
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
  if constexpr (D / 64 == 2)
    *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t *>(o) = w[0];
  if (a.lse && lane == 0) a.lse[t * a.Hq + hq] = none ? -INFINITY : (m + __log2f(L)) * 0.6931471805599453f;
}

}  // namespace paged
}  // namespace tq
