// Attention of ragged query rows over a paged 4-bit TurboQuant cache
// (sm_100a): the general kernel and the host launch.
//
// For row t of request r, at position p = kv_len - q_len + i of its request,
// and cached token j (j <= p when causal, j > p - window with a window):
//   logit_j = scale n_j <H(sigma_K q) / sqrt d, c_K[idx_j]>,
//   o = sigma_V H(sum_j softmax_j n'_j c_V[idx'_j]) / sqrt d,
// the softmax kept as a running maximum and sum in base 2, all in fp32.

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"

#include <float.h>

namespace tq {
namespace {

constexpr int kWarps = 4;

struct GeneralParams {
  PagedAttentionArgs a;
  unsigned *faults;
};

// Last r in [0, R) with cu[r] <= t (cu ascending).
__device__ __forceinline__ int find_request(const int32_t *cu, int R, int64_t t) {
  int i = 0, j = R;
  while (j - i > 1) {
    const int m = (i + j) >> 1;
    if (__ldg(cu + m) <= t) i = m; else j = m;
  }
  return i;
}

template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  if constexpr (DT == TQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(static_cast<const __half *>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
  if constexpr (DT == TQ_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// One block per (query row, head): its warps take every fourth run of 32
// tokens, a token per lane for the scores and D/32 coordinates per lane for
// the values, and merge in shared memory.
template <int D, int DT>
__global__ void __launch_bounds__(kWarps * 32) paged_general_kernel(GeneralParams p) {
  constexpr int C = D / 32;  // coordinates per lane
  __shared__ float s_q[D], s_ck[16], s_cv[16], s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
  const PagedAttentionArgs &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int hq = blockIdx.y, h = hq / (a.Hq / a.Hkv);
  int r = (int)t, q0 = (int)t, q1 = (int)t + 1;
  if (a.cu_q) {
    r = find_request(a.cu_q, a.R, t);
    q0 = a.cu_q[r];
    q1 = a.cu_q[r + 1];
    if (t < q0 || t >= q1) return;  // behind the last sequence
  }
  int kv = max(a.kv_lens[r], 0);
  if (kv > a.max_pages * a.page_size) {
    if (threadIdx.x == 0) atomicOr(p.faults, kFaultIndex);
    kv = a.max_pages * a.page_size;
  }
  const int64_t pos = (int64_t)kv - (q1 - t);
  const int hi = a.causal ? (int)max((int64_t)0, pos + 1) : kv;
  const int lo = a.window > 0 ? (int)max((int64_t)0, pos + 1 - a.window) : 0;

  if (warp == 0) {
    float x[C];
#pragma unroll
    for (int e = 0; e < C; ++e) {
      const int i = lane * C + e;
      x[e] = load1<DT>(a.q, t * a.q_st + hq * a.q_sh + i) * (float)a.kq.signs[i];
    }
    dev::fwht<32, C>(x, lane);
    const float f = a.scale * 1.4426950408889634f / a.kq.sqrt_d;
#pragma unroll
    for (int e = 0; e < C; ++e) s_q[lane * C + e] = x[e] * f;
  }
  if (threadIdx.x < 16) {
    s_ck[threadIdx.x] = a.kq.centroids[threadIdx.x];
    s_cv[threadIdx.x] = a.vq.centroids[threadIdx.x];
  }
  __syncthreads();

  float m = -FLT_MAX, l = 0.f, o[C];
#pragma unroll
  for (int e = 0; e < C; ++e) o[e] = 0.f;
  const int32_t *row = a.table + (int64_t)r * a.table_stride;
  for (int j0 = (lo & ~31) + 32 * warp; j0 < hi; j0 += 32 * kWarps) {
    const int j = j0 + lane;
    bool seen = j >= lo && j < hi;
    float z = -INFINITY, nv = 0.f;
    int64_t vrec = 0;
    if (seen) {
      const int page = j / a.page_size, off = j - page * a.page_size;
      const int id = row[page];
      seen = (unsigned)id < (unsigned)a.n_pages;
      if (!seen) atomicOr(p.faults, kFaultIndex);
      if (seen) {
        const int64_t krec = id * a.k.sb + h * a.k.sh + off * a.k.sn;
        vrec = id * a.v.sb + h * a.v.sh + off * a.v.sn;
        const uint4 *c = reinterpret_cast<const uint4 *>(a.k.codes + krec * (D / 2));
        float s = 0.f;
#pragma unroll 2
        for (int b = 0; b < D / 32; ++b) {
          const uint4 u = __ldg(c + b);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(s_q[32 * b + 8 * i + e], s_ck[(w[i] >> (4 * e)) & 15], s);
        }
        z = s * a.k.norms[krec];
        nv = a.v.norms[vrec];
      }
    }
    float mx = z;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(dev::kFull, mx, x));
    if (!__any_sync(dev::kFull, seen)) continue;
    const float mn = fmaxf(m, mx);
    const float w = seen ? exp2f(z - mn) : 0.f, scale = mn == m ? 1.f : exp2f(m - mn);
    m = mn;
    l = l * scale + w;
#pragma unroll
    for (int e = 0; e < C; ++e) o[e] *= scale;
    const float wv = seen ? w * nv : 0.f;
    const unsigned have = __ballot_sync(dev::kFull, seen);
    for (int i = 0; i < 32; ++i) {
      const float wi = __shfl_sync(dev::kFull, wv, i);
      const int64_t rec = __shfl_sync(dev::kFull, vrec, i);
      if (!(have >> i & 1)) continue;
      const uint8_t *c = a.v.codes + rec * (D / 2) + lane * (C / 2);
#pragma unroll
      for (int e = 0; e < C; e += 2) {
        const int b = __ldg(c + e / 2);
        o[e] = fmaf(wi, s_cv[b & 15], o[e]);
        o[e + 1] = fmaf(wi, s_cv[b >> 4], o[e + 1]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(dev::kFull, l, x);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < C; ++e) s_o[warp][lane * C + e] = o[e];
  __syncthreads();
  if (warp != 0) return;
  float M = s_m[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  float L = 0.f, y[C];
#pragma unroll
  for (int e = 0; e < C; ++e) y[e] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = exp2f(s_m[w] - M);
    L += f * s_l[w];
#pragma unroll
    for (int e = 0; e < C; ++e) y[e] += f * s_o[w][lane * C + e];
  }
  dev::fwht<32, C>(y, lane);
  const bool none = L == 0.f;  // no token seen
  const float inv = none ? 0.f : 1.f / (L * a.vq.sqrt_d);
#pragma unroll
  for (int e = 0; e < C; ++e) {
    const int i = lane * C + e;
    store1<DT>(a.out, (t * a.Hq + hq) * D + i, none ? 0.f : y[e] * inv * (float)a.vq.signs[i]);
  }
  if (a.lse && lane == 0) a.lse[t * a.Hq + hq] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int D>
cudaError_t run_general(const GeneralParams &p, cudaStream_t s) {
  const dim3 grid((unsigned)p.a.T, (unsigned)p.a.Hq);
  if (p.a.dtype == TQ_BF16)
    paged_general_kernel<D, TQ_BF16><<<grid, kWarps * 32, 0, s>>>(p);
  else
    paged_general_kernel<D, TQ_F16><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t paged_attention_workspace(int R, int64_t T, int Hq, int Hkv, int d) {
  if (d == 256) return 16;
  const size_t rows = paged_rows_workspace(d), tile = paged_tile_workspace(R, T, Hq, Hkv, d);
  return rows > tile ? rows : tile;
}

cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t s) {
  // Query rows of a request and KV head.  The small tiles decode the cache once for 8 rows, the large ones for 128 or
  // 256, with more work around each block: 64 requests of up to 4001 tokens, 64 / 8 heads, us, small and large tiles:
  // 16 rows 173 and 303 (bf16), 174 and 424 (fp16); 32 rows 243 and 308, 243 and 435; 64 rows 481 and 313, 481 and 436.
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv);
  if (a.kq.d != 256) return rows <= 32 ? launch_paged_rows(a, s) : launch_paged_tile(a, s);
  GeneralParams p{a, nullptr};
  const cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  return run_general<256>(p, s);
}

}  // namespace tq
