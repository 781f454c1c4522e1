// Paged cache write and read-back for sm_100a: rotary positions on several
// axes, the 4-bit TurboQuant_mse records of the batch's K and V rows written
// at their slots, and cached rows reconstructed from their slots.
//
// Append, per row (one head of one token): K and Q pairs (x1, x2) turn by
// theta_i = position[axis_i] * inv_freq_i; Q is rounded to its type and
// stored; K goes on in fp32 (no rounding in between).  Then, for K and V, the
// canonical encode ("TurboQuant của Google: nén KV cache 6 lần", sections
// "Trick đầu tiên" and "Lloyd-Max quantizer"): norm, sign flips + FWHT, scale,
// nearest of 16 levels, packed nibbles -- the same fp32 steps in the same
// order as tq_encode, so without positions the records are bit-identical.
//
// Work layout: a block takes a few tokens; D/16 lanes hold a row, 16
// coordinates each, so a warp works on 512/D rows of one kind (Q, K or V) at
// a time.  The block first forms cos and sin of its tokens' angles once for
// all heads, laid out per coordinate in the order the lanes read them.  The
// angle is formed in double as a number of turns and only its fraction goes
// on in fp32, so positions up to 2^31 keep their phase.
// A pair's other half comes from the row itself through L1 when it lies in
// another lane (pairs half a head apart).
//
// Both kernels are bound by the shared-memory pipe, which does the shuffles too:
// 48 of them per four rows of 128 for the transform's stages across lanes; 72%
// of its rate in the read-back.  A row in two lanes (64 coordinates each) needs
// a third of the shuffles but scatters the loads: 66 us against 61 (read-back of
// 65536 rows of 8 heads, 2.8 TB/s), 218 against 163 (append of 16384 tokens, 32
// / 8 heads, and its two read-backs).

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_paged.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 4;  // tokens per block
constexpr int E = 16;          // coordinates per lane

// The transform of tq_device.cuh with the same steps and roundings; a stage
// across lanes is one multiply-add by +1 or -1 a pair (the product is exact),
// without flipping a sign first.
template <int T>
__device__ __forceinline__ void fwht_row(float (&a)[E], int t) {
#pragma unroll
  for (int P = T / 2; P >= 1; P >>= 1) {
    const float sign = t & P ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float o0 = __shfl_xor_sync(dev::kFull, a[i], P), o1 = __shfl_xor_sync(dev::kFull, a[i + 1], P);
      dev::fma_x2(a[i], a[i + 1], a[i], a[i + 1], sign, sign, o0, o1);
    }
  }
  dev::fwht_local<E>(a);
}

// Neither a slot of the cache nor -1, which is none.
__device__ __forceinline__ bool bad_slot(int64_t slot, int64_t n_slots) {
  return (uint64_t)slot + 1 > (uint64_t)n_slots;
}

// The lane's signs of a rotation as +1 and -1.
__device__ __forceinline__ void load_signs(const int8_t *signs, float (&s)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) s[i] = signs[i] < 0 ? -1.f : 1.f;
}

// The values of a 16-byte word.
template <int DT>
__device__ __forceinline__ void widen(const uint4 &u, float *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == TQ_F32) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = DT == TQ_BF16 ? dev::bf16lo(w[i]) : dev::f16lo(w[i]);
      x[2 * i + 1] = DT == TQ_BF16 ? dev::bf16hi(w[i]) : dev::f16hi(w[i]);
    }
  }
}

struct AppendParams {
  PagedAppendArgs a;
  int tokens;          // tokens per block
  int gq, gk;          // warp groups per block: of Q rows, of K (and of V) rows
  unsigned *faults;
};

__device__ __forceinline__ void store16(void *dst, int dt, const float (&v)[E]) {
  if (dt == TQ_F32) {
    float4 *o = static_cast<float4 *>(dst);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    return;
  }
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    if (dt == TQ_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
      const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
  }
  uint4 *o = static_cast<uint4 *>(dst);
  o[0] = make_uint4(w[0], w[1], w[2], w[3]);
  o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, DT == TQ_F32 ? 2 : 3) paged_append_kernel(AppendParams p) {
  constexpr int T = D / E;           // lanes per row
  constexpr int RPW = 32 / T;        // rows per warp
  constexpr int ES = DT == TQ_F32 ? 4 : 2;
  // (cos, signed sin) per coordinate: chunk c of 4 coordinates of lane t at
  // float4 c * T + t, so the lanes of a row read consecutive 16-byte words
  __shared__ float4 s_cos[kMaxTokens][D / 4], s_sin[kMaxTokens][D / 4];
  __shared__ int64_t s_krec[kMaxTokens], s_vrec[kMaxTokens];  // record of head 0, or -1
  __shared__ float4 s_flip[2][D / 4];  // the rotations' signs, laid out alike

  const PagedAppendArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t tok0 = (int64_t)blockIdx.x * p.tokens;
  const int ntok = (int)min((int64_t)p.tokens, a.T - tok0);

  for (int i = tid; i < 2 * D; i += kThreads) {
    const int c = i % D;
    const int8_t *signs = i < D ? a.kq.signs : a.vq.signs;
    reinterpret_cast<float *>(&s_flip[i / D][((c % E) / 4) * T + c / E])[c & 3] = signs[c] < 0 ? -1.f : 1.f;
  }
  if (tid >= kThreads - kMaxTokens) {
    const int k = tid - (kThreads - kMaxTokens);
    if (k < ntok) {
      const int64_t slot = a.slots[tok0 + k];
      int64_t kr = -1, vr = -1;
      if (bad_slot(slot, a.n_slots)) {
        if (blockIdx.y == 0) atomicOr(p.faults, kFaultIndex);
      } else if (slot >= 0) {
        const int64_t page = slot / a.page_size, off = slot - page * a.page_size;
        kr = page * a.kc.sb + off * a.kc.sn;
        vr = page * a.vc.sb + off * a.vc.sn;
      }
      s_krec[k] = kr;
      s_vrec[k] = vr;
    }
  }
  const int half = a.rot_dim / 2;
  for (int i = tid; i < ntok * half; i += kThreads) {
    const int k = i / half, f = i - k * half;
    const int ax = a.axis ? min(max(__ldg(a.axis + f), 0), a.n_axes - 1) : 0;
    const int pos = a.positions[ax * a.pos_stride + tok0 + k];
    double turns = (double)pos * (double)__ldg(a.inv_freq + f) * 0.15915494309189533577;
    turns -= rint(turns);
    float sn, cs;
    sincospif((float)(2.0 * turns), &sn, &cs);
    const int i0 = a.adjacent ? 2 * f : f, i1 = a.adjacent ? 2 * f + 1 : f + half;
    auto at = [&](float4 *s, int c) -> float & {
      return reinterpret_cast<float *>(s + ((c % E) / 4) * T + c / E)[c & 3];
    };
    at(s_cos[k], i0) = cs;
    at(s_cos[k], i1) = cs;
    at(s_sin[k], i0) = -sn;
    at(s_sin[k], i1) = sn;
  }
  __syncthreads();

  const int t = lane % T, rw = lane / T;
  const int groups = p.gq + 2 * p.gk;
  // A group's rows: what kind, which token and head of the lane's row, and where that lies.
  struct Group {
    int kind, k, h;  // Q, K, V
    bool active;
    const char *src;
  };
  auto group = [&](int g) {
    Group r;
    r.kind = g < p.gq ? 0 : g < p.gq + p.gk ? 1 : 2;
    const int H = r.kind == 0 ? a.Hq : a.Hkv;
    int row = (g - (r.kind == 0 ? 0 : r.kind == 1 ? p.gq : p.gq + p.gk)) * RPW + rw;
    r.active = row < ntok * H;
    if (!r.active) row = 0;  // idle lanes still take part in the shuffles
    r.k = (ntok > 1 && row >= H) + (ntok > 2 && row >= 2 * H) + (ntok > 3 && row >= 3 * H);
    r.h = row - r.k * H;
    const int64_t tok = tok0 + r.k;
    if (r.kind == 0)
      r.src = static_cast<const char *>(a.q) + (tok * a.q_st + r.h * a.q_sh) * ES;
    else if (r.kind == 1)
      r.src = static_cast<const char *>(a.k) + (tok * a.k_st + r.h * a.k_sh) * ES;
    else
      r.src = static_cast<const char *>(a.v) + (tok * a.v_st + r.h * a.v_sh) * ES;
    return r;
  };
  constexpr int NR = E * ES / 16;  // 16-byte words of a lane
  uint4 ahead[NR];
  auto fetch = [&](const Group &r) {
#pragma unroll
    for (int i = 0; i < NR; ++i) ahead[i] = __ldg(reinterpret_cast<const uint4 *>(r.src + t * E * ES) + i);
  };
  const int step = gridDim.y * kWarps;
  int g = blockIdx.y * kWarps + warp;
  Group cur = group(min(g, groups - 1));
  if (g < groups) fetch(cur);
  for (; g < groups; g += step) {
    const int kind = cur.kind, k = cur.k, h = cur.h;
    const bool active = cur.active;
    const char *src = cur.src;
    const int64_t tok = tok0 + k;
    float x[E];
#pragma unroll
    for (int i = 0; i < NR; ++i) widen<DT>(ahead[i], x + i * (16 / ES));
    if (g + step < groups) {  // the next group's rows, while this one is worked on
      cur = group(g + step);
      fetch(cur);
    }

    if (kind != 2 && t * E < a.rot_dim) {
      float y[E];  // each coordinate's partner
      if (a.adjacent) {
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = x[i ^ 1];
      } else if (a.rot_dim == D) {
        // half a row away: the same coordinates of another lane
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = __shfl_xor_sync(dev::kFull, x[i], T / 2);
      } else {
        // half is a multiple of 8, so a chunk of 8 lies on one side of it
#pragma unroll
        for (int c = 0; c < E / 8; ++c) {
          const int i = t * E + 8 * c;
          const int j = i < half ? i + half : i < a.rot_dim ? i - half : i;
          float z[8];
          dev::load_block<DT, 8>(src + j * ES, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[8 * c + e] = z[e];
        }
      }
#pragma unroll
      for (int c = 0; c < E / 4; ++c) {
        // rot_dim is a multiple of 16: a lane's block is turned or not
        const float4 cs = s_cos[k][c * T + t], sn = s_sin[k][c * T + t];
        x[4 * c] = fmaf(x[4 * c], cs.x, y[4 * c] * sn.x);
        x[4 * c + 1] = fmaf(x[4 * c + 1], cs.y, y[4 * c + 1] * sn.y);
        x[4 * c + 2] = fmaf(x[4 * c + 2], cs.z, y[4 * c + 2] * sn.z);
        x[4 * c + 3] = fmaf(x[4 * c + 3], cs.w, y[4 * c + 3] * sn.w);
      }
    }
    if (kind == 0) {
      if (active)
        store16(static_cast<char *>(a.q_out) + ((tok * a.Hq + h) * D + t * E) * (int64_t)ES, DT, x);
      continue;
    }

    // the canonical encode (tq_encode.cu), 16 levels
    const QuantParams &q = kind == 1 ? a.kq : a.vq;
    uint32_t P[8];
#pragma unroll
    for (int m = 0; m < 7; ++m) P[m] = __float_as_uint(__ldg(q.thresholds + 8 + m));
    P[7] = 0;
    const float nrm = __fsqrt_rn(dev::fold_halves_sumsq<T, E>(x));
#pragma unroll
    for (int c = 0; c < E / 4; ++c) {
      const float4 sg = s_flip[kind - 1][c * T + t];
      dev::mul_x2(x[4 * c], x[4 * c + 1], x[4 * c], x[4 * c + 1], sg.x, sg.y);
      dev::mul_x2(x[4 * c + 2], x[4 * c + 3], x[4 * c + 2], x[4 * c + 3], sg.z, sg.w);
    }
    fwht_row<T>(x, t);
    const float wsc = __fmul_rn(nrm, q.sqrt_d);
    const float inv = wsc > 0.0f ? __frcp_rn(wsc) : 0.0f;
    dev::scale_x2<E>(x, inv);
    uint32_t W[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < E; ++i) dev::put_field<4>(W, i, (uint32_t)dev::quantize_sym<4>(x[i], P));
    const CacheView &c = kind == 1 ? a.kc : a.vc;
    const int64_t base = kind == 1 ? s_krec[k] : s_vrec[k];
    if (active && base >= 0) {
      const int64_t rec = base + h * c.sh;
      *reinterpret_cast<uint2 *>(c.codes + rec * (D / 2) + t * 8) = make_uint2(W[0], W[1]);
      if (t == 0) c.norms[rec] = nrm;
    }
  }
}

struct ReadParams {
  PagedDequantArgs a;
  dev::IndexSplit rows;    // row -> (token, head)
  uint32_t page_mul;       // slot / page_size = (slot * page_mul) >> page_shift below 2^31 slots
  int page_shift;
  bool small;              // so many
  unsigned *faults;
};

// x_hat = n sigma H(c[idx]) / sqrt(d) of the record at each row's slot; zeros
// for a row without one.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_dequant_kernel(ReadParams p) {
  constexpr int T = D / E, RPW = 32 / T;
  __shared__ float s_cent[16];
  const PagedDequantArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 16) s_cent[tid] = a.q.centroids[tid];
  float sign[E];
  load_signs(a.q.signs + (lane % T) * E, sign);
  __syncthreads();
  const int t = lane % T;
  const int64_t rows = a.T * a.H;
  const int64_t step = (int64_t)gridDim.x * kWarps * RPW;
  for (int64_t r0 = ((int64_t)blockIdx.x * kWarps + warp) * RPW; r0 < rows; r0 += step) {
    int64_t row = r0 + lane / T;
    const bool active = row < rows;
    if (!active) row = r0;
    int64_t none, tok, h;
    dev::split_bhn(p.rows, row, none, tok, h);
    const int64_t slot = a.slots[tok];
    int64_t rec = -1;
    if (bad_slot(slot, a.n_slots)) {
      if (t == 0 && h == 0) atomicOr(p.faults, kFaultIndex);
    } else if (slot >= 0) {
      const int64_t page = p.small ? (int64_t)(((uint64_t)slot * p.page_mul) >> p.page_shift) : slot / a.page_size;
      rec = page * a.c.sb + (slot - page * a.page_size) * a.c.sn + h * a.c.sh;
    }
    float x[E], sc = 0.f;
    uint32_t W[2] = {0u, 0u};
    if (rec >= 0) {
      dev::load_words<2>(a.c.codes + rec * (D / 2) + t * 8, W);
      sc = __fdiv_rn(__ldg(a.c.norms + rec), a.q.sqrt_d);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = s_cent[dev::get_field<4>(W, i)];
    fwht_row<T>(x, t);
#pragma unroll
    for (int i = 0; i < E; i += 2) {  // sc is 0 for a row without a record
      dev::mul_x2(x[i], x[i + 1], x[i], x[i + 1], sign[i], sign[i + 1]);
      dev::mul_x2(x[i], x[i + 1], x[i], x[i + 1], sc, sc);
    }
    if (active)
      store16(static_cast<char *>(a.out) + (row * D + t * E) * (a.out_dtype == TQ_F32 ? 4 : 2), a.out_dtype, x);
  }
}

template <int D>
cudaError_t append_d(const AppendParams &p, dim3 grid, cudaStream_t s) {
  switch (p.a.dtype) {
    case TQ_F32: paged_append_kernel<D, TQ_F32><<<grid, kThreads, 0, s>>>(p); break;
    case TQ_BF16: paged_append_kernel<D, TQ_BF16><<<grid, kThreads, 0, s>>>(p); break;
    default: paged_append_kernel<D, TQ_F16><<<grid, kThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t s) {
  AppendParams p{a, 1, 0, 0, nullptr};
  cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  const int rpw = 512 / a.kq.d, sms = decode_ctas();
  // more tokens to a block once that still leaves a few blocks an SM
  while (p.tokens < kMaxTokens && a.T / (2 * p.tokens) >= 4 * sms) p.tokens *= 2;
  p.gq = (p.tokens * a.Hq + rpw - 1) / rpw;
  p.gk = (p.tokens * a.Hkv + rpw - 1) / rpw;
  const int64_t bx = (a.T + p.tokens - 1) / p.tokens;
  // few tokens: their rows spread over several blocks
  const int most = (p.gq + 2 * p.gk + kWarps - 1) / kWarps;
  const int by = (int)max((int64_t)1, min((int64_t)most, (2 * sms + bx - 1) / bx));
  const dim3 grid((unsigned)bx, (unsigned)by);
  switch (a.kq.d) {
    case 64: return append_d<64>(p, grid, s);
    case 128: return append_d<128>(p, grid, s);
    case 256: return append_d<256>(p, grid, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_dequant(const PagedDequantArgs &a, cudaStream_t s) {
  ReadParams p{};
  p.a = a;
  p.rows = dev::make_index_split(a.T, a.H, a.T * a.H);
  p.small = a.n_slots < ((int64_t)1 << 31);
  dev::magic31_div(a.page_size, p.page_mul, p.page_shift);
  cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  const int rpb = kWarps * (512 / a.q.d);
  const int64_t blocks = min((a.T * a.H + rpb - 1) / rpb, (int64_t)decode_ctas() * 16);
  switch (a.q.d) {
    case 64: paged_dequant_kernel<64><<<(unsigned)blocks, kThreads, 0, s>>>(p); break;
    case 128: paged_dequant_kernel<128><<<(unsigned)blocks, kThreads, 0, s>>>(p); break;
    case 256: paged_dequant_kernel<256><<<(unsigned)blocks, kThreads, 0, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace tq
