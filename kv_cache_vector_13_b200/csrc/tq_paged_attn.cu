// Attention of ragged query rows over a paged 4-bit TurboQuant cache
// (sm_100a): which kernel takes a call.
//
// For row t of request r, at position p = kv_len - q_len + i of its request,
// and cached token j (j <= p when causal, j > p - window with a window):
//   logit_j = scale n_j <H(sigma_K q) / sqrt d, c_K[idx_j]>,
//   o = sigma_V H(sum_j softmax_j n'_j c_V[idx'_j]) / sqrt d,
// the softmax kept as a running reference and sum in base 2, all in fp32.

#include "../../include/tq.h"
#include "tq_paged.h"

namespace tq {

size_t paged_attention_workspace(int R, int64_t T, int Hq, int Hkv, int d) {
  const size_t rows = paged_rows_workspace(d), tile = d == 256 ? 0 : paged_tile_workspace(R, T, Hq, Hkv, d);
  return rows > tile ? rows : tile;
}

cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t s) {
  // Query rows of a request and KV head.  The small tiles decode the cache once for 16 rows, the large ones for 128 or
  // 256, with more work around each block: 64 requests of up to 4001 tokens, 64 / 8 heads, us, small and large tiles:
  // bf16 16 rows 89 and 204, 32 rows 149 and 207, 40 rows 194 and 210, 48 rows 216 and 211; fp16 (large tiles of 128
  // rows, and twice the products) 32 rows 181 and 284, 48 rows 261 and 289, 64 rows 293 and 292.
  // The large tiles' operands and tables have no room for d = 256.
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv);
  return rows <= (a.dtype == TQ_BF16 ? 40 : 48) || a.kq.d == 256 ? launch_paged_rows(a, s) : launch_paged_tile(a, s);
}

}  // namespace tq
