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
  // Query rows of a request and KV head.  The small tiles decode the cache once for 16 rows, or 32 in two groups of
  // warps, and again beyond that; the large ones for 128 or 256, with more work around each block.  us, small and large
  // tiles, 8 KV heads:
  //   64 requests of 1 to 4001 tokens and of up to so many rows each, d = 128: bf16 16 rows 89 and 204, 32 rows 149 and
  //   207, 40 rows 194 and 210, 48 rows 216 and 211; fp16 (large tiles of 128 rows, and twice the products) 32 rows 181
  //   and 284, 48 rows 261 and 289, 64 rows 293 and 292.
  //   So many rows in every request, 32 and 40 rows (bf16), 32 and 48 rows (fp16): d = 128, 1 request of 32768 tokens
  //   47|62 and 67|63, 55|80 and 83|81; 16 of up to 4001 64|72 and 92|73, 71|92 and 105|92; 128 of up to 4001 306|388
  //   and 493|396, 361|543 and 610|565.  d = 64: 33|49 and 46|48, 38|57 and 56|57; 46|52 and 69|53, 50|65 and 76|65;
  //   216|275 and 349|279, 247|367 and 416|377.
  // So up to 32 rows the small tiles win everywhere; between 33 and the limits they win where requests have fewer rows
  // than max_q says, and lose up to a quarter where all have as many.
  // The large tiles' shapes are for d = 64 and 128: with blocks of 128 tokens their operands and tables have no room for
  // d = 256 (blocks of 64 would).
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv);
  return rows <= (a.dtype == TQ_BF16 ? 40 : 48) || a.kq.d == 256 ? launch_paged_rows(a, s) : launch_paged_tile(a, s);
}

}  // namespace tq
