// Page plan of a batch (sm_100a): block-table rows, slots and positions of
// the tokens a step adds, from the requests' cached and new lengths.
//
// With cu the exclusive prefix sum of the new lengths and pages(l) =
// ceil(l / P), request r needs pages(lens + new) - pages(lens) pages, and the
// exclusive prefix sum of the needs is its place in the free list, which is
// popped from its end.  Token t of request r stands at lens_r + t - cu_r.
//
// One launch: every block takes a range of token rows and repeats the two
// prefix sums for the requests up to that range, a request per thread and a
// tile of requests at a time, so nothing is exchanged between blocks.  The
// tokens of a tile find their request by binary search in the tile's sums.  A
// new page's first token is always one of this call's tokens, and its thread
// writes the page's block-table entry; a page's id is read from the free list
// itself by every token of a new page, and from the table only for pages that
// were there before, so no thread reads an entry that another one writes.

#include "tq_paged.h"

namespace tq {
namespace {

constexpr int kThreads = 512;        // requests per tile
constexpr int kTokens = 2 * kThreads;  // token rows per block


// Exclusive prefix sum over the block; *total gets the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *s_warp, int64_t *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[w] = x;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int64_t y = s_warp[i];
    if (i < w) base += y;
    all += y;
  }
  *total = all;
  __syncthreads();
  return base + x - v;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(PagePlanArgs p) {
  __shared__ int64_t s_warp[kThreads / 32];
  __shared__ int64_t s_begin[kThreads + 1];  // first token of each request of the tile
  __shared__ int64_t s_before[kThreads];     // its place in the free list
  __shared__ int32_t s_len[kThreads];
  __shared__ bool s_ok[kThreads];
  const int tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int64_t t1 = min(t0 + kTokens, p.max_tokens);
  int64_t n_free = *p.n_free;
  n_free = n_free < 0 ? 0 : min(n_free, p.free_cap);

  int64_t tokens = 0, pages = 0, taken = 0;  // sums over the tiles before
  for (int r0 = 0; r0 < p.R; r0 += kThreads) {
    // block 0 goes through all requests; another block stops behind its range
    if (!first && tokens >= t1) break;
    const int r = r0 + tid, n = min(kThreads, p.R - r0);
    int64_t len = 0, add = 0;
    if (tid < n) {
      len = max(p.lens[r], 0);
      add = max(p.new_lens[r], 0);
    }
    int64_t all;
    const int64_t begin = tokens + block_scan(add, s_warp, &all);
    const int64_t had = (len + p.page_size - 1) / p.page_size;
    const int64_t has = (len + add + p.page_size - 1) / p.page_size;
    const bool fits = has <= p.max_pages && begin + add <= p.max_tokens;
    const int64_t need = fits ? has - had : 0;
    int64_t all_need;
    const int64_t before = pages + block_scan(need, s_warp, &all_need);
    const bool paid = need == 0 || before + need <= n_free;
    s_begin[tid] = begin;
    s_before[tid] = before;
    s_len[tid] = (int32_t)len;
    s_ok[tid] = fits && paid;
    if (tid == 0) s_begin[n] = tokens + all;
    if (first) {
      if (tid < n) {
        p.cu_new[r] = (int32_t)min(begin, (int64_t)INT32_MAX);
        p.seq_lens[r] = (int32_t)(fits && paid ? len + add : len);
        p.status[r] = !fits ? 2 : paid ? 0 : 1;
      }
      int64_t all_taken;
      block_scan(fits && paid ? need : 0, s_warp, &all_taken);
      taken += all_taken;
    }
    __syncthreads();
    // the block's tokens among this tile's
    const int64_t lo = max(t0, tokens), hi = min(t1, tokens + all);
    for (int64_t t = lo + tid; t < hi; t += kThreads) {
      int i = 0, j = n;  // the last request i of the tile with s_begin[i] <= t
      while (j - i > 1) {
        const int m = (i + j) >> 1;
        if (s_begin[m] <= t) i = m; else j = m;
      }
      const uint32_t l = (uint32_t)s_len[i];
      const uint32_t pos = l + (uint32_t)(t - s_begin[i]);
      int64_t slot = -1;
      if (s_ok[i]) {
        const uint32_t page = pos / (uint32_t)p.page_size, off = pos - page * (uint32_t)p.page_size;
        const uint32_t old = l / (uint32_t)p.page_size + (l % (uint32_t)p.page_size != 0);
        int32_t *row = p.table + (int64_t)(r0 + i) * p.table_stride;
        int32_t id;
        if (page >= old) {
          id = p.free_pages[n_free - 1 - s_before[i] - (page - old)];
          if (off == 0) row[page] = id;
        } else {
          id = row[page];
        }
        slot = id < 0 ? -1 : (int64_t)id * p.page_size + off;
      }
      p.slots[t] = slot;
      p.positions[t] = (int32_t)pos;
    }
    tokens += all;
    pages += all_need;
    __syncthreads();
  }
  // rows behind the last token
  for (int64_t t = max(t0, tokens) + tid; t < t1; t += kThreads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
  if (first && tid == 0) {
    p.cu_new[p.R] = (int32_t)min(tokens, (int64_t)INT32_MAX);
    *p.n_free_out = (int32_t)(n_free - taken);
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
  const int64_t blocks = a.max_tokens > 0 ? (a.max_tokens + kTokens - 1) / kTokens : 1;
  page_plan_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
