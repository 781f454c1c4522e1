// Page plan of a batch (sm_100a): block-table rows, slots and positions of
// the tokens a step adds, from the requests' cached and new lengths.
//
// With cu the exclusive prefix sum of the new lengths and pages(l) =
// ceil(l / P), request r needs pages(lens + new) - pages(lens) pages, and the
// exclusive prefix sum of the needs is its place in the free list, which is
// popped from its end.  Token t of request r stands at lens_r + t - cu_r.
//
// One launch: every block takes a range of token rows and repeats the two
// prefix sums (both in one pass, but where token rows run out) for the
// requests up to that range, four requests per thread and a tile of 2048 at a
// time, so nothing is exchanged between blocks.  The
// tokens of a tile find their request by binary search in the tile's sums.  A
// new page's first token is always one of this call's tokens, and its thread
// writes the page's block-table entry; a page's id is read from the free list
// itself by every token of a new page, and from the table only for pages that
// were there before, so no thread reads an entry that another one writes.
//
// Bound by its launch and the chain of loads, scan and search, not by bytes:
// 16 requests 5.1 us, 257 requests 6.5 us, 2048 requests with new prompts (5 MB
// in and out) 14.4 us.

#include "tq_paged.h"

namespace tq {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;                // requests per thread
constexpr int kTile = kThreads * kPer; // requests per tile
constexpr int kTokens = 2 * kThreads;  // token rows per block

// Exclusive prefix sums of two values over the block, and their totals.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t (*s_warp)[2], int64_t &ta, int64_t &tb) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    s_warp[w][0] = x;
    s_warp[w][1] = y;
  }
  __syncthreads();
  int64_t ba = 0, bb = 0;
  ta = tb = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int64_t u = s_warp[i][0], v = s_warp[i][1];
    if (i < w) {
      ba += u;
      bb += v;
    }
    ta += u;
    tb += v;
  }
  a = ba + x - a;
  b = bb + y - b;
}

__device__ __forceinline__ uint32_t pages(uint32_t tokens, uint32_t page) {
  return tokens / page + (tokens % page != 0);
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(PagePlanArgs p) {
  __shared__ int64_t s_warp[kThreads / 32][2];
  __shared__ int32_t s_begin[kTile];   // first token of each request of the tile (INT32_MAX at most)
  __shared__ int32_t s_before[kTile];  // its place in the free list, -1 where it was refused
  __shared__ int32_t s_len[kTile];
  __shared__ int s_taken;
  const int tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int64_t t1 = min(t0 + kTokens, p.max_tokens);
  const uint32_t P = (uint32_t)p.page_size;
  const int64_t n_free = min((int64_t)max(*p.n_free, 0), p.free_cap);
  if (tid == 0) s_taken = 0;

  int64_t tokens = 0, taken = 0;  // token rows and wanted pages of the tiles before
  for (int r0 = 0; r0 < p.R; r0 += kTile) {
    // block 0 goes through all requests; another block stops behind its range
    if (!first && tokens >= t1) break;
    const int n = min(kTile, p.R - r0);
    uint32_t len[kPer], add[kPer], had[kPer], need[kPer];
    bool fits[kPer];
    int64_t sum_t = 0, sum_p = 0, all_t, all_p;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid * kPer + k;
      len[k] = i < n ? (uint32_t)max(p.lens[r0 + i], 0) : 0u;
      add[k] = i < n ? (uint32_t)max(p.new_lens[r0 + i], 0) : 0u;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      had[k] = pages(len[k], P);
      const uint32_t has = pages(len[k] + add[k], P);  // at most 2^32 - 2 tokens
      fits[k] = has <= (uint32_t)p.max_pages;
      need[k] = fits[k] ? has - had[k] : 0u;
      sum_t += add[k];
      sum_p += need[k];
    }
    int64_t begin = sum_t, before = sum_p;
    block_scan2(begin, before, s_warp, all_t, all_p);
    begin += tokens;
    // too few token rows: the pages of the requests that do not fit them are not wanted
    bool over = false;
    int64_t at = begin;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      at += add[k];
      if (at > p.max_tokens && fits[k]) {
        over = true;
        fits[k] = false;
        sum_p -= need[k];
        need[k] = 0;
      }
    }
    if (__syncthreads_or(over)) {
      int64_t none = 0, t;
      before = sum_p;
      block_scan2(before, none, s_warp, all_p, t);
    }
    before += taken;
    int most = 0;  // pages taken up to here
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = tid * kPer + k;
      const bool paid = need[k] == 0 || before + need[k] <= n_free, ok = fits[k] && paid;
      if (ok && need[k]) most = (int)(before + need[k]);
      s_begin[i] = (int32_t)min(begin, (int64_t)INT32_MAX);
      s_before[i] = ok ? (int32_t)min(before, (int64_t)INT32_MAX) : -1;
      s_len[i] = (int32_t)len[k];
      if (first && i < n) {
        p.cu_new[r0 + i] = (int32_t)min(begin, (int64_t)INT32_MAX);
        p.seq_lens[r0 + i] = (int32_t)(ok ? len[k] + add[k] : len[k]);
        p.status[r0 + i] = !fits[k] ? 2 : paid ? 0 : 1;
      }
      begin += add[k];
      before += need[k];
    }
    if (first && most) atomicMax(&s_taken, most);
    __syncthreads();
    // the block's tokens among this tile's
    const int64_t lo = max(t0, tokens), hi = min(t1, tokens + all_t);
    for (int64_t t = lo + tid; t < hi; t += kThreads) {
      int i = 0, j = n;  // the last request i of the tile with s_begin[i] <= t
      while (j - i > 1) {
        const int m = (i + j) >> 1;
        if (s_begin[m] <= t) i = m; else j = m;
      }
      const uint32_t l = (uint32_t)s_len[i], pos = l + (uint32_t)(t - s_begin[i]);
      const int32_t free_at = s_before[i];
      int64_t slot = -1;
      if (free_at >= 0) {
        const uint32_t page = pos / P, off = pos - page * P, old = pages(l, P);
        int32_t *row = p.table + (int64_t)(r0 + i) * p.table_stride;
        int32_t id;
        if (page >= old) {
          id = p.free_pages[n_free - 1 - free_at - (page - old)];
          if (off == 0) row[page] = id;
        } else {
          id = row[page];
        }
        slot = id < 0 ? -1 : (int64_t)id * P + off;
        if (id < 0) atomicOr(p.faults, kFaultIndex);  // an accepted token without a place
      }
      p.slots[t] = slot;
      p.positions[t] = (int32_t)pos;
    }
    tokens += all_t;
    taken += all_p;
    __syncthreads();
  }
  // rows behind the last token
  for (int64_t t = max(t0, tokens) + tid; t < t1; t += kThreads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
  if (first) {
    __syncthreads();
    if (tid == 0) {
      p.cu_new[p.R] = (int32_t)min(tokens, (int64_t)INT32_MAX);
      *p.n_free_out = (int32_t)(n_free - s_taken);
    }
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
  const int64_t blocks = a.max_tokens > 0 ? (a.max_tokens + kTokens - 1) / kTokens : 1;
  PagePlanArgs p = a;
  const cudaError_t e = fault_word(&p.faults);
  if (e != cudaSuccess) return e;
  page_plan_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tq
