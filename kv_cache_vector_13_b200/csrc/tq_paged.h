// Internal interface of the paged-cache calls: tq_host.cpp validates, the
// tq_paged_*.cu launchers run.  Not installed.
#pragma once

#include "tq_internal.h"

namespace tq {

// A slot or a block-table entry outside the cache: the access is skipped.
constexpr unsigned kFaultIndex = 4u;

struct PagePlanArgs {
  int R, page_size, max_pages;
  const int32_t *lens, *new_lens, *free_pages, *n_free;
  int64_t free_cap;
  int32_t *table;
  int64_t table_stride;
  int64_t max_tokens;
  int64_t *slots;
  int32_t *positions, *cu_new, *seq_lens, *status, *n_free_out;
  unsigned *faults;       // the launcher's
};

struct PagedAppendArgs {
  QuantParams kq, vq;
  int dtype;
  int64_t T;
  int Hq, Hkv;            // Hq = 0: no query rows
  const void *q, *k, *v;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // element strides (token, head)
  void *q_out;            // [T][Hq][d]
  CacheView kc, vc;       // sb = page stride
  int64_t n_slots;        // n_pages * page_size
  int page_size;
  const int64_t *slots;
  int rot_dim;            // 0: no rotary positions
  bool adjacent;
  const float *inv_freq;  // rot_dim / 2
  const int32_t *axis;    // rot_dim / 2, or NULL (all 0)
  int n_axes;
  const int32_t *positions;  // [n_axes][T], row stride pos_stride
  int64_t pos_stride;
};

struct PagedDequantArgs {
  QuantParams q;
  CacheView c;
  int64_t T;
  int H;
  int64_t n_slots;
  int page_size;
  const int64_t *slots;
  int out_dtype;
  void *out;              // [T][H][d]
};

struct PagedAttentionArgs {
  QuantParams kq, vq;
  int dtype;
  const void *q;
  int64_t T;
  int Hq, Hkv;
  int64_t q_st, q_sh;
  CacheView k, v;
  int64_t n_pages;
  int page_size;
  const int32_t *table;
  int64_t table_stride;
  int R, max_pages;
  const int32_t *kv_lens;
  const int32_t *cu_q;    // NULL: one query row per request
  int max_q;
  float scale;
  bool causal;
  int window;             // 0: none
  void *out;              // [T][Hq][d], q's dtype
  float *lse;             // [T][Hq] or NULL
  void *ws;
};

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s);
cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t s);
cudaError_t launch_paged_dequant(const PagedDequantArgs &a, cudaStream_t s);
size_t paged_attention_workspace(int R, int64_t T, int Hq, int Hkv, int d);
cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t s);
// d = 64 and 128 on tensor cores, a few query rows a unit (tq_paged_rows.cu)
size_t paged_rows_workspace(int d);
cudaError_t launch_paged_rows(const PagedAttentionArgs &a, cudaStream_t s);
// d = 64 and 128 on the fifth-generation tensor cores, 128 or 256 query rows a unit (tq_paged_tile.cu)
size_t paged_tile_workspace(int R, int64_t T, int Hq, int Hkv, int d);
cudaError_t launch_paged_tile(const PagedAttentionArgs &a, cudaStream_t s);

}  // namespace tq
