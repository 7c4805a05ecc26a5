// paged_call.h — the paged-cache operators as the entry points call them (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_attn.h"
#include "params.h"

namespace gqa {

// An extent of a pool with more than one entry, in bytes; below: what the narrower extents reach, at most `stride`.
struct PagedExtent {
  long long n, stride, below;
};

}  // namespace gqa

struct gqa_paged {
  int device, n_kv, dtype;
  gqa::PagedPool pool;
  int n_extents;
  gqa::PagedExtent extents[3];  // the narrowest first
  int log_box;             // slots of the maps' boxes: a power of two, at most 64, that divides the page
  CUtensorMap map_k, map_v;
};

namespace gqa {

struct PagedAppendCall {
  const void* k;
  const void* v;
  int B, T;
  long long stride_b, stride_t;
  const gqa_rope* rope;  // null: no rotation
  const int* rope_pos;   // null: kv_len
  const int* page_table;
  int max_pages;
  const int* kv_len;
  const int* n_new;      // null: T
};

// Whether the description goes with the context and a table of max_pages pages a sequence.
gqa_status check_paged(gqa_ctx* c, const gqa_paged* paged, int max_pages);

// Makes room for the attention's scratch: a caller that enqueues other work first does so before, as
// a refusal enqueues nothing.
gqa_status reserve_paged_attn(gqa_ctx* c, cudaStream_t s);

// Arguments already checked; enqueue on `s`.
gqa_status run_paged_append(gqa_ctx* c, const gqa_paged* paged, const PagedAppendCall& a, cudaStream_t s);
gqa_status run_paged_attn(gqa_ctx* c, const gqa_paged* paged, const void* q, int B, const int* page_table,
                          int max_pages, const int* kv_len, int n_new, void* h, cudaStream_t s);

}  // namespace gqa
