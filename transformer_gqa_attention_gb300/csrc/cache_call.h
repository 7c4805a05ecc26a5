// cache_call.h — the attention over caches of per-sequence length as the entry points call it
// (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_attn.h"

namespace gqa {

struct CacheAttnCall {
  int B, T, n_new, S_max;
  const uint32_t* mask;  // null: every key visible
  const int* kv_len;
  const void* q;
  const void* cache_k;
  const void* cache_v;
  void* h;
  float* weights;        // T = 1 only; null: none
};

// Makes room for the call's scratch: a caller that enqueues other work first does so before, as a
// refusal enqueues nothing.
gqa_status reserve_cache_attn(gqa_ctx* c, const CacheAttnCall& a, cudaStream_t s);

// Arguments already checked; enqueues the attention on `s`.
gqa_status run_cache_attn(gqa_ctx* c, const CacheAttnCall& a, cudaStream_t s);

}  // namespace gqa
