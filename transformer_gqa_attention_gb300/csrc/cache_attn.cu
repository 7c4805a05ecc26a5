// cache_attn.cu — instantiations of the attention over caches of per-sequence length.
#include "cache_attn.cuh"
#include "cache_attn_pair.cuh"
#include "cache_decode.cuh"
#include "cache_merge.cuh"
#include "launch.h"

namespace gqa {

namespace {

// The attention kernel of a call: the decode step with key weights, one 128-row tile of up to 32
// positions, or CTA pairs.
using CacheAttnFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CacheAttnParams);
struct CacheAttnKernel {
  CacheAttnFn fn;
  int smem;
};

CacheAttnKernel attn_of(const CacheAttnParams& p) {
  if (p.weights) return {cache_decode_kernel, CacheDecodeSmem::kBytes};
  if (p.T <= kOneTilePos) return {cache_attn_kernel, CacheAttnSmem::kBytes};
  return {cache_attn_pair_kernel, CachePairSmem::kBytes};
}

}  // namespace

cudaError_t configure_cache_attn() {
  cudaError_t e = cudaFuncSetAttribute(cache_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       CacheDecodeSmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(cache_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CacheAttnSmem::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(cache_attn_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CachePairSmem::kBytes);
}

cudaError_t launch_cache_attn(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              const CacheAttnParams& p, int n_ctas, cudaStream_t s) {
  const CacheAttnKernel a = attn_of(p);
  return launch_pdl(a.fn, dim3(n_ctas), dim3(384), a.smem, s, 0, q, k, v, p);
}

cudaError_t launch_cache_merge(const CacheAttnParams& p, int workers, cudaStream_t s) {
  return launch_pdl(cache_merge_kernel, dim3(workers, kMergeY), dim3(256), 0, s, 0, p);
}

cudaError_t launch_cache_weights(const CacheAttnParams& p, int workers, int n_blocks, cudaStream_t s) {
  return launch_pdl(cache_weights_kernel, dim3(workers + n_blocks), dim3(256), 0, s, 0, p, workers);
}

}  // namespace gqa
