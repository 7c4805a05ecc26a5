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

// Blocks per worker: a warp of eight for each task of 32 rows x 16 columns that a unit may have.  With 2,
// 4 and 8, us: 9.8, 10.1, 10.2 for one sequence of 300 keys and 8 tokens (a block has all its tasks), 25.7, 23.6, 24.9 for
// 8 ragged ones and 26 (four), 18.8, 14.7, 12.5 for one of 300 and 64 (eight).
static int merge_blocks(const CacheAttnParams& p) { return p.part_rows / 32; }

cudaError_t launch_cache_merge(const CacheAttnParams& p, int workers, cudaStream_t s) {
  return launch_pdl(cache_merge_kernel, dim3(workers, merge_blocks(p)), dim3(256), 0, s, 0, p);
}

cudaError_t launch_cache_weights(const CacheAttnParams& p, int workers, int n_blocks, cudaStream_t s) {
  return launch_pdl(cache_weights_kernel, dim3(workers + n_blocks), dim3(256), 0, s, 0, p, workers);
}

}  // namespace gqa
