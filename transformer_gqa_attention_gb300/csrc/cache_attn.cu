// cache_attn.cu — instantiations of the attention over caches of per-sequence length.
#include "cache_attn.cuh"
#include "launch.h"

namespace gqa {

cudaError_t configure_cache_attn() {
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       CacheAttnSmem<false>::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(cache_attn_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           CacheAttnSmem<false>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(cache_attn_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              CacheAttnSmem<true>::kBytes);
}

cudaError_t launch_cache_attn(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              const CacheAttnParams& p, int n_ctas, cudaStream_t s) {
  const dim3 grid(n_ctas), block(384);
  if (p.group_pos > 32) return launch_pdl(cache_attn_kernel<true, false>, grid, block, CacheAttnSmem<true>::kBytes, s, 0, q, k, v, p);
  if (p.weights) return launch_pdl(cache_attn_kernel<false, true>, grid, block, CacheAttnSmem<false>::kBytes, s, 0, q, k, v, p);
  return launch_pdl(cache_attn_kernel<false, false>, grid, block, CacheAttnSmem<false>::kBytes, s, 0, q, k, v, p);
}

cudaError_t launch_cache_finish(const CacheAttnParams& p, int n_ctas, cudaStream_t s) {
  if (p.weights) return launch_pdl(cache_finish_kernel<true>, dim3(n_ctas), dim3(256), 0, s, 0, p);
  return launch_pdl(cache_finish_kernel<false>, dim3(n_ctas, p.part_rows / 32), dim3(256), 0, s, 0, p);
}

}  // namespace gqa
