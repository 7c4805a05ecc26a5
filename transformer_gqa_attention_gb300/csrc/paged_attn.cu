// paged_attn.cu — instantiations of the attention over a paged cache.
#include "paged_attn.cuh"

#include "launch.h"

namespace gqa {

cudaError_t configure_paged_attn() {
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PagedSmem::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(paged_attn_kernel<uint8_t>, cudaFuncAttributeMaxDynamicSharedMemorySize, PagedSmem::kBytes);
}

cudaError_t launch_paged_attn(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnParams& p, int dtype, int n_ctas,
                              cudaStream_t s) {
  auto* kernel = dtype == GQA_CACHE_BF16 ? paged_attn_kernel<__nv_bfloat16> : paged_attn_kernel<uint8_t>;
  return launch_pdl(kernel, dim3(n_ctas), dim3(kPagedThreads), PagedSmem::kBytes, s, 0, k, v, p);
}

}  // namespace gqa
