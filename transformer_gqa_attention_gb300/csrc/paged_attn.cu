// paged_attn.cu — instantiations of the attention over a paged cache.
#include "paged_attn.cuh"

#include "launch.h"

namespace gqa {

cudaError_t configure_paged_attn() {
  for (auto* kernel : {paged_attn_kernel<__nv_bfloat16, false>, paged_attn_kernel<__nv_bfloat16, true>,
                       paged_attn_kernel<uint8_t, false>, paged_attn_kernel<uint8_t, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PagedSmem::kBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_paged_attn(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnParams& p, int dtype, int n_ctas,
                              bool groups, cudaStream_t s) {
  auto* kernel = dtype == GQA_CACHE_BF16 ? groups ? paged_attn_kernel<__nv_bfloat16, true> : paged_attn_kernel<__nv_bfloat16, false>
                 : groups                ? paged_attn_kernel<uint8_t, true>
                                         : paged_attn_kernel<uint8_t, false>;
  return launch_pdl(kernel, dim3(n_ctas), dim3(kPagedThreads), PagedSmem::kBytes, s, 0, k, v, p);
}

}  // namespace gqa
