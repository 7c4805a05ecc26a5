// paged_attn.cu — instantiations of the attention over a paged cache.
#include "paged_attn.cuh"

#include "launch.h"

namespace gqa {

cudaError_t configure_paged_attn() { return cudaSuccess; }

cudaError_t launch_paged_attn(const PagedAttnParams& p, int dtype, cudaStream_t s) {
  const dim3 grid(p.n_kv, p.B);
  return dtype == GQA_CACHE_BF16 ? launch_pdl(paged_attn_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 0, p)
                                 : launch_pdl(paged_attn_kernel<uint8_t>, grid, dim3(256), 0, s, 0, p);
}

}  // namespace gqa
