// cache_attn.cu — instantiations of the attention over caches of per-sequence length.
#include <algorithm>

#include "cache_attn.cuh"
#include "cache_attn_few.cuh"
#include "cache_attn_pair.cuh"
#include "cache_merge.cuh"
#include "launch.h"

namespace gqa {

namespace {

// The attention kernel of a call and its shared memory: by positions per sequence, up to 16 keys on
// the tensor core's rows, up to 32 one row tile, above CTA pairs.
using CacheAttnFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CacheAttnParams);
constexpr CacheAttnFn kAttn[] = {cache_attn_few_kernel<4, true>,   cache_attn_few_kernel<4, false>,
                                 cache_attn_few_kernel<16, false>, cache_attn_few_kernel<32, false>,
                                 cache_attn_few_kernel<64, false>, cache_attn_kernel,
                                 cache_attn_pair_kernel};
constexpr int kFewKernels = 5;

int attn_of(const CacheAttnParams& p) {
  if (p.T == 1) return p.weights ? 0 : 1;
  return p.T <= 4 ? 2 : p.T <= 8 ? 3 : p.T <= kFewPos ? 4 : p.T <= kOneTilePos ? 5 : 6;
}

int smem_of(int kernel) {
  return kernel < kFewKernels ? CacheFewSmem::kBytes : kernel == kFewKernels ? CacheAttnSmem::kBytes : CachePairSmem::kBytes;
}

}  // namespace

cudaError_t configure_cache_attn() {
  for (int i = 0; i < static_cast<int>(sizeof(kAttn) / sizeof(kAttn[0])); ++i) {
    cudaError_t e = cudaFuncSetAttribute(kAttn[i], cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(i));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Positions of a query tensor map's box: the rows that the kernel's queries take, / 4.
int cache_attn_box(const CacheAttnParams& p) {
  constexpr int box[] = {1, 1, 4, 8, 16, 32, 32};
  return box[attn_of(p)];
}

cudaError_t launch_cache_attn(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              const CacheAttnParams& p, int n_ctas, cudaStream_t s) {
  const int i = attn_of(p);
  return launch_pdl(kAttn[i], dim3(n_ctas), dim3(384), smem_of(i), s, 0, q, k, v, p);
}

cudaError_t launch_cache_merge(const CacheAttnParams& p, int workers, cudaStream_t s) {
  if (p.T <= kFewPos)
    return launch_pdl(cache_merge_kernel<true>, dim3(workers, std::min(p.T, kMergeFewY)), dim3(256), 0, s, 0, p);
  return launch_pdl(cache_merge_kernel<false>, dim3(workers, kMergeY), dim3(256), 0, s, 0, p);
}

cudaError_t launch_cache_weights(const CacheAttnParams& p, int workers, int n_blocks, cudaStream_t s) {
  return launch_pdl(cache_weights_kernel, dim3(workers + n_blocks), dim3(256), 0, s, 0, p, workers);
}

}  // namespace gqa
