// gemm_launch.cu — instantiations of the tcgen05 GEMMs: CTA-pair kernels for many tokens,
// split-K kernels (with their fused reductions) for few tokens.
#include "gemm_rings.cuh"

namespace gqa {

cudaError_t configure_gemm_kernels() {
  cudaError_t e;
  e = cudaFuncSetAttribute(gemm_tc_pair_kernel<6, kQkvRope>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           PairSmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_tc_pair_kernel<6, kStoreF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           PairSmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_splitk_cluster_kernel<kSplitKQkv, kSkinnyStages, 64>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, SkinnySmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_splitk_cluster_kernel<kSplitKOut, kDeepStages, 64>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, DeepSmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_splitk_cluster_kernel<kSplitKQkv, kNarrowStages, 32>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowSmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_splitk_cluster_kernel<kSplitKOut, kNarrowStages, 32>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowSmem::kBytes);
  if (e != cudaSuccess) return e;
  return configure_gemm_seq_kernels();
}

int gemm_pair_max_clusters() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(192, 1, 1);
  cfg.dynamicSmemBytes = PairSmem::kBytes;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_tc_pair_kernel<6, kQkvRope>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_gemm_qkv_rope(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& bt,
                                 const GemmParams& p, int grid, cudaStream_t s) {
  return launch_pdl(gemm_tc_pair_kernel<6, kQkvRope>, dim3(grid), dim3(192), PairSmem::kBytes, s, 0, a, b, bt, p);
}

cudaError_t launch_gemm_store_f32(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& bt,
                                  const GemmParams& p, int grid, cudaStream_t s) {
  return launch_pdl(gemm_tc_pair_kernel<6, kStoreF32>, dim3(grid), dim3(192), PairSmem::kBytes, s, 0, a, b, bt, p);
}

int splitk_token_tile(int n_tok) { return n_tok <= 32 ? 32 : 64; }

cudaError_t launch_gemm_splitk_qkv(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p,
                                   cudaStream_t s) {
  return launch_splitk<kSplitKQkv>(a, b, p, s);
}

cudaError_t launch_gemm_splitk_out(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p,
                                   cudaStream_t s) {
  return launch_splitk<kSplitKOut>(a, b, p, s);
}

}  // namespace gqa
