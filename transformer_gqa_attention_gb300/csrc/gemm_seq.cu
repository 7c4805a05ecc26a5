// gemm_seq.cu — the Q/K/V projections whose sequences have their own starts in the cache
// (GemmSeqParams::seq_start).  A translation unit of their own: beside them in gemm_launch.cu the other
// instantiations start 0.2 to 0.5 us later in steps of 32 to 139 us.
#include "gemm_rings.cuh"

namespace gqa {

cudaError_t configure_gemm_seq_kernels() {
  cudaError_t e = cudaFuncSetAttribute(gemm_tc_pair_kernel<6, kQkvRopeSeq>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PairSmem::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_splitk_cluster_kernel<kSplitKQkvSeq, kSkinnyStages, 64>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, SkinnySmem::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gemm_splitk_cluster_kernel<kSplitKQkvSeq, kNarrowStages, 32>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowSmem::kBytes);
}

cudaError_t launch_gemm_qkv_rope_seq(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& bt,
                                     const GemmSeqParams& p, int grid, cudaStream_t s) {
  return launch_pdl(gemm_tc_pair_kernel<6, kQkvRopeSeq>, dim3(grid), dim3(192), PairSmem::kBytes, s, 0, a, b, bt, p);
}

cudaError_t launch_gemm_splitk_qkv_seq(const CUtensorMap& a, const CUtensorMap& b, const GemmSeqParams& p,
                                       cudaStream_t s) {
  return launch_splitk<kSplitKQkvSeq>(a, b, p, s);
}

}  // namespace gqa
