// The FP8 forms' products that write and read H and U kept in 8 bits (kept8.cu): per-row e4m3 and block-scaled operands.
#include "internal.h"

namespace vgg {

cudaError_t run_gate_up_swiglu_e4m3_kept8(int BN, int cn, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (BN == 256) {
    if (cn == 2)
      return launch_grouped_gemm<256, 4, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU_Q, false, 2, X_KEPT8>(p, m, grid, s);
    return launch_grouped_gemm<256, 4, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU_Q, false, 1, X_KEPT8>(p, m, grid, s);
  }
  return launch_grouped_gemm<128, 6, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU_Q, false, 1, X_KEPT8>(p, m, grid, s);
}

cudaError_t run_gate_up_swiglu_mx_kept8(int cn, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (cn == 2)
    return launch_grouped_gemm<kMxBN, 4, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU, false, 2, X_MX_KEPT8>(p, m, grid,
                                                                                                              s);
  return launch_grouped_gemm<kMxBN, 4, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU, false, 1, X_MX_KEPT8>(p, m, grid, s);
}

cudaError_t run_dact_dswiglu_e4m3_kept8(int BN, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (BN == 256 && SmemLayout<256, 4, 8, 1>::bytes(p.groups, VAR_M) <= kMaxSmem)
    return launch_grouped_gemm<256, 4, 8, 1, A_TMA_K, B_TMA_K3, VAR_M, EPI_DSWIGLU_Q, false, 1, X_KEPT8>(p, m, grid, s);
  if (BN == 256)
    return launch_grouped_gemm<256, 3, 8, 2, A_TMA_K, B_TMA_K3, VAR_M, EPI_DSWIGLU_Q, false, 1, X_KEPT8>(p, m, grid, s);
  return launch_grouped_gemm<128, 4, 8, 2, A_TMA_K, B_TMA_K3, VAR_M, EPI_DSWIGLU_Q, false, 1, X_KEPT8>(p, m, grid, s);
}

cudaError_t run_dact_dswiglu_mx_kept8(int BN, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (BN == 128)
    return launch_grouped_gemm<128, 4, 8, 2, A_TMA_K, B_TMA_K3, VAR_M, EPI_DSWIGLU, false, 1, X_MX_KEPT8>(p, m, grid, s);
  return launch_grouped_gemm<kMxBN, 4, 8, 1, A_TMA_K, B_TMA_K3, VAR_M, EPI_DSWIGLU, false, 1, X_MX_KEPT8>(p, m, grid, s);
}

}  // namespace vgg
