// Activations kept in 8 bits between the forward and the backward: the gate/up products that write H and U so (bf16 operands;
// gemm_kept8_fp8.cu has the FP8 forms'), the dSwiGLU products that read them, and the passes over whole matrices.
//
// A training step keeps X, H and U of every layer.  In fp32 H and U are 8 bytes a pair and column, the largest part by far;
// as whole numbers of 8 bits with a bf16 scale for 32 columns they are 2.125.  A thread of an epilogue holds 32 columns
// of a row, one block, so quantizing costs no exchange and the step moves 5.9 bytes a pair and column less each way.
// Against fp32 H and U (4096 x 2048 x 128 x 512 and 32768 x 1536 x 512 x 256): gate/up 182 and 508 us (186 and 529), dSwiGLU
// 155 and 528 (166 and 521; with 256 columns a tile and whole reductions in the accumulators 152 and 448), dX 154 and
// 404 (150 and 388).
#include "internal.h"

namespace vgg {

cudaError_t run_gate_up_swiglu_kept8(int BN, int cn, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (BN == 256) {
    if (cn == 2)
      return launch_grouped_gemm<256, 4, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU, false, 2, X_KEPT8>(p, m, grid, s);
    return launch_grouped_gemm<256, 4, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU, false, 1, X_KEPT8>(p, m, grid, s);
  }
  return launch_grouped_gemm<128, 6, 4, 1, A_GATHER_K, B_TMA_K3_GU, VAR_M, EPI_SWIGLU, false, 1, X_KEPT8>(p, m, grid, s);
}

cudaError_t run_dact_dswiglu_kept8(int BN, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (BN == 256 && SmemLayout<256, 4, 8, 1>::bytes(p.groups, VAR_M) <= kMaxSmem)
    return launch_grouped_gemm<256, 4, 8, 1, A_TMA_K, B_TMA_MN3, VAR_M, EPI_DSWIGLU, false, 1, X_KEPT8>(p, m, grid, s);
  if (BN == 256)
    return launch_grouped_gemm<256, 3, 8, 2, A_TMA_K, B_TMA_MN3, VAR_M, EPI_DSWIGLU, false, 1, X_KEPT8>(p, m, grid, s);
  return launch_grouped_gemm<128, 4, 8, 2, A_TMA_K, B_TMA_MN3, VAR_M, EPI_DSWIGLU, false, 1, X_KEPT8>(p, m, grid, s);
}

// dXp = [dH | dU] [W_gate[e]; W_up[e]] in scaled fp16 for the sum over a token's pairs.
cudaError_t run_dx_store_f16s(int BN, const GemmParams& p, const Maps& m, int grid, cudaStream_t s) {
  if (BN == 256) return launch_grouped_gemm<256, 4, 4, 1, A_TMA_K, B_TMA_MN3, VAR_M, EPI_STORE, false, 1, X_F16S>(p, m, grid, s);
  return launch_grouped_gemm<128, 6, 4, 1, A_TMA_K, B_TMA_MN3, VAR_M, EPI_STORE, false, 1, X_F16S>(p, m, grid, s);
}

// A matrix of bf16 values to codes and scales.  Four lanes have a block's 32 columns, 8 (16 bytes) each: loads and stores
// are contiguous over the warp.  Rows are whole blocks, so the matrix is one run of them.  32768 x 1536 35 us with its
// events (154 MB, 4.4 TB/s, two thirds of the copy rate), the way back 30: a thread has one load in flight, and two
// exchanges and a division behind it before the next.
__global__ void __launch_bounds__(256) keep_rows8_kernel(const __nv_bfloat16* __restrict__ M, long long n8,
                                                         uint8_t* __restrict__ q, __nv_bfloat16* __restrict__ scale) {
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < n8; i += step) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(M) + i);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16x2(w[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
    float amax = max_abs_nan(v);
    // n8 and the step are multiples of 4: the four lanes of a block are in the loop together
    const unsigned quad = 0xFu << (threadIdx.x & 28);
    amax = max_abs_nan(amax, __shfl_xor_sync(quad, amax, 1));
    amax = max_abs_nan(amax, __shfl_xor_sync(quad, amax, 2));
    float inv;
    const uint32_t bits = kept8_scale(amax, inv);
    reinterpret_cast<uint2*>(q)[i] =
        make_uint2(kept8_x4(v[0], v[1], v[2], v[3], inv), kept8_x4(v[4], v[5], v[6], v[7], inv));
    if ((threadIdx.x & 3) == 0) reinterpret_cast<uint16_t*>(scale)[i >> 2] = static_cast<uint16_t>(bits);
  }
}

__global__ void __launch_bounds__(256) read_rows8_kernel(const uint8_t* __restrict__ q, const __nv_bfloat16* __restrict__ scale,
                                                         long long n8, __nv_bfloat16* __restrict__ M) {
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < n8; i += step) {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(q) + i);
    const float s = __bfloat162float(__ldg(scale + (i >> 2)));
    const uint2 a = kept8_values4(c.x, s), b = kept8_values4(c.y, s);
    reinterpret_cast<uint4*>(M)[i] = make_uint4(a.x, a.y, b.x, b.y);
  }
}

static unsigned rows8_grid(long long n8) {
  const long long want = (n8 + 255) / 256;
  return static_cast<unsigned>(want < 152 * 64 ? want : 152 * 64);
}

cudaError_t launch_keep_rows8(const __nv_bfloat16* M, long long n, uint8_t* q, __nv_bfloat16* scale, cudaStream_t s) {
  if (n > 0) keep_rows8_kernel<<<rows8_grid(n / 8), 256, 0, s>>>(M, n / 8, q, scale);
  return cudaGetLastError();
}

cudaError_t launch_read_rows8(const uint8_t* q, const __nv_bfloat16* scale, long long n, __nv_bfloat16* M, cudaStream_t s) {
  if (n > 0) read_rows8_kernel<<<rows8_grid(n / 8), 256, 0, s>>>(q, scale, n / 8, M);
  return cudaGetLastError();
}

}  // namespace vgg
