// The elementwise steps of the router's gradient products: dlogits into two bf16 parts, and the split-K sums.
#include "internal.h"

namespace vgg {

// Four values a thread (E is a multiple of 8).
__global__ void __launch_bounds__(256) split_dlogits_kernel(const float* __restrict__ dl, long long n, long long np,
                                                            __nv_bfloat16* __restrict__ hi,
                                                            __nv_bfloat16* __restrict__ lo) {
  const long long step = 4ll * gridDim.x * blockDim.x;
  for (long long i = 4ll * (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x); i < np; i += step) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < n) v = __ldcs(reinterpret_cast<const float4*>(dl + i));
    const uint2 h = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    const float2 a = unpack_bf16x2(h.x), b = unpack_bf16x2(h.y);
    *reinterpret_cast<uint2*>(hi + i) = h;
    *reinterpret_cast<uint2*>(lo + i) = make_uint2(pack_bf16x2(v.x - a.x, v.y - a.y), pack_bf16x2(v.z - b.x, v.w - b.y));
  }
}

cudaError_t launch_split_dlogits(const float* dlogits, long long T, long long Tp, int E, __nv_bfloat16* hi,
                                 __nv_bfloat16* lo, cudaStream_t s) {
  const long long np = Tp * E, want = (np / 4 + 255) / 256;
  if (np > 0) split_dlogits_kernel<<<static_cast<unsigned>(want < 8192 ? want : 8192), 256, 0, s>>>(dlogits, T * E, np, hi, lo);
  return cudaGetLastError();
}

__global__ void __launch_bounds__(256) splitk_reduce_add_kernel(const float* __restrict__ part, int splits, long long n,
                                                                const float* in, float* out) {
  const long long i = 4ll * (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x);
  if (i >= n) return;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < splits; ++s) {
    const float4 b = __ldcs(reinterpret_cast<const float4*>(part + s * n + i));
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  if (in) {
    const float4 b = *reinterpret_cast<const float4*>(in + i);
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  *reinterpret_cast<float4*>(out + i) = a;
}

cudaError_t launch_splitk_reduce_add(const float* part, int splits, long long n, const float* in, float* out,
                                     cudaStream_t s) {
  if (n > 0)
    splitk_reduce_add_kernel<<<static_cast<unsigned>((n / 4 + 255) / 256), 256, 0, s>>>(part, splits, n, in, out);
  return cudaGetLastError();
}

}  // namespace vgg
