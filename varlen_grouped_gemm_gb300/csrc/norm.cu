// Residual addition with root-mean-square norm and an optional 8-bit output, and its backward.
//
//   h = r + x (rounded to the residual stream's type),  rstd = (mean_j h_j^2 + eps)^(-1/2),
//   y_j = h_j rstd g_j  (bf16),  q = e4m3 codes of the fp32 y with one fp32 scale a row (max|y| / 448), or
//   with one power of two for every 32 columns.
//
// The codes come from the fp32 y, not from its bf16 rounding: one rounding instead of two.
//
// Both directions move every element once and are bound by HBM.  A row's values stay in registers between the
// reduction and the output: thread i of the row's TPR threads holds the 16-byte vectors i, i + TPR, ... (NV of
// them).
#include "internal.h"

namespace vgg {

namespace {

// Eight consecutive values of a bf16 or fp32 row (16-byte aligned), as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* base, long long off, float (&v)[8]) {
  if (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16x2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, long long off, const float (&v)[8]) {
  if (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 q;
    q.x = pack_bf16x2(v[0], v[1]);
    q.y = pack_bf16x2(v[2], v[3]);
    q.z = pack_bf16x2(v[4], v[5]);
    q.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) = q;
  }
}

// V = 8 consecutive values by vector accesses, or V = 1 value (rows of any width and alignment).
template <int V, bool F32>
__device__ __forceinline__ void load_v(const void* base, long long off, float (&v)[V]) {
  if constexpr (V == 8) load8<F32>(base, off, v);
  else v[0] = F32 ? static_cast<const float*>(base)[off] : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off]);
}

template <int V, bool F32>
__device__ __forceinline__ void store_v(void* base, long long off, const float (&v)[V]) {
  if constexpr (V == 8) store8<F32>(base, off, v);
  else if (F32) static_cast<float*>(base)[off] = v[0];
  else static_cast<__nv_bfloat16*>(base)[off] = __float2bfloat16_rn(v[0]);
}

template <int V>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int j, float (&v)[V]) {
  if (f32) {
    if constexpr (V == 8) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + j);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = __ldg(static_cast<const float*>(w) + j);
    }
  } else {
    if constexpr (V == 8) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + j));
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
      v[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(w)[j]);
    }
  }
}

// Sum (or maximum) of v over the blockDim.x threads of a row, the same value in every one of them.  `red` holds a
// float for each warp of the block; one __syncthreads when a row has more than one warp, so the next use of
// the same `red` needs another barrier in between.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  const int w0 = threadIdx.y * nw, lane = threadIdx.x & 31;
  if (lane == 0) red[w0 + (threadIdx.x >> 5)] = v;
  __syncthreads();
  v = lane < nw ? red[w0 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  return v;
}

enum NormForm { NORM_BF16 = 0, NORM_E4M3 = 1, NORM_MX = 2 };

template <int V, int NV, bool RES32, int FORM>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormFwd a) {
  __shared__ float red_sum[32], red_max[32];
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool row_ok = t < a.T;
  const int nvec = a.d / V;
  float h[NV][V];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (row_ok && j < nvec) {
      load_v<V, RES32>(a.res, t * a.ld_res + static_cast<long long>(j) * V, h[i]);
      if (a.x) {
        float x[V];
        load_v<V, false>(a.x, t * a.ld_x + static_cast<long long>(j) * V, x);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          h[i][k] += x[k];
          if (!RES32) h[i][k] = bf16_round(h[i][k]);  // the norm's input is the stream as it is stored
        }
      }
      if (a.h) store_v<V, RES32>(a.h, t * a.ld_h + static_cast<long long>(j) * V, h[i]);
#pragma unroll
      for (int k = 0; k < V; ++k) ss += h[i][k] * h[i][k];
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) h[i][k] = 0.0f;
    }
  }
  ss = row_reduce<false>(ss, red_sum);
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
  if (a.rstd && row_ok && threadIdx.x == 0) a.rstd[t] = rstd;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (row_ok && j < nvec) {
      float g[V];
      load_weight<V>(a.weight, a.weight_f32 != 0, j * V, g);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        h[i][k] = h[i][k] * rstd * g[k];
        amax = fmaxf(amax, fabsf(h[i][k]));
      }
      if (a.y) store_v<V, false>(a.y, t * a.ld_y + static_cast<long long>(j) * V, h[i]);
    }
  }
  if constexpr (FORM == NORM_E4M3 && V == 8) {
    amax = row_reduce<true>(amax, red_max);
    const float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (row_ok && threadIdx.x == 0) a.scales[t] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (row_ok && j < nvec) {
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] = __fdiv_rn(h[i][k], s);
        *reinterpret_cast<uint2*>(a.q + t * a.d + 8ll * j) =
            make_uint2(e4m3x4(h[i][0], h[i][1], h[i][2], h[i][3]), e4m3x4(h[i][4], h[i][5], h[i][6], h[i][7]));
      }
    }
  }
  if constexpr (FORM == NORM_MX && V == 8) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      // four neighbouring lanes hold a block of 32 columns
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) m = fmaxf(m, fabsf(h[i][k]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = mx_exponent(m);
      const float inv = mx_inv_scale(e);
      if (row_ok && j < nvec) {
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] *= inv;
        *reinterpret_cast<uint2*>(a.q + t * a.d + 8ll * j) =
            make_uint2(e4m3x4(h[i][0], h[i][1], h[i][2], h[i][3]), e4m3x4(h[i][4], h[i][5], h[i][6], h[i][7]));
        if ((j & 3) == 0) a.sf[t * a.sf_ld + (j >> 2)] = static_cast<uint8_t>(e + 127);
      }
    }
    // bytes past the last block of the row hold scale 1
    for (int b = (a.d >> 5) + threadIdx.x; row_ok && b < a.sf_ld; b += blockDim.x) a.sf[t * a.sf_ld + b] = 127;
  }
}

template <int V, int NV, bool RES32>
cudaError_t run_norm_form(const NormFwd& a, int tpr, int rows, cudaStream_t s) {
  const dim3 block(tpr, rows);
  const unsigned grid = static_cast<unsigned>((a.T + rows - 1) / rows);
  if (V == 1 || a.form == NORM_BF16) add_rmsnorm_kernel<V, NV, RES32, NORM_BF16><<<grid, block, 0, s>>>(a);
  else if (a.form == NORM_E4M3) add_rmsnorm_kernel<V, NV, RES32, NORM_E4M3><<<grid, block, 0, s>>>(a);
  else add_rmsnorm_kernel<V, NV, RES32, NORM_MX><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

template <int V, int NV>
cudaError_t run_norm(const NormFwd& a, int tpr, int rows, cudaStream_t s) {
  return a.res_f32 ? run_norm_form<V, NV, true>(a, tpr, rows, s) : run_norm_form<V, NV, false>(a, tpr, rows, s);
}

inline int round32(int x) { return (x + 31) & ~31; }

}  // namespace

cudaError_t launch_add_rmsnorm(const NormFwd& a, bool vec, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  if (!vec) return run_norm<1, 16>(a, round32((a.d + 15) / 16), 1, s);
  const int nvec = a.d / 8;
  if (nvec <= 1024) return run_norm<8, 1>(a, round32(nvec), 1, s);
  return run_norm<8, 2>(a, round32((nvec + 1) / 2), 1, s);
}

// ------------------------------------------------------------------------------------------- backward
//
//   xhat = h rstd,  c = mean_j(dy_j g_j xhat_j),  dh_j = up_j + rstd (dy_j g_j - c xhat_j),
//   dg_j = sum_t dy_tj xhat_tj
//
// A block takes the rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps its share of dg in registers (a thread's
// columns never change); the shares go to part[block][d] and a second launch adds them in block order, so dg
// has one summation order whatever runs first.

namespace {

template <int V, int NV, bool RES32>
__global__ void __launch_bounds__(512) add_rmsnorm_bwd_kernel(const NormBwd a) {
  __shared__ float red[2][32];
  const int nvec = a.d / V;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float g[NV][V], dg[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
#pragma unroll
    for (int k = 0; k < V; ++k) g[i][k] = dg[i][k] = 0.0f;
    if (j < nvec) load_weight<V>(a.weight, a.weight_f32 != 0, j * V, g[i]);
  }
  int it = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++it) {
    const float rstd = __ldg(a.rstd + t);
    float dy[NV][V], h[NV][V];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < nvec) {
        load_v<V, false>(a.dy, t * a.ld_dy + static_cast<long long>(j) * V, dy[i]);
        load_v<V, RES32>(a.h, t * a.ld_h + static_cast<long long>(j) * V, h[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          h[i][k] *= rstd;
          dg[i][k] += dy[i][k] * h[i][k];
          dy[i][k] *= g[i][k];
          c += dy[i][k] * h[i][k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) dy[i][k] = h[i][k] = 0.0f;
      }
    }
    c = row_reduce<false>(c, red[it & 1]) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < nvec) {
        float o[V];
        if (a.dh) load_v<V, RES32>(a.dh, t * a.ld_dh + static_cast<long long>(j) * V, o);
        else {
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] += rstd * (dy[i][k] - c * h[i][k]);
        if (a.dx) store_v<V, false>(a.dx, t * a.ld_dx + static_cast<long long>(j) * V, o);
        if (a.dres) store_v<V, RES32>(a.dres, t * a.ld_dres + static_cast<long long>(j) * V, o);
      }
    }
  }
  float* out = gridDim.x == 1 ? a.dweight : a.part + static_cast<long long>(blockIdx.x) * a.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (j < nvec) {
#pragma unroll
      for (int k = 0; k < V; ++k) out[static_cast<long long>(j) * V + k] = dg[i][k];
    }
  }
}

// out[j] = sum_b part[b][j]: 32 columns a block, 32 threads of partial sums each, added in a fixed order.
__global__ void __launch_bounds__(1024) reduce_rows_kernel(const float* __restrict__ part, int parts, int d,
                                                           float* __restrict__ out) {
  __shared__ float sm[32][33];
  const int j = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (j < d)
    for (int b = threadIdx.y; b < parts; b += 32) v += part[static_cast<long long>(b) * d + j];
  sm[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = sm[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int jo = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && jo < d) out[jo] = v;
}

template <int V, int NV>
cudaError_t run_norm_bwd(const NormBwd& a, int tpr, int grid, cudaStream_t s) {
  if (a.res_f32) add_rmsnorm_bwd_kernel<V, NV, true><<<grid, tpr, 0, s>>>(a);
  else add_rmsnorm_bwd_kernel<V, NV, false><<<grid, tpr, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm_bwd(const NormBwd& a, bool vec, int parts, cudaStream_t s) {
  if (a.T <= 0) return cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.d, s);
  cudaError_t e;
  if (!vec) {
    e = run_norm_bwd<1, 32>(a, round32((a.d + 31) / 32), parts, s);
  } else {
    const int nvec = a.d / 8;
    if (nvec <= 512) e = run_norm_bwd<8, 1>(a, round32(nvec), parts, s);
    else if (nvec <= 1024) e = run_norm_bwd<8, 2>(a, round32((nvec + 1) / 2), parts, s);
    else e = run_norm_bwd<8, 4>(a, round32((nvec + 3) / 4), parts, s);
  }
  if (e != cudaSuccess || parts == 1) return e;
  reduce_rows_kernel<<<(a.d + 31) / 32, dim3(32, 32), 0, s>>>(a.part, parts, a.d, a.dweight);
  return cudaGetLastError();
}

}  // namespace vgg
