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

// Vector j of a row in shared memory.
template <bool F32>
__device__ __forceinline__ void load_smem8(const uint8_t* row, int j, float (&v)[8]) {
  if (F32) {
    const float4 a = *reinterpret_cast<const float4*>(row + 32 * j), b = *reinterpret_cast<const float4*>(row + 32 * j + 16);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(row + 16 * j);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16x2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
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

// What follows a row's rstd: h (with HOUT, else it has been stored), y and the codes.  h holds the row's stream and is
// used up; row_max gives the maximum over the row's threads (all of them call it).
template <int V, int NV, bool RES32, int FORM, bool HOUT, class RowMax>
__device__ __forceinline__ void norm_row_out(const NormFwd& a, long long t, int tx, int tpr, int nvec, bool row_ok, float rstd,
                                             float (&h)[NV][V], const float (&g)[NV][V], RowMax row_max) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
    if (row_ok && j < nvec) {
      if (HOUT && a.h) store_v<V, RES32>(a.h, t * a.ld_h + static_cast<long long>(j) * V, h[i]);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        h[i][k] = h[i][k] * rstd * g[i][k];
        amax = fmaxf(amax, fabsf(h[i][k]));
      }
      if (a.y) store_v<V, false>(a.y, t * a.ld_y + static_cast<long long>(j) * V, h[i]);
    }
  }
  if constexpr (FORM == NORM_E4M3) {
    amax = row_max(amax);
    const float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (row_ok && tx == 0) a.scales[t] = s;
    // one reciprocal a row; where it would overflow, a quotient for every value
    const bool tiny = amax < 1e-30f;
    const float inv = tiny ? 1.0f : __fdiv_rn(448.0f, amax);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (row_ok && j < nvec) {
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] = tiny ? __fdiv_rn(h[i][k], s) : h[i][k] * inv;
        *reinterpret_cast<uint2*>(a.q + t * a.d + 8ll * j) =
            make_uint2(e4m3x4(h[i][0], h[i][1], h[i][2], h[i][3]), e4m3x4(h[i][4], h[i][5], h[i][6], h[i][7]));
      }
    }
  }
  if constexpr (FORM == NORM_MX) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
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
    for (int b = (a.d >> 5) + tx; row_ok && b < a.sf_ld; b += tpr) a.sf[t * a.sf_ld + b] = 127;
  }
}

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
  float g[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (row_ok && j < nvec) load_weight<V>(a.weight, a.weight_f32 != 0, j * V, g[i]);
  }
  norm_row_out<V, NV, RES32, FORM, false>(a, t, threadIdx.x, blockDim.x, nvec, row_ok, rstd, h, g,
                                          [&](float m) { return row_reduce<true>(m, red_max); });
}

// ---- rows through a ring of bulk copies
//
// Each of the RG = blockDim.y row groups of a persistent block has a ring of `stages` rows in shared memory, filled ahead
// by the group's first thread, so the bytes in flight do not depend on registers or on how many warps are waiting.
// A stage is free again at the group's first barrier of a row (by then its values are in registers).  Every wait is
// bounded; a group that gave up runs on with what it has, so that its barriers stay matched, and leaves once its
// copies have landed.
constexpr int kRingGroups = 8, kRingStages = 4;

struct RingShared {
  float red[2][kRingGroups][16];  // 16-byte aligned: read as float4
  float red2[2][kRingGroups][16];
  uint64_t full[kRingGroups][kRingStages];
  int abort;
};

__device__ __forceinline__ void ring_init(RingShared& sh, int stages) {
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, n = blockDim.x * blockDim.y;
  if (tid == 0) sh.abort = 0;
  if (threadIdx.x < stages) mbar_init(&sh.full[threadIdx.y][threadIdx.x], 1);
  for (int i = tid; i < 2 * kRingGroups * 16; i += n) (&sh.red[0][0][0])[i] = (&sh.red2[0][0][0])[i] = 0.0f;
  fence_mbar_init();
  __syncthreads();
}

// After the last row: when some wait gave up, let every copy of this group still in flight land.
__device__ __forceinline__ void ring_drain(RingShared& sh, int stages, int rows_done) {
  __syncthreads();
  if (!sh.abort) return;
  volatile int never = 0;
  if (threadIdx.x == 0)
    for (int k = rows_done > stages ? rows_done - stages : 0; k < rows_done; ++k)
      mbar_wait(&sh.full[threadIdx.y][k % stages], (k / stages) & 1, &never, 20000000ull, nullptr);
  __syncthreads();
}

// Sum (or maximum of values that are not negative) over the blockDim.x threads of a row group; `red` is the group's 16
// floats for this parity of rows (those past its warps stay 0), so that one barrier a row is enough.
template <bool MAX>
__device__ __forceinline__ float group_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) {
    __syncwarp();
    return v;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.y) + 1), "r"(static_cast<int>(blockDim.x)) : "memory");
  v = 0.0f;
  for (int w = 0; w < nw; w += 4) {
    const float4 r = *reinterpret_cast<const float4*>(red + w);
    v = MAX ? fmaxf(fmaxf(v, fmaxf(r.x, r.y)), fmaxf(r.z, r.w)) : v + ((r.x + r.y) + (r.z + r.w));
  }
  return v;
}

// Launch shape of a ring kernel for rows of d columns and `row` bytes a stage: NV vectors a thread, up to 512 threads as
// row groups of tpr, at least three stages for each group within `bytes` (two for one group), at most four.
struct RingShape {
  int tpr, rgs, stages, grid;
  size_t smem;
};
inline int round32(int x) { return (x + 31) & ~31; }
inline RingShape ring_shape(long long T, int d, int NV, size_t row, size_t bytes, int blocks) {
  RingShape r;
  r.tpr = round32((d / 8 + NV - 1) / NV);
  r.rgs = 512 / r.tpr;
  if (r.rgs > kRingGroups) r.rgs = kRingGroups;
  while (r.rgs > 1 && 3 * r.rgs * row > bytes) --r.rgs;
  r.stages = static_cast<int>(bytes / (r.rgs * row));
  if (r.stages > kRingStages) r.stages = kRingStages;
  if (r.stages < 2) r.stages = 2;
  r.smem = r.rgs * r.stages * row;
  const long long want = (T + r.rgs - 1) / r.rgs;
  r.grid = static_cast<int>(want < blocks ? want : blocks);
  return r;
}

template <int NV, bool RES32, int FORM>
__global__ void __launch_bounds__(512) add_rmsnorm_ring_kernel(const NormFwd a, int stages) {
  constexpr int V = 8, ES = RES32 ? 4 : 2;
  extern __shared__ __align__(128) uint8_t nf_ring[];
  __shared__ __align__(16) RingShared sh;
  const int rg = threadIdx.y, tx = threadIdx.x, tpr = blockDim.x;
  const int nvec = a.d / V;
  const uint32_t xb = a.x ? 2u * a.d : 0u, rb = static_cast<uint32_t>(ES) * a.d, sb = xb + rb;
  uint8_t* ring = nf_ring + static_cast<size_t>(rg) * stages * sb;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.y + rg;
  ring_init(sh, stages);
  auto issue = [&](long long t, int st) {
    uint8_t* dst = ring + static_cast<size_t>(st) * sb;
    uint64_t* bar = &sh.full[rg][st];
    mbar_arrive_expect_tx(bar, sb);
    bulk_load(dst, static_cast<const uint8_t*>(a.res) + t * a.ld_res * ES, rb, bar);
    if (a.x) bulk_load(dst + rb, static_cast<const __nv_bfloat16*>(a.x) + t * a.ld_x, xb, bar);
  };
  if (tx == 0)
    for (int k = 0; k < stages; ++k)
      if (t0 + k * step < a.T) issue(t0 + k * step, k);
  float g[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
    if (j < nvec) load_weight<V>(a.weight, a.weight_f32 != 0, j * V, g[i]);
  }
  int it = 0, st = 0, ph = 0;
  for (long long t = t0; t < a.T; t += step, ++it) {
    mbar_wait(&sh.full[rg][st], ph, &sh.abort, a.timeout_ns, a.err);
    const uint8_t* src = ring + static_cast<size_t>(st) * sb;
    float h[NV][V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (j < nvec) {
        load_smem8<RES32>(src, j, h[i]);
        if (a.x) {
          float x[V];
          load_smem8<false>(src + rb, j, x);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            h[i][k] += x[k];
            if (!RES32) h[i][k] = bf16_round(h[i][k]);
          }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) ss += h[i][k] * h[i][k];
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) h[i][k] = 0.0f;
      }
    }
    ss = group_reduce<false>(ss, sh.red[it & 1][rg]);
    if (tx == 0 && t + stages * step < a.T) issue(t + stages * step, st);
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
    if (a.rstd && tx == 0) a.rstd[t] = rstd;
    norm_row_out<V, NV, RES32, FORM, true>(a, t, tx, tpr, nvec, true, rstd, h, g, [&](float m) {
      return group_reduce<true>(m, sh.red2[it & 1][rg]);
    });
  }
  ring_drain(sh, stages, it);
}

template <int V, int NV, bool RES32>
cudaError_t run_norm_form(const NormFwd& a, int tpr, int rows, cudaStream_t s) {
  const dim3 block(tpr, rows);
  const unsigned grid = static_cast<unsigned>((a.T + rows - 1) / rows);
  if constexpr (V == 8) {
    if (a.form == NORM_E4M3) {
      add_rmsnorm_kernel<V, NV, RES32, NORM_E4M3><<<grid, block, 0, s>>>(a);
      return cudaGetLastError();
    }
    if (a.form == NORM_MX) {
      add_rmsnorm_kernel<V, NV, RES32, NORM_MX><<<grid, block, 0, s>>>(a);
      return cudaGetLastError();
    }
  }
  add_rmsnorm_kernel<V, NV, RES32, NORM_BF16><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

template <int V, int NV>
cudaError_t run_norm(const NormFwd& a, int tpr, int rows, cudaStream_t s) {
  return a.res_f32 ? run_norm_form<V, NV, true>(a, tpr, rows, s) : run_norm_form<V, NV, false>(a, tpr, rows, s);
}

template <bool RES32, int FORM>
cudaError_t run_norm_ring(const NormFwd& a, const RingShape& r, cudaStream_t s) {
  auto kern = add_rmsnorm_ring_kernel<2, RES32, FORM>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(r.smem));
  if (e != cudaSuccess) return e;
  kern<<<r.grid, dim3(r.tpr, r.rgs), r.smem, s>>>(a, r.stages);
  return cudaGetLastError();
}

template <bool RES32>
cudaError_t run_norm_ring_form(const NormFwd& a, const RingShape& r, cudaStream_t s) {
  return a.form == NORM_E4M3 ? run_norm_ring<RES32, NORM_E4M3>(a, r, s)
         : a.form == NORM_MX ? run_norm_ring<RES32, NORM_MX>(a, r, s)
                             : run_norm_ring<RES32, NORM_BF16>(a, r, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormFwd& a, bool vec, int num_sms, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  // Rows of more than 4096 columns, four for every SM: two ring blocks an SM.  At 8192 x 7168 with per-row codes 87.6 us
  // against 116 us for a block a row (few such wide blocks fit an SM, and all of one waits at each of its barriers);
  // at 500 rows 9.2 against 9.8 us.  Narrower rows are as fast or faster with a block a row (4096 x 2048: 14.3 against
  // 14.5 us, 32768 x 1536 fp32: 96 against 100 us), single rows need fewer threads' work each.
  if (vec && a.d > 4096 && a.d <= 8192 && a.T >= 4ll * num_sms) {
    const size_t row = static_cast<size_t>(a.d) * ((a.x ? 2 : 0) + (a.res_f32 ? 4 : 2));
    const RingShape r = ring_shape(a.T, a.d, 2, row, 106 * 1024, 2 * num_sms);
    return a.res_f32 ? run_norm_ring_form<true>(a, r, s) : run_norm_ring_form<false>(a, r, s);
  }
  if (!vec) return run_norm<1, 16>(a, round32((a.d + 15) / 16), 1, s);
  const int nvec = a.d / 8;
  // Narrow rows share a block of 128 threads.
  if (nvec <= 1024) return run_norm<8, 1>(a, round32(nvec), nvec <= 32 ? 4 : nvec <= 64 ? 2 : 1, s);
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

// Rows of any width and alignment, straight from global memory; the weight and dh are read where they are needed.
template <int V, int NV, bool RES32>
__global__ void __launch_bounds__(512) add_rmsnorm_bwd_kernel(const NormBwd a) {
  __shared__ float red[2][32];
  const int nvec = a.d / V;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float dg[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dg[i][k] = 0.0f;
  int it = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++it) {
    const float rstd = __ldg(a.rstd + t);
    float dy[NV][V], h[NV][V];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < nvec) {
        float g[V];
        load_v<V, false>(a.dy, t * a.ld_dy + static_cast<long long>(j) * V, dy[i]);
        load_v<V, RES32>(a.h, t * a.ld_h + static_cast<long long>(j) * V, h[i]);
        load_weight<V>(a.weight, a.weight_f32 != 0, j * V, g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          h[i][k] *= rstd;
          dg[i][k] += dy[i][k] * h[i][k];
          dy[i][k] *= g[k];
          c += dy[i][k] * h[i][k];
        }
      }
    }
    c = row_reduce<false>(c, red[it & 1]) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < nvec) {
        float o[V];
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = 0.0f;
        if (a.dh) load_v<V, RES32>(a.dh, t * a.ld_dh + static_cast<long long>(j) * V, o);
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

// The same with the rows (dy, h and dh side by side) through the ring.
template <int NV, bool RES32>
__global__ void __launch_bounds__(512) add_rmsnorm_bwd_ring_kernel(const NormBwd a, int stages) {
  constexpr int V = 8, ES = RES32 ? 4 : 2;
  extern __shared__ __align__(128) uint8_t nb_ring[];
  __shared__ __align__(16) RingShared sh;
  const int rg = threadIdx.y, RG = blockDim.y, tx = threadIdx.x, tpr = blockDim.x;
  const int nvec = a.d / V;
  const uint32_t dyb = 2u * a.d, hb = static_cast<uint32_t>(ES) * a.d, sb = dyb + hb + (a.dh ? hb : 0u);
  uint8_t* ring = nb_ring + static_cast<size_t>(rg) * stages * sb;
  const long long step = static_cast<long long>(gridDim.x) * RG, t0 = static_cast<long long>(blockIdx.x) * RG + rg;
  ring_init(sh, stages);
  auto issue = [&](long long t, int st) {
    uint8_t* dst = ring + static_cast<size_t>(st) * sb;
    uint64_t* bar = &sh.full[rg][st];
    mbar_arrive_expect_tx(bar, sb);
    bulk_load(dst, static_cast<const __nv_bfloat16*>(a.dy) + t * a.ld_dy, dyb, bar);
    bulk_load(dst + dyb, static_cast<const uint8_t*>(a.h) + t * a.ld_h * ES, hb, bar);
    if (a.dh) bulk_load(dst + dyb + hb, static_cast<const uint8_t*>(a.dh) + t * a.ld_dh * ES, hb, bar);
  };
  if (tx == 0)
    for (int k = 0; k < stages; ++k)
      if (t0 + k * step < a.T) issue(t0 + k * step, k);
  float g[NV][V], dg[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
#pragma unroll
    for (int k = 0; k < V; ++k) g[i][k] = dg[i][k] = 0.0f;
    if (j < nvec) load_weight<V>(a.weight, a.weight_f32 != 0, j * V, g[i]);
  }
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float rstd_next = t0 < a.T ? __ldg(a.rstd + t0) : 0.0f;
  int it = 0, st = 0, ph = 0;
  for (long long t = t0; t < a.T; t += step, ++it) {
    const float rstd = rstd_next;
    if (t + step < a.T) rstd_next = __ldg(a.rstd + t + step);
    mbar_wait(&sh.full[rg][st], ph, &sh.abort, a.timeout_ns, a.err);
    const uint8_t* src = ring + static_cast<size_t>(st) * sb;
    float dy[NV][V], h[NV][V], o[NV][V];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (j < nvec) {
        load_smem8<false>(src, j, dy[i]);
        load_smem8<RES32>(src + dyb, j, h[i]);
        if (a.dh) load_smem8<RES32>(src + dyb + hb, j, o[i]);
        else {
#pragma unroll
          for (int k = 0; k < V; ++k) o[i][k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
          h[i][k] *= rstd;
          dg[i][k] += dy[i][k] * h[i][k];
          dy[i][k] *= g[i][k];
          c += dy[i][k] * h[i][k];
        }
      }
    }
    c = group_reduce<false>(c, sh.red[it & 1][rg]) * inv_d;
    if (tx == 0 && t + stages * step < a.T) issue(t + stages * step, st);
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (j < nvec) {
#pragma unroll
        for (int k = 0; k < V; ++k) o[i][k] += rstd * (dy[i][k] - c * h[i][k]);
        if (a.dx) store8<false>(a.dx, t * a.ld_dx + static_cast<long long>(j) * V, o[i]);
        if (a.dres) store8<RES32>(a.dres, t * a.ld_dres + static_cast<long long>(j) * V, o[i]);
      }
    }
  }
  ring_drain(sh, stages, it);
  // the groups' shares, added in group order
  float* share = reinterpret_cast<float*>(nb_ring);
  float* out = gridDim.x == 1 ? a.dweight : a.part + static_cast<long long>(blockIdx.x) * a.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
    if (j < nvec) store8<true>(RG > 1 ? share + static_cast<size_t>(rg) * a.d : out, static_cast<long long>(j) * V, dg[i]);
  }
  if (RG == 1) return;
  __syncthreads();
  for (int j = rg * tpr + tx; j < a.d; j += RG * tpr) {
    float v = 0.0f;
    for (int r = 0; r < RG; ++r) v += share[static_cast<size_t>(r) * a.d + j];
    out[j] = v;
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

template <int NV, bool RES32>
cudaError_t run_norm_bwd_ring(const NormBwd& a, const RingShape& r, cudaStream_t s) {
  auto kern = add_rmsnorm_bwd_ring_kernel<NV, RES32>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(r.smem));
  if (e != cudaSuccess) return e;
  kern<<<r.grid, dim3(r.tpr, r.rgs), r.smem, s>>>(a, r.stages);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm_bwd(const NormBwd& a, bool vec, int num_sms, cudaStream_t s) {
  if (a.T <= 0) return cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.d, s);
  const size_t row = static_cast<size_t>(a.d) * (2 + (a.res_f32 ? 4 : 2) * (a.dh ? 2 : 1));
  cudaError_t e;
  int parts;
  if (vec && a.d <= 8192) {
    // 150 KB of rows in flight on an SM: with the whole shared memory 8192 x 7168 fp32 took 164 us against 155 and
    // 8192 x 5120 fp32 116 against 103, with two stages 8192 x 7168 bf16 81 against 74.
    const bool narrow = a.d <= 1024;
    const RingShape r = ring_shape(a.T, a.d, narrow ? 1 : 2, row, 150 * 1024, num_sms);
    parts = r.grid;
    if (narrow) e = a.res_f32 ? run_norm_bwd_ring<1, true>(a, r, s) : run_norm_bwd_ring<1, false>(a, r, s);
    else e = a.res_f32 ? run_norm_bwd_ring<2, true>(a, r, s) : run_norm_bwd_ring<2, false>(a, r, s);
  } else {
    const long long most = 4ll * num_sms < kMaxNormParts ? 4ll * num_sms : kMaxNormParts;
    parts = static_cast<int>(a.T < most ? a.T : most);
    if (!vec) e = run_norm_bwd<1, 32>(a, round32((a.d + 31) / 32), parts, s);
    else e = run_norm_bwd<8, 4>(a, round32((a.d / 8 + 3) / 4), parts, s);
  }
  if (e != cudaSuccess || parts == 1) return e;
  reduce_rows_kernel<<<(a.d + 31) / 32, dim3(32, 32), 0, s>>>(a.part, parts, a.d, a.dweight);
  return cudaGetLastError();
}

}  // namespace vgg
