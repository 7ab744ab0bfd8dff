// Residual addition with root-mean-square norm and an optional 8-bit output, and its backward.
//
//   h = r + x (rounded to the residual stream's type),  rstd = (mean_j h_j^2 + eps)^(-1/2),
//   y_j = h_j rstd g_j  (bf16),  q = e4m3 codes of the fp32 y with one fp32 scale a row (max|y| / 448), or
//   with one power of two for every 32 columns.
//
// The codes come from the fp32 y, not from its bf16 rounding: one rounding instead of two.
//
// Both directions move every element once and are bound by HBM and, with rows of 2 bytes an element, nearly as much by
// issue slots (hence the packed arithmetic).  A row's values stay in registers between the reduction and the
// output: thread i of a row's tpr threads holds the vectors of eight values i, i + tpr, ... (NV of them).
// Forward: 8192 x 7168 with per-row codes 83 us (529 MB, 6.4 TB/s), 32768 x 1536 fp32 with block-scaled codes 98 us
// (656 MB, 6.7 TB/s), a copy running at 6.7; 61 rows of 2048 2.2 us, one row of 7168 3.0 us (a launch and a row's latency).
// Backward: 8192 x 7168 fp32 155 us (940 MB, 6.0 TB/s), 4096 x 2048 18.4 us with its second launch (67 MB).
#include <type_traits>

#include "internal.h"

namespace vgg {

namespace {

struct Vec8 {
  f32x2 p[4];
};

__device__ __forceinline__ Vec8 zero8() {
  Vec8 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v.p[k] = pack2(0.0f, 0.0f);
  return v;
}

__device__ __forceinline__ Vec8 from_bf16(const uint4 q) {
  Vec8 v;
  v.p[0] = bf16x2_to_f32x2(q.x);
  v.p[1] = bf16x2_to_f32x2(q.y);
  v.p[2] = bf16x2_to_f32x2(q.z);
  v.p[3] = bf16x2_to_f32x2(q.w);
  return v;
}

__device__ __forceinline__ Vec8 from_f32(const float4 a, const float4 b) {
  Vec8 v;
  v.p[0] = pack2(a.x, a.y);
  v.p[1] = pack2(a.z, a.w);
  v.p[2] = pack2(b.x, b.y);
  v.p[3] = pack2(b.z, b.w);
  return v;
}

__device__ __forceinline__ uint4 to_bf16(const Vec8& v) {
  return make_uint4(f32x2_to_bf16x2(v.p[0]), f32x2_to_bf16x2(v.p[1]), f32x2_to_bf16x2(v.p[2]), f32x2_to_bf16x2(v.p[3]));
}

// Eight values of a bf16 or fp32 row from element off (16-byte aligned), in global memory (read once) or shared memory.
template <bool F32>
__device__ __forceinline__ Vec8 load8(const void* base, long long off) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    return from_f32(__ldcs(p), __ldcs(p + 1));
  } else {
    return from_bf16(__ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off)));
  }
}

template <bool F32>
__device__ __forceinline__ Vec8 load_smem8(const uint8_t* row, int j) {
  if constexpr (F32)
    return from_f32(*reinterpret_cast<const float4*>(row + 32 * j), *reinterpret_cast<const float4*>(row + 32 * j + 16));
  else return from_bf16(*reinterpret_cast<const uint4*>(row + 16 * j));
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, long long off, const Vec8& v) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
    const float2 a = unpack2(v.p[0]), b = unpack2(v.p[1]), c = unpack2(v.p[2]), d = unpack2(v.p[3]);
    p[0] = make_float4(a.x, a.y, b.x, b.y);
    p[1] = make_float4(c.x, c.y, d.x, d.y);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) = to_bf16(v);
  }
}

__device__ __forceinline__ Vec8 load_weight8(const void* w, int f32, int j) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + 8 * j);
    return from_f32(__ldg(p), __ldg(p + 1));
  }
  return from_bf16(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + 8 * j)));
}

// One value of a row of any alignment.
template <bool F32>
__device__ __forceinline__ float load1(const void* base, long long off) {
  return F32 ? static_cast<const float*>(base)[off] : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off]);
}

template <bool F32>
__device__ __forceinline__ void store1(void* base, long long off, float v) {
  if (F32) static_cast<float*>(base)[off] = v;
  else static_cast<__nv_bfloat16*>(base)[off] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float load_weight1(const void* w, int f32, int j) {
  return f32 ? __ldg(static_cast<const float*>(w) + j) : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[j]);
}

// The stream's next value from its packed parts: the sum of two bf16 values rounded once.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}

// Sum (or maximum of values that are not negative) of v over the blockDim.x threads of a row, the same in every one of
// them.  `red`: a float for each warp of the block; one __syncthreads when a row has more than one warp, so the next
// use of the same `red` needs another barrier in between.
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

// The stream's vector as it is stored: four packed bf16 pairs, or eight fp32 values.
template <bool F32>
using Raw8 = std::conditional_t<F32, Vec8, uint4>;

__device__ __forceinline__ Vec8 values(const Vec8& r) { return r; }
__device__ __forceinline__ Vec8 values(const uint4& r) { return from_bf16(r); }

__device__ __forceinline__ Vec8 add_x(const Vec8& r, const uint4& x) {
  const Vec8 xv = from_bf16(x);
  Vec8 h;
#pragma unroll
  for (int k = 0; k < 4; ++k) h.p[k] = add2(r.p[k], xv.p[k]);
  return h;
}
__device__ __forceinline__ uint4 add_x(const uint4& r, const uint4& x) {
  return make_uint4(add_bf16x2(r.x, x.x), add_bf16x2(r.y, x.y), add_bf16x2(r.z, x.z), add_bf16x2(r.w, x.w));
}

__device__ __forceinline__ void store_raw(void* base, long long off, const Vec8& r) { store8<true>(base, off, r); }
__device__ __forceinline__ void store_raw(void* base, long long off, const uint4& r) {
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) = r;
}

__device__ __forceinline__ uint4 ldcs4(const void* base, long long off) {
  return __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
}

// 1 / sqrt(x): the approximation (2 steps) and one Newton step.  Every thread of a row computes it, so a correctly rounded
// root and two quotients cost a thread as many issue slots as its values do.
__device__ __forceinline__ float inv_root(float x) {
  const float r = rsqrtf(x);
  const float e = fmaf(-x * r, r, 1.0f);
  return x < 1e30f && x > 1e-30f ? fmaf(0.5f * r, e, r) : r;  // (out there the step's products would leave the range)
}

__device__ __forceinline__ f32x2 squares(const Vec8& h, f32x2 ss) {
#pragma unroll
  for (int k = 0; k < 4; ++k) ss = fma2(h.p[k], h.p[k], ss);
  return ss;
}

__device__ __forceinline__ float amax8(const Vec8& v, float m) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2(v.p[k]);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return m;
}

__device__ __forceinline__ void store_codes8(uint8_t* q, const Vec8& v, float scale) {
  const f32x2 s = pack2(scale, scale);
  const float2 a = unpack2(mul2(v.p[0], s)), b = unpack2(mul2(v.p[1], s)), c = unpack2(mul2(v.p[2], s)),
               d = unpack2(mul2(v.p[3], s));
  *reinterpret_cast<uint2*>(q) = make_uint2(e4m3x4(a.x, a.y, b.x, b.y), e4m3x4(c.x, c.y, d.x, d.y));
}

// Where a thread's first vector of a row goes in h, y and q (null: nowhere), and the row's other outputs.
struct RowOut {
  uint8_t *h, *y, *q, *sf;
  float *rstd, *scale;
};
template <bool RES32>
__device__ __forceinline__ RowOut row_out(const NormFwd& a, long long t, int tx) {
  RowOut o;
  o.h = a.h ? static_cast<uint8_t*>(a.h) + (t * a.ld_h + 8ll * tx) * (RES32 ? 4 : 2) : nullptr;
  o.y = a.y ? static_cast<uint8_t*>(a.y) + (t * a.ld_y + 8ll * tx) * 2 : nullptr;
  o.q = a.q + t * a.d + 8ll * tx;
  o.sf = a.sf + t * a.sf_ld;
  o.rstd = a.rstd ? a.rstd + t : nullptr;
  o.scale = a.scales + t;
  return o;
}
// The same `rows` rows further on.
template <bool RES32>
__device__ __forceinline__ void advance(const NormFwd& a, RowOut& o, long long rows) {
  if (o.h) o.h += rows * a.ld_h * (RES32 ? 4 : 2);
  if (o.y) o.y += rows * a.ld_y * 2;
  o.q += rows * a.d;
  o.sf += rows * a.sf_ld;
  if (o.rstd) o.rstd += rows;
  o.scale += rows;
}

// What follows a row's rstd, first half: h and y leave, h becomes y in fp32; the largest |y| of the thread's columns.
// raw holds the row's stream, weight(i, j) gives the weight's vector j.
template <int NV, bool RES32, int FORM, class Weight>
__device__ __forceinline__ float norm_row_y(const RowOut& o, int tx, int tpr, int nvec, bool row_ok, float rstd,
                                            const Raw8<RES32> (&raw)[NV], Vec8 (&h)[NV], Weight weight) {
  float amax = 0.0f;
  const f32x2 r2 = pack2(rstd, rstd);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
    h[i] = zero8();
    if (row_ok && j < nvec) {
      if (o.h) store_raw(o.h, 8 * tpr * i, raw[i]);
      const Vec8 g = weight(i, j), v = values(raw[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[i].p[k] = mul2(mul2(v.p[k], r2), g.p[k]);
      if (FORM == NORM_E4M3) amax = amax8(h[i], amax);
      if (o.y) store8<false>(o.y, 8 * tpr * i, h[i]);
    }
  }
  return amax;
}

// Second half: the codes, from the fp32 y and, with one scale a row, the row's largest |y|.
template <int NV, int FORM>
__device__ __forceinline__ void norm_row_codes(const NormFwd& a, const RowOut& o, int tx, int tpr, int nvec, bool row_ok,
                                               float amax, Vec8 (&h)[NV]) {
  if constexpr (FORM == NORM_E4M3) {
    if (row_ok && tx == 0) *o.scale = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    // one factor a row; values so small that it would overflow are brought up first
    const bool tiny = amax < 1e-30f;
    const float up = tiny ? 0x1p100f : 1.0f;
    const float inv = amax > 0.0f ? __fdiv_rn(448.0f, amax * up) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (row_ok && j < nvec) {
        if (tiny) {
#pragma unroll
          for (int k = 0; k < 4; ++k) h[i].p[k] = mul2(h[i].p[k], pack2(up, up));
        }
        store_codes8(o.q + 8 * tpr * i, h[i], inv);
      }
    }
  }
  if constexpr (FORM == NORM_MX) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      // four neighbouring lanes hold a block of 32 columns
      float m = amax8(h[i], 0.0f);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = mx_exponent(m);
      if (row_ok && j < nvec) {
        store_codes8(o.q + 8 * tpr * i, h[i], mx_inv_scale(e));
        if ((j & 3) == 0) o.sf[j >> 2] = static_cast<uint8_t>(e + 127);
      }
    }
    // bytes past the last block of the row hold scale 1
    const int b = (a.d >> 5) + tx;
    if (row_ok && b < a.sf_ld) o.sf[b] = 127;
  }
}

// blockDim.y rows a block.  32 registers keep 2048 threads on an SM; the fp32 stream with per-row codes spills 20 bytes
// for that (32768 x 1536 107.0 us, with 40 registers and none 108.1; 8192 x 4096 77.1 and 80.2).
template <int NV, bool RES32, int FORM>
__global__ void __launch_bounds__(1024, NV == 1 ? 2 : 1) add_rmsnorm_kernel(const NormFwd a) {
  __shared__ float red_sum[32], red_max[32];
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool row_ok = t < a.T;
  const int nvec = a.d / 8;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  Raw8<RES32> raw[NV];
  f32x2 s2 = pack2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (row_ok && j < nvec) {
      if constexpr (RES32) raw[i] = load8<true>(a.res, t * a.ld_res + 8ll * j);
      else raw[i] = ldcs4(a.res, t * a.ld_res + 8ll * j);
      if (a.x) raw[i] = add_x(raw[i], ldcs4(a.x, t * a.ld_x + 8ll * j));
      if (a.h) store_raw(a.h, t * a.ld_h + 8ll * j, raw[i]);
      s2 = squares(values(raw[i]), s2);
    }
  }
  const float2 sf = unpack2(s2);
  const float ss = row_reduce<false>(sf.x + sf.y, red_sum);
  const float rstd = inv_root(fmaf(ss, inv_d, a.eps));
  if (a.rstd && row_ok && threadIdx.x == 0) a.rstd[t] = rstd;
  RowOut o = row_out<RES32>(a, t, threadIdx.x);
  o.h = nullptr;  // stored above
  Vec8 h[NV];
  float amax = norm_row_y<NV, RES32, FORM>(o, threadIdx.x, blockDim.x, nvec, row_ok, rstd, raw, h,
                                           [&](int, int j) { return load_weight8(a.weight, a.weight_f32, j); });
  if (FORM == NORM_E4M3) amax = row_reduce<true>(amax, red_max);
  norm_row_codes<NV, FORM>(a, o, threadIdx.x, blockDim.x, nvec, row_ok, amax, h);
}

// Rows that are not aligned and too wide for a vector a thread (more than about 8100 columns): a block a row, 16 values a
// thread, each a load of its own.
template <bool RES32>
__global__ void __launch_bounds__(1024) add_rmsnorm_any_kernel(const NormFwd a) {
  constexpr int N = 16;
  __shared__ float red[32];
  const long long t = blockIdx.x;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float h[N], ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    h[i] = 0.0f;
    if (j < a.d) {
      h[i] = load1<RES32>(a.res, t * a.ld_res + j);
      if (a.x) {
        h[i] += load1<false>(a.x, t * a.ld_x + j);
        if (!RES32) h[i] = bf16_round(h[i]);  // the norm's input is the stream as it is stored
      }
      if (a.h) store1<RES32>(a.h, t * a.ld_h + j, h[i]);
      ss += h[i] * h[i];
    }
  }
  ss = row_reduce<false>(ss, red);
  const float rstd = inv_root(fmaf(ss, inv_d, a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (j < a.d) store1<false>(a.y, t * a.ld_y + j, h[i] * rstd * load_weight1(a.weight, a.weight_f32, j));
  }
}

// ---- rows that start anywhere
//
// A row's phase is the element mod 8 at which it begins; tensors of a call mostly have it in common (addresses and strides
// alike).  In its phase a row's vectors begin at its first aligned column and are aligned in all of those tensors;
// the others are read and written a value at a time.
// A row group takes rows whose numbers differ by multiples of eight, so that its phase, and with it every thread's
// columns, stay the same: the weight's vector is read once, and the backward's share of dg stays in registers.  The next
// row's loads are on their way while a row is reduced.
// Against the kernels that load a value at a time: 8192 x 4001 bf16 forward 48 us and 161 (262 MB, 39 us of them), backward
// 70 and 495; 16384 x 999 26 and 72, 42 and 740; 300 x 1501 3.1 and 8.2, 7.0 and 17.6.  One tensor out of phase: 61 and 95
// us at 8192 x 4001.
struct Phase {
  int first, step;  // of row 0, and from one row to the next
  unsigned in;      // bit i: the call's tensor i has this phase
  __device__ int of(long long t) const { return (first + static_cast<int>(t & 7) * step) & 7; }
  __device__ bool has(int i) const { return in >> i & 1; }
};
struct PhaseOf {
  const void* p;
  long long ld;
  bool f32;
};
// The phase of a bf16 tensor, and which of n tensors have it (a missing one does; four fp32 values fill 16 bytes).
inline Phase phase_of(const void* p, long long ld, const PhaseOf* t, int n) {
  Phase f{static_cast<int>(reinterpret_cast<uintptr_t>(p) / 2 & 7), static_cast<int>(ld & 7), 0};
  for (int i = 0; i < n; ++i) {
    const long long m = t[i].f32 ? 3 : 7, at = static_cast<long long>(reinterpret_cast<uintptr_t>(t[i].p) / (t[i].f32 ? 4 : 2));
    if (!t[i].p || (((at - f.first) & m) == 0 && ((t[i].ld - f.step) & m) == 0)) f.in |= 1u << i;
  }
  return f;
}
// Threads of a row: the fewest vectors that a phase leaves, and a thread for every column outside them.
inline int phase_threads(int d) { return d < 8 ? d : d - 7 * ((d - 7) / 8); }

// What a thread has of such a row: columns c .. c + n - 1, a vector (n = 8) or one of the up to 14 columns at the ends
// (n = 1; as the first value of a vector of zeros), or nothing.  A thread with a part of a vector instead takes eight
// turns at loading and storing, and the row waits for it (8192 x 2049 bf16: forward 53 us against 34).
struct Cols {
  int c, n;
  __device__ Cols(int phase, int d, int i) {
    const int head = min(d, (8 - phase) & 7), full = (d - head) / 8, tail = d - head - 8 * full, e = i - full;
    n = e < 0 ? 8 : e < head + tail ? 1 : 0;
    c = e < 0 ? head + 8 * i : e < head ? e : 8 * full + e;
  }
};
struct Pair4 {
  float4 a, b;
};
// As loaded, so that nothing waits for the load before the values are used.
template <bool F32>
using Cols8 = std::conditional_t<F32, Pair4, uint4>;
template <bool F32>
__device__ __forceinline__ Cols8<F32> load_cols(const void* base, long long off, const Cols& w, bool in_phase) {
  Cols8<F32> v{};
  if constexpr (F32) {
    const float* p = static_cast<const float*>(base) + off + w.c;
    if (w.n == 8 && in_phase) {
      v.a = __ldcs(reinterpret_cast<const float4*>(p));
      v.b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    } else if (w.n == 8) {
      v.a = make_float4(p[0], p[1], p[2], p[3]);
      v.b = make_float4(p[4], p[5], p[6], p[7]);
    } else if (w.n) {
      v.a.x = *p;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off + w.c;
    if (w.n == 8 && in_phase) {
      v = ldcs4(base, off + w.c);
    } else if (w.n == 8) {
      v = make_uint4(p[0] | static_cast<uint32_t>(p[1]) << 16, p[2] | static_cast<uint32_t>(p[3]) << 16,
                     p[4] | static_cast<uint32_t>(p[5]) << 16, p[6] | static_cast<uint32_t>(p[7]) << 16);
    } else if (w.n) {
      v.x = *p;
    }
  }
  return v;
}
__device__ __forceinline__ Vec8 values(const Pair4& r) { return from_f32(r.a, r.b); }
template <bool F32>
__device__ __forceinline__ void store_cols(void* base, long long off, const Cols& w, bool in_phase, const Vec8& v) {
  if (w.n == 8 && in_phase) return store8<F32>(base, off + w.c, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 p = unpack2(v.p[k / 2]);
    if (k < w.n) store1<F32>(base, off + w.c + k, k % 2 ? p.y : p.x);
  }
}
__device__ __forceinline__ Vec8 weight_cols(const void* w, int f32, const Cols& l) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = k < l.n ? load_weight1(w, f32, l.c + k) : 0.0f;
  return from_f32(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]));
}

// Sum over the blockDim.x threads of a row group, which has a barrier of its own; red: 32 floats a group, another set
// for every other row.
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (nw == 1) return v;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.y) + 1), "r"(static_cast<int>(blockDim.x)) : "memory");
  v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Launch shape: row groups of tpr threads, up to 512 threads a block, `threads` on an SM.
struct PhaseShape {
  int tpr, rows, grid;
};
inline PhaseShape phase_shape(long long T, int d, int threads, int num_sms) {
  PhaseShape r;
  r.tpr = (phase_threads(d) + 31) & ~31;
  r.rows = r.tpr >= 512 ? 1 : 512 / r.tpr < 8 ? 512 / r.tpr : 8;
  const long long want = (T + r.rows - 1) / r.rows;
  const int most = (num_sms * (threads / (r.tpr * r.rows)) + 7) & ~7;  // a multiple of eight rows from one to the next
  r.grid = static_cast<int>(want < most ? want : most);
  return r;
}

template <bool RES32>
__global__ void __launch_bounds__(1024) add_rmsnorm_phase_kernel(const NormFwd a, Phase f) {
  __shared__ float red[2][8][32];
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  if (t0 >= a.T) return;
  const int d = a.d;
  const Cols w(f.of(t0), d, threadIdx.x);
  const Vec8 g = weight_cols(a.weight, a.weight_f32, w);
  const float inv_d = 1.0f / static_cast<float>(d);
  Cols8<RES32> res{};
  uint4 x{};
  auto fetch = [&](long long t) {  // a row ahead
    if (t >= a.T) return;
    res = load_cols<RES32>(a.res, t * a.ld_res, w, f.has(0));
    if (a.x) x = load_cols<false>(a.x, t * a.ld_x, w, f.has(1));
  };
  fetch(t0);
  int it = 0;
  for (long long t = t0; t < a.T; t += step, ++it) {
    Vec8 h;
    if constexpr (RES32) h = a.x ? add_x(values(res), x) : values(res);
    else h = values(a.x ? add_x(res, x) : res);
    if (a.h) store_cols<RES32>(a.h, t * a.ld_h, w, f.has(2), h);
    fetch(t + step);
    const float2 sq = unpack2(squares(h, pack2(0.0f, 0.0f)));
    const float rstd = inv_root(fmaf(group_sum(sq.x + sq.y, red[it & 1][threadIdx.y]), inv_d, a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
    const f32x2 r2 = pack2(rstd, rstd);
#pragma unroll
    for (int k = 0; k < 4; ++k) h.p[k] = mul2(mul2(h.p[k], r2), g.p[k]);
    store_cols<false>(a.y, t * a.ld_y, w, f.has(3), h);
  }
}

// ---- rows through a ring of bulk copies
//
// Each of the RG = blockDim.y row groups of a persistent block has a ring of `stages` rows in shared memory, filled ahead
// by the group's first thread, so the bytes in flight do not depend on registers or on how many warps are waiting.
// A stage is free again at the group's one barrier a row (by then its values are in registers).  Every wait is
// bounded; a group that gave up runs on with what it has, so that its barriers stay matched, and leaves once its
// copies have landed.
constexpr int kRingGroups = 8, kRingStages = 4;

struct RingShared {
  float red[2][kRingGroups][16];
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

// The sum of v and, with MAX, the maximum of m (not negative) over the threads of a row group, which has a barrier of
// its own; red and redm are the group's 16 floats for this parity of rows (those past its warps stay 0), so that one
// barrier a row is enough.
template <bool MAX>
__device__ __forceinline__ void group_reduce(float& v, float& m, float* red, float* redm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    if (MAX) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) {
    __syncwarp();
    return;
  }
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = v;
    if (MAX) redm[threadIdx.x >> 5] = m;
  }
  asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.y) + 1), "r"(static_cast<int>(blockDim.x)) : "memory");
  v = red[threadIdx.x & 15];
  if (MAX) m = redm[threadIdx.x & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    if (MAX) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
}

// Launch shape of a ring kernel for rows of d columns and `row` bytes a stage: NV vectors a thread, up to 512 threads as
// row groups of tpr, at least three stages for each group within `bytes` (two for one group), at most four.
struct RingShape {
  int tpr, rgs, stages, grid;
  size_t smem;
};
// The most that a shape takes: two of the backward's widest rows (8192 columns in bf16 and twice in fp32).  The kernels'
// attribute is always set to it: with a call's own size one thread could lower it between another's setting and launch.
constexpr int kRingMost = 2 * 8192 * (2 + 4 + 4);
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
__global__ void __launch_bounds__(512, 1) add_rmsnorm_ring_kernel(const NormFwd a, int stages) {
  constexpr int ES = RES32 ? 4 : 2;
  extern __shared__ __align__(128) uint8_t nf_ring[];
  __shared__ __align__(16) RingShared sh;
  const int rg = threadIdx.y, tx = threadIdx.x, tpr = blockDim.x;
  const int nvec = a.d / 8;
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
  Vec8 g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tx + tpr * i < nvec) g[i] = load_weight8(a.weight, a.weight_f32, tx + tpr * i);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  // The group's next row into registers, and this thread's share of its sum of squares.
  int st = 0, ph = 0;
  auto fetch = [&](Raw8<RES32> (&raw)[NV]) {
    mbar_wait(&sh.full[rg][st], ph, &sh.abort, a.timeout_ns, a.err);
    const uint8_t* src = ring + static_cast<uint32_t>(st) * sb;
    f32x2 s2 = pack2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (j < nvec) {
        if constexpr (RES32) raw[i] = load_smem8<true>(src, j);
        else raw[i] = *reinterpret_cast<const uint4*>(src + 16 * j);
        if (a.x) raw[i] = add_x(raw[i], *reinterpret_cast<const uint4*>(src + rb + 16 * j));
        s2 = squares(values(raw[i]), s2);
      }
    }
    const float2 f = unpack2(s2);
    return f.x + f.y;
  };
  long long t_in = t0 + stages * step;  // the next row to ask for
  auto refill = [&]() {  // the stage that the last fetch has emptied
    if (tx == 0 && t_in < a.T) issue(t_in, st);
    t_in += step;
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  };
  // The next row's sum of squares and this row's largest value go through one barrier, and this row's arithmetic fills
  // the time that the reduction takes.
  int it = 0;
  if (t0 < a.T) {
    Raw8<RES32> raw[NV];
    float ss = fetch(raw), none = 0.0f;
    group_reduce<false>(ss, none, sh.red[0][rg], sh.red2[0][rg]);
    refill();
    RowOut o = row_out<RES32>(a, t0, tx);
    for (long long t = t0;; t += step) {
      const float rstd = inv_root(fmaf(ss, inv_d, a.eps));
      if (o.rstd && tx == 0) *o.rstd = rstd;
      const bool more = t + step < a.T;
      Raw8<RES32> next[NV];
      Vec8 h[NV];
      if (more) ss = fetch(next);
      float amax = norm_row_y<NV, RES32, FORM>(o, tx, tpr, nvec, true, rstd, raw, h, [&](int i, int) { return g[i]; });
      ++it;
      if (FORM == NORM_E4M3 || more) group_reduce<FORM == NORM_E4M3>(ss, amax, sh.red[it & 1][rg], sh.red2[it & 1][rg]);
      if (more) refill();
      norm_row_codes<NV, FORM>(a, o, tx, tpr, nvec, true, amax, h);
      if (!more) break;
      advance<RES32>(a, o, step);
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[i] = next[i];
    }
  }
  ring_drain(sh, stages, it);
}

template <int NV, bool RES32>
cudaError_t run_norm_form(const NormFwd& a, int tpr, int rows, cudaStream_t s) {
  const dim3 block(tpr, rows);
  const unsigned grid = static_cast<unsigned>((a.T + rows - 1) / rows);
  if (a.form == NORM_E4M3) add_rmsnorm_kernel<NV, RES32, NORM_E4M3><<<grid, block, 0, s>>>(a);
  else if (a.form == NORM_MX) add_rmsnorm_kernel<NV, RES32, NORM_MX><<<grid, block, 0, s>>>(a);
  else add_rmsnorm_kernel<NV, RES32, NORM_BF16><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

template <int NV>
cudaError_t run_norm(const NormFwd& a, int tpr, int rows, cudaStream_t s) {
  return a.res_f32 ? run_norm_form<NV, true>(a, tpr, rows, s) : run_norm_form<NV, false>(a, tpr, rows, s);
}

template <bool RES32, int FORM>
cudaError_t run_norm_ring(const NormFwd& a, const RingShape& r, cudaStream_t s) {
  auto kern = add_rmsnorm_ring_kernel<3, RES32, FORM>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMost);
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
  // Rows of more than 4096 columns, four for every SM: through the ring, one row in work and 90 KB of them in flight on
  // an SM.  At 8192 x 7168 with per-row codes 83 us against 105 us for a block a row (few such wide blocks fit an SM, and
  // all of one waits at each of its barriers); two rows in work 95 us, two vectors a thread instead of three 95 us.
  // Narrower rows are as fast or faster with a block a row (32768 x 1536 fp32: 96 against 104 us).
  if (vec && a.d > 4096 && a.d <= 8192 && a.T >= 4ll * num_sms) {
    const size_t row = static_cast<size_t>(a.d) * ((a.x ? 2 : 0) + (a.res_f32 ? 4 : 2));
    const RingShape r = ring_shape(a.T, a.d, 3, row, 90 * 1024, num_sms);
    return a.res_f32 ? run_norm_ring_form<true>(a, r, s) : run_norm_ring_form<false>(a, r, s);
  }
  if (!vec) {
    if (phase_threads(a.d) <= 1024) {
      const PhaseOf t[] = {{a.res, a.ld_res, a.res_f32 != 0}, {a.x, a.ld_x, false}, {a.h, a.ld_h, a.res_f32 != 0}, {a.y, a.ld_y, false}};
      const PhaseOf& lead = a.x ? t[1] : a.res_f32 ? t[3] : t[0];  // what is read, if it is bf16
      const Phase f = phase_of(lead.p, lead.ld, t, 4);
      const PhaseShape p = phase_shape(a.T, a.d, 2048, num_sms);
      if (a.res_f32) add_rmsnorm_phase_kernel<true><<<p.grid, dim3(p.tpr, p.rows), 0, s>>>(a, f);
      else add_rmsnorm_phase_kernel<false><<<p.grid, dim3(p.tpr, p.rows), 0, s>>>(a, f);
      return cudaGetLastError();
    }
    const int tpr = round32((a.d + 15) / 16);
    if (a.res_f32) add_rmsnorm_any_kernel<true><<<static_cast<unsigned>(a.T), tpr, 0, s>>>(a);
    else add_rmsnorm_any_kernel<false><<<static_cast<unsigned>(a.T), tpr, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int nvec = a.d / 8;
  // Narrow rows share a block of 128 threads.
  if (nvec <= 1024) return run_norm<1>(a, round32(nvec), nvec <= 32 ? 4 : nvec <= 64 ? 2 : 1, s);
  return run_norm<2>(a, round32((nvec + 1) / 2), 1, s);
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

// A vector of xhat, of dy g and of the row's sum for c; dg's share grows.
__device__ __forceinline__ void bwd8(Vec8& dy, Vec8& h, const Vec8& g, Vec8& dg, f32x2 rstd2, f32x2& c) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h.p[k] = mul2(h.p[k], rstd2);
    dg.p[k] = fma2(dy.p[k], h.p[k], dg.p[k]);
    dy.p[k] = mul2(dy.p[k], g.p[k]);
    c = fma2(dy.p[k], h.p[k], c);
  }
}

// o += rstd (dy g) - rstd c xhat, stored in both forms asked for (dx, dres: the vector's places, null: nowhere).
template <bool RES32>
__device__ __forceinline__ void bwd_out8(void* dx, void* dres, Vec8& o, const Vec8& dy, const Vec8& h, f32x2 rstd2, f32x2 nc2) {
#pragma unroll
  for (int k = 0; k < 4; ++k) o.p[k] = fma2(nc2, h.p[k], fma2(rstd2, dy.p[k], o.p[k]));
  if (dx) store8<false>(dx, 0, o);
  if (dres) store8<RES32>(dres, 0, o);
}

template <int ES>
__device__ __forceinline__ uint8_t* place(void* base, long long t, long long ld, int j) {
  return base ? static_cast<uint8_t*>(base) + (t * ld + 8ll * j) * ES : nullptr;
}

// Rows wider than the ring takes, straight from global memory; the weight and dh are read where they are needed.
template <int NV, bool RES32>
__global__ void __launch_bounds__(512) add_rmsnorm_bwd_wide_kernel(const NormBwd a) {
  __shared__ float red[2][32];
  const int nvec = a.d / 8;
  Vec8 dg[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) dg[i] = zero8();
  griddep_launch();
  int it = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++it) {
    const float rstd = __ldg(a.rstd + t);
    const f32x2 rstd2 = pack2(rstd, rstd);
    Vec8 dy[NV], h[NV];
    f32x2 c2 = pack2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < nvec) {
        dy[i] = load8<false>(a.dy, t * a.ld_dy + 8ll * j);
        h[i] = load8<RES32>(a.h, t * a.ld_h + 8ll * j);
        bwd8(dy[i], h[i], load_weight8(a.weight, a.weight_f32, j), dg[i], rstd2, c2);
      }
    }
    const float2 cf = unpack2(c2);
    const float c = row_reduce<false>(cf.x + cf.y, red[it & 1]) / static_cast<float>(a.d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < nvec) {
        Vec8 o = a.dh ? load8<RES32>(a.dh, t * a.ld_dh + 8ll * j) : zero8();
        bwd_out8<RES32>(place<2>(a.dx, t, a.ld_dx, j), place<RES32 ? 4 : 2>(a.dres, t, a.ld_dres, j), o, dy[i], h[i], rstd2,
                        pack2(-rstd * c, -rstd * c));
      }
    }
  }
  // dweight may begin at any float, the shares' rows are aligned
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (j >= nvec) continue;
    if (gridDim.x > 1) {
      store8<true>(a.part + static_cast<long long>(blockIdx.x) * a.d, 8ll * j, dg[i]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 p = unpack2(dg[i].p[k / 2]);
        a.dweight[8 * j + k] = k % 2 ? p.y : p.x;
      }
    }
  }
}

// Rows that are not aligned and too wide for a vector a thread, 32 values a thread.
template <bool RES32>
__global__ void __launch_bounds__(512) add_rmsnorm_bwd_any_kernel(const NormBwd a) {
  constexpr int N = 32;
  __shared__ float red[2][32];
  float dg[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = 0.0f;
  griddep_launch();
  int it = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++it) {
    const float rstd = __ldg(a.rstd + t);
    float dy[N], h[N], c = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < a.d) {
        dy[i] = load1<false>(a.dy, t * a.ld_dy + j);
        h[i] = load1<RES32>(a.h, t * a.ld_h + j) * rstd;
        dg[i] += dy[i] * h[i];
        dy[i] *= load_weight1(a.weight, a.weight_f32, j);
        c += dy[i] * h[i];
      }
    }
    c = row_reduce<false>(c, red[it & 1]) / static_cast<float>(a.d);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = threadIdx.x + blockDim.x * i;
      if (j < a.d) {
        const float o = (a.dh ? load1<RES32>(a.dh, t * a.ld_dh + j) : 0.0f) + rstd * (dy[i] - c * h[i]);
        if (a.dx) store1<false>(a.dx, t * a.ld_dx + j, o);
        if (a.dres) store1<RES32>(a.dres, t * a.ld_dres + j, o);
      }
    }
  }
  float* out = gridDim.x == 1 ? a.dweight : a.part + static_cast<long long>(blockIdx.x) * a.d;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = threadIdx.x + blockDim.x * i;
    if (j < a.d) out[j] = dg[i];
  }
}

// Rows that start anywhere (see the forward).  1024 threads of 64 registers an SM: the bf16 form spills 36 bytes and takes
// 72 us at 8192 x 4001, without spills in 80 registers, and fewer rows in work, 89.
template <bool RES32>
__global__ void __launch_bounds__(1024) add_rmsnorm_bwd_phase_kernel(const NormBwd a, Phase f) {
  extern __shared__ __align__(16) float4 weights[];  // every thread's, which registers have no room for; then the shares
  __shared__ float red[2][8][32];
  griddep_launch();
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  const int d = a.d;
  const Cols w(f.of(t0), d, threadIdx.x);
  const int threads = blockDim.x * blockDim.y, me = threadIdx.y * blockDim.x + threadIdx.x;
  {
    const Vec8 g = weight_cols(a.weight, a.weight_f32, w);
    const float2 p0 = unpack2(g.p[0]), p1 = unpack2(g.p[1]), p2 = unpack2(g.p[2]), p3 = unpack2(g.p[3]);
    weights[me] = make_float4(p0.x, p0.y, p1.x, p1.y);
    weights[threads + me] = make_float4(p2.x, p2.y, p3.x, p3.y);
  }
  const float inv_d = 1.0f / static_cast<float>(d);
  Vec8 dg = zero8();
  uint4 dy_in{};
  Cols8<RES32> h_in{}, dh_in{};
  float rstd_in = 0.0f;
  constexpr bool kAhead = !RES32;
  auto fetch = [&](long long t) {  // a row ahead where the registers suffice (1024 threads of 64)
    if (t >= a.T) return;
    rstd_in = __ldg(a.rstd + t);
    dy_in = load_cols<false>(a.dy, t * a.ld_dy, w, true);
    h_in = load_cols<RES32>(a.h, t * a.ld_h, w, f.has(0));
    if (a.dh) dh_in = load_cols<RES32>(a.dh, t * a.ld_dh, w, f.has(1));
  };
  if (kAhead) fetch(t0);
  int it = 0;
  for (long long t = t0; t < a.T; t += step, ++it) {
    if (!kAhead) fetch(t);
    const float rstd = rstd_in;
    const f32x2 rstd2 = pack2(rstd, rstd);
    Vec8 dy = values(dy_in), h = values(h_in), o = values(dh_in);
    if (kAhead) fetch(t + step);
    f32x2 c2 = pack2(0.0f, 0.0f);
    bwd8(dy, h, from_f32(weights[me], weights[threads + me]), dg, rstd2, c2);
    const float2 cf = unpack2(c2);
    const float m = group_sum(cf.x + cf.y, red[it & 1][threadIdx.y]) * inv_d;
    const f32x2 nc2 = pack2(-rstd * m, -rstd * m);
#pragma unroll
    for (int k = 0; k < 4; ++k) o.p[k] = fma2(nc2, h.p[k], fma2(rstd2, dy.p[k], o.p[k]));
    if (a.dx) store_cols<false>(a.dx, t * a.ld_dx, w, f.has(2), o);
    if (a.dres) store_cols<RES32>(a.dres, t * a.ld_dres, w, f.has(3), o);
  }
  // the groups' shares, each in its own phase, added in group order
  float* out = gridDim.x == 1 ? a.dweight : a.part + static_cast<long long>(blockIdx.x) * d;
  float* shares = reinterpret_cast<float*>(weights + 2 * threads);
  float* mine = blockDim.y > 1 ? shares + threadIdx.y * d : out;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 p = unpack2(dg.p[k / 2]);
    if (k < w.n) mine[w.c + k] = k % 2 ? p.y : p.x;
  }
  if (blockDim.y == 1) return;
  __syncthreads();
  for (int j = me; j < d; j += threads) {
    float v = 0.0f;
    for (int r = 0; r < static_cast<int>(blockDim.y); ++r) v += shares[r * d + j];
    out[j] = v;
  }
}

// Rows (dy, h and dh side by side) through the ring.
template <int NV, bool RES32>
__global__ void __launch_bounds__(512, 1) add_rmsnorm_bwd_ring_kernel(const NormBwd a, int stages) {
  constexpr int ES = RES32 ? 4 : 2;
  extern __shared__ __align__(128) uint8_t nb_ring[];
  __shared__ __align__(16) RingShared sh;
  const int rg = threadIdx.y, RG = blockDim.y, tx = threadIdx.x, tpr = blockDim.x;
  const int nvec = a.d / 8;
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
  griddep_launch();  // the launch that adds the blocks' shares waits for this one's end
  Vec8 g[NV], dg[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
    g[i] = dg[i] = zero8();
    if (j < nvec) g[i] = load_weight8(a.weight, a.weight_f32, j);
  }
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float rstd_next = t0 < a.T ? __ldg(a.rstd + t0) : 0.0f;
  uint8_t *dx = place<2>(a.dx, t0, a.ld_dx, tx), *dres = place<ES>(a.dres, t0, a.ld_dres, tx);
  int it = 0, st = 0, ph = 0;
  for (long long t = t0; t < a.T; t += step, ++it) {
    const float rstd = rstd_next;
    const f32x2 rstd2 = pack2(rstd, rstd);
    if (t + step < a.T) rstd_next = __ldg(a.rstd + t + step);
    mbar_wait(&sh.full[rg][st], ph, &sh.abort, a.timeout_ns, a.err);
    const uint8_t* src = ring + static_cast<size_t>(st) * sb;
    Vec8 dy[NV], h[NV], o[NV];
    f32x2 c2 = pack2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (j < nvec) {
        dy[i] = load_smem8<false>(src, j);
        h[i] = load_smem8<RES32>(src + dyb, j);
        o[i] = a.dh ? load_smem8<RES32>(src + dyb + hb, j) : zero8();
        bwd8(dy[i], h[i], g[i], dg[i], rstd2, c2);
      }
    }
    const float2 cf = unpack2(c2);
    float c = cf.x + cf.y, none = 0.0f;
    group_reduce<false>(c, none, sh.red[it & 1][rg], sh.red2[it & 1][rg]);
    c *= inv_d;
    if (tx == 0 && t + stages * step < a.T) issue(t + stages * step, st);
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
    const f32x2 nc2 = pack2(-rstd * c, -rstd * c);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = tx + tpr * i;
      if (j < nvec)
        bwd_out8<RES32>(dx ? dx + 16 * tpr * i : nullptr, dres ? dres + 8 * ES * tpr * i : nullptr, o[i], dy[i], h[i], rstd2, nc2);
    }
    if (dx) dx += step * a.ld_dx * 2;
    if (dres) dres += step * a.ld_dres * ES;
  }
  ring_drain(sh, stages, it);
  // the groups' shares, added in group order; a block of one group stores its vectors itself, but not to dweight, which
  // may begin at any float
  float* share = reinterpret_cast<float*>(nb_ring);
  float* out = gridDim.x == 1 ? a.dweight : a.part + static_cast<long long>(blockIdx.x) * a.d;
  const bool direct = RG == 1 && gridDim.x > 1;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tx + tpr * i;
    if (j < nvec) store8<true>(direct ? out : share + static_cast<size_t>(rg) * a.d, 8ll * j, dg[i]);
  }
  if (direct) return;
  __syncthreads();
  for (int j = rg * tpr + tx; j < a.d; j += RG * tpr) {
    float v = 0.0f;
    for (int r = 0; r < RG; ++r) v += share[static_cast<size_t>(r) * a.d + j];
    out[j] = v;
  }
}

// out[j] = sum_b part[b][j]: 32 columns a block, 32 threads of partial sums each, four loads in flight, added in a fixed
// order.  A dependent launch: it is set up while the rows are still worked on.
__global__ void __launch_bounds__(1024) reduce_rows_kernel(const float* __restrict__ part, int parts, int d,
                                                           float* __restrict__ out) {
  __shared__ float sm[32][33];
  griddep_wait();
  const int j = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  for (int b0 = threadIdx.y; b0 < parts; b0 += 128) {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = j < d && b0 + 32 * k < parts ? part[static_cast<long long>(b0 + 32 * k) * d + j] : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) v += x[k];
  }
  sm[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = sm[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int jo = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && jo < d) out[jo] = v;
}

template <int NV, bool RES32>
cudaError_t run_norm_bwd_ring(const NormBwd& a, const RingShape& r, cudaStream_t s) {
  auto kern = add_rmsnorm_bwd_ring_kernel<NV, RES32>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMost);
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
    // 144 KB of rows in flight on an SM: 8192 x 5120 fp32 (51 KB a row) takes 105 us with two rows and 116 with three,
    // 8192 x 7168 bf16 (43 KB) 74 us with three and 80 with two.  One vector a thread for narrow rows and for fp32
    // streams, which bring twice the work a vector (32768 x 1536 fp32: 119 us against 140 with two), else two (8192 x
    // 1024 bf16: 17.9 against 19.5).
    const bool one = a.d <= (a.res_f32 ? 4096 : 256);
    const RingShape r = ring_shape(a.T, a.d, one ? 1 : 2, row, 144 * 1024, num_sms);
    parts = r.grid;
    if (one) e = a.res_f32 ? run_norm_bwd_ring<1, true>(a, r, s) : run_norm_bwd_ring<1, false>(a, r, s);
    else e = a.res_f32 ? run_norm_bwd_ring<2, true>(a, r, s) : run_norm_bwd_ring<2, false>(a, r, s);
  } else if (!vec && phase_threads(a.d) <= 1024) {
    const bool f32 = a.res_f32 != 0;
    const PhaseOf t[] = {{a.h, a.ld_h, f32}, {a.dh, a.ld_dh, f32}, {a.dx, a.ld_dx, false}, {a.dres, a.ld_dres, f32}};
    const Phase f = phase_of(a.dy, a.ld_dy, t, 4);
    const PhaseShape p = phase_shape(a.T, a.d, 1024, num_sms < 256 ? num_sms : 256);
    parts = p.grid;
    const size_t smem = 32 * static_cast<size_t>(p.tpr) * p.rows + (p.rows > 1 ? sizeof(float) * p.rows * a.d : 0);  // up to 32 KB
    if (a.res_f32) add_rmsnorm_bwd_phase_kernel<true><<<p.grid, dim3(p.tpr, p.rows), smem, s>>>(a, f);
    else add_rmsnorm_bwd_phase_kernel<false><<<p.grid, dim3(p.tpr, p.rows), smem, s>>>(a, f);
    e = cudaGetLastError();
  } else {
    const long long most = 4ll * num_sms < kMaxNormParts ? 4ll * num_sms : kMaxNormParts;
    parts = static_cast<int>(a.T < most ? a.T : most);
    const int tpr = vec ? round32((a.d / 8 + 3) / 4) : round32((a.d + 31) / 32);
    if (vec && a.res_f32) add_rmsnorm_bwd_wide_kernel<4, true><<<parts, tpr, 0, s>>>(a);
    else if (vec) add_rmsnorm_bwd_wide_kernel<4, false><<<parts, tpr, 0, s>>>(a);
    else if (a.res_f32) add_rmsnorm_bwd_any_kernel<true><<<parts, tpr, 0, s>>>(a);
    else add_rmsnorm_bwd_any_kernel<false><<<parts, tpr, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || parts == 1) return e;
  return launch_dependent(reduce_rows_kernel, dim3((a.d + 31) / 32), dim3(32, 32), 0, s, static_cast<const float*>(a.part), parts,
                          a.d, a.dweight);
}

}  // namespace vgg
