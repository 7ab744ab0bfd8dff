// The router's products for an additional logit gradient: dlogits into three bf16 parts, dW_r = X^T dlogits from them
// (dX = dlogits W_r^T runs on the shared GEMM template, on two of them).  The launches of one call follow one another as dependent
// launches: each sets itself up while the one ahead of it drains.
#include "internal.h"

namespace vgg {

namespace {

// x = hi + mid + lo with hi = bf16(x), mid = bf16(x - hi), lo = bf16(x - hi - mid): three times 8 bits hold an fp32
// significand, so a product with a bf16 matrix in three bf16 multiplications has fp32 operands' precision (two parts
// leave 2^-17 of a value, 2.4e-6 normwise, ten times the error of an fp32 product's sums).  parts: [PARTS][np].
// A value that rounds to infinity has bf16's largest number as its high part, an infinite one no other parts (infinity
// less itself would make NaN of every product).
template <int PARTS>
__global__ void __launch_bounds__(256) split_dlogits_kernel(const float* __restrict__ dl, long long n, long long np,
                                                            __nv_bfloat16* __restrict__ parts) {
  griddep_launch();
  const long long step = 4ll * gridDim.x * blockDim.x;
  for (long long i = 4ll * (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x); i < np; i += step) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < n) v = __ldcs(reinterpret_cast<const float4*>(dl + i));
    const bool far = is_far(v.x) || is_far(v.y) || is_far(v.z) || is_far(v.w);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      uint2 h = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      if (p == 0 && far) {
        const float4 f = make_float4(is_far(v.x) ? far_high(v.x) : v.x, is_far(v.y) ? far_high(v.y) : v.y,
                                     is_far(v.z) ? far_high(v.z) : v.z, is_far(v.w) ? far_high(v.w) : v.w);
        h = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
      }
      *reinterpret_cast<uint2*>(parts + p * np + i) = h;
      const float2 a = unpack_bf16x2(h.x), b = unpack_bf16x2(h.y);
      v = make_float4(v.x - a.x, v.y - a.y, v.z - b.x, v.w - b.y);
      if (p == 0 && far)
        v = make_float4(isinf(a.x) ? 0.0f : v.x, isinf(a.y) ? 0.0f : v.y, isinf(b.x) ? 0.0f : v.z, isinf(b.y) ? 0.0f : v.w);
    }
  }
}

// D[e, i] = sum_t dlogits[t, e] X[t, i] over a split's tokens: tiles of 128 experts x 256 columns, both operands read with
// the tokens outermost.  A step of 64 tokens takes the X tile once (32 KB) and multiplies it with the three parts' tiles
// (16 KB each) into one accumulator: 80 KB of shared memory filled for 1536 cycles of tensor work, where a reduction
// over three times the tokens (every part with its own copy of X) fills 144 KB and was bound by that (32768 x 1536 x 512:
// 102 us).  X and the parts have rings of their own, each slot free again as soon as its last product has run.
//
// The tensor cores' fp32 accumulator drops the bits that an addition shifts out, always towards zero: sums over 5461
// tokens in one accumulator came out 1.6e-5 too small.  So an accumulator takes two steps only (24 additions); the
// epilogue warps add it, rounded to nearest, to sums in registers while the next two run into the other one.
// Four steps cost 5 us less at 32768 x 1536 x 512 and leave 9.5e-7 normwise instead of 5.6e-7, one accumulator for all
// 10 us less and 1.9e-5.
//
// 32768 x 1536 x 512: 95 us, 155 GFLOP in the three products (1.6 PFLOP/s, tensor pipe 67% busy by its counter).
// 4096 x 2048 x 128: 12 us for four or five steps a block, their latency.
constexpr int kDwChunk = 2;                   // steps an accumulator takes
constexpr int kDwX = 3, kDwP = 6;             // slots of the rings
constexpr int kDwXBytes = 32768, kDwPBytes = 16384, kDwBox = 64 * 128;
constexpr size_t kDwSmem = 1024 + kDwX * kDwXBytes + kDwP * kDwPBytes + 8 * kStgBuf;
constexpr int kDwThreads = 352;  // 8 epilogue warps, X's and the parts' producers, the issuer

struct DwArgs {
  int E, d, Tp, chunk;  // chunk: tokens of a split, a multiple of 64
  int etiles, tiles, items;
  int wait_first;
  int* err;
  unsigned long long timeout_ns;
};

// Maps: X, the parts, the sums [splits][E][d].
__global__ void __launch_bounds__(kDwThreads, 1) router_dw_kernel(const DwArgs a, const __grid_constant__ CUtensorMap mx,
                                                                  const __grid_constant__ CUtensorMap mp,
                                                                  const __grid_constant__ CUtensorMap mo) {
  extern __shared__ uint8_t dw_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dw_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xs = smem;
  uint8_t* ps = smem + kDwX * kDwXBytes;
  __shared__ uint64_t full_x[kDwX], empty_x[kDwX], full_p[kDwP], empty_p[kDwP], tfull[2], tempty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kDwX; ++i) {
      mbar_init(&full_x[i], 1);
      mbar_init(&empty_x[i], 1);
    }
    for (int i = 0; i < kDwP; ++i) {
      mbar_init(&full_p[i], 1);
      mbar_init(&empty_p[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 256);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    if (lane == 0) {
      tma_prefetch_desc(&mx);
      tma_prefetch_desc(&mp);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // The kernel ahead is the split, or router_dx, which lets this one start only when the split has ended.  Only in the
  // first case is there something to wait for before the loads; the wait at the end keeps the launches' order.
  griddep_launch();
  if (a.wait_first) griddep_wait();
  // an item: a split (its tokens k0..) of a tile (its experts e0.., its columns i0..)
  struct Item {
    int sp, e0, i0, k0, steps;
  };
  auto item = [&](int n) {
    Item it;
    it.sp = n / a.tiles;
    const int tile = n % a.tiles;
    it.e0 = tile % a.etiles * 128;
    it.i0 = tile / a.etiles * 256;
    it.k0 = it.sp * a.chunk;
    it.steps = (min(a.Tp, it.k0 + a.chunk) - it.k0) / 64;
    return it;
  };
  if (warp == 8 && lane == 0) {  // X
    int n = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < a.items && ok; id += gridDim.x) {
      const Item it = item(id);
      for (int k = 0; k < it.steps; ++k, ++n) {
        const int s = n % kDwX;
        ok = mbar_wait(&empty_x[s], (n / kDwX & 1) ^ 1, &s_abort, a.timeout_ns, a.err);
        if (!ok) break;
        mbar_arrive_expect_tx(&full_x[s], kDwXBytes);
        tma_load_3d(xs + s * kDwXBytes, &mx, &full_x[s], 0, it.k0 + 64 * k, it.i0 / 64);
      }
    }
  } else if (warp == 9 && lane == 0) {  // the parts
    int n = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < a.items && ok; id += gridDim.x) {
      const Item it = item(id);
      for (int k = 0; k < it.steps && ok; ++k) {
        for (int p = 0; p < 3; ++p, ++n) {
          const int s = n % kDwP;
          ok = mbar_wait(&empty_p[s], (n / kDwP & 1) ^ 1, &s_abort, a.timeout_ns, a.err);
          if (!ok) break;
          mbar_arrive_expect_tx(&full_p[s], kDwPBytes);
          const int row = p * a.Tp + it.k0 + 64 * k;
          tma_load_2d(ps + s * kDwPBytes, &mp, &full_p[s], it.e0, row);
          tma_load_2d(ps + s * kDwPBytes + kDwBox, &mp, &full_p[s], it.e0 + 64, row);
        }
      }
    }
  } else if (warp == 10 && lane == 0) {  // the products
    constexpr uint32_t kIdesc = idesc_bf16(128, 256, 1, 1);
    int nx = 0, np = 0, acc = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < a.items && ok; id += gridDim.x) {
      const Item it = item(id);
      for (int k0 = 0; k0 < it.steps && ok; k0 += kDwChunk, ++acc) {
        const int buf = acc & 1;
        ok = mbar_wait(&tempty[buf], (acc >> 1 & 1) ^ 1, &s_abort, a.timeout_ns, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dt = tmem + buf * 256;
        for (int k = k0; k < min(k0 + kDwChunk, it.steps) && ok; ++k, ++nx) {
          const int sx = nx % kDwX;
          ok = mbar_wait(&full_x[sx], nx / kDwX & 1, &s_abort, a.timeout_ns, a.err);
          const uint32_t xb = smem_u32(xs + sx * kDwXBytes);
          for (int p = 0; p < 3 && ok; ++p, ++np) {
            const int sp = np % kDwP;
            ok = mbar_wait(&full_p[sp], np / kDwP & 1, &s_abort, a.timeout_ns, a.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t pb = smem_u32(ps + sp * kDwPBytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16(dt, sdesc_sw128(pb + kk * 2048, kDwBox, 1024), sdesc_sw128(xb + kk * 2048, kDwBox, 1024), kIdesc,
                        ((k - k0) | p | kk) != 0 ? 1u : 0u);
            umma_commit(&empty_p[sp]);
          }
          if (ok) umma_commit(&empty_x[sx]);
        }
        if (ok) umma_commit(&tfull[buf]);
      }
    }
    if (!ok) {  // the products in flight read shared memory and write TMEM
      umma_commit(&drain);
      volatile int never = 0;
      mbar_wait(&drain, 0, &never, 20000000ull, nullptr);
    }
  } else if (warp < 8) {  // the sums: a thread holds 128 columns of an expert, which leave through shared memory
    const int quarter = warp & 3, c0 = (warp >> 2) * 128;
    uint8_t* stg = ps + kDwP * kDwPBytes + warp * kStgBuf;
    int acc = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < a.items && ok; id += gridDim.x) {
      const Item it = item(id);
      float v[4][32];
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int q = 0; q < 32; ++q) v[b][q] = 0.0f;
      for (int k0 = 0; k0 < it.steps; k0 += kDwChunk, ++acc) {
        const int buf = acc & 1;
        // one verdict for the warp: what follows are its loads of the accumulator
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[buf], acc >> 1 & 1, &s_abort, a.timeout_ns, a.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t t0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * 256 + c0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t r[32];
          tmem_ld32(t0 + 32 * b, r);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q) v[b][q] += __uint_as_float(r[q]);
        }
        tc_fence_before();
        mbar_arrive(&tempty[buf]);
      }
      if (!ok) break;
      if (it.e0 + quarter * 32 >= a.E) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (it.i0 + c0 + 32 * b >= a.d) break;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        stage_row32(stg, lane, v[b], true);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&mo, stg, it.i0 + c0 + 32 * b, it.e0 + quarter * 32, it.sp);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait0();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_abort) linger();
  if (warp == 8) tmem_dealloc(tmem, 512);
  griddep_wait();
}

// out[i][e] = in[i][e] (or 0) + sum_s part[s][e][i]: tiles of 64 columns x 8 experts (whole 32-byte sectors on both
// sides), turned in shared memory.  Two threads share a place's splits and have theirs in flight at once: with one
// thread and four at a time 16 splits of 2048 x 128 took 5 us more.
__global__ void __launch_bounds__(256) router_dw_reduce_kernel(const float* __restrict__ part, int splits, int E, int d,
                                                               const float* in, float* out) {
  constexpr int kHalf = kMaxRouterSplit / 2;
  __shared__ __align__(16) float tile[2][8][68];
  griddep_wait();
  const int i0 = blockIdx.x * 64, e0 = blockIdx.y * 8, tx = threadIdx.x & 15, ty = threadIdx.x >> 4 & 7, tz = threadIdx.x >> 7;
  const long long plane = static_cast<long long>(E) * d;
  const float* src = part + tz * kHalf * plane + static_cast<long long>(e0 + ty) * d + i0 + 4 * tx;
  float4 x[kHalf], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int s = 0; s < kHalf; ++s)
    x[s] = tz * kHalf + s < splits ? __ldcs(reinterpret_cast<const float4*>(src + s * plane)) : v;
#pragma unroll
  for (int s = 0; s < kHalf; ++s) {
    v.x += x[s].x; v.y += x[s].y; v.z += x[s].z; v.w += x[s].w;
  }
  *reinterpret_cast<float4*>(&tile[tz][ty][4 * tx]) = v;
  __syncthreads();
  const int te = threadIdx.x & 7;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int ti = (threadIdx.x >> 3) + 32 * r;
    const long long at = static_cast<long long>(i0 + ti) * E + e0 + te;
    out[at] = (in ? in[at] : 0.0f) + (tile[0][te][ti] + tile[1][te][ti]);
  }
}

}  // namespace

cudaError_t launch_split_dlogits(const float* dlogits, long long T, long long Tp, int E, int nparts, __nv_bfloat16* parts,
                                 cudaStream_t s) {
  const long long np = Tp * E, want = (np / 4 + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want < 8192 ? want : 8192);
  if (np <= 0) return cudaSuccess;
  if (nparts == 2) split_dlogits_kernel<2><<<grid, 256, 0, s>>>(dlogits, T * E, np, parts);
  else split_dlogits_kernel<3><<<grid, 256, 0, s>>>(dlogits, T * E, np, parts);
  return cudaGetLastError();
}

cudaError_t launch_router_dw(const __nv_bfloat16* X, const __nv_bfloat16* parts, int T, int Tp, int d, int E, bool after_split,
                             int num_sms, float* sums, int* splits, int* err, unsigned long long timeout_ns, cudaStream_t s) {
  CUtensorMap mx, mp, mo;
  if (!make_chunked_map_2d(&mx, X, d, T, 4) || !make_map_2d(&mp, parts, E, 3 * static_cast<uint64_t>(Tp), E, 64))
    return cudaErrorInvalidValue;
  DwArgs a{};
  a.E = E;
  a.d = d;
  a.Tp = Tp;
  a.etiles = (E + 127) / 128;
  a.tiles = a.etiles * ((d + 255) / 256);
  const int steps = Tp / 64;
  int split = num_sms / a.tiles;  // about a tile for every SM, two steps of tokens each at least
  if (split > kMaxRouterSplit) split = kMaxRouterSplit;
  if (split > steps / 2) split = steps / 2;
  if (split < 1) split = 1;
  a.chunk = (steps + split - 1) / split * 64;
  split = (Tp + a.chunk - 1) / a.chunk;
  a.items = a.tiles * split;
  a.wait_first = after_split;
  a.err = err;
  a.timeout_ns = timeout_ns;
  *splits = split;
  if (!make_store_map_3d(&mo, sums, true, d, E, split, 32)) return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(router_dw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kDwSmem));
  if (e != cudaSuccess) return e;
  return launch_dependent(router_dw_kernel, dim3(a.items < num_sms ? a.items : num_sms), dim3(kDwThreads), kDwSmem, s, a, mx, mp, mo);
}

cudaError_t launch_router_dw_reduce(const float* sums, int splits, int d, int E, const float* in, float* out, cudaStream_t s) {
  return launch_dependent(router_dw_reduce_kernel, dim3(d / 64, E / 8), dim3(256), 0, s, sums, splits, E, d, in, out);
}

}  // namespace vgg
