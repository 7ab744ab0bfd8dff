// The whole layer for a few tokens (a decoding step): router, choice, the chosen experts' products, weighted sum, in
// two launches.
//
//   logits = X W_r + b;  the K largest, w = softmax over them;  O[t] = sum_k w_k W_down[e_k] (silu(W_gate[e_k] x) W_up[e_k] x)
//
// A call reads every chosen expert's weights once and computes little on them, so it is bound by HBM; what costs beside
// that is the chain of dependent steps.  The design follows from both:
//   * the weights are the 128-row operand of the tensor cores and the tokens the narrow one (N = 16 .. 128 columns), so a
//     weight tile moves once through shared memory whatever the number of tokens;
//   * the stages (128 weight rows x 128 bytes of the reduction) of all chosen experts form one list, of which each of the
//     persistent blocks takes an equal, contiguous share: blocks finish together whatever the sizes and the choice.
//     An output tile that several blocks share is summed from their parts in block order, so results do not depend
//     on which of them ends last;
//   * both products run in one launch, and the loads of the second do not wait for the first: the producers go on to
//     W_down's stages while the activations are still being made, so HBM keeps working through that step.
//
// bf16: A = silu(H) U enters the second product as its bf16 value and the bf16 rounding of the rest, as further columns
// of the same tile (they cost nothing: the products are far below the tensor cores' rate).  e4m3: X quantized per token
// and A (rounded to bf16) per pair, as moe_quantize_rows_e4m3 does.  Sums are fp32; O is rounded once.
#include <cuda_fp8.h>

#include "internal.h"

namespace vgg {

namespace {

constexpr int kEpi = 4;      // epilogue warps 0..3 (TMEM lanes 32 w ..)
constexpr int kGath = 8;     // gather warps
constexpr int kProd = 4;     // TMA producers: loads issued by one thread complete one after another
constexpr int kGath0 = kEpi, kMma = kEpi + kGath, kProd0 = kMma + 1;
constexpr int kWarps = kProd0 + kProd;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 128;             // weight rows of a tile
constexpr int kWBytes = kRows * 128;   // weight bytes of a stage
constexpr int kMaxPairs = kFewMaxTokens * 8;
constexpr int kMaxStages = 12;
// Every block finds the choice of so few tokens itself; of more, each is found by one block behind a barrier (a block
// reads splits x T x E partial logits otherwise).
constexpr int kOwnChoice = 8;

struct Lists {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  uint32_t tmem;
  volatile int abort;
  int active, last, ok;
  float pw[kMaxPairs];         // [token][rank]: combine weight, experts of a token ascending
  uint16_t act_e[kMaxPairs];   // expert of each chosen expert's index, ascending
  uint16_t act_off[kMaxPairs + 1];  // its first pair
  uint16_t tok_pair[kMaxPairs], tok_a[kMaxPairs];  // [token][rank]: pair, index of its expert
  uint8_t ptok[kMaxPairs];     // token of a pair
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 -> +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

__device__ __forceinline__ void red_release(int* p) { asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory"); }

// Waits (bounded) until *p >= target, acquiring what the arrivals released.
__device__ __forceinline__ bool wait_count(const int* p, int target, volatile int* abort_flag, unsigned long long timeout_ns,
                                           int* err) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= target) return true;
    if ((i & 15u) != 15u) continue;
    if (*abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > timeout_ns) {
      *abort_flag = 1;
      set_error(err, DERR_TIMEOUT);
      return false;
    }
  }
}

// The blocks' shares of a list of S stages: block b has [b S / G, (b + 1) S / G).
struct Share {
  long long S;
  int G;
  __device__ __forceinline__ long long begin(int b) const { return b >= G ? S : b * S / G; }
  __device__ __forceinline__ int owner(long long s) const { return static_cast<int>(((s + 1) * G - 1) / S); }
};

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpi) : "memory"); }

// The same barrier; true when every epilogue thread says so.
__device__ __forceinline__ bool epi_all(bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(v)), "n"(32 * kEpi)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  return amax_bits ? __fdiv_rn(__uint_as_float(amax_bits), 448.0f) : 1.0f;
}

// 16 bf16 values to 16 codes of a row with scale s.
__device__ __forceinline__ uint4 codes16(const uint4 x, const uint4 y, float s) {
  const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_bf16x2(v[2 * i]), b = unpack_bf16x2(v[2 * i + 1]);
    w[i] = e4m3x4(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s), __fdiv_rn(b.x, s), __fdiv_rn(b.y, s));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

// ---- first launch: parts of the logits, X's codes, cleared counters -------------------------------------------------
// Blocks [0, strips * splits): 16 experts (32 bytes of every row of W_r, a memory sector) times a share of d: part[split][t][e].
// Thread: two experts (tid & 7) and every 32nd row of the share; NT tokens at a time.  The blocks behind clear the counters
// and, for the e4m3 form, quantize a token each.
template <int NT>
__global__ void __launch_bounds__(256) few_router_kernel(const __grid_constant__ FewArgs a) {
  __shared__ float red[8][NT][16];
  __shared__ float s_top[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int strips = (a.E + 15) / 16;
  const int b = blockIdx.x;
  if (b >= strips * a.splits) {
    const int q = b - strips * a.splits;
    if (q == 0) {
      for (int i = tid; i < a.nctr; i += 256) a.ctr[i] = 0;
      for (int i = tid; i < a.T * a.K; i += 256) a.amax[i] = 0;
    }
    if (!a.xq) return;
    for (int t = q; t < a.T; t += gridDim.x - strips * a.splits) {
      const uint4* row = reinterpret_cast<const uint4*>(a.X + t * a.ld_x);
      const int vecs = a.d / 16;  // pairs of vectors, 16 codes each
      float top = 0.0f;
      for (int v = tid; v < 2 * vecs; v += 256) {
        const uint4 x = __ldg(row + v);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack_bf16x2(w[i]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      __syncthreads();
      if (lane == 0) s_top[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) top = fmaxf(top, s_top[w]);
      const float s = row_scale(__float_as_uint(top));
      if (tid == 0) a.xs[t] = s;
      uint4* dst = reinterpret_cast<uint4*>(a.xq + static_cast<long long>(t) * a.d);
      for (int v = tid; v < vecs; v += 256) dst[v] = codes16(__ldg(row + 2 * v), __ldg(row + 2 * v + 1), s);
    }
    return;
  }
  const int strip = b % strips, split = b / strips;
  const int r0 = static_cast<int>(static_cast<long long>(a.d) * split / a.splits);
  const int r1 = static_cast<int>(static_cast<long long>(a.d) * (split + 1) / a.splits);
  const int e0 = strip * 16 + 2 * (tid & 7);
  const bool in = e0 < a.E;  // E is a multiple of 8: a pair is in or out
  const int rg = tid >> 3;
  for (int t0 = 0; t0 < a.T; t0 += NT) {
    float acc[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = 0.0f;
    if (in) {
#pragma unroll 4
      for (int r = r0 + rg; r < r1; r += 32) {
        const float2 w = unpack_bf16x2(__ldg(reinterpret_cast<const uint32_t*>(a.W_r + static_cast<long long>(r) * a.E + e0)));
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float x = t0 + i < a.T ? __bfloat162float(__ldg(a.X + (t0 + i) * a.ld_x + r)) : 0.0f;
          acc[i][0] = fmaf(x, w.x, acc[i][0]);
          acc[i][1] = fmaf(x, w.y, acc[i][1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], 8);
        acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], 16);
      }
      if (lane < 8) {
        red[warp][i][2 * lane] = acc[i][0];
        red[warp][i][2 * lane + 1] = acc[i][1];
      }
    }
    __syncthreads();
    for (int i = tid; i < NT * 16; i += 256) {
      const int t = t0 + i / 16, e = strip * 16 + i % 16;
      if (t < a.T && e < a.E) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += red[w][i / 16][i % 16];
        a.part[(static_cast<long long>(split) * a.T + t) * a.E + e] = s;
      }
    }
    __syncthreads();
  }
}

// One warp finds token t's choice: its logits as order keys in keys[E] (shared memory), then K rounds of the largest key, the
// lower expert among equal ones (the rule of moe_route).  Lane k < K returns the k-th choice and its weight.
__device__ __forceinline__ void choose(const FewArgs& a, int t, uint32_t* keys, int& id, float& w) {
  const int lane = threadIdx.x & 31;
  const long long plane = static_cast<long long>(a.T) * a.E;
  const float* row = a.part + static_cast<long long>(t) * a.E;
  for (int e = lane; e < a.E; e += 32) {
    float v = __ldcg(row + e);
#pragma unroll 8
    for (int sp = 1; sp < a.splits; ++sp) v += __ldcg(row + sp * plane + e);
    if (a.bias) v += __ldg(a.bias + e);
    keys[e] = max(order_key(v), 1u);
  }
  float vmax = 0.0f, sum = 0.0f, ex_k = 0.0f;
  id = 0;
  for (int k = 0; k < a.K; ++k) {
    uint32_t bk = 0;
    int be = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32) {
      const uint32_t q = keys[e];
      if (q > bk) {
        bk = q;
        be = e;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    const int e = __reduce_min_sync(0xffffffffu, bk == top ? be : 0x7fffffff);
    if ((e & 31) == lane) keys[e] = 0;
    const float v = key_value(top);
    if (k == 0) vmax = v;
    const float ex = expf(v - vmax);
    sum += ex;
    if (lane == k) {
      id = e;
      ex_k = ex;
    }
  }
  w = ex_k / sum;
}

template <bool F8>
__global__ void __launch_bounds__(kThreads, 1) few_layer_kernel(const __grid_constant__ FewArgs a,
                                                               const __grid_constant__ CUtensorMap mg,
                                                               const __grid_constant__ CUtensorMap mu,
                                                               const __grid_constant__ CUtensorMap md) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kWBytes + a.nrows * 128;
  Lists& L = *reinterpret_cast<Lists*>(ring + a.stages * stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x, b = blockIdx.x;
  const int P = a.T * a.K;
  const int acc_cols = a.nrows <= 16 ? 16 : a.nrows <= 32 ? 32 : a.nrows <= 64 ? 64 : 128;  // of an accumulator
  const uint32_t tmem_cols = 2 * acc_cols;  // two of them: a power of two, 32 at least

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&L.full[s], 1 + 32 * kGath);
      mbar_init(&L.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&L.tfull[i], 1);
      mbar_init(&L.tempty[i], 32 * kEpi);
    }
    mbar_init(&L.drain, 1);
    L.abort = 0;
    L.ok = 1;
    fence_mbar_init();
    tma_prefetch_desc(&mg);
    tma_prefetch_desc(&mu);
    tma_prefetch_desc(&md);
  }
  if (warp == kMma) tmem_alloc(&L.tmem, tmem_cols);

  // ---- the choice, and the pairs grouped by expert (the ring's memory is scratch until the first load) ----
  uint32_t* keys = reinterpret_cast<uint32_t*>(ring) + warp * a.E;
  int* s_ids = reinterpret_cast<int*>(ring) + kWarps * a.E;  // [P]
  float* s_w = reinterpret_cast<float*>(s_ids + kMaxPairs);
  uint64_t* s_mask = reinterpret_cast<uint64_t*>(s_w + kMaxPairs);  // [E] tokens of each expert
  uint16_t* s_eoff = reinterpret_cast<uint16_t*>(s_mask + a.E);      // [E] first pair, index
  uint16_t* s_ea = s_eoff + a.E;
  for (int e = tid; e < a.E; e += kThreads) s_mask[e] = 0;
  if (a.T <= kOwnChoice) {
    if (warp < a.T) {
      int id;
      float w;
      choose(a, warp, keys, id, w);
      if (lane < a.K) {
        s_ids[warp * a.K + lane] = id;
        s_w[warp * a.K + lane] = w;
        if (b == 0) {
          a.ids[warp * a.K + lane] = id;
          a.w[warp * a.K + lane] = w;
        }
      }
    }
    __syncthreads();
  } else {
    for (int t = b + warp * G; t < a.T; t += kWarps * G) {
      int id;
      float w;
      choose(a, t, keys, id, w);
      if (lane < a.K) {
        a.ids[t * a.K + lane] = id;
        a.w[t * a.K + lane] = w;
      }
      __syncwarp();
      if (lane == 0) red_release(&a.ctr[0]);
    }
    if (tid == 0) L.ok = wait_count(&a.ctr[0], a.T, &L.abort, a.timeout_ns, a.err) ? 1 : 0;
    __syncthreads();
    if (L.ok)
      for (int i = tid; i < P; i += kThreads) {
        s_ids[i] = __ldcg(a.ids + i);
        s_w[i] = __ldcg(a.w + i);
      }
    __syncthreads();
  }
  const bool ok = L.ok != 0;  // the wait gave up: nothing below runs
  if (ok)
    for (int i = tid; i < P; i += kThreads)
      atomicOr(reinterpret_cast<unsigned long long*>(&s_mask[s_ids[i]]), 1ull << (i / a.K));
  __syncthreads();
  if (warp == 0) {
    int run = 0, act = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int cnt = (ok && e < a.E) ? __popcll(s_mask[e]) : 0;
      int v = cnt | (cnt ? 1 << 16 : 0), incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int excl = incl - v;
      if (cnt) {
        const int ai = act + (excl >> 16);
        s_eoff[e] = static_cast<uint16_t>(run + (excl & 0xffff));
        s_ea[e] = static_cast<uint16_t>(ai);
        L.act_e[ai] = static_cast<uint16_t>(e);
        L.act_off[ai] = static_cast<uint16_t>(run + (excl & 0xffff));
      }
      const int tot = __shfl_sync(0xffffffffu, incl, 31);
      run += tot & 0xffff;
      act += tot >> 16;
    }
    if (lane == 0) {
      L.active = act;
      L.act_off[act] = static_cast<uint16_t>(run);
    }
  }
  __syncthreads();
  if (ok)
    for (int i = tid; i < P; i += kThreads) {
      const int t = i / a.K, e = s_ids[i];
      const int p = s_eoff[e] + __popcll(s_mask[e] & ((1ull << t) - 1ull));
      L.ptok[p] = static_cast<uint8_t>(t);
      int rank = 0;
      for (int k = 0; k < a.K; ++k) rank += s_ids[t * a.K + k] < e;
      L.tok_pair[t * a.K + rank] = static_cast<uint16_t>(p);
      L.tok_a[t * a.K + rank] = s_ea[e];
      L.pw[t * a.K + rank] = s_w[i];
    }
  fence_proxy_async_smem();  // the scratch's uses come before the copies that overwrite it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = L.tmem;
  const int A = L.active;

  // ---- the two lists of stages ----
  const int es = F8 ? 1 : 2;
  const int t1 = a.n / 64, c1 = (a.d * es + 127) / 128;           // tiles of an expert, stages of a tile
  const int t2 = (a.d + kRows - 1) / kRows, c2 = (a.n * es + 127) / 128;
  Share sh[2];
  sh[0].S = static_cast<long long>(A) * t1 * c1;
  sh[1].S = static_cast<long long>(A) * t2 * c2;
  sh[0].G = static_cast<int>(sh[0].S < G ? sh[0].S : G);
  sh[1].G = static_cast<int>(sh[1].S < G ? sh[1].S : G);
  auto columns = [&](int ph, int m) { return (!F8 && ph == 1) ? 2 * ((m + 7) & ~7) : (m + 15) & ~15; };

  if (warp >= kProd0) {
    // ---------------------------------------------------------------- weights (lane 0 of each producer warp)
    if (lane == 0) {
      const int pj = warp - kProd0;
      int it = 0, s = 0;
      uint32_t par = 1;  // parity of the empty barrier's wait
      bool stop = false;
      for (int ph = 0; ph < 2 && !stop; ++ph) {
        const int c = ph ? c2 : c1;
        const long long end = sh[ph].begin(b + 1);
        for (long long q = sh[ph].begin(b); q < end && !stop; ++q, ++it) {
          if ((it & (kProd - 1)) == pj) {
            const long long item = q / c;
            const int k = static_cast<int>(q - item * c) * 64;
            if (!mbar_wait(&L.empty[s], par, &L.abort, a.timeout_ns, a.err)) {
              stop = true;
              break;
            }
            uint8_t* dst = ring + s * stage_bytes;
            mbar_arrive_expect_tx(&L.full[s], kWBytes);
            if (ph == 0) {
              const int ai = static_cast<int>(item / t1), tile = static_cast<int>(item - static_cast<long long>(ai) * t1);
              const int e = L.act_e[ai];
              tma_load_3d(dst, &mg, &L.full[s], k, tile * 64, e);
              tma_load_3d(dst + kWBytes / 2, &mu, &L.full[s], k, tile * 64, e);
            } else {
              const int tile = static_cast<int>(item / A), ai = static_cast<int>(item - static_cast<long long>(tile) * A);
              tma_load_3d(dst, &md, &L.full[s], k, tile * kRows, L.act_e[ai]);
            }
          }
          if (++s == a.stages) {
            s = 0;
            par ^= 1;
          }
        }
      }
      if (stop) {  // let the copies in flight land before the block goes away
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp >= kGath0 && warp < kGath0 + kGath) {
    // ---------------------------------------------------------------- the tokens' rows
    // Thread: the 16-byte piece c16 of rows rsub and rsub + 32 of every stage.  Rows past the expert's tokens hold
    // whatever was there: they are columns of their own in the product.
    const int ptid = tid - 32 * kGath0, c16 = ptid & 7, rsub = ptid >> 3;
    int s = 0;
    uint32_t par = 1;
    bool stop = false;
    for (int ph = 0; ph < 2 && !stop; ++ph) {
      const int c = ph ? c2 : c1;
      const long long end = sh[ph].begin(b + 1);
      long long q = sh[ph].begin(b);
      if (ph == 1 && q < end) {
        // every pair's activations are there
        int go = 0;
        if (lane == 0) go = wait_count(&a.ctr[1], A * t1, &L.abort, a.timeout_ns, a.err) ? 1 : 0;
        __syncwarp();
        stop = !__shfl_sync(0xffffffffu, go, 0);
      }
      while (q < end && !stop) {
        const long long item = q / c;
        int k = static_cast<int>(q - item * c);
        const int k1 = static_cast<int>(min(static_cast<long long>(c), k + (end - q)));
        const int ai = ph == 0 ? static_cast<int>(item / t1) : static_cast<int>(item % A);
        const int p0 = L.act_off[ai], m = L.act_off[ai + 1] - p0;
        const int mh = (m + 7) & ~7;
        // this thread's rows of the tile: source row and, of the second product's e4m3 form, its scale
        const uint8_t* src[4];
        float sc[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        const int rows = (!F8 && ph == 1) ? mh + m : m;
        const int kbytes = ph == 0 ? a.d * es : a.n * (F8 ? 1 : 2);  // bytes of an operand row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int r = rsub + 32 * i;
          src[i] = nullptr;
          if (r >= rows) continue;
          if (ph == 0) {
            const long long t = L.ptok[p0 + r];
            src[i] = F8 ? a.xq + t * a.d : reinterpret_cast<const uint8_t*>(a.X + t * a.ld_x);
          } else if (F8) {
            src[i] = reinterpret_cast<const uint8_t*>(a.A + static_cast<long long>(p0 + r) * a.n);
            sc[i] = row_scale(__ldcg(a.amax + p0 + r));
          } else if (r < m) {
            src[i] = reinterpret_cast<const uint8_t*>(a.A + static_cast<long long>(p0 + r) * a.n);
          } else if (r >= mh) {
            src[i] = reinterpret_cast<const uint8_t*>(a.A_lo + static_cast<long long>(p0 + r - mh) * a.n);
          }
        }
        for (; k < k1; ++k, ++q) {
          if (!mbar_wait(&L.empty[s], par, &L.abort, a.timeout_ns, a.err)) {
            stop = true;
            break;
          }
          uint8_t* tok = ring + s * stage_bytes + kWBytes;
          const int off = k * 128 + c16 * 16;
          const bool in = off < kbytes;  // a last stage half past the reduction reads zeros (the weights do, too)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!src[i]) continue;
            const uint32_t o = sw128_offset(rsub + 32 * i, c16);
            if (F8 && ph == 1) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (in) {
                const uint4* x = reinterpret_cast<const uint4*>(src[i] + 2 * off);
                v = codes16(__ldcg(x), __ldcg(x + 1), sc[i]);
              }
              *reinterpret_cast<uint4*>(tok + o) = v;
            } else {
              cp_async_16(smem_u32(tok) + o, in ? src[i] + off : src[i], in ? 16u : 0u);
            }
          }
          if (F8 && ph == 1) {
            fence_proxy_async_smem();
            mbar_arrive(&L.full[s]);
          } else {
            cp_async_mbar_arrive_noinc(&L.full[s]);
          }
          if (++s == a.stages) {
            s = 0;
            par ^= 1;
          }
        }
      }
    }
    cp_async_wait_all();
  } else if (warp == kMma) {
    // ---------------------------------------------------------------- the products (lane 0)
    if (lane == 0) {
      int s = 0, acc = 0;
      uint32_t par = 0;
      bool stop = false;
      for (int ph = 0; ph < 2 && !stop; ++ph) {
        const int c = ph ? c2 : c1;
        const long long end = sh[ph].begin(b + 1);
        for (long long q = sh[ph].begin(b); q < end && !stop; ++acc) {
          const long long item = q / c;
          const int k0 = static_cast<int>(q - item * c);
          const int k1 = static_cast<int>(min(static_cast<long long>(c), k0 + (end - q)));
          const int ai = ph == 0 ? static_cast<int>(item / t1) : static_cast<int>(item % A);
          const int N = columns(ph, L.act_off[ai + 1] - L.act_off[ai]);
          const uint32_t idesc = F8 ? idesc_e4m3(kRows, N, 0, 0) : idesc_bf16(kRows, N, 0, 0);
          if (!mbar_wait(&L.tempty[acc & 1], ((acc >> 1) & 1) ^ 1, &L.abort, a.timeout_ns, a.err)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + (acc & 1) * acc_cols;
          for (int k = k0; k < k1; ++k, ++q) {
            if (!mbar_wait(&L.full[s], par, &L.abort, a.timeout_ns, a.err)) {
              stop = true;
              break;
            }
            fence_proxy_async_smem();  // cp.async writes -> operand reads
            tc_fence_after();
            const uint32_t sa = smem_u32(ring + s * stage_bytes), sb = sa + kWBytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_step<F8>(d_tmem, sdesc_sw128(sa + kk * 32, 16, 1024), sdesc_sw128(sb + kk * 32, 16, 1024), idesc,
                            (k != k0 || kk) ? 1u : 0u);
            umma_commit(&L.empty[s]);
            if (++s == a.stages) {
              s = 0;
              par ^= 1;
            }
          }
          if (!stop) umma_commit(&L.tfull[acc & 1]);
        }
      }
      if (L.abort) {
        umma_commit(&L.drain);
        volatile int never = 0;
        mbar_wait(&L.drain, 0, &never, 20000000ull, nullptr);
      }
    }
  } else {
    // ---------------------------------------------------------------- accumulators out (warps 0..3)
    // Warp w's lanes hold rows 32 w .. of the tile, a column per token.  The part of the block that has an item's first
    // stage goes to the item's place, another block's to that block's own overflow rows (a block goes on with at most one
    // item that began elsewhere).
    const int row = tid;
    int acc = 0;
    bool stop = false;
    for (int ph = 0; ph < 2 && !stop; ++ph) {
      const int c = ph ? c2 : c1;
      const long long end = sh[ph].begin(b + 1);
      long long q = sh[ph].begin(b);
      const bool any = q < end;
      const long long ld = ph ? static_cast<long long>(t2) * kRows : static_cast<long long>(t1) * kRows;
      for (; q < end; ++acc) {
        const long long item = q / c;
        const int k0 = static_cast<int>(q - item * c);
        const int k1 = static_cast<int>(min(static_cast<long long>(c), k0 + (end - q)));
        q += k1 - k0;
        const int ai = ph == 0 ? static_cast<int>(item / t1) : static_cast<int>(item % A);
        const int tile = ph == 0 ? static_cast<int>(item % t1) : static_cast<int>(item / A);
        const int p0 = L.act_off[ai], m = L.act_off[ai + 1] - p0, mh = (m + 7) & ~7;
        // one verdict for all: a thread alone at the barriers below would wait for ever
        if (!epi_all(mbar_wait(&L.tfull[acc & 1], (acc >> 1) & 1, &L.abort, a.timeout_ns, a.err))) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem + (static_cast<uint32_t>(warp * 32) << 16) + (acc & 1) * acc_cols;
        float* dst;
        long long step;
        if (k0 == 0) {
          dst = (ph ? a.y : a.hu) + p0 * ld + tile * kRows + row;
          step = ld;
        } else {
          dst = (ph ? a.ov2 : a.ov1) + static_cast<long long>(b) * a.T * kRows + row;
          step = kRows;
        }
        for (int j0 = 0; j0 < m; j0 += 8) {
          float v[8];
          tmem_ld8(tb + j0, v);
          if (!F8 && ph == 1) {
            float lo[8];
            tmem_ld8(tb + mh + j0, lo);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += lo[i];
          } else {
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (j0 + i < m) __stcg(dst + (j0 + i) * step, v[i]);
        }
        tc_fence_before();
        mbar_arrive(&L.tempty[acc & 1]);
        if (ph == 1) continue;
        // first product: who completes the item makes its activations
        int b0 = b, b1 = b;
        epi_sync();
        if (k1 - k0 < c) {
          b0 = sh[0].owner(item * c);
          b1 = sh[0].owner(item * c + c - 1);
          if (tid == 0) {
            __threadfence();
            L.last = atomicAdd(&a.ctr[4 + b0], 1) == b1 - b0;
            __threadfence();
          }
          epi_sync();
          if (!L.last) continue;
        }
        const int e = L.act_e[ai];
        for (int i = tid; i < m * 64; i += 32 * kEpi) {
          const int j = i >> 6, r = i & 63;
          const float* hu = a.hu + (p0 + j) * ld + tile * kRows + r;
          float h = __ldcg(hu), u = __ldcg(hu + 64);
          for (int o = b0 + 1; o <= b1; ++o) {
            const float* ov = a.ov1 + (static_cast<long long>(o) * a.T + j) * kRows + r;
            h += __ldcg(ov);
            u += __ldcg(ov + 64);
          }
          if (F8) {
            const float sx = __ldcg(a.xs + L.ptok[p0 + j]);
            const long long col = static_cast<long long>(e) * a.n + tile * 64 + r;
            h *= sx * __ldg(a.wg_scale + col);
            u *= sx * __ldg(a.wu_scale + col);
          }
          const float act = h * sigmoidf_(h) * u;
          const __nv_bfloat16 hi = __float2bfloat16_rn(act);
          const long long at = static_cast<long long>(p0 + j) * a.n + tile * 64 + r;
          a.A[at] = hi;
          if (F8) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(__bfloat162float(hi))));
            if (lane == 0) atomicMax(a.amax + p0 + j, top);
          } else {
            a.A_lo[at] = __float2bfloat16_rn(act - __bfloat162float(hi));
          }
        }
        epi_sync();
        if (tid == 0) red_release(&a.ctr[1]);
      }
      if (ph == 1 && any && !stop) {
        epi_sync();
        if (tid == 0) red_release(&a.ctr[2]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, tmem_cols);
  // ---- the weighted sums, once every block's parts are there: eight lanes a token and four columns, one a choice ----
  if (tid == 0) L.ok = ok && !L.abort && wait_count(&a.ctr[2], sh[1].G, &L.abort, a.timeout_ns, a.err) ? 1 : 0;
  __syncthreads();
  if (!L.ok) return;
  const int quads = a.d / 4;
  const long long units = static_cast<long long>(a.T) * quads;
  const long long u1 = units * (b + 1) / G;
  for (long long u0 = units * b / G + 4 * warp; u0 < u1; u0 += 4 * kWarps) {
    const long long u = u0 + (lane >> 3);
    const int k = lane & 7;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int t = static_cast<int>(u < u1 ? u / quads : 0), col = static_cast<int>(u < u1 ? u - static_cast<long long>(t) * quads : 0) * 4;
    if (u < u1 && k < a.K) {
      const int p = L.tok_pair[t * a.K + k], ai = L.tok_a[t * a.K + k];
      const int tile = col / kRows, r = col % kRows;
      v = __ldcg(reinterpret_cast<const float4*>(a.y + static_cast<long long>(p) * t2 * kRows + col));
      const long long item = static_cast<long long>(tile) * A + ai;
      const int b0 = sh[1].owner(item * c2), b1 = sh[1].owner(item * c2 + c2 - 1);
      for (int o = b0 + 1; o <= b1; ++o) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(
            a.ov2 + (static_cast<long long>(o) * a.T + (p - L.act_off[ai])) * kRows + r));
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      float w = L.pw[t * a.K + k];
      if (F8) {
        w *= row_scale(__ldcg(a.amax + p));
        const float4 c = __ldg(reinterpret_cast<const float4*>(a.wd_scale + static_cast<long long>(L.act_e[ai]) * a.d + col));
        v.x *= c.x; v.y *= c.y; v.z *= c.z; v.w *= c.w;
      }
      v.x *= w; v.y *= w; v.z *= w; v.w *= w;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
      v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
    if (k == 0 && u < u1)
      *reinterpret_cast<uint2*>(a.O + t * a.ld_o + col) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

// ---- host -----------------------------------------------------------------------------------------------------------
int few_blocks(int num_sms) { return num_sms < kFewMaxBlocks ? num_sms : kFewMaxBlocks; }

FewLayout few_layout(int T, int d, int E, int n, int K) {
  FewLayout l{};
  size_t p = 0;
  auto take = [&](size_t bytes) {
    const size_t r = p;
    p += (bytes + 255) & ~static_cast<size_t>(255);
    return r;
  };
  const size_t P = static_cast<size_t>(T) * K;
  l.nctr = 4 + kFewMaxBlocks;
  l.ctr = take(sizeof(int) * l.nctr);
  l.amax = take(sizeof(uint32_t) * P);
  l.part = take(sizeof(float) * static_cast<size_t>(kFewMaxSplits) * T * E);
  l.xq = take(static_cast<size_t>(T) * d);
  l.xs = take(sizeof(float) * T);
  l.hu = take(sizeof(float) * P * 2 * n);
  l.A = take(sizeof(__nv_bfloat16) * P * n);
  l.A_lo = take(sizeof(__nv_bfloat16) * P * n);
  l.y = take(sizeof(float) * P * ((d + kRows - 1) / kRows) * kRows);
  l.ov1 = take(sizeof(float) * static_cast<size_t>(kFewMaxBlocks) * T * kRows);
  l.ov2 = take(sizeof(float) * static_cast<size_t>(kFewMaxBlocks) * T * kRows);
  l.bytes = p;
  return l;
}

cudaError_t launch_few_router(const FewArgs& args, int num_sms, cudaStream_t s) {
  const int strips = (args.E + 15) / 16;
  const int grid = strips * args.splits + (args.xq ? args.T : 1);
  if (args.T == 1) few_router_kernel<1><<<grid, 256, 0, s>>>(args);
  else few_router_kernel<8><<<grid, 256, 0, s>>>(args);
  return cudaGetLastError();
}

int few_splits(int d, int E, int num_sms) {
  const int strips = (E + 15) / 16;
  int sp = num_sms / strips;
  sp = sp < 1 ? 1 : sp > kFewMaxSplits ? kFewMaxSplits : sp;
  return sp > d / 64 ? d / 64 : sp;
}

template <bool F8>
static cudaError_t launch(FewArgs args, const CUtensorMap& mg, const CUtensorMap& mu, const CUtensorMap& md, int num_sms,
                          cudaStream_t s) {
  auto kern = few_layer_kernel<F8>;
  // rows of the narrow operand: as many columns as an expert's product may have
  args.nrows = F8 ? (args.T + 15) / 16 * 16 : (args.T + 7) / 8 * 16;
  const int stage_bytes = kWBytes + args.nrows * 128;
  const int room = static_cast<int>(kMaxSmem) - 1024 - static_cast<int>(sizeof(Lists));
  args.stages = room / stage_bytes < kMaxStages ? room / stage_bytes : kMaxStages;
  const size_t smem = 1024 + static_cast<size_t>(args.stages) * stage_bytes + sizeof(Lists);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // blocks wait for one another's parts: all of them resident at once
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3(few_blocks(num_sms), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args, mg, mu, md);
}

cudaError_t launch_few_layer(const FewArgs& args, bool f8, const CUtensorMap& mg, const CUtensorMap& mu,
                             const CUtensorMap& md, int num_sms, cudaStream_t s) {
  return f8 ? launch<true>(args, mg, mu, md, num_sms, s) : launch<false>(args, mg, mu, md, num_sms, s);
}

}  // namespace vgg
