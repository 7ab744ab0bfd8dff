// The whole layer for a few tokens (a decoding step): router, choice, the chosen experts' products, weighted sum, in
// two launches.
//
//   logits = X W_r + b;  the K largest, w = softmax over them;  O[t] = sum_k w_k W_down[e_k] (silu(W_gate[e_k] x) W_up[e_k] x)
//
// A call reads every chosen expert's weights once and computes little on them, so it is bound by HBM; what costs beside
// that is the chain of dependent steps.  The design follows from both:
//   * the weights are the 128-row operand of the tensor cores and the tokens the narrow one (N = 16 .. 128 columns), so a
//     weight tile moves once through shared memory whatever the number of tokens;
//   * the stages (256 weight rows x 128 bytes of the reduction) of all chosen experts form one list, of which each of the
//     persistent blocks takes an equal, contiguous share: blocks finish together whatever the sizes and the choice.
//     An output tile that several blocks share is summed from their parts in block order, so results do not depend
//     on which of them ends last;
//   * both products run in one launch, and the loads of the second do not wait for the first: the producers go on to
//     W_down's stages while the activations are still being made, so HBM keeps working through that step.
//
// A block runs through most of the code once or a few times, and fetches it from memory as it goes: loops are kept short rather
// than unrolled.
//
// Measured, a layer of a captured stack whose weights come from HBM (bf16, e4m3; tokens x d x experts x n): 1 x 2048 x 128 x 512
// 23.4 and 22 us, a chain of latencies (its 50 MB take 7.6); 4 tokens 44 and 35; 61 x 1536 x 512 x 256 134 to 136 us (5.5 TB/s) and 88;
// 24 x 2880 x 128 x 2880 with 4 choices 505 us (6.7 TB/s, what a copy reaches) and 284.  The layer's own path, 128 rows of
// tokens a tile in seven launches, takes 127 us for one token and 371 for the 61.
//
// bf16: A = silu(H) U enters the second product as its bf16 value and the bf16 rounding of the rest, as further columns
// of the same tile (they cost nothing: the products are far below the tensor cores' rate).  e4m3: X quantized per token
// and A (rounded to bf16) per pair, as moe_quantize_rows_e4m3 does.  Sums are fp32; O is rounded once.
#include <cuda_fp8.h>

#include "internal.h"

namespace vgg {

namespace {

constexpr int kEpi = 4;      // epilogue warps 0..3 (TMEM lanes 32 w ..)
constexpr int kGath = 6;     // gather warps: a stage of the ring each
constexpr int kProd = 2;     // TMA producers (loads issued by one thread complete one after another)
constexpr int kGath0 = kEpi, kMma = kEpi + kGath, kProd0 = kMma + 1;
constexpr int kWarps = kProd0 + kProd;
constexpr int kThreads = 32 * kWarps;
// A tile is two halves of 128 weight rows: the same rows of W_gate and W_up, so that the thread that holds a row of H holds that
// of U; or 256 rows of W_down.  The halves share the tokens' operand: its rows are gathered, and every step of the roles
// made, once for 32 KB of weights (with halves of 64 rows, 16 KB a stage: 61 x 1536 x 512 x 256 e4m3 101 us).
constexpr int kRows = 128;             // weight rows of a half
constexpr int kTile = 2 * kRows;
constexpr int kHBytes = kRows * 128;   // weight bytes of a half's stage
constexpr int kWBytes = 2 * kHBytes;
constexpr int kMaxPairs = kFewMaxTokens * 8;
// Tiles' accumulators, where TMEM has room: the second product's items may be as short as a stage, and a pair of accumulators
// leaves the products waiting for the epilogue's latency.
constexpr int kMaxAccs = 4;
// In lists of less than 100 stages a block, the bf16 form of up to so many tokens leaves the parts of H and U as they are, and the
// gather warps of the second product add them up and make the activations as they fill a stage: an atomic and a round trip through
// L2 fewer in the chain, for a sum that every row tile of W_down repeats (layers of a stack: 1 x 2048 x 128 x 512 24.9 -> 23.4 us,
// 4 x the same 44.9 -> 43.2, 3 x 192 x 8 x 64 13.6 -> 12.6, 24 x 320 x 24 x 448 25.1 -> 23.3, 32 x 512 x 8 x 256 24.8 -> 24.5; but 64 x
// 512 x 16 x 128 30.8 -> 32.2, 32 x 2048 x 128 x 512 123.1 -> 126.1, 8 x 7168 x 64 x 2048 480 -> 485).  e4m3 cannot: a code
// needs the largest magnitude of its whole row.
constexpr int kDirect = 32;
constexpr int kMaxStages = 6, kMinStages = 4;  // (the producers take stages in turn, too)
static_assert(kProd <= kMinStages && kMinStages >= 3, "the ring");
// Every block finds the choice of so few tokens itself; of more, each is found by one block behind a barrier (a block
// reads splits x T x E partial logits otherwise).
constexpr int kOwnChoice = 8;
static_assert(kOwnChoice <= kWarps, "a warp for each token of a choice");
// counters: choices made, items with activations of each half, blocks done, then one for each shared item
constexpr int kCtrChoice = 0, kCtrItems = 1, kCtrDone = 3, kCtrShared = 4;

// landed, full, empty: a stage's weights are there, its tokens' rows, its place is free.
struct Lists {
  uint64_t landed[kMaxStages], full[kMaxStages], empty[kMaxStages], tfull[kMaxAccs], tempty[kMaxAccs], drain;
  uint32_t tmem;
  volatile int abort;
  int active, last, ok;
  uint32_t chunk[32];          // pairs and experts (<< 16) of 32 experts each
  float xs[kFewMaxTokens];     // scales of X's codes (e4m3)
  float pw[kMaxPairs];         // combine weight of a pair
  float factor[2][kFewMaxTokens];  // of the second product's columns, for two experts in turn
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

__device__ __forceinline__ void red_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int atom_acq_rel(int* p) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

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

// The work as lists of stages: the first product of the first half of the chosen experts, of the second half, then the second
// product of either.  A list's items (an expert's 128-row tiles) are c stages each; block b of its G takes the stages
// [b S / G, (b + 1) S / G).  With halves the activations that a block waits for at the second product's start have been
// complete for half a product's time; a short list is one, since a further list is a further chain of steps (a block's
// stages of the first product times 0.76 us against about 10 us: 1 x 2048 x 128 x 512, 7 stages, 33 us and in halves 41.5).
struct List {
  int ph, half, a0, tiles, c, S, G;
  __device__ __forceinline__ int begin(int b) const {
    return b >= G ? S : static_cast<int>(static_cast<long long>(b) * S / G);
  }
  // the block that has stage s (the host refuses sizes where S G would pass 32 bits)
  __device__ __forceinline__ int owner(int s) const {
    return static_cast<int>((static_cast<uint32_t>(s + 1) * static_cast<uint32_t>(G) - 1u) / static_cast<uint32_t>(S));
  }
};
constexpr int kLists = 4;
constexpr int kHalves = 16;  // stages of a block in the first product from which there are halves

struct Plan {
  int A, cut, G, t1, c1, t2, c2;  // cut: the second half's first expert
  __device__ __forceinline__ List list(int l) const {
    List x;
    x.ph = l >> 1;
    x.half = l & 1;
    x.a0 = x.half ? cut : 0;
    x.tiles = x.ph ? t2 : t1;
    x.c = x.ph ? c2 : c1;
    x.S = ((x.half ? A : cut) - x.a0) * x.tiles * x.c;
    x.G = min(x.S, G);
    return x;
  }
};

// A block's way through a list: stage q is reduction step k of tile `tile` of the chosen expert ai.
struct Walk {
  int q, end, k, tile, ai;
  __device__ __forceinline__ void start(const List& x, int b) {
    q = x.begin(b);
    end = x.begin(b + 1);
    const int item = q / x.c;
    k = q - item * x.c;
    const int i = item / x.tiles;
    ai = x.a0 + i;
    tile = item - i * x.tiles;
  }
  __device__ __forceinline__ void next_item(const List& x) {
    k = 0;
    if (++tile == x.tiles) {
      tile = 0;
      ++ai;
    }
  }
  __device__ __forceinline__ void next(const List& x) {
    ++q;
    if (++k == x.c) next_item(x);
  }
  __device__ __forceinline__ int item(const List& x) const { return (ai - x.a0) * x.tiles + tile; }
};

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

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

__device__ __forceinline__ void tmem_ld1(uint32_t taddr, float& v) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  v = __uint_as_float(r);
}

__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  return amax_bits ? __fdiv_rn(__uint_as_float(amax_bits), 448.0f) : 1.0f;
}

// x / s, correctly rounded, for many x with one s: Markstein's correction of a product with the correctly rounded reciprocal
// (P. Markstein, IBM J. Res. Dev. 34, 1990).  Scales from 2^-60 to 2^60; a quotient so small that the remainder
// underflows is far below the smallest code.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, s, x), inv, q);
}

// 16 bf16 values to 16 codes of a row with scale s.
__device__ __forceinline__ uint4 codes16(const uint4 x, const uint4 y, float s, float inv) {
  const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_bf16x2(v[2 * i]), b = unpack_bf16x2(v[2 * i + 1]);
    w[i] = e4m3x4(quotient(a.x, s, inv), quotient(a.y, s, inv), quotient(b.x, s, inv), quotient(b.y, s, inv));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same for any scale.
__device__ __noinline__ uint4 codes16_any(const uint4 x, const uint4 y, float s) {
  const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_bf16x2(v[2 * i]), b = unpack_bf16x2(v[2 * i + 1]);
    w[i] = e4m3x4(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s), __fdiv_rn(b.x, s), __fdiv_rn(b.y, s));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 codes16(const uint4 x, const uint4 y, float s) {
  if (s >= 8.673617379884035e-19f && s <= 1.152921504606847e18f) return codes16(x, y, s, __frcp_rn(s));
  return codes16_any(x, y, s);
}

}  // namespace

// ---- first launch: parts of the logits, X's codes, cleared counters -------------------------------------------------
// Block (x, y), x < strips * splits: 16 experts (32 bytes of every row of W_r, a memory sector) times a share of d, for the
// tokens NT y .. : part[split][t][e].  Thread: two experts (tid & 7) and four rows of every 128, R times 128 rows at a time.  The blocks behind (y = 0)
// clear the counters and, for the e4m3 form, quantize a token each.  The chunk ahead is loaded while one is multiplied.  A
// token of 2048 x 128 (0.5 MB): 4.7 us by itself with cold caches, 1.8 of a captured stack's layer, latencies of two chunks.
template <int NT, int R>
__global__ void __launch_bounds__(256) few_router_kernel(const __grid_constant__ FewArgs a) {
  __shared__ float red[8][NT][16];
  constexpr int kRtRows = 128 * R;
  __shared__ __align__(16) float s_x[NT][kRtRows];
  __shared__ float s_top[8];
  griddep_wait();    // a dependent launch too: eager calls in a row 24.6 -> 22.6 us (a token of 2048 x 128 x 512)
  griddep_launch();  // the second launch's start may overlap; it waits for this one's end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int strips = (a.E + 15) / 16;
  const int b = blockIdx.x;
  if (b >= strips * a.splits) {
    if (blockIdx.y > 0) return;
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
  const int strip = b % strips, split = b / strips, t0 = blockIdx.y * NT;
  const int d8 = a.d / 8;
  const int r0 = d8 * split / a.splits * 8, r1 = d8 * (split + 1) / a.splits * 8;
  const int e0 = strip * 16 + 2 * (tid & 7);
  const bool in = e0 < a.E;  // E is a multiple of 8: a pair is in or out
  const int rg = 4 * (tid >> 3);
  float acc[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = 0.0f;
  // a chunk's rows of W_r and of X in registers while the one before is multiplied
  constexpr int kXv = NT * (kRtRows / 8), kXn = (kXv + 255) / 256;
  uint32_t w[R][4];
  uint4 xr[kXn];
  auto load = [&](int c) {
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = c + 128 * q + rg + j;
        w[q][j] = (in && r < r1) ? __ldg(reinterpret_cast<const uint32_t*>(a.W_r + static_cast<long long>(r) * a.E + e0)) : 0u;
      }
#pragma unroll
    for (int q = 0; q < kXn; ++q) {
      const int i = tid + 256 * q, t = i / (kRtRows / 8), v = i % (kRtRows / 8) * 8;
      xr[q] = make_uint4(0, 0, 0, 0);
      if (i < kXv && t0 + t < a.T && c + v < r1)
        xr[q] = __ldg(reinterpret_cast<const uint4*>(a.X + (t0 + t) * a.ld_x + c + v));
    }
  };
  load(r0);
  for (int c = r0; c < r1; c += kRtRows) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kXn; ++q) {
      const int i = tid + 256 * q, t = i / (kRtRows / 8), v = i % (kRtRows / 8) * 8;
      const float2 f0 = unpack_bf16x2(xr[q].x), f1 = unpack_bf16x2(xr[q].y), f2 = unpack_bf16x2(xr[q].z),
                   f3 = unpack_bf16x2(xr[q].w);
      if (i < kXv) {
        *reinterpret_cast<float4*>(&s_x[t][v]) = make_float4(f0.x, f0.y, f1.x, f1.y);
        *reinterpret_cast<float4*>(&s_x[t][v + 4]) = make_float4(f2.x, f2.y, f3.x, f3.y);
      }
    }
    float2 f[R][4];  // zero past the share, as X's values there
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) f[q][j] = unpack_bf16x2(w[q][j]);
    __syncthreads();
    if (c + kRtRows < r1) load(c + kRtRows);
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(&s_x[i][128 * q + rg]);
        const float xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][0] = fmaf(xv[j], f[q][j].x, acc[i][0]);
          acc[i][1] = fmaf(xv[j], f[q][j].y, acc[i][1]);
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
}

// The choice of the tokens first .. first + count - 1, kOwnChoice at most: the block adds up their logits as order keys in
// keys [.][E] (shared memory), then one warp a token takes K times the largest key, the lower expert among equal ones (the rule
// of moe_route).  put(t, k, id, w) receives each.
template <class Put>
__device__ __forceinline__ void choose(const FewArgs& a, int first, int count, uint32_t* keys, const Put& put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long plane = static_cast<long long>(a.T) * a.E;
  for (int x = threadIdx.x; x < count * a.E; x += kThreads) {
    const int i = x / a.E, e = x - i * a.E;
    const float* p = a.part + static_cast<long long>(first + i) * a.E + e;
    float v = a.bias ? __ldg(a.bias + e) : 0.0f;
    for (int s0 = 0; s0 < a.splits; s0 += 16) {  // sixteen loads in flight
      float y[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = s0 + j < a.splits ? __ldcg(p + (s0 + j) * plane) : 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) v += y[j];
    }
    keys[x] = max(order_key(v), 1u);
  }
  __syncthreads();
  if (warp < count) {
    uint32_t* key = keys + warp * a.E;
    float vmax = 0.0f, sum = 0.0f, ex_k = 0.0f;
    int id = 0;
    for (int k = 0; k < a.K; ++k) {
      uint32_t bk = 0;
      int be = 0x7fffffff;
#pragma unroll 4
      for (int e = lane; e < a.E; e += 32) {
        const uint32_t q = key[e];
        if (q > bk) {
          bk = q;
          be = e;
        }
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
      const int e = __reduce_min_sync(0xffffffffu, bk == top ? be : 0x7fffffff);
      if ((e & 31) == lane) key[e] = 0;
      const float v = key_value(top);
      if (k == 0) vmax = v;
      const float ex = expf(v - vmax);
      sum += ex;
      if (lane == k) {
        id = e;
        ex_k = ex;
      }
    }
    if (lane < a.K) put(first + warp, lane, id, ex_k / sum);
  }
  __syncthreads();
}

// A = silu(H) U of one column (a lane's) of pair p: bf16 and the bf16 rounding of the rest, or, for the e4m3 form, bf16 and the
// pair's largest magnitude.  Lanes past the last column (in false) have none.
template <bool F8>
__device__ __forceinline__ void activate(const FewArgs& a, long long p, int col, bool in, float h, float u) {
  const float act = h * sigmoidf_(h) * u;
  const __nv_bfloat16 hi = __float2bfloat16_rn(act);
  const long long at = p * a.n + col;
  if (in) a.A[at] = hi;
  if (F8) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, in ? __float_as_uint(fabsf(__bfloat162float(hi))) : 0u);
    if ((threadIdx.x & 31) == 0) atomicMax(a.amax + p, top);
  } else if (in) {
    a.A_lo[at] = __float2bfloat16_rn(act - __bfloat162float(hi));
  }
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
  const int half_cols = a.nrows <= 16 ? 16 : a.nrows <= 32 ? 32 : a.nrows <= 64 ? 64 : 128;  // of a half's accumulator
  const int accs = a.nrows <= 64 ? kMaxAccs : kMaxAccs / 2, acc_bit = a.nrows <= 64 ? 2 : 1;  // 512 columns at most
  const uint32_t tmem_cols = accs * 2 * half_cols;  // a power of two

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&L.landed[s], 1);
      mbar_init(&L.full[s], 32);
      mbar_init(&L.empty[s], 1);
    }
    for (int i = 0; i < accs; ++i) {
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
  uint32_t* keys = reinterpret_cast<uint32_t*>(ring);              // [kOwnChoice][E]
  uint64_t* s_mask = reinterpret_cast<uint64_t*>(keys + kOwnChoice * a.E);  // [E] tokens of each expert
  int* s_ids = reinterpret_cast<int*>(s_mask + a.E);                // [P]
  float* s_w = reinterpret_cast<float*>(s_ids + kMaxPairs);
  uint16_t* s_eoff = reinterpret_cast<uint16_t*>(s_w + kMaxPairs);  // [E] first pair, index
  uint16_t* s_ea = s_eoff + a.E;
  if (P > 32)
    for (int e = tid; e < a.E; e += kThreads) s_mask[e] = 0;
  griddep_wait();  // the first launch's parts and cleared counters
  if (F8)
    for (int t = tid; t < a.T; t += kThreads) L.xs[t] = __ldcg(a.xs + t);
  if (a.T <= kOwnChoice) {
    choose(a, 0, a.T, keys, [&](int t, int k, int id, float w) {
      s_ids[t * a.K + k] = id;
      s_w[t * a.K + k] = w;
      if (b == 0) {
        a.ids[t * a.K + k] = id;
        a.w[t * a.K + k] = w;
      }
    });
  } else {
    for (int t = b; t < a.T; t += G) {
      choose(a, t, 1, keys, [&](int t2, int k, int id, float w) {
        a.ids[t2 * a.K + k] = id;
        a.w[t2 * a.K + k] = w;
      });
      if (tid == 0) red_release(&a.ctr[kCtrChoice], 1);
    }
    if (tid == 0) L.ok = wait_count(&a.ctr[kCtrChoice], a.T, &L.abort, a.timeout_ns, a.err) ? 1 : 0;
    __syncthreads();
    if (L.ok)
      for (int i = tid; i < P; i += kThreads) {
        s_ids[i] = __ldcg(a.ids + i);
        s_w[i] = __ldcg(a.w + i);
      }
    __syncthreads();
  }
  const bool ok = L.ok != 0;  // the wait gave up: nothing below runs
  if (P <= 32) {
    // one warp, a lane a pair: its place is the number of pairs before it by (expert, token)
    if (warp == 0) {
      const int t = lane / a.K, e = lane < P ? s_ids[lane] : 0x7fff;
      int p = 0, ai = 0, rank = 0;
      bool head = true;
      for (int j = 0; j < P; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j), tj = j / a.K;
        p += ej < e || (ej == e && tj < t);
        rank += tj == t && ej < e;
        head = head && !(ej == e && tj < t);
      }
      for (int j = 0; j < P; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j), hj = __shfl_sync(0xffffffffu, static_cast<int>(head), j);
        ai += hj && ej < e;
      }
      if (lane < P) {
        if (head) {
          L.act_e[ai] = static_cast<uint16_t>(e);
          L.act_off[ai] = static_cast<uint16_t>(p);
        }
        L.ptok[p] = static_cast<uint8_t>(t);
        L.tok_pair[t * a.K + rank] = static_cast<uint16_t>(p);
        L.tok_a[t * a.K + rank] = static_cast<uint16_t>(ai);
        L.pw[p] = s_w[lane];
      }
      const int act = __popc(__ballot_sync(0xffffffffu, lane < P && head));
      if (lane == 0) {
        L.active = ok ? act : 0;
        L.act_off[act] = static_cast<uint16_t>(P);
      }
    }
  } else {
  if (ok)
    for (int i = tid; i < P; i += kThreads)
      atomicOr(reinterpret_cast<unsigned long long*>(&s_mask[s_ids[i]]), 1ull << (i / a.K));
  __syncthreads();
  const int chunks = (a.E + 31) / 32;
  for (int c = warp; c < chunks; c += kWarps) {
    const int e = 32 * c + lane;
    const int cnt = (ok && e < a.E) ? __popcll(s_mask[e]) : 0;
    const uint32_t tot = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(cnt | (cnt ? 1 << 16 : 0)));
    if (lane == 0) L.chunk[c] = tot;
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += kWarps) {
    const int e = 32 * c + lane;
    const uint64_t mask = (ok && e < a.E) ? s_mask[e] : 0;
    const int cnt = __popcll(mask);
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < c ? L.chunk[lane] : 0u);
    const uint32_t v = cnt | (cnt ? 1u << 16 : 0u);
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t at = before + incl - v;
    if (cnt) {
      s_eoff[e] = static_cast<uint16_t>(at);
      s_ea[e] = static_cast<uint16_t>(at >> 16);
      L.act_e[at >> 16] = static_cast<uint16_t>(e);
      L.act_off[at >> 16] = static_cast<uint16_t>(at);
    }
    if (c == chunks - 1 && lane == 31) {
      L.active = static_cast<int>((before + incl) >> 16);
      L.act_off[(before + incl) >> 16] = static_cast<uint16_t>(before + incl);
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
      L.pw[p] = s_w[i];
    }
  }
  fence_proxy_async_smem();  // the scratch's uses come before the copies that overwrite it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = L.tmem;

  const int es = F8 ? 1 : 2;
  Plan plan;
  plan.A = L.active;
  plan.G = G;
  plan.t1 = (a.n + kRows - 1) / kRows;
  plan.c1 = (a.d * es + 127) / 128;
  plan.t2 = (a.d + kTile - 1) / kTile;
  plan.c2 = (a.n * es + 127) / 128;
  plan.cut = plan.A * plan.t1 * plan.c1 >= kHalves * G ? plan.A / 2 : 0;
  // Stages of weights asked for and not there yet.  HBM needs about 100 KB a block in flight; what is asked for beyond waits in
  // the memory system, and everything else behind it: the activations' way through L2 takes several times as long.  Long
  // lists gain by the deeper queue, short ones by the shorter way (two and all six stages: 4 x 2048 x 128 x 512 51.7 and
  // 59.0 us, 64 tokens e4m3 94 and 99, bf16 152 and 144; 24 x 2880 x 128 x 2880 553 and 518; three: 1 x 7168 x 64 x 2048 e4m3
  // 74.1 and 77.5).  The shortest of few tokens keep HBM busy for a moment only, their way included: there the queue starts the
  // stream sooner (layers of a stack, two and four: 1 x 2048 x 128 x 512 25.5 and 24.8 us, but 4 x the same 44.9 and 48.0, and 64 x
  // 2048 x 8 x 512, with many rows to gather, 90 and 102).  The ring is as deep all the same: it fills while a block waits for
  // the activations.
  // The number is odd where the ring's is: the stage whose landing a producer waits for is then its own to fill again, and its
  // barrier cannot go on by a second phase, of the same parity, before the wait has seen the first.
  static_assert(kProd == 2, "the parity of ahead");
  const int share = plan.A * (plan.t1 * plan.c1 + plan.t2 * plan.c2) / G;
  const int want = share < 20 && a.stages == kMaxStages ? 4 : share < 100 ? 2 : share < 150 ? 3 : a.stages;
  const int ahead = want + ((a.stages - want) & 1);
  const int ld_hu = plan.t1 * kTile, ld_y = plan.t2 * kTile;
  const bool direct = !F8 && share < 100 && a.T <= kDirect;
  // a last tile of W_down may have rows in its first half alone
  auto halves = [&](const List& x, int tile) { return x.ph == 1 && a.d - tile * kTile <= kRows ? 1 : 2; };

  if (warp >= kProd0) {
    // ---------------------------------------------------------------- weights (lane 0 of each producer warp)
    if (lane == 0) {
      const int pj = warp - kProd0;
      int it = 0, s = 0;
      uint32_t par = 1;  // parity of the empty barrier's wait
      bool stop = false;
      for (int l = 0; l < kLists && !stop; ++l) {
        const List x = plan.list(l);
        if (b >= x.G) continue;
        Walk w;
        for (w.start(x, b); w.q < w.end; w.next(x), ++it) {
          if ((it & (kProd - 1)) == pj) {
            if (!mbar_wait(&L.empty[s], par, &L.abort, a.timeout_ns, a.err)) {
              stop = true;
              break;
            }
            // not more than `ahead` stages on their way: the one that many back has landed
            const int back = s - ahead;
            if (it >= ahead && !mbar_wait(&L.landed[back < 0 ? back + a.stages : back], back < 0 ? par : par ^ 1, &L.abort,
                                           a.timeout_ns, a.err)) {
              stop = true;
              break;
            }
            uint8_t* dst = ring + s * stage_bytes;
            const int e = L.act_e[w.ai];
            const int hs = halves(x, w.tile);
            mbar_arrive_expect_tx(&L.landed[s], hs * kHBytes);
            if (x.ph == 0) {
              tma_load_3d(dst, &mg, &L.landed[s], w.k * 64, w.tile * kRows, e);
              tma_load_3d(dst + kHBytes, &mu, &L.landed[s], w.k * 64, w.tile * kRows, e);
            } else {
              tma_load_3d(dst, &md, &L.landed[s], w.k * 64, w.tile * kTile, e);
              if (hs == 2) tma_load_3d(dst + kHBytes, &md, &L.landed[s], w.k * 64, w.tile * kTile + kRows, e);
            }
          }
          if (++s == a.stages) {
            s = 0;
            par ^= 1;
          }
        }
      }
    }
  } else if (warp >= kGath0 && warp < kGath0 + kGath) {
    // ---------------------------------------------------------------- the tokens' rows
    // The warps take stages in turn, so that several stages' loads are in flight whatever each waits for.  No more warps
    // than the ring has stages: a warp's next stage must not lie more than one turn of the ring ahead of its last, or the
    // parity that it waits for could be that of two turns before.  Lane: the 16-byte piece c16 of every fourth row.  Rows past
    // the expert's tokens hold whatever was there: they are columns of their own in the product.
    const int gj = warp - kGath0, c16 = lane & 7, rsub = lane >> 3;
    const int turns = a.stages < kGath ? a.stages : kGath;
    int turn = 0, s = 0;
    uint32_t par = 1;
    bool stop = false;
    for (int l = 0; l < kLists && !stop; ++l) {
      const List x = plan.list(l);
      if (b >= x.G) continue;
      if (x.ph == 1) {
        // every pair's activations of this half are there
        const List first = plan.list(x.half);
        int go = 0;
        if (lane == 0)
          go = wait_count(&a.ctr[kCtrItems + x.half], direct ? first.G : first.S / first.c, &L.abort, a.timeout_ns, a.err) ? 1 : 0;
        __syncwarp();
        if (!__shfl_sync(0xffffffffu, go, 0)) {
          stop = true;
          break;
        }
      }
      Walk w;
      for (w.start(x, b); w.q < w.end; w.next(x)) {
        if (turn == gj) {
          const int p0 = L.act_off[w.ai], m = L.act_off[w.ai + 1] - p0;
          if (!mbar_wait(&L.empty[s], par, &L.abort, a.timeout_ns, a.err)) stop = true;
          stop = __any_sync(0xffffffffu, stop);
          if (stop) break;
          uint8_t* tok = ring + s * stage_bytes + kWBytes;
          const int off = w.k * 128 + c16 * 16;  // bytes of the operand's row; half a last stage may be past its end: zeros
          if (x.ph == 0) {
            const bool in = off < a.d * es;
            const uint8_t* src = (F8 ? a.xq : reinterpret_cast<const uint8_t*>(a.X)) + (in ? off : 0);
            const long long ld = F8 ? a.d : a.ld_x * 2;
            for (int r = rsub; r < m; r += 4)
              cp_async_16(smem_u32(tok) + sw128_offset(r, c16), src + L.ptok[p0 + r] * ld, in ? 16u : 0u);
            cp_async_mbar_arrive_noinc(&L.full[s]);
          } else if (!F8 && direct) {
            // lane: two of the stage's columns; their parts of H and U lie where the first product's blocks left them
            const List made = plan.list(x.half);
            const int mh = (m + 7) & ~7, c0 = w.k * 64 + 2 * lane, tile = c0 / kRows, s0 = ((w.ai - made.a0) * plan.t1 + tile) * plan.c1;
            const int b0 = made.owner(s0), parts = made.owner(s0 + plan.c1 - 1) - b0 + 1;
            const float* main = a.hu + static_cast<long long>(p0) * ld_hu + tile * kTile + c0 % kRows;
            const float* over = a.ov1 + (static_cast<long long>(x.half) * kFewMaxBlocks + b0) * a.T * kTile + c0 % kRows;
#pragma unroll 1
            for (int r = 0; r < m; ++r) {
              float2 h = make_float2(0.0f, 0.0f), u = h;
#pragma unroll 1
              for (int o0 = 0; o0 < parts; o0 += 8) {
                float2 yh[8], yu[8];
#pragma unroll
                for (int o = 0; o < 8; ++o) {
                  const float* at = o0 + o == 0 ? main + static_cast<long long>(r) * ld_hu
                                                : over + (static_cast<long long>(o0 + o) * a.T + r) * kTile;
                  const bool has = o0 + o < parts;
                  yh[o] = has ? __ldcg(reinterpret_cast<const float2*>(at)) : make_float2(0.0f, 0.0f);
                  yu[o] = has ? __ldcg(reinterpret_cast<const float2*>(at + kRows)) : make_float2(0.0f, 0.0f);
                }
#pragma unroll
                for (int o = 0; o < 8; ++o) {
                  h.x += yh[o].x; h.y += yh[o].y;
                  u.x += yu[o].x; u.y += yu[o].y;
                }
              }
              const float ax = h.x * sigmoidf_(h.x) * u.x, ay = h.y * sigmoidf_(h.y) * u.y;
              const uint32_t hi = pack_bf16x2(ax, ay);
              const float2 back = unpack_bf16x2(hi);
              uint8_t* to = tok + 4 * (lane & 3);
              *reinterpret_cast<uint32_t*>(to + sw128_offset(r, lane >> 2)) = hi;
              *reinterpret_cast<uint32_t*>(to + sw128_offset(mh + r, lane >> 2)) = pack_bf16x2(ax - back.x, ay - back.y);
            }
            fence_proxy_async_smem();
            mbar_arrive(&L.full[s]);
          } else if (!F8) {
            const int mh = (m + 7) & ~7;
            const uint8_t* hi = reinterpret_cast<const uint8_t*>(a.A + static_cast<long long>(p0) * a.n) + off;
            const uint8_t* lo = reinterpret_cast<const uint8_t*>(a.A_lo + static_cast<long long>(p0) * a.n) + off;
            for (int r = rsub; r < m; r += 4) {
              const long long o = static_cast<long long>(r) * a.n * 2;
              cp_async_16(smem_u32(tok) + sw128_offset(r, c16), hi + o, 16u);
              cp_async_16(smem_u32(tok) + sw128_offset(mh + r, c16), lo + o, 16u);
            }
            cp_async_mbar_arrive_noinc(&L.full[s]);
          } else {
            const bool in = off < a.n;
            const uint4* src = reinterpret_cast<const uint4*>(a.A + static_cast<long long>(p0) * a.n + (in ? off : 0));
            const int ld = a.n / 8;
            uint4 v0, v1;
            uint32_t top = 0;
            auto load = [&](int r) {
              const uint4* at = src + static_cast<long long>(r) * ld;
              v0 = __ldcg(at);
              v1 = __ldcg(at + 1);
              top = __ldcg(a.amax + p0 + r);
            };
            if (rsub < m) load(rsub);
#pragma unroll 1
            for (int r = rsub; r < m; r += 4) {
              const uint4 x0 = v0, x1 = v1;
              const float sc = row_scale(top);
              if (r + 4 < m) load(r + 4);
              *reinterpret_cast<uint4*>(tok + sw128_offset(r, c16)) = in ? codes16(x0, x1, sc) : make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            mbar_arrive(&L.full[s]);
          }
        }
        if (++turn == turns) turn = 0;
        if (++s == a.stages) {
          s = 0;
          par ^= 1;
        }
      }
    }
    cp_async_wait_all();
  } else if (warp == kMma) {
    // ---------------------------------------------------------------- the products
    // The whole warp goes through the stages, one lane issues: operands that all lanes agree on stay in uniform registers
    // (issued out of a branch of lane 0's, a stage's four products took 300 cycles).
    const bool one = elect_one();
    int s = 0, acc = 0;
    uint32_t par = 0;
    bool stop = false;
    for (int l = 0; l < kLists && !stop; ++l) {
      const List x = plan.list(l);
      if (b >= x.G) continue;
      Walk w;
      for (w.start(x, b); w.q < w.end && !stop; ++acc) {
        const int k1 = min(x.c, w.k + (w.end - w.q));
        const int m = L.act_off[w.ai + 1] - L.act_off[w.ai];
        const int N = (!F8 && x.ph == 1) ? 2 * ((m + 7) & ~7) : (m + 15) & ~15;
        const uint32_t idesc = F8 ? idesc_e4m3(kRows, N, 0, 0) : idesc_bf16(kRows, N, 0, 0);
        stop = __any_sync(0xffffffffu, !mbar_wait(&L.tempty[acc & (accs - 1)], ((acc >> acc_bit) & 1) ^ 1, &L.abort, a.timeout_ns, a.err));
        if (stop) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (acc & (accs - 1)) * 2 * half_cols;
        const bool two = halves(x, w.tile) == 2;
        uint32_t more = 0;
        for (; w.k < k1; ++w.k, ++w.q) {
          stop = __any_sync(0xffffffffu, !mbar_wait(&L.landed[s], par, &L.abort, a.timeout_ns, a.err) ||
                                             !mbar_wait(&L.full[s], par, &L.abort, a.timeout_ns, a.err));
          if (stop) break;
          fence_proxy_async_smem();  // cp.async writes -> operand reads
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + s * stage_bytes);
          const uint64_t ad = sdesc_sw128(sa, 16, 1024), bd = sdesc_sw128(sa + kWBytes, 16, 1024);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_step<F8>(d_tmem, ad + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : more);
            if (two) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_step<F8>(d_tmem + half_cols, ad + (kHBytes >> 4) + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : more);
            }
            umma_commit(&L.empty[s]);
          }
          more = 1;
          if (++s == a.stages) {
            s = 0;
            par ^= 1;
          }
        }
        if (!stop && one) umma_commit(&L.tfull[acc & (accs - 1)]);
        if (w.k == x.c) w.next_item(x);
      }
    }
    if (L.abort && one) {
      umma_commit(&L.drain);
      volatile int never = 0;
      mbar_wait(&L.drain, 0, &never, 20000000ull, nullptr);
    }
  } else {
    // ---------------------------------------------------------------- accumulators out (warps 0..3)
    // A thread has a row of either half, a column per token.  Of an item that other blocks share, the part with the first
    // stage goes to the item's place, another block's to that block's own overflow rows (in a list a block goes on with at
    // most one item that began elsewhere).
    const int row = tid;
    int acc = 0, last = -1, turn = 0;
    bool stop = false;
    for (int l = 0; l < kLists && !stop; ++l) {
      const List x = plan.list(l);
      if (b >= x.G) continue;
      const int ld = x.ph ? ld_y : ld_hu;
      float* const first = x.ph ? a.y : a.hu;
      float* const over = (x.ph ? a.ov2 : a.ov1) + static_cast<long long>(x.half) * kFewMaxBlocks * a.T * kTile;
      int items = 0;  // completed here, of the first product
      if (F8 && x.ph == 1) {  // the factors below need the pairs' largest magnitudes
        const List made = plan.list(x.half);
        const bool go = tid > 0 || wait_count(&a.ctr[kCtrItems + x.half], made.S / made.c, &L.abort, a.timeout_ns, a.err);
        if (!epi_all(go)) {
          stop = true;
          break;
        }
      }
      Walk w;
      for (w.start(x, b); w.q < w.end; ++acc) {
        const int k0 = w.k, k1 = min(x.c, k0 + (w.end - w.q));
        const int ai = w.ai, tile = w.tile, item = w.item(x);
        w.q += k1 - k0;
        if (k1 == x.c) w.next_item(x);
        const int p0 = L.act_off[ai], m = L.act_off[ai + 1] - p0, mh = (m + 7) & ~7;
        const bool whole = k1 - k0 == x.c, two = halves(x, tile) == 2;
        const int slot = acc & (accs - 1);
        const uint32_t tb = tmem + (static_cast<uint32_t>(warp * 32) << 16) + slot * 2 * half_cols;
        const int col = tile * kRows + row;  // the first product's column of this thread
        const bool in = col < a.n;
        // e4m3: scales of this thread's two rows of weights; H and U take their token's, the second product's columns a factor
        float s0 = 1.0f, s1 = 1.0f;
        if (F8 && x.ph == 0 && in) {
          const long long at = static_cast<long long>(L.act_e[ai]) * a.n + col;
          s0 = __ldg(a.wg_scale + at);
          s1 = __ldg(a.wu_scale + at);
        }
        if (x.ph == 1) {
          if (F8) {
            const int r = tile * kTile + row;
            const float* at = a.wd_scale + static_cast<long long>(L.act_e[ai]) * a.d + r;
            s0 = r < a.d ? __ldg(at) : 0.0f;
            s1 = r + kRows < a.d ? __ldg(at + kRows) : 0.0f;
          }
          if (ai != last) {  // the factors are the expert's: one load for all of its tiles
            last = ai;
            turn ^= 1;
            if (row < m) L.factor[turn][row] = L.pw[p0 + row] * (F8 ? row_scale(__ldcg(a.amax + p0 + row)) : 1.0f);
          }
        }
        float* dst;
        int step;
        if (k0 == 0) {
          dst = first + static_cast<long long>(p0) * ld + tile * kTile + row;
          step = ld;
        } else {
          dst = over + static_cast<long long>(b) * a.T * kTile + row;
          step = kTile;
        }
        // one verdict for all: a thread alone at the barriers below would wait for ever
        if (!epi_all(mbar_wait(&L.tfull[slot], (acc >> acc_bit) & 1, &L.abort, a.timeout_ns, a.err))) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (x.ph == 0 && whole && !direct) {
#pragma unroll 1
          for (int j = 0; j < m; ++j) {
            float h, u;
            tmem_ld1(tb + j, h);
            tmem_ld1(tb + half_cols + j, u);
            tmem_ld_wait();
            const float sx = F8 ? L.xs[L.ptok[p0 + j]] : 1.0f;
            activate<F8>(a, p0 + j, col, in, h * (sx * s0), u * (sx * s1));
          }
        } else {
          const float* factor = L.factor[turn];
#pragma unroll 1
          for (int j0 = 0; j0 < m; j0 += 8) {
            float v[2][8];
            tmem_ld8(tb + j0, v[0]);
            if (two) tmem_ld8(tb + half_cols + j0, v[1]);
            if (!F8 && x.ph == 1) {
              float lo[2][8];
              tmem_ld8(tb + mh + j0, lo[0]);
              if (two) tmem_ld8(tb + half_cols + mh + j0, lo[1]);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                v[0][i] += lo[0][i];
                v[1][i] += lo[1][i];
              }
            } else {
              tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (j0 + i < m) {
                const float f = x.ph ? factor[j0 + i] : 1.0f;
                float* to = dst + static_cast<long long>(j0 + i) * step;
                __stcg(to, v[0][i] * (F8 && x.ph ? f * s0 : f));
                if (two) __stcg(to + kRows, v[1][i] * (F8 && x.ph ? f * s1 : f));
              }
          }
        }
        tc_fence_before();
        mbar_arrive(&L.tempty[slot]);
        if (x.ph == 1 || direct) continue;
        if (whole) {
          ++items;
          continue;
        }
        // an item in parts: the block that brings the last of them adds them up in block order, eight loads at a time: four
        // parts of two pairs, or eight of the only one (short lists are cut into many parts and have few pairs)
        const int b0 = x.owner(item * x.c), parts = x.owner(item * x.c + x.c - 1) - b0 + 1;
        epi_sync();
        if (tid == 0) L.last = atom_acq_rel(&a.ctr[kCtrShared + x.half * kFewMaxBlocks + b0]) == parts - 1;
        epi_sync();
        if (!L.last) continue;
        ++items;
#pragma unroll 1
        for (int j0 = 0; j0 < m; j0 += 2) {
          float h[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
          const bool one = m == 1;
#pragma unroll 1
          for (int o0 = 0; o0 < parts; o0 += one ? 8 : 4) {
            float y[8][2];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const int j = one ? 0 : j0 + (r >> 2), o = o0 + (one ? r : r & 3);
              const bool has = j < m && o < parts;
              const float* at = o == 0 ? a.hu + static_cast<long long>(p0 + j) * ld + tile * kTile + row
                                       : over + (static_cast<long long>(b0 + o) * a.T + j) * kTile + row;
              y[r][0] = has ? __ldcg(at) : 0.0f;
              y[r][1] = has ? __ldcg(at + kRows) : 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              if (r < 4 || one) {
                h[0] += y[r][0];
                u[0] += y[r][1];
              } else {
                h[1] += y[r][0];
                u[1] += y[r][1];
              }
            }
          }
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (j0 + q < m) {
              const float sx = F8 ? L.xs[L.ptok[p0 + j0 + q]] : 1.0f;
              activate<F8>(a, p0 + j0 + q, col, in, h[q] * (sx * s0), u[q] * (sx * s1));
            }
        }
      }
      if (stop || x.ph == 1) continue;
      epi_sync();
      if (tid == 0 && (direct || items > 0)) red_release(&a.ctr[kCtrItems + x.half], direct ? 1 : items);
    }
    if (!stop) {
      epi_sync();
      if (tid == 0) red_release(&a.ctr[kCtrDone], 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool gave_up = L.abort;  // (every thread sees so)
  if (gave_up) linger();
  if (warp == kMma) tmem_dealloc(tmem, tmem_cols);
  // ---- the sums over a token's choices, once every block's parts are there: eight lanes a token and four columns, one a choice ----
  if (gave_up) return;
  __syncthreads();  // (the wait below may raise the flag)
  if (tid == 0) L.ok = ok && wait_count(&a.ctr[kCtrDone], G, &L.abort, a.timeout_ns, a.err) ? 1 : 0;
  __syncthreads();
  if (!L.ok) return;
  const int quads = a.d / 4, units = a.T * quads, t2 = plan.t2, c2 = plan.c2;
  const List y0 = plan.list(2), y1 = plan.list(3);
  const int u1 = static_cast<int>(static_cast<long long>(units) * (b + 1) / G);
  constexpr int kU = 2;  // units of a lane group at a time, and four parts: their loads in flight together
#pragma unroll 1
  for (int u0 = static_cast<int>(static_cast<long long>(units) * b / G) + 4 * kU * warp; u0 < u1; u0 += 4 * kU * kWarps) {
    const int k = lane & 7;
    float4 v[kU];
    const float *main[kU], *over[kU];
    int t[kU], col[kU], parts[kU];
#pragma unroll
    for (int q = 0; q < kU; ++q) {
      const int u = u0 + 4 * q + (lane >> 3);
      v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      t[q] = u / quads;
      col[q] = (u - t[q] * quads) * 4;
      parts[q] = 0;
      main[q] = over[q] = a.y;
      if (u < u1 && k < a.K) {
        const int p = L.tok_pair[t[q] * a.K + k], ai = L.tok_a[t[q] * a.K + k];
        const bool h = ai >= y1.a0;
        const int s0 = ((ai - (h ? y1.a0 : 0)) * t2 + col[q] / kTile) * c2;
        const int b0 = (h ? y1 : y0).owner(s0);
        parts[q] = (h ? y1 : y0).owner(s0 + c2 - 1) - b0 + 1;
        main[q] = a.y + static_cast<long long>(p) * ld_y + col[q];
        over[q] = a.ov2 + ((static_cast<long long>(h) * kFewMaxBlocks + b0) * a.T + (p - L.act_off[ai])) * kTile + col[q] % kTile;
      }
    }
    const int most = __reduce_max_sync(0xffffffffu, max(parts[0], parts[1]));
#pragma unroll 1
    for (int o = 0; o < most; o += 4) {
      float4 z[kU][4];
#pragma unroll
      for (int q = 0; q < kU; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          z[q][r] = o + r < parts[q] ? __ldcg(reinterpret_cast<const float4*>(
                                           o + r == 0 ? main[q] : over[q] + static_cast<long long>(o + r) * a.T * kTile))
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < kU; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[q].x += z[q][r].x; v[q].y += z[q][r].y; v[q].z += z[q][r].z; v[q].w += z[q][r].w;
        }
    }
#pragma unroll
    for (int q = 0; q < kU; ++q) {
      float4 x = v[q];
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, o);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
      }
      if (k == 0 && u0 + 4 * q + (lane >> 3) < u1)
        *reinterpret_cast<uint2*>(a.O + t[q] * a.ld_o + col[q]) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
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
  l.nctr = kCtrShared + 2 * kFewMaxBlocks;
  l.ctr = take(sizeof(int) * l.nctr);
  l.amax = take(sizeof(uint32_t) * P);
  l.part = take(sizeof(float) * static_cast<size_t>(kFewMaxSplits) * T * E);
  l.xq = take(static_cast<size_t>(T) * d);
  l.xs = take(sizeof(float) * T);
  l.hu = take(sizeof(float) * P * ((n + kRows - 1) / kRows) * kTile);
  l.A = take(sizeof(__nv_bfloat16) * P * n);
  l.A_lo = take(sizeof(__nv_bfloat16) * P * n);
  l.y = take(sizeof(float) * P * ((d + kTile - 1) / kTile) * kTile);
  l.ov1 = take(sizeof(float) * 2 * static_cast<size_t>(kFewMaxBlocks) * T * kTile);
  l.ov2 = take(sizeof(float) * 2 * static_cast<size_t>(kFewMaxBlocks) * T * kTile);
  l.bytes = p;
  return l;
}

// Shares of d in the router's product: about four blocks an SM over all tokens, 64 rows a share at least.
int few_splits(int T, int d, int E, int num_sms) {
  const int blocks = (E + 15) / 16 * ((T + 7) / 8);
  int sp = 4 * num_sms / blocks;
  sp = sp < 1 ? 1 : sp > kFewMaxSplits ? kFewMaxSplits : sp;
  return sp > d / 64 ? d / 64 : sp;
}

cudaError_t launch_few_router(const FewArgs& args, cudaStream_t s) {
  const int strips = (args.E + 15) / 16;
  const dim3 grid(strips * args.splits + (args.xq ? args.T : 1), (args.T + 7) / 8);
  if (args.T == 1) return launch_dependent(few_router_kernel<1, 4>, grid, dim3(256), 0, s, args);
  return launch_dependent(few_router_kernel<8, 1>, grid, dim3(256), 0, s, args);
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
  if (args.stages < kMinStages) return cudaErrorInvalidConfiguration;
  const size_t smem = 1024 + static_cast<size_t>(args.stages) * stage_bytes + sizeof(Lists);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // blocks wait for one another's parts: all of them resident at once
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its start overlaps the first launch's end
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(few_blocks(num_sms), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args, mg, mu, md);
}

cudaError_t launch_few_layer(const FewArgs& args, bool f8, const CUtensorMap& mg, const CUtensorMap& mu,
                             const CUtensorMap& md, int num_sms, cudaStream_t s) {
  return f8 ? launch<true>(args, mg, mu, md, num_sms, s) : launch<false>(args, mg, mu, md, num_sms, s);
}

}  // namespace vgg
