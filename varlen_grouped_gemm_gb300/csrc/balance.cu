// The router's balance and z losses with their gradient, and the per-expert counts.
//
// For the counted tokens of every sequence b (n_b of them; n in all, B' sequences with any), p_t = softmax(l_t):
//   f_be = E / (K n_b) #{(t, k): id_tk = e},   P_be = 1 / n_b sum_t p_te
//   loss = alpha / B' sum_b sum_e f_be P_be  +  beta / n sum_t lse_t^2
//   dl_te = p_te (c_be - sum_j p_tj c_bj) + 2 beta / n lse_t p_te,   c_be = alpha f_be / (B' n_b)
//
// f depends on the choices alone, so once the counts are known one pass over the logits gives P, both losses and the
// gradient: 8 bytes an element, bound by HBM for long batches and by the barriers between the phases for short ones.
// A shift of c_b by a constant leaves dl unchanged (p sums to one), so the kernel works with u_be = f_be - 1 =
// (counts_be E - K n_b) / (K n_b): its numerator is a whole number, and a nearly even load loses nothing to
// cancellation.  A token's share of the balance loss is 1 + <p_t, u_b>, which the gradient needs anyway.
//
// One launch: (1) counts by shared-memory histograms, added with integer atomics (any order, one result); (2) the
// pass over the logits; (3) the probabilities' sums and the loss.  Block c takes the tokens of chunk c; where a
// chunk crosses into another sequence it closes a piece.  The piece of (chunk c, sequence b) has the index c + b,
// unique because every next piece moves on by a chunk, a sequence or both.  Sums over tokens run in a fixed order,
// so equal calls give equal bits.
// 64 x 8 7.8 us and 4096 x 128 11.5 us (the phases' latency and the barriers between them); 32768 x 512 in 37
// sequences 40.3 us (135 MB, 20 us of them): launch and clearing 3, counting under the first loads 6, barriers 3, blocks
// that memory serves unevenly 5, the last phase 3.  Without the gradient 26 us there (35 with it for sequences of one length
// and no mask), 10.9 us at 4096 x 128.  The widest form (513 to 1024 experts) spills 104 bytes at the 128 registers that 512
// threads leave it: 16384 x 1024 35.9 us.
#include "internal.h"

namespace vgg {

namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxBlocks = 1024;  // bounds the number of pieces, and with it the workspace
constexpr int kBalCluster = 16;      // up to so many blocks wait for one another as a cluster, more as a whole grid
// What one cluster takes: T (E + 16), the 16 standing for a token's choices and reductions, below kBalOneCluster, and at
// most kBalClusterSeqs sequences, each of which a block closes with two barriers.  Eager calls in a cluster and as a
// cooperative grid with the clearing ahead of it: 2048 x 128 12.3 and 15.4 us, 4096 x 128 16.4 and 15.4, 8192 x 16 14.4 and
// 15.4, 16384 x 16 16.4 and 15.4; 1500 x 64 in 32 sequences 24.2 and 25.6, in 48 27.3 and 26.5.
constexpr long long kBalOneCluster = 3 << 17;
constexpr int kBalClusterSeqs = 40;

inline size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BalWs {
  int* ctrl;      // [0] grid barrier
  int* nvalid;    // [B]
  float* zpart;   // [pieces] sums of lse^2
  float* bpart;   // [pieces] sums of the balance loss's shares, over n_b
  int* cnt;       // [B][E]
  float* ppart;   // [pieces][E]
  size_t zeroed;  // bytes from ctrl up to ppart
  size_t bytes;
};

BalWs carve_balance(void* ws, long long T, int E, int B) {
  // a launch has at most max(T, kBalCluster) blocks
  const size_t pieces = static_cast<size_t>(T < kBalCluster ? kBalCluster : T < kBalMaxBlocks ? T : kBalMaxBlocks) + B;
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = p + at;
    at += al256(bytes);
    return r;
  };
  BalWs w{};
  w.ctrl = reinterpret_cast<int*>(take(sizeof(int)));
  w.nvalid = reinterpret_cast<int*>(take(sizeof(int) * B));
  w.zpart = reinterpret_cast<float*>(take(sizeof(float) * pieces));
  w.bpart = reinterpret_cast<float*>(take(sizeof(float) * pieces));
  w.cnt = reinterpret_cast<int*>(take(sizeof(int) * static_cast<size_t>(B) * E));
  w.zeroed = at;
  w.ppart = reinterpret_cast<float*>(take(sizeof(float) * pieces * E));
  w.bytes = at;
  return w;
}

__device__ __forceinline__ int seq_begin(const BalanceArgs& a, int b) {
  if (!a.seq_off) return b == 0 ? 0 : static_cast<int>(a.T);
  return max(0, min(__ldg(a.seq_off + b), static_cast<int>(a.T)));
}

// A chunk's pieces in order: the sequence b and its tokens [t0, t1) within the chunk.  Always ends, and stays
// within the chunk, whatever the offsets hold (the last sequence reaches to T).
struct Piece {
  int b, t0, t1;
  // b0: the last sequence that begins at c0 or before
  __device__ void first(int b0, int c0) {
    b = b0;
    t0 = t1 = c0;
  }
  __device__ bool next(const BalanceArgs& a, int c1) {
    if (t1 >= c1) return false;
    t0 = t1;
    while (b + 1 < a.B && seq_begin(a, b + 1) <= t0) ++b;
    t1 = b + 1 < a.B ? min(c1, seq_begin(a, b + 1)) : c1;
    return true;
  }
};

// A warp's tiles of up to kTile tokens in order: each kBalWarps-th of the chunk's, whose count runs on from one piece into
// the next, so that the warps' shares differ by one tile at most however many pieces there are.
template <int kTile>
struct Tiles {
  Piece pc;
  int tb;
  int nth;  // the chunk's tiles before this piece
  bool ok;
  static __device__ int first_of(const Piece& p, int nth, int warp) {  // the warp's first tile of a piece begins here
    return p.t0 + ((warp - nth) & (kBalWarps - 1)) * kTile;
  }
  static __device__ int count(const Piece& p) { return (p.t1 - p.t0 + kTile - 1) / kTile; }
  __device__ void skip(const BalanceArgs& a, int c1, int warp) {
    while (ok && tb >= pc.t1) {
      nth += count(pc);
      ok = pc.next(a, c1);
      tb = first_of(pc, nth, warp);
    }
  }
  __device__ void first(const BalanceArgs& a, int b0, int c0, int c1, int warp) {
    pc.first(b0, c0);
    nth = 0;
    ok = true;
    tb = pc.t1;
    skip(a, c1, warp);
  }
  __device__ void next(const BalanceArgs& a, int c1, int warp) {
    tb += kBalWarps * kTile;
    skip(a, c1, warp);
  }
};

// Sums of two values over the block, the same in every thread.
__device__ __forceinline__ float2 block_sum2(float x, float y, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(x, y);
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kBalWarps; ++i) {
    s.x += red[i].x;
    s.y += red[i].y;
  }
  __syncthreads();
  return s;
}

// 2^x, at most 2 steps off; results below 2^-126 are 0.  As e^(l - m) from x = (l - m) log2 e the three roundings of x come
// first, 3 (m - l) 2^-24 of the value: an exact exponential of the rounded l - m would keep one of them.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest of v over LPT neighbouring lanes.
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LPT == 32) {
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(v) : "f"(v));
    return v;
  }
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// VEC: LPT lanes a token (32 / LPT tokens in a warp), NV vectors of four logits a lane; a warp's tiles of kTile tokens come
// through a ring of ST stages of its own, one bulk copy a tile (the tokens' rows are contiguous), so the bytes in
// flight do not depend on registers, and the ring runs on from one piece into the next.  Else one value a load, a warp
// a token, NV values a lane.
template <bool VEC, int LPT, int NV, int UN, int ST>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(const BalanceArgs a, const BalWs w, int chunk) {
  constexpr int kPairs = VEC ? 2 * NV : NV / 2;
  constexpr int kTok = 32 / LPT, kTile = kTok * UN;
  extern __shared__ __align__(128) uint8_t bal_smem[];
  __shared__ float2 s_red[kBalWarps];
  __shared__ float s_tile[kBalWarps][33];
  __shared__ __align__(8) uint64_t full[kBalWarps][ST];
  __shared__ int s_n[kBalWarps], s_ok, s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, E = a.E, K = a.K, T = static_cast<int>(a.T);
  const int c0 = min(T, static_cast<int>(blockIdx.x) * chunk), c1 = min(T, c0 + chunk);
  float* sums = reinterpret_cast<float*>(bal_smem);                // [kBalWarps][E] partial sums (phase 1: the histogram)
  float* su = sums + kBalWarps * E;                                // [E] u of the current sequence
  float* ring = su + (E + 3) / 4 * 4 + static_cast<size_t>(warp) * ST * kTile * E;
  auto barrier = [&](int nth) -> bool {
    if (G == 1) {
      __syncthreads();
      return true;
    }
    if (G <= kBalCluster) {
      cluster_sync();
      return true;
    }
    return grid_barrier(w.ctrl, nth * G, a.timeout_ns, a.err, &s_ok);
  };
  if (tid == 0) s_abort = 0;
  if (tid < kBalWarps) s_n[tid] = 0;
  if (VEC && lane < ST) mbar_init(&full[warp][lane], 1);
  fence_mbar_init();
  int* hist = reinterpret_cast<int*>(sums);
  for (int i = tid; i < (a.B > 1 ? kBalWarps : 1) * E; i += kBalThreads) hist[i] = 0;
  if (G <= kBalCluster) {  // a small grid clears its own workspace
    int* z = w.ctrl;
    for (size_t i = blockIdx.x * kBalThreads + tid; i < w.zeroed / sizeof(int); i += static_cast<size_t>(G) * kBalThreads)
      z[i] = 0;
    barrier(0);
  } else {
    __syncthreads();
  }
  // the chunk's first sequence: every thread looks at some of them (a search would take a memory latency a step)
  int b0 = 0;
  for (int k = 0; k < a.B; k += kBalThreads) {
    const int begun = __syncthreads_count(k + tid < a.B && seq_begin(a, k + tid) <= c0);
    b0 += begun;
    if (begun < kBalThreads) break;
  }
  b0 = max(b0 - 1, 0);
  // the first tiles of logits come while the choices are counted and the blocks wait for one another
  Tiles<kTile> in;  // lane 0's next tile to ask for
  int st_in = 0;
  auto issue = [&]() {
    const uint32_t bytes = static_cast<uint32_t>(min(kTile, in.pc.t1 - in.tb)) * E * 4;
    mbar_arrive_expect_tx(&full[warp][st_in], bytes);
    bulk_load(ring + static_cast<size_t>(st_in) * kTile * E, a.logits + static_cast<long long>(in.tb) * E, bytes,
              &full[warp][st_in]);
    if (++st_in == ST) st_in = 0;
    in.next(a, c1, warp);
  };
  if (VEC && lane == 0) {
    in.first(a, b0, c0, c1, warp);
    for (int k = 0; k < ST && in.ok; ++k) issue();
  }
  // (1) counts: choices and mask bytes four ahead, all loads of a round before its first addition (an error's record
  // would hold the loads behind it back).  The chunk's first kBalWarps sequences have a histogram each in shared memory,
  // their rows as in cnt; those of further ones go straight there.
  Piece pc;
  pc.first(b0, c0);
  if (pc.next(a, c1)) {
    int last = pc.b;  // the last sequence that begins in the chunk, or the last with a histogram
    while (last + 1 < a.B && last - pc.b < kBalWarps && seq_begin(a, last + 1) < c1) ++last;
    const int pairs = (c1 - c0) * K;
    const int32_t* ids = a.topk_ids + static_cast<long long>(c0) * K;
    int* cnt = w.cnt + static_cast<long long>(pc.b) * E;
    int b = pc.b;
    for (int i0 = tid; i0 < pairs; i0 += 4 * kBalThreads) {
      int id[4], tok[4];
      bool on[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kBalThreads;
        tok[k] = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(K));
        on[k] = i < pairs && (!a.mask || __ldg(a.mask + c0 + tok[k]));
        id[k] = i < pairs ? __ldg(ids + i) : 0;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!on[k]) continue;
        if (last > pc.b)
          while (b + 1 < a.B && seq_begin(a, b + 1) <= c0 + tok[k]) ++b;
        const int r = b - pc.b;
        const bool token = i0 + k * kBalThreads == tok[k] * K;  // a token is counted at its first choice
        if (id[k] < 0 || id[k] >= E) set_error(a.err, DERR_BAD_EXPERT);
        else atomicAdd((r < kBalWarps ? hist : cnt) + r * E + id[k], 1);
        if (token) atomicAdd(r < kBalWarps ? s_n + r : w.nvalid + b, 1);
      }
    }
    __syncthreads();
    const int rows = min(last - pc.b + 1, kBalWarps);
    for (int i = tid; i < rows * E; i += kBalThreads)
      if (hist[i]) atomicAdd(cnt + i, hist[i]);
    if (tid < rows && s_n[tid]) atomicAdd(w.nvalid + pc.b + tid, s_n[tid]);
  }
  const bool counted = barrier(1);  // where it gave up: run on, so that every copy is waited for
  // (2) the pass over the logits
  // the counts of a piece's sequence are fetched while the piece before it is worked on (experts tid and tid + 512)
  Piece pn;
  int nb_next = 0, cnt_next[2] = {0, 0};
  auto fetch = [&]() {
    if (!pn.next(a, c1)) return;
    nb_next = __ldcg(w.nvalid + pn.b);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int e = tid + k * kBalThreads;
      if (e < E) cnt_next[k] = __ldcg(w.cnt + static_cast<long long>(pn.b) * E + e);
    }
  };
  pn.first(b0, c0);
  fetch();
  float2 nu = make_float2(0.0f, 0.0f);  // counted tokens, sequences with any
  if (a.B == 1) {
    nu.x = static_cast<float>(__ldcg(w.nvalid));
    nu.y = nu.x > 0.0f ? 1.0f : 0.0f;
  } else {
    for (int b = tid; b < a.B; b += kBalThreads) {
      const int n = __ldcg(w.nvalid + b);
      nu.x += static_cast<float>(n);
      nu.y += n > 0 ? 1.0f : 0.0f;
    }
    nu = block_sum2(nu.x, nu.y, s_red);
  }
  const float scale = a.dloss ? __ldg(a.dloss) : 1.0f;
  const float zc = nu.x > 0.0f ? 2.0f * a.z_coef * scale / nu.x : 0.0f;
  constexpr float kLog2e = 1.4426950408889634f;
  const int sl = lane & (LPT - 1), sub = lane / LPT;
  auto expert = [&](int i) { return VEC ? 4 * (sl + LPT * (i / 4)) + i % 4 : sl + LPT * i; };  // of a lane's i-th logit
  int st = 0, ph = 0;
  pc.first(b0, c0);
  for (int nth = 0; pc.next(a, c1); nth += Tiles<kTile>::count(pc)) {
    const int nb = nb_next;
    const float inv_kn = nb > 0 ? 1.0f / (static_cast<float>(K) * static_cast<float>(nb)) : 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int e = tid + k * kBalThreads;
      if (e < E)
        su[e] = static_cast<float>(static_cast<long long>(cnt_next[k]) * E - static_cast<long long>(K) * nb) * inv_kn;
    }
    __syncthreads();
    fetch();
    f32x2 acc[kPairs], u[kPairs];  // a lane's logits in pairs
    float zs = 0.0f, bs = 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int e0 = expert(2 * i), e1 = expert(2 * i + 1);
      acc[i] = pack2(0.0f, 0.0f);
      u[i] = pack2(e0 < E ? su[e0] : 0.0f, e1 < E ? su[e1] : 0.0f);
    }
    const float cb = nb > 0 ? a.balance_coef * scale / (nu.y * static_cast<float>(nb)) : 0.0f;
    // which of a tile's tokens count, looked up a tile ahead
    auto counts_here = [&](int t) { return lane < kTile && t + lane < pc.t1 && (!a.mask || a.mask[t + lane]); };
    const int tb0 = Tiles<kTile>::first_of(pc, nth, warp);
    bool mine = counts_here(tb0);
    for (int tb = tb0; tb < pc.t1; tb += kBalWarps * kTile) {
      const float* src = ring + static_cast<size_t>(st) * kTile * E;
      const unsigned here = __ballot_sync(0xffffffffu, mine);
      mine = counts_here(tb + kBalWarps * kTile);
      if (VEC) mbar_wait(&full[warp][st], ph, &s_abort, a.timeout_ns, a.err);
      // the UN tokens of a lane go through every step together, which hides the latency of the lane sums
      f32x2 v[UN][kPairs];
      float m[UN], z[UN], dot[UN];
#pragma unroll
      for (int g = 0; g < UN; ++g) {
        const int r = g * kTok + sub;
        const bool on = (here >> r) & 1;
        m[g] = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) {
          float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          if constexpr (VEC) {
            if (on && expert(2 * i) < E) q = *reinterpret_cast<const float4*>(src + r * E + expert(2 * i));
          } else {
            const float* row = a.logits + static_cast<long long>(tb + r) * E;
            if (on && expert(2 * i) < E) q.x = __ldcs(row + expert(2 * i));
            if (on && expert(2 * i + 1) < E) q.y = __ldcs(row + expert(2 * i + 1));
            if (on && expert(2 * i + 2) < E) q.z = __ldcs(row + expert(2 * i + 2));
            if (on && expert(2 * i + 3) < E) q.w = __ldcs(row + expert(2 * i + 3));
          }
          m[g] = fmaxf(m[g], fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)));
          v[g][i] = pack2(q.x, q.y);
          v[g][i + 1] = pack2(q.z, q.w);
        }
      }
#pragma unroll
      for (int g = 0; g < UN; ++g) {
        m[g] = lanes_max<LPT>(m[g]);
        if (m[g] == -INFINITY) m[g] = 0.0f;  // a token that does not count, or without a finite logit: all terms are zero
        const f32x2 nm = pack2(-m[g], -m[g]), l2e = pack2(kLog2e, kLog2e);
        f32x2 zz = pack2(0.0f, 0.0f), dd = zz;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 x = unpack2(mul2(add2(v[g][i], nm), l2e));  // the difference first: m may be the type's lowest value
          v[g][i] = pack2(exp2_approx(x.x), exp2_approx(x.y));
          zz = add2(zz, v[g][i]);
          dd = fma2(v[g][i], u[i], dd);
        }
        const float2 zf = unpack2(zz), df = unpack2(dd);
        z[g] = zf.x + zf.y;
        dot[g] = df.x + df.y;
      }
#pragma unroll
      for (int o = LPT / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int g = 0; g < UN; ++g) {
          z[g] += __shfl_xor_sync(0xffffffffu, z[g], o);
          dot[g] += __shfl_xor_sync(0xffffffffu, dot[g], o);
        }
      }
      // The fast logarithm is off by 2^-21.4 near 1, too much for a log-sum that the z loss drives towards 0.  The exact one
      // is taken once for the UN tokens, each in lanes of its own.
      float logz = z[0];
#pragma unroll
      for (int g = 1; g < UN; ++g)
        if ((sl & (UN - 1)) == g) logz = z[g];
      logz = logf(logz);
#pragma unroll
      for (int g = 0; g < UN; ++g) {
        const int t = tb + g * kTok + sub;
        const float inv = z[g] == 0.0f ? 0.0f : __fdividef(1.0f, z[g]);  // z is between 1 and E
        const float lz = __shfl_sync(0xffffffffu, logz, (lane & ~(LPT - 1)) + g);  // (by every lane)
        const float lse = z[g] == 0.0f ? 0.0f : m[g] + lz;
        dot[g] *= inv;
        if (sl == 0) {
          zs += lse * lse;
          bs += z[g] == 0.0f ? 0.0f : 1.0f + dot[g];
        }
        // dl = p (cb (u - dot) + zc lse) with p = v / z
        const float g0 = inv * (zc * lse - cb * dot[g]), c1 = inv * cb;
        const f32x2 inv2 = pack2(inv, inv), g2 = pack2(g0, g0), c2 = pack2(c1, c1);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          acc[i] = fma2(v[g][i], inv2, acc[i]);
          v[g][i] = mul2(v[g][i], fma2(c2, u[i], g2));
        }
        if (a.dlogits && t < pc.t1) {
          float* out = a.dlogits + static_cast<long long>(t) * E;
#pragma unroll
          for (int i = 0; i < kPairs; i += 2) {
            const float2 lo = unpack2(v[g][i]), hi = unpack2(v[g][i + 1]);
            if constexpr (VEC) {
              if (expert(2 * i) < E)
                *reinterpret_cast<float4*>(out + expert(2 * i)) = make_float4(lo.x, lo.y, hi.x, hi.y);
            } else {
              if (expert(2 * i) < E) out[expert(2 * i)] = lo.x;
              if (expert(2 * i + 1) < E) out[expert(2 * i + 1)] = lo.y;
              if (expert(2 * i + 2) < E) out[expert(2 * i + 2)] = hi.x;
              if (expert(2 * i + 3) < E) out[expert(2 * i + 3)] = hi.y;
            }
          }
        }
      }
      if (VEC) {
        __syncwarp();  // the stage has been read
        if (lane == 0 && in.ok) issue();
        if (++st == ST) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    // close the piece: lane groups, then warps in order
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float2 x = unpack2(acc[i]);
#pragma unroll
      for (int o = LPT; o < 32; o <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
      }
      if (sub == 0 && expert(2 * i) < E) sums[warp * E + expert(2 * i)] = x.x;
      if (sub == 0 && expert(2 * i + 1) < E) sums[warp * E + expert(2 * i + 1)] = x.y;
    }
    const float2 part = block_sum2(zs, bs, s_red);
    const long long piece = static_cast<long long>(blockIdx.x) + pc.b;
    for (int e = tid; e < E; e += kBalThreads) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kBalWarps; ++i) s += sums[i * E + e];
      w.ppart[piece * E + e] = s;
    }
    if (tid == 0) {
      w.zpart[piece] = part.x;
      w.bpart[piece] = nb > 0 ? part.y / static_cast<float>(nb) : 0.0f;
    }
  }
  if (a.seq_off) {  // offsets: from 0 to T, never falling
    for (int b = blockIdx.x * kBalThreads + tid; b <= a.B; b += G * kBalThreads) {
      const int o = a.seq_off[b];
      if ((b == 0 && o != 0) || (b == a.B && o != T) || (b > 0 && a.seq_off[b - 1] > o)) set_error(a.err, DERR_BAD_OFFSETS);
    }
  }
  if (VEC && s_abort) {  // a wait gave up: let this warp's copies in flight land
    volatile int never = 0;
    if (lane == 0)
      for (int k = 0; k < ST; ++k) mbar_wait(&full[warp][k], k < st ? ph : ph ^ 1, &never, 20000000ull, nullptr);
    __syncwarp();
  }
  if (!barrier(2) || !counted || s_abort) return;
  // (3) mean probabilities and counts, 32 experts of one sequence at a time: a block for such a unit, its warps sharing
  // the pieces, while there are no more units than blocks, else a warp
  float2 l = make_float2(0.0f, 0.0f);
  if (blockIdx.x == G - 1) {  // the last block also adds the losses' shares
    for (int i = tid; i < G + a.B; i += kBalThreads) {
      l.x += __ldcg(w.zpart + i);
      l.y += __ldcg(w.bpart + i);
    }
  }
  const int et = (E + 31) / 32;
  const long long units = static_cast<long long>(a.B) * et;
  const bool shared = units <= G;
  const long long u0 = shared ? blockIdx.x : blockIdx.x + static_cast<long long>(warp) * G;
  for (long long un = u0; un < units; un += shared ? G : static_cast<long long>(G) * kBalWarps) {
    const int b = static_cast<int>(un / et), e = static_cast<int>(un % et) * 32 + lane;
    const int o0 = seq_begin(a, b), o1 = seq_begin(a, b + 1);
    const int n = __ldcg(w.nvalid + b), count = e < E ? __ldcg(w.cnt + static_cast<long long>(b) * E + e) : 0;
    float s = 0.0f;
    if (o1 > o0 && e < E) {
      const float* src = w.ppart + static_cast<long long>(b) * E + e;
      const int last = (o1 - 1) / chunk, by = shared ? kBalWarps : 1;
      int c = o0 / chunk + (shared ? warp : 0);
      for (; c + 3 * by <= last; c += 4 * by) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __ldcg(src + static_cast<long long>(c + k * by) * E);
        s += (x[0] + x[1]) + (x[2] + x[3]);
      }
      for (; c <= last; c += by) s += __ldcg(src + static_cast<long long>(c) * E);
    }
    if (shared) {
      s_tile[warp][lane] = s;
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < kBalWarps; ++i) s += s_tile[i][lane];
    }
    if ((!shared || warp == 0) && e < E) {
      a.probs[static_cast<long long>(b) * E + e] = n > 0 ? s / static_cast<float>(n) : 0.0f;
      a.counts[static_cast<long long>(b) * E + e] = count;
    }
    if (shared) __syncthreads();
  }
  if (blockIdx.x != G - 1) return;
  l = block_sum2(l.x, l.y, s_red);
  if (tid == 0) {
    const float bl = nu.y > 0.0f ? l.y / nu.y : 0.0f, zl = nu.x > 0.0f ? l.x / nu.x : 0.0f;
    // a loss that is switched off adds nothing, whatever its value
    a.loss[0] = (a.balance_coef != 0.0f ? a.balance_coef * bl : 0.0f) + (a.z_coef != 0.0f ? a.z_coef * zl : 0.0f);
    a.loss[1] = bl;
    a.loss[2] = zl;
  }
}

template <bool VEC, int LPT, int NV, int UN, int ST>
cudaError_t run_balance(const BalanceArgs& a, void* ws, int num_sms, cudaStream_t s) {
  auto kern = balance_kernel<VEC, LPT, NV, UN, ST>;
  constexpr int kTile = 32 / LPT * UN;
  auto bytes = [](int E) {
    return sizeof(float) * (kBalWarps * static_cast<size_t>(E) * (1 + (VEC ? ST * kTile : 0)) + (E + 3) / 4 * 4);
  };
  const size_t smem = bytes(a.E);
  // the attribute is the kernel's, whichever thread launches it with however many experts: always the same value
  cudaError_t st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(bytes(VEC ? 4 * LPT * NV : LPT * NV)));
  if (st != cudaSuccess) return st;
  if ((st = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return st;
  const BalWs w = carve_balance(ws, a.T, a.E, a.B);
  // blocks that give every warp a tile, or every sequence a block where that is more (a block works on one sequence after
  // the other: 42 tokens in 34 sequences took 93 us in one block, 15 us in sixteen)
  const long long seqs = a.T < a.B ? a.T : a.B, tiles = (a.T + kBalWarps * kTile - 1) / (kBalWarps * kTile);
  const long long want = tiles > seqs ? tiles : seqs;
  long long G;
  if (a.T * (a.E + 16) < kBalOneCluster && seqs <= kBalClusterSeqs) {
    for (G = 1; G < kBalCluster && G < want; G *= 2) {
    }
  } else {
    G = want < num_sms ? want : num_sms;  // one block an SM: all of them resident
    if (G > kBalMaxBlocks) G = kBalMaxBlocks;
    if (G <= kBalCluster) G = kBalCluster;
  }
  const int chunk = a.T > 0 ? static_cast<int>((a.T + G - 1) / G) : 1;
  if (G > kBalCluster && (st = cudaMemsetAsync(w.ctrl, 0, w.zeroed, s)) != cudaSuccess) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  if (G > kBalCluster) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(G);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(G), 1, 1);
  cfg.blockDim = dim3(kBalThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, w, chunk);
}

}  // namespace

size_t balance_ws_bytes(long long T, int E, int B) { return carve_balance(nullptr, T, E, B).bytes; }

cudaError_t launch_balance_loss(const BalanceArgs& a, void* ws, int num_sms, cudaStream_t s) {
  const bool vec = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.dlogits) & 15) == 0;
  if (!vec)
    return a.E <= 128 ? run_balance<false, 32, 4, 1, 1>(a, ws, num_sms, s) : run_balance<false, 32, 32, 1, 1>(a, ws, num_sms, s);
  if (a.E <= 32) return run_balance<true, 8, 1, 4, 4>(a, ws, num_sms, s);
  if (a.E <= 64) return run_balance<true, 16, 1, 4, 4>(a, ws, num_sms, s);
  if (a.E <= 128) return run_balance<true, 32, 1, 4, 4>(a, ws, num_sms, s);
  if (a.E <= 256) return run_balance<true, 32, 2, 2, 4>(a, ws, num_sms, s);
  if (a.E <= 512) return run_balance<true, 32, 4, 2, 2>(a, ws, num_sms, s);
  return run_balance<true, 32, 8, 1, 2>(a, ws, num_sms, s);
}

}  // namespace vgg
