// The router's balance and z losses with their gradient, and the per-expert counts.
//
// For the valid tokens of every sequence b (n_b of them; n in all, B' sequences with any), p_t = softmax(l_t):
//   f_be = E / (K n_b) #{(t, k): id_tk = e},   P_be = 1 / n_b sum_t p_te
//   loss = alpha / B' sum_b sum_e f_be P_be  +  beta / n sum_t lse_t^2
//   dl_te = p_te (c_be - sum_j p_tj c_bj) + 2 beta / n lse_t p_te,   c_be = alpha f_be / (B' n_b)
//
// f depends on the choices alone, so once the counts are known one pass over the logits gives P, the z loss and
// the gradient: 8 bytes an element, bound by HBM for long batches and by the grid barriers for short ones.
// A shift of c_b by a constant leaves dl unchanged (p sums to one): with c' = alpha E / (B' n_b) (counts_be / (K n_b) -
// 1 / E), whose numerator counts_be E - K n_b is a whole number, a nearly even load loses nothing to cancellation.
//
// One cooperative launch: (1) counts by shared-memory histograms, added with integer atomics (any order, one
// result); (2) the pass over the logits; (3) the probabilities' sums and the loss.  Block c takes the tokens of
// chunk c; where a chunk crosses into another sequence it closes a piece.  The piece of (chunk c, sequence b) has
// the index c + b, unique because every next piece moves on by a chunk, a sequence or both.  Sums over tokens run
// in a fixed order, so equal calls give equal bits.
#include "internal.h"

namespace vgg {

namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxBlocks = 1024;  // bounds the number of pieces, and with it the workspace

inline size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BalWs {
  int* ctrl;      // [0] grid barrier, [1] blocks that have finished phase 3
  int* nvalid;    // [B]
  float* zpart;   // [pieces]
  int* cnt;       // [B][E]
  float* ppart;   // [pieces][E]
  float* lpart;   // [B][ceil(E / 32)]
  size_t zeroed;  // bytes from ctrl up to ppart
  size_t bytes;
};

BalWs carve_balance(void* ws, long long T, int E, int B) {
  const size_t pieces = static_cast<size_t>(T < kBalMaxBlocks ? (T > 0 ? T : 1) : kBalMaxBlocks) + B;
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = p + at;
    at += al256(bytes);
    return r;
  };
  BalWs w{};
  w.ctrl = reinterpret_cast<int*>(take(2 * sizeof(int)));
  w.nvalid = reinterpret_cast<int*>(take(sizeof(int) * B));
  w.zpart = reinterpret_cast<float*>(take(sizeof(float) * pieces));
  w.cnt = reinterpret_cast<int*>(take(sizeof(int) * static_cast<size_t>(B) * E));
  w.zeroed = at;
  w.ppart = reinterpret_cast<float*>(take(sizeof(float) * pieces * E));
  w.lpart = reinterpret_cast<float*>(take(sizeof(float) * static_cast<size_t>(B) * ((E + 31) / 32)));
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
  __device__ void first(const BalanceArgs& a, int c0) {
    int lo = 0, hi = a.B;  // the last b with seq_begin(b) <= c0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seq_begin(a, mid) <= c0) lo = mid;
      else hi = mid;
    }
    b = lo;
    t1 = c0;
  }
  __device__ bool next(const BalanceArgs& a, int c1) {
    if (t1 >= c1) return false;
    t0 = t1;
    while (b + 1 < a.B && seq_begin(a, b + 1) <= t0) ++b;
    t1 = b + 1 < a.B ? min(c1, seq_begin(a, b + 1)) : c1;
    return true;
  }
};

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kBalWarps; ++i) s += red[i];
  __syncthreads();
  return s;
}

// VEC: a token's row by 16-byte loads, LPT lanes a token (32 / LPT tokens in a warp), NV vectors a lane; else one
// value a load, a warp a token, NV values a lane.  UN tokens a lane group are in flight at once.
template <bool VEC, int LPT, int NV, int UN>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(const BalanceArgs a, const BalWs w, int chunk) {
  constexpr int W = VEC ? 4 : 1;
  constexpr int kTok = 32 / LPT;
  extern __shared__ float bal_smem[];  // [kBalWarps][E] partial sums; phase 1: the histogram
  __shared__ float s_red[kBalWarps];
  __shared__ float s_tile[kBalWarps][33];
  __shared__ int s_n, s_ok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, E = a.E, K = a.K, T = static_cast<int>(a.T);
  const int c0 = min(T, static_cast<int>(blockIdx.x) * chunk), c1 = min(T, c0 + chunk);
  auto barrier = [&](int nth) -> bool {
    if (G == 1) {
      __syncthreads();
      return true;
    }
    return grid_barrier(w.ctrl, nth * G, a.timeout_ns, a.err, &s_ok);
  };
  if (G == 1) {  // nothing was cleared for a single block
    int* z = w.ctrl;
    for (size_t i = tid; i < w.zeroed / sizeof(int); i += kBalThreads) z[i] = 0;
    __syncthreads();
  }
  if (a.seq_off) {  // offsets: from 0 to T, never falling
    for (int b = blockIdx.x * kBalThreads + tid; b <= a.B; b += G * kBalThreads) {
      const int o = a.seq_off[b];
      if ((b == 0 && o != 0) || (b == a.B && o != T) || (b > 0 && a.seq_off[b - 1] > o)) set_error(a.err, DERR_BAD_OFFSETS);
    }
  }
  Piece pc;
  // (1) counts
  int* hist = reinterpret_cast<int*>(bal_smem);
  for (int e = tid; e < E; e += kBalThreads) hist[e] = 0;
  if (tid == 0) s_n = 0;
  __syncthreads();
  pc.first(a, c0);
  while (pc.next(a, c1)) {
    const int pairs = (pc.t1 - pc.t0) * K;
    const int32_t* ids = a.topk_ids + static_cast<long long>(pc.t0) * K;
    int n = 0;
    for (int i = tid; i < pairs; i += kBalThreads) {
      const int t = i / K;
      if (a.mask && !a.mask[pc.t0 + t]) continue;
      if (i - t * K == 0) ++n;
      const int id = __ldg(ids + i);
      if (id < 0 || id >= E) set_error(a.err, DERR_BAD_EXPERT);
      else atomicAdd(&hist[id], 1);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n) atomicAdd(&s_n, n);
    __syncthreads();
    for (int e = tid; e < E; e += kBalThreads) {
      const int v = hist[e];
      if (v) {
        atomicAdd(w.cnt + static_cast<long long>(pc.b) * E + e, v);
        hist[e] = 0;
      }
    }
    if (tid == 0) {
      if (s_n) atomicAdd(w.nvalid + pc.b, s_n);
      s_n = 0;
    }
    __syncthreads();
  }
  if (!barrier(1)) return;
  // (2) the pass over the logits
  float nf = 0.0f, used = 0.0f;  // valid tokens, sequences with any
  for (int b = tid; b < a.B; b += kBalThreads) {
    const int n = __ldcg(w.nvalid + b);
    nf += static_cast<float>(n);
    used += n > 0 ? 1.0f : 0.0f;
  }
  nf = block_sum(nf, s_red);
  used = block_sum(used, s_red);
  const float scale = a.dloss ? __ldg(a.dloss) : 1.0f;
  const float zc = nf > 0.0f ? 2.0f * a.z_coef * scale / nf : 0.0f;
  const int sl = lane & (LPT - 1), sub = lane / LPT;
  pc.first(a, c0);
  while (pc.next(a, c1)) {
    const int nb = __ldcg(w.nvalid + pc.b);
    float acc[NV * W], cf[NV * W];
    float zs = 0.0f;
#pragma unroll
    for (int i = 0; i < NV * W; ++i) acc[i] = cf[i] = 0.0f;
    if (a.dlogits && nb > 0) {
      // alpha E / (B' n_b) (counts / (K n_b) - 1 / E), from the whole number counts E - K n_b
      const float kn = static_cast<float>(K) * static_cast<float>(nb);
      const float s0 = a.balance_coef * scale / (used * static_cast<float>(nb) * kn);
#pragma unroll
      for (int i = 0; i < NV * W; ++i) {
        const int e = VEC ? 4 * (sl + LPT * (i / W)) + i % W : sl + LPT * i;
        if (e < E) {
          const long long c = __ldcg(w.cnt + static_cast<long long>(pc.b) * E + e);
          cf[i] = s0 * static_cast<float>(c * E - static_cast<long long>(K) * nb);
        }
      }
    }
    for (int tb = pc.t0 + (warp * kTok + sub); tb - sub < pc.t1; tb += kBalWarps * kTok * UN) {
      float v[UN][NV * W];
      bool ok[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int t = tb + u * kBalWarps * kTok;
        ok[u] = t < pc.t1;
        const bool on = ok[u] && (!a.mask || a.mask[t]);
        const float* row = a.logits + static_cast<long long>(t) * E;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = VEC ? 4 * (sl + LPT * i) : sl + LPT * i;
          if (on && e < E) {
            if constexpr (VEC) {
              const float4 q = __ldcs(reinterpret_cast<const float4*>(row + e));
              v[u][4 * i] = q.x; v[u][4 * i + 1] = q.y; v[u][4 * i + 2] = q.z; v[u][4 * i + 3] = q.w;
            } else {
              v[u][i] = __ldcs(row + e);
            }
          } else {
#pragma unroll
            for (int k = 0; k < W; ++k) v[u][W * i + k] = -INFINITY;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int t = tb + u * kBalWarps * kTok;
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV * W; ++i) m = fmaxf(m, v[u][i]);
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -INFINITY) m = 0.0f;  // a masked token, or one without a finite logit: all terms are zero
        float z = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * W; ++i) {
          v[u][i] = expf(v[u][i] - m);
          z += v[u][i];
          dot += v[u][i] * cf[i];
        }
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) {
          z += __shfl_xor_sync(0xffffffffu, z, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float inv = z == 0.0f ? 0.0f : 1.0f / z;
        const float lse = z == 0.0f ? 0.0f : m + logf(z);
        if (sl == 0) zs += lse * lse;
        const float g0 = zc * lse - dot * inv;
#pragma unroll
        for (int i = 0; i < NV * W; ++i) {
          v[u][i] *= inv;
          acc[i] += v[u][i];
        }
        if (a.dlogits && ok[u]) {
          float* out = a.dlogits + static_cast<long long>(t) * E;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = VEC ? 4 * (sl + LPT * i) : sl + LPT * i;
            if (e < E) {
              if constexpr (VEC)
                *reinterpret_cast<float4*>(out + e) =
                    make_float4(v[u][4 * i] * (cf[4 * i] + g0), v[u][4 * i + 1] * (cf[4 * i + 1] + g0),
                                v[u][4 * i + 2] * (cf[4 * i + 2] + g0), v[u][4 * i + 3] * (cf[4 * i + 3] + g0));
              else
                out[e] = v[u][i] * (cf[i] + g0);
            }
          }
        }
      }
    }
    // close the piece: lane groups, then warps in order
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1) {
      zs += __shfl_xor_sync(0xffffffffu, zs, o);
#pragma unroll
      for (int i = 0; i < NV * W; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < NV * W; ++i) {
        const int e = VEC ? 4 * (sl + LPT * (i / W)) + i % W : sl + LPT * i;
        if (e < E) bal_smem[warp * E + e] = acc[i];
      }
    }
    const float zsum = block_sum(lane == 0 ? zs : 0.0f, s_red);
    const long long piece = static_cast<long long>(blockIdx.x) + pc.b;
    for (int e = tid; e < E; e += kBalThreads) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kBalWarps; ++i) s += bal_smem[i * E + e];
      w.ppart[piece * E + e] = s;
    }
    if (tid == 0) w.zpart[piece] = zsum;
    __syncthreads();
  }
  if (!barrier(2)) return;
  // (3) mean probabilities, counts, the loss: 32 experts of one sequence at a time, a warp for every 16th piece
  const int et = (E + 31) / 32;
  const long long units = static_cast<long long>(a.B) * et;
  for (long long un = blockIdx.x; un < units; un += G) {
    const int b = static_cast<int>(un / et), e = static_cast<int>(un % et) * 32 + lane;
    const int o0 = seq_begin(a, b), o1 = seq_begin(a, b + 1);
    float s = 0.0f;
    if (o1 > o0 && e < E)
      for (int c = o0 / chunk + warp; c <= (o1 - 1) / chunk; c += kBalWarps)
        s += __ldcg(w.ppart + (static_cast<long long>(c) + b) * E + e);
    s_tile[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < kBalWarps; ++i) s += s_tile[i][lane];
      const int n = __ldcg(w.nvalid + b);
      float term = 0.0f;
      if (e < E) {
        const int cnt = __ldcg(w.cnt + static_cast<long long>(b) * E + e);
        const float p = n > 0 ? s / static_cast<float>(n) : 0.0f;
        a.probs[static_cast<long long>(b) * E + e] = p;
        a.counts[static_cast<long long>(b) * E + e] = cnt;
        if (n > 0) term = static_cast<float>(cnt) * p * (static_cast<float>(E) / (static_cast<float>(K) * static_cast<float>(n)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
      if (lane == 0) w.lpart[un] = term;
    }
    __syncthreads();
  }
  if (tid == 0) {
    __threadfence();
    s_n = atomicAdd(w.ctrl + 1, 1);
    __threadfence();
  }
  __syncthreads();
  if (s_n != G - 1) return;
  float bl = 0.0f, zl = 0.0f;
  for (long long i = tid; i < units; i += kBalThreads) bl += __ldcg(w.lpart + i);
  for (int i = tid; i < G + a.B; i += kBalThreads) zl += __ldcg(w.zpart + i);
  bl = block_sum(bl, s_red);
  zl = block_sum(zl, s_red);
  if (tid == 0) {
    bl = used > 0.0f ? bl / used : 0.0f;
    zl = nf > 0.0f ? zl / nf : 0.0f;
    a.loss[0] = a.balance_coef * bl + a.z_coef * zl;
    a.loss[1] = bl;
    a.loss[2] = zl;
  }
}

template <bool VEC, int LPT, int NV, int UN>
cudaError_t run_balance(const BalanceArgs& a, void* ws, int num_sms, cudaStream_t s) {
  auto kern = balance_kernel<VEC, LPT, NV, UN>;
  const size_t smem = sizeof(float) * kBalWarps * a.E;
  cudaError_t st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (st != cudaSuccess) return st;
  const BalWs w = carve_balance(ws, a.T, a.E, a.B);
  const long long per = static_cast<long long>(kBalWarps) * (32 / LPT);  // tokens a block takes at once
  long long G = (a.T + per - 1) / per;
  if (G > num_sms) G = num_sms;  // one block an SM: all of them resident
  if (G > kBalMaxBlocks) G = kBalMaxBlocks;
  if (G < 1) G = 1;
  const int chunk = a.T > 0 ? static_cast<int>((a.T + G - 1) / G) : 1;
  if (G > 1 && (st = cudaMemsetAsync(w.ctrl, 0, w.zeroed, s)) != cudaSuccess) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(G), 1, 1);
  cfg.blockDim = dim3(kBalThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = G > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, w, chunk);
}

}  // namespace

size_t balance_ws_bytes(long long T, int E, int B) { return carve_balance(nullptr, T, E, B).bytes; }

cudaError_t launch_balance_loss(const BalanceArgs& a, void* ws, int num_sms, cudaStream_t s) {
  const bool vec = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.dlogits) & 15) == 0;
  if (!vec) return a.E <= 128 ? run_balance<false, 32, 4, 2>(a, ws, num_sms, s) : run_balance<false, 32, 32, 1>(a, ws, num_sms, s);
  if (a.E <= 32) return run_balance<true, 8, 1, 2>(a, ws, num_sms, s);
  if (a.E <= 128) return run_balance<true, 32, 1, 2>(a, ws, num_sms, s);
  if (a.E <= 256) return run_balance<true, 32, 2, 2>(a, ws, num_sms, s);
  if (a.E <= 512) return run_balance<true, 32, 4, 2>(a, ws, num_sms, s);
  return run_balance<true, 32, 8, 1>(a, ws, num_sms, s);
}

}  // namespace vgg
