// few.cu -- the whole MoE layer for at most 16 tokens in one cooperative launch (moe_forward_few).
//
//   z = x W_r ; s = sigma(z) ; selected = top_k(s + b) ; G_i = gate_scale * s_i / sum_sel s_j
//   E_i(x) = (SiLU(x W1_i) * (x W3_i)) W2_i ;  y = sum_sel G_i E_i(x) + E_shared(x)
//   latent: experts on x W_down; y = RMSNorm(sum_sel G_i E_i) W_up + E_shared(x)
//
// With T tokens a weight is used at most T times, so the layer is one pass over the selected experts'
// weights, bound by memory (4-bit weights: by their conversion).  Two kernels, both one CTA per SM,
// equal calls giving equal bits: few_stream_kernel (bf16 activations) keeps that pass going through
// all steps; few_kernel (fp32, small models) is plain.  Steps, each needing what every CTA wrote in
// the one before:
//   A  router scores; W_down rows; the shared expert's W1|W3 rows
//   B  every CTA repeats the selection, then W1|W3 rows of the distinct selected experts, each
//      read once for all of its tokens; h = G SiLU(g) u per (expert, token) row
//   C  W2: each output feature's sum over every selected expert (and the shared one)
//   D  (latent) W_up rows and the shared expert's W2 rows
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxT = MOE_FEW_MAX_TOKENS;
constexpr int kMaxE = 1023;
constexpr int kMaxPairs = kMaxT * 32;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;  // consumers of the stream, too
static_assert(kWarps >= kMaxT, "one for each token");

struct FewParams {
  int T, d, E, k, I, L;  // L: latent width, 0 on the K2 path
  int n_shared;
  int latent_norm;
  float gate_scale, eps;
  const void* x;
  const float* W_r;
  const float* b;
  const void *W13, *W2, *Ws13, *Ws2, *W_down, *W_up;
  const void *s13, *s2, *ss13, *ss2;
  void* out;
  uint32_t* err;
  uint32_t* bar;   // one arrival counter per barrier, zeroed before the launch
  float* scores;   // [T][E] sigma(z), zeroed before the launch
  // fp32 kernel
  float* x_lat;    // [T][L]
  float* h;        // [T * k + T][I]: routed rows expert by expert, then the shared rows
  float* y_lat;    // [T][L]
  // bf16 kernel: the same as two bf16 planes, value = plane 0 + plane 1 to 16 bits or more
  __nv_bfloat16 *x_lat2, *h2, *y_lat2;
  float* y_sh;     // [T][d] shared expert's output
  // e4m3 experts: the tokens in fp16, each divided by a power of two, and those powers
  __half* x16;
  float* x_scale;  // [16]
  float* ssq;      // [CTAs][16] sums of squares of each CTA's latent features
};

struct Selection {
  uint32_t mask[kMaxE + 1];      // tokens of each expert
  union {
    float bias[kMaxE + 1];       // b, until the choice
    int16_t slot[kMaxE + 1];     // then each expert's place in active
  };
  int16_t active[kMaxPairs];     // distinct selected experts, ascending
  uint16_t active_mask[kMaxPairs];  // their tokens
  int16_t row0[kMaxPairs + 1];   // first h row of each
  int16_t pair_e[kMaxPairs];
  float pair_g[kMaxPairs];
  float row_gate[kMaxPairs];
  uint8_t row_token[kMaxPairs];
  int n_active;
  // The stream's split of the selected experts' W1|W3 features over the CTAs: what a feature of each
  // place costs, and the sums before it.
  uint16_t cost[kMaxPairs], before[kMaxPairs + 1];
};

// Waits (bounded) until `counter` reaches `want`; one thread.
__device__ __forceinline__ bool counter_reached(const uint32_t* counter, uint32_t want) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
  return v >= want;
}
__device__ bool counter_wait(const uint32_t* counter, uint32_t want, volatile int* abort,
                             uint32_t* err) {
  const uint64_t t0 = globaltimer_ns();
  while (!counter_reached(counter, want)) {
    if (abort && *abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      if (abort) *abort = 1;
      raise_flag(err, kErrTimeout);
      return false;
    }
  }
  return true;
}

// Arrive and wait until every CTA of the (cooperative) grid has; false once the wait expires.
__device__ bool grid_barrier(uint32_t* counter, uint32_t* err) {
  __shared__ int ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1u);
    ok = counter_wait(counter, gridDim.x, nullptr, err);
    __threadfence();
  }
  __syncthreads();
  const bool r = ok != 0;
  __syncthreads();
  return r;
}

// Order-preserving map of a key to an unsigned integer >= 1; NaN keys count as -infinity.
__device__ __forceinline__ uint32_t key_bits(float v) {
  if (isnan(v)) v = -INFINITY;
  if (v == 0.0f) v = 0.0f;  // -0 ties with +0
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One warp selects the experts of token t: k rounds of the largest key, ties to the lower index.
// Lane l holds experts l, l + 32, ... in registers (N >= ceil(E / 32) of them).  The scores may still
// be on their way: the launch starts with zeros in their place, no score is stored as +0, and the
// warp reads until none is left (one trip to memory instead of a counter's and then the scores').
template <int N>
__device__ bool select_token(const FewParams& p, int t, Selection& sel, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  uint32_t key[N];
  float z[N];
  const float* sc = p.scores + (int64_t)t * p.E + lane;
  uint64_t since = 0;
  while (true) {
    bool all = true;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      z[j] = -0.0f;
      if (lane + 32 * j < p.E)
        asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(z[j]) : "l"(sc + 32 * j));
    }
#pragma unroll
    for (int j = 0; j < N; ++j) all = all && __float_as_uint(z[j]) != 0u;
    if (__all_sync(0xffffffffu, all)) break;
    const uint64_t now = globaltimer_ns();
    if (since == 0) since = now;
    bool stop = abort && *abort;
    if (now - since > kWaitLimitNs) {
      if (abort) *abort = 1;
      raise_flag(p.err, kErrTimeout);
      stop = true;
    }
    if (__any_sync(0xffffffffu, stop)) return false;
  }
  uint32_t top = 0;  // this lane's largest key left, its place j (the lowest) and score
  int top_j = 0;
  float top_s = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    key[j] = lane + 32 * j < p.E ? key_bits(z[j] + sel.bias[lane + 32 * j]) : 0u;
    if (key[j] > top) {
      top = key[j];
      top_j = j;
      top_s = z[j];
    }
  }
  float my_s = 0.0f, den = 0.0f;
  int my_e = 0;
  for (int slot = 0; slot < p.k; ++slot) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, top);  // >= 1: an expert is left
    const uint32_t e = __reduce_min_sync(0xffffffffu, top == best ? (uint32_t)(lane + 32 * top_j) : 0xffffffffu);
    const float s = __shfl_sync(0xffffffffu, top_s, e & 31);
    if (lane == slot) {
      my_e = (int)e;
      my_s = s;
    }
    den += s;
    if (lane == (int)(e & 31)) {
      const int was = top_j;
      top = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j == was) key[j] = 0;
        if (key[j] > top) {
          top = key[j];
          top_j = j;
          top_s = z[j];
        }
      }
    }
    __syncwarp();
  }
  if (lane < p.k) {
    sel.pair_e[t * p.k + lane] = (int16_t)my_e;
    sel.pair_g[t * p.k + lane] = p.gate_scale * my_s / den;
  }
  return true;
}

// The CTA's copy of the selection, by the kWarps warps of which this thread is number tid (barrier 1
// is theirs), one for each token: per-expert token masks, the distinct experts in index order, the
// first h row of each and each row's gate.  False when a wait for the scores gave up.
__device__ bool build_selection(const FewParams& p, Selection& sel, int tid, volatile int* abort) {
  constexpr int n = kWarps * 32, bar = 1;
  const int lane = tid & 31, t = tid >> 5;
  for (int e = tid; e < p.E; e += n) {
    sel.mask[e] = 0;
    sel.bias[e] = __ldg(p.b + e);
  }
  named_barrier(bar, n);
  bool ok = true;
  if (t < p.T)
    ok = p.E <= 64    ? select_token<2>(p, t, sel, abort)
         : p.E <= 384 ? select_token<12>(p, t, sel, abort)
                      : select_token<32>(p, t, sel, abort);
  if (!named_barrier_and(bar, n, ok)) return false;
  if (p.T * p.k <= 32) {  // few pairs: one lane each, ordered by comparing every two
    if (tid < 32) {
      const int P = p.T * p.k, tok = lane / p.k;
      const int e = lane < P ? sel.pair_e[lane] : 0x7fff;
      int rows = 0, place = 0;  // pairs and distinct experts before this one's
      uint32_t mask = 0, first = 0xffffffffu;
      for (int j = P - 1; j >= 0; --j) {
        const int ej = __shfl_sync(0xffffffffu, e, j);
        if (ej == e) {
          mask |= 1u << (j / p.k);
          first = j;
        }
        rows += ej < e;
      }
      const uint32_t leaders = __ballot_sync(0xffffffffu, lane < P && (int)first == lane);
      for (uint32_t m = leaders; m; m &= m - 1)
        place += __shfl_sync(0xffffffffu, e, __ffs(m) - 1) < e;
      if (lane < P) {
        if ((int)first == lane) {
          sel.active[place] = (int16_t)e;
          sel.active_mask[place] = (uint16_t)mask;
          sel.row0[place] = (int16_t)rows;
        }
        sel.row_gate[rows + __popc(mask & ((1u << tok) - 1u))] = sel.pair_g[lane];
        sel.row_token[rows + __popc(mask & ((1u << tok) - 1u))] = (uint8_t)tok;
      }
      if (lane == 0) {
        sel.n_active = __popc(leaders);
        sel.row0[__popc(leaders)] = (int16_t)P;
      }
    }
    named_barrier(bar, n);
    return true;
  }
  for (int i = tid; i < p.T * p.k; i += n) atomicOr(&sel.mask[sel.pair_e[i]], 1u << (i / p.k));
  named_barrier(bar, n);
  if (tid < 32) {  // compact: 32 experts at a time
    int na = 0, row = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const uint32_t m = e0 + lane < p.E ? sel.mask[e0 + lane] : 0u;
      const uint32_t act = __ballot_sync(0xffffffffu, m != 0);
      int incl = __popc(m);  // rows up to and including this expert
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      if (m) {
        const int a = na + __popc(act & ((1u << lane) - 1u));
        sel.active[a] = (int16_t)(e0 + lane);
        sel.active_mask[a] = (uint16_t)m;
        sel.row0[a] = (int16_t)(row + incl - __popc(m));
        sel.slot[e0 + lane] = (int16_t)a;
      }
      na += __popc(act);
      row += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      sel.row0[na] = (int16_t)row;
      sel.n_active = na;
    }
  }
  named_barrier(bar, n);
  for (int i = tid; i < p.T * p.k; i += n) {
    const int e = sel.pair_e[i], tok = i / p.k;
    const int row = sel.row0[sel.slot[e]] + __popc(sel.mask[e] & ((1u << tok) - 1u));
    sel.row_gate[row] = sel.pair_g[i];
    sel.row_token[row] = (uint8_t)tok;
  }
  named_barrier(bar, n);
  return true;
}

// sigma of a logit as it is stored: +0 marks one that is not computed yet.
__device__ __forceinline__ float stored_score(float z) {
  const float s = 1.0f / (1.0f + expf(-z));
  return s == 0.0f ? -0.0f : s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The n-th token of a mask.
__device__ __forceinline__ int nth_token(uint32_t mask, int n) {
  for (; n > 0; --n) mask &= mask - 1u;
  return __ffs(mask) - 1;
}

// acc[r][n] += this lane's part of dot(w[r], act(n)) for R weight rows and N activation rows of K.
template <int R, int N, typename Act>
__device__ __forceinline__ void dot_rows(float (&acc)[R][N], const float* const (&w)[R], int K,
                                         Act act) {
  const float* a[N];
#pragma unroll
  for (int n = 0; n < N; ++n) a[n] = act(n);
#pragma unroll(N <= 2 ? 4 : N <= 4 ? 2 : 1)
  for (int c = (threadIdx.x & 31) * 4; c < K; c += 128) {
    float4 wv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = __ldg(reinterpret_cast<const float4*>(w[r] + c));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a[n] + c));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r][n] = fmaf(wv[r].x, v.x, acc[r][n]);
        acc[r][n] = fmaf(wv[r].y, v.y, acc[r][n]);
        acc[r][n] = fmaf(wv[r].z, v.z, acc[r][n]);
        acc[r][n] = fmaf(wv[r].w, v.w, acc[r][n]);
      }
    }
  }
}

// The same for n rows, n known at run time, in passes of 8, 4 or 1 rows; out(sums, n) on every
// lane, with the warp's sums.
template <int R, typename Act, typename Out>
__device__ __forceinline__ void dots(const float* const (&w)[R], int K, int n, Act act, Out out) {
  auto pass = [&](auto width, int n0) {
    constexpr int N = decltype(width)::value;
    float acc[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[r][i] = 0.0f;
    // rows past the last read the last and are dropped
    dot_rows<R, N>(acc, w, K, [&](int i) { return act(min(n0 + i, n - 1)); });
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (n0 + i >= n) break;
      float v[R];
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = warp_sum(acc[r][i]);
      out(v, n0 + i);
    }
  };
  if (n == 1)
    pass(std::integral_constant<int, 1>{}, 0);
  else if (n <= 4)
    pass(std::integral_constant<int, 4>{}, 0);
  else
    for (int n0 = 0; n0 < n; n0 += 8) pass(std::integral_constant<int, 8>{}, n0);
}

// The fp32 layer, for small models: a warp computes a feature of W1|W3 for all tokens of its expert,
// and a feature of the sums over experts is split over up to 16 warps of a CTA when there are fewer
// features than warps.  Bound by the steps' latency as long as the weights sit in L2.
__global__ void __launch_bounds__(kThreads) few_kernel(const FewParams p) {
  __shared__ Selection sel;
  __shared__ float inv_rms[kMaxT];
  __shared__ float red[2][kWarps][kMaxT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // features in CTA-major order: neighbours of a step with few features land on different SMs
  const int gw = warp * gridDim.x + blockIdx.x, nw = gridDim.x * kWarps;
  const int de = p.L ? p.L : p.d;
  const int P = p.T * p.k;
  const float* x = static_cast<const float*>(p.x);
  const float *W13 = static_cast<const float*>(p.W13), *W2 = static_cast<const float*>(p.W2),
              *Ws13 = static_cast<const float*>(p.Ws13), *Ws2 = static_cast<const float*>(p.Ws2),
              *W_down = static_cast<const float*>(p.W_down),
              *W_up = static_cast<const float*>(p.W_up);
  float* out = static_cast<float*>(p.out);

  // A
  const int nA = p.E + p.L + (p.n_shared ? p.I : 0);
  auto token = [&](int n) { return x + (int64_t)n * p.d; };
  for (int u = gw; u < nA; u += nw) {
    if (u < p.E + p.L) {
      const float* w[1] = {u < p.E ? p.W_r + (int64_t)u * p.d : W_down + (int64_t)(u - p.E) * p.d};
      dots<1>(w, p.d, p.T, token, [&](const float (&v)[1], int n) {
        if (lane) return;
        if (u < p.E)
          p.scores[(int64_t)n * p.E + u] = stored_score(v[0]);
        else
          p.x_lat[(int64_t)n * p.L + u - p.E] = v[0];
      });
    } else {
      const int f = u - p.E - p.L;
      const float* w[2] = {Ws13 + (int64_t)f * p.d, Ws13 + (int64_t)(p.I + f) * p.d};
      dots<2>(w, p.d, p.T, token, [&](const float (&v)[2], int n) {
        if (lane == 0) p.h[(int64_t)(P + n) * p.I + f] = silu_accurate(v[0]) * v[1];
      });
    }
  }
  // the scores are waited for by themselves; x_lat needs the barrier
  if (p.L && !grid_barrier(p.bar, p.err)) return;

  // B
  if (!build_selection(p, sel, threadIdx.x, nullptr)) return;
  for (int u = gw; u < sel.n_active * p.I; u += nw) {
    const int a = u / p.I, f = u - a * p.I;
    const int64_t e = sel.active[a];
    const int row0 = sel.row0[a], n_e = sel.row0[a + 1] - row0;
    const uint32_t mask = sel.active_mask[a];
    const float* w[2] = {W13 + (e * 2 * p.I + f) * de, W13 + (e * 2 * p.I + p.I + f) * de};
    dots<2>(
        w, de, n_e,
        [&](int n) { return (p.L ? p.x_lat : x) + (int64_t)nth_token(mask, n) * de; },
        [&](const float (&v)[2], int n) {
          if (lane == 0)
            p.h[(int64_t)(row0 + n) * p.I + f] = sel.row_gate[row0 + n] * (silu_accurate(v[0]) * v[1]);
        });
  }
  if (!grid_barrier(p.bar + 1, p.err)) return;

  // Sums over segments: feature f of a step is the sum of segments 0 .. n_seg (seg(s, f, acc) adds
  // one to acc), taken by S <= most warps of a CTA by the segments' keys and joined in warp order;
  // store(t, f, v).  Neither S nor a segment's warp depends on the other tokens' experts, so neither
  // does the order of a token's sum.
  auto features = [&](int n_f, int n_seg, int most, auto key, auto seg, auto store) {
    int S = 1;
    while (S < kWarps && S < most && 2 * S * n_f <= nw) S *= 2;
    const int at_once = kWarps / S * gridDim.x;  // features of all CTAs
    int turn = 0;
    for (int f0 = 0; f0 < n_f; f0 += at_once, turn ^= 1) {
      const int f = f0 + warp / S * gridDim.x + blockIdx.x;
      float mine = 0.0f;  // lane t: token t
      if (f < n_f)
        for (int s = 0; s < n_seg; ++s)
          if (key(s) % S == warp % S) seg(s, f, mine);
      if (S > 1) {
        if (lane < kMaxT) red[turn][warp][lane] = mine;
        __syncthreads();
        if (warp % S == 0 && lane < kMaxT)
          for (int i = 1; i < S; ++i) mine += red[turn][warp + i][lane];
      }
      if (f < n_f && warp % S == 0 && lane < p.T) store(lane, f, mine);
    }
  };
  auto expert_seg = [&](int a, int f, float& mine) {
    const int64_t e = sel.active[a];
    const int row0 = sel.row0[a], n_e = sel.row0[a + 1] - row0;
    const uint32_t mask = sel.active_mask[a];
    const float* w[1] = {W2 + (e * de + f) * p.I};
    dots<1>(
        w, p.I, n_e, [&](int n) { return p.h + (int64_t)(row0 + n) * p.I; },
        [&](const float (&v)[1], int n) {
          if (lane == nth_token(mask, n)) mine += v[0];
        });
  };
  auto shared_seg = [&](int f, float& mine) {
    const float* w[1] = {Ws2 + (int64_t)f * p.I};
    dots<1>(
        w, p.I, p.T, [&](int n) { return p.h + (int64_t)(P + n) * p.I; },
        [&](const float (&v)[1], int n) {
          if (lane == n) mine += v[0];
        });
  };

  // C: per token the sum over its experts, in expert order (K2: then the shared expert)
  if (!p.L) {
    features(
        p.d, sel.n_active + p.n_shared, P + p.n_shared,
        [&](int s) { return s < sel.n_active ? (int)sel.active[s] : p.E; },
        [&](int s, int f, float& mine) {
          if (s < sel.n_active)
            expert_seg(s, f, mine);
          else
            shared_seg(f, mine);
        },
        [&](int t, int f, float v) { out[(int64_t)t * p.d + f] = v; });
    return;
  }
  features(p.L, sel.n_active, P, [&](int s) { return (int)sel.active[s]; }, expert_seg,
           [&](int t, int f, float v) { p.y_lat[(int64_t)t * p.L + f] = v; });
  if (!grid_barrier(p.bar + 2, p.err)) return;

  // D
  if (warp < p.T) {
    float ss = 0.0f;
    for (int c = lane; c < p.L; c += 32) {
      const float v = __ldcg(p.y_lat + (int64_t)warp * p.L + c);
      ss = fmaf(v, v, ss);
    }
    ss = warp_sum(ss);
    if (lane == 0) inv_rms[warp] = p.latent_norm ? 1.0f / sqrtf(ss / (float)p.L + p.eps) : 1.0f;
  }
  __syncthreads();
  features(
      p.d, 1 + p.n_shared, 2, [](int s) { return s; },
      [&](int s, int f, float& mine) {
        if (s == 1) {
          shared_seg(f, mine);
          return;
        }
        const float* w[1] = {W_up + (int64_t)f * p.L};
        dots<1>(
            w, p.L, p.T, [&](int n) { return p.y_lat + (int64_t)n * p.L; },
            [&](const float (&v)[1], int n) {
              if (lane == n) mine += v[0] * inv_rms[n];
            });
      },
      [&](int t, int f, float v) { out[(int64_t)t * p.d + f] = v; });
}

// ---------------------------------------------------------------------------------------------
// bf16 activations: one stream of weights through shared memory per SM.
//
// Producer warps walk the CTA's share of every step and copy it (bulk asynchronous copies, a row
// piece each) into a ring of slots: 16 weight rows times as many input channels as 22-24 KB hold, and
// the same channels of the activations they meet.  Consumer warps split a slot's channels and
// multiply 16 rows by 8 tokens with mma.sync m16n8k16; when a tile of rows is complete, reducer warps
// add the partial sums in a fixed order and store.  The products' K index may be permuted as long as
// both operands agree, so a lane takes 16 consecutive bytes of its row (8 bf16, 16 e4m3 or 32 4-bit
// weights) and the same channels of its token: shared memory is read in 16-byte words with no
// transposition.  (A tcgen05 product would want 16 token rows in shared memory and a trip through
// tensor memory for the one or two tokens that an expert has; products bound nothing here.)
//
// The stream does not stop at the steps' barriers.  Weights are copied ahead of them and only the
// activations' copies wait (each slot's barrier counts two arrivals, weights and activations); the
// selection runs on the consumer warps, a warp a token, while the ring fills with the shared expert's
// weights; and the shared expert's W2 stands where the last CTAs of a step are waited for.
//
// Measured (384 experts of d 7168, I 2048, top 8; in brackets the bytes at the measured copy bandwidth):
// one token 130 us (118), 16 tokens 1230 us (1240), four tokens with e4m3 weights 238-247 us (200), 16
// 812 us (626), one token with 4-bit weights 83 us (35); latent width 3584, four tokens 247-258 us (222).
//
// Values that one step leaves to the next (h, the latent activations) are kept as two bf16 planes,
// hi = bf16(v) and lo = bf16(v - hi), and multiplied plane by plane into the same fp32 sum: 16 bits
// or more of each, where one bf16 would add a rounding of 2^-9.
// ---------------------------------------------------------------------------------------------
constexpr int kCons = kWarps;  // consumer warps
// Four lanes of the stream, each four consumer warps and two slots, of which one fills while the other
// is multiplied: one slot after another on all sixteen warps left the latencies of a slot's few
// products and of its bookkeeping in the open (int4, one token: 128 us instead of 93 at
// that time).
constexpr int kLanes = 4;
constexpr int kBufs = 2;
constexpr int kSlots = kLanes * kBufs;  // one producer warp each
constexpr int kRedWarps = 2;   // sums of the finished tiles
constexpr int kFirstCons = kSlots + kRedWarps;
constexpr int kStreamThreads = 32 * (kFirstCons + kCons);
constexpr int kRed = 2;        // tiles whose partial sums wait for the reducers
// What is left of one CTA's shared memory, for 8 or 16 tokens.
constexpr int slot_bytes(int nt) { return nt == 1 ? 24064 : 22016; }
static_assert(kCons == 4 * kLanes && (kSlots & (kSlots - 1)) == 0, "four consumer warps to a lane");

// Counters of the launch (FewParams::bar): arrivals of CTAs at the end of each part.
enum : int { kCntDown = 0, kCntH = 1, kCntLat = 2, kCntShared = 3, kCntX = 4, kCounters = 5 };
constexpr int kNoDep = -1;

template <int WD>
struct Wt {
  static constexpr int kBits = WD == MOE_BF16 ? 16 : WD == MOE_FP8_E4M3 ? 8 : 4;
  static constexpr int kChunk = 128 / kBits;     // channels of a lane's 16 bytes
  static constexpr int kStep = 4 * kChunk;       // channels of a warp's 16-byte loads
  static constexpr int kUnit = WD == MOE_BF16 ? 32 : 128;  // channels a warp takes at a time
  static constexpr int kGran = WD == MOE_BF16 ? 64 : WD == MOE_FP8_E4M3 ? 128 : 256;
  static __device__ __forceinline__ int bytes(int cols) { return cols * kBits / 8; }
};

// Row pitch in a slot: past a multiple of 128 bytes by what keeps the 16-byte loads of eight lanes
// (two rows, four words each) on different banks: 64 bytes where the words follow one another (weights,
// bf16 layer's activations), 16 where they are 32 bytes apart (e4m3 layer's activations).  4-bit
// layer's activations: 64 bytes apart, two words meet, with 16 not also the rows.
__device__ __forceinline__ int slot_pitch(int bytes, int past) {
  return ((bytes + 127) & ~127) + past;
}

// Channels a slot of a segment takes (K in all, nr activation rows), cut evenly.
template <int WD, int NT>
__device__ __forceinline__ int slot_cols(int K, int nr) {
  constexpr int per16 = 16 * Wt<WD>::kBits / 8 + (WD == MOE_INT4 ? 1 : 0);
  constexpr int round = 4 * Wt<WD>::kUnit;  // a round of the lane's four consumer warps
  int c = (slot_bytes(NT) - (16 + nr) * 64) / (per16 + 2 * nr);
  const int gran = c >= round ? round : Wt<WD>::kGran;
  c = c / gran * gran;
  const int n = (K + c - 1) / c;
  return ((K + n - 1) / n + gran - 1) / gran * gran;
}

// The most activation rows (both planes of every token) leave room for one unit of channels at least.
template <int WD>
constexpr bool slot_fits(int nt) {
  return (slot_bytes(nt) - (16 + 16 * nt) * 64) /
             (16 * Wt<WD>::kBits / 8 + (WD == MOE_INT4 ? 1 : 0) + 2 * 16 * nt) >= Wt<WD>::kGran;
}
static_assert(slot_fits<MOE_BF16>(1) && slot_fits<MOE_FP8_E4M3>(1) && slot_fits<MOE_INT4>(1) &&
                  slot_fits<MOE_BF16>(2) && slot_fits<MOE_FP8_E4M3>(2) && slot_fits<MOE_INT4>(2),
              "a slot takes one unit of channels");

// What a slot holds, written by its producer for the consumers.
enum : int { kScaled = 1, kStop = 2 };  // kStop: no data, the stream ends
struct alignas(16) SlotInfo {  // written in four 16-byte stores
  int cols, wpitch, apitch, aoff;
  int soff, plane;   // int4 scales; distance of the activations' second plane (0: one plane)
  uint32_t mask;     // sums over segments: the tokens; else one bit for each
  int flags;
  int f0, cnt;
  const float* s;    // e4m3: scale of the matrix's row block 0 and the slot's first channel
  int s_ld, u_off;   // scales per row block; distance of the W3 rows (0: no pairs)
  uint32_t tile;     // the tile it belongs to; the ones before it are complete in the stream
  int pad_;
};
static_assert(sizeof(SlotInfo) == 64, "four 16-byte stores");

// A tile of features in stream order; kPublish: the CTA's share of a part is complete, add it to
// counter f0; kEnd: the last.
enum Kind { kDown, kHid, kLat, kShOut, kOut, kPublish, kEnd };
struct Tile {
  int f0;
  uint16_t row0, mask;  // first h row, columns in use
  uint8_t kind, cnt, gated, pad_;
};
// Between two pieces of one producer the stream has kSlots - 1 others: at most kSlots tiles begin, and
// twice that while it is a piece ahead, with the publishings and the end: fewer than kTiles.
constexpr int kTiles = 32;

struct StreamHead {
  uint64_t info_bar[kSlots], full[kSlots], empty[kSlots], red_full[kRed], red_empty[kRed];
  uint64_t sel_bar, inv_bar, start_bar;
  SlotInfo info[kSlots];
  Tile tile[kSlots][kTiles];  // each producer's own, for its consumers
  Tile red_tile[kRed];        // for the reducers
  uint4 zeros[4];
  uint32_t x_top;             // bits of the token's largest magnitude (token_to_f16)
  float inv[kMaxT];
  int abort;
  uint32_t done[kCounters];  // reducer warps through each part
  Selection sel;
};
constexpr size_t head_bytes() { return (sizeof(StreamHead) + 127) & ~size_t(127); }
constexpr size_t stream_smem(int nt) {
  return 128 + head_bytes() + (size_t)kRed * kCons * nt * 512 + (size_t)kSlots * slot_bytes(nt);
}
static_assert(stream_smem(1) <= 227 * 1024 && stream_smem(2) <= 227 * 1024, "one CTA's memory");

// The parts of the layer in stream order, each split evenly over the CTAs by features.
// The shared expert's W2 needs nothing of the step before it: its weights pass by while the last CTAs
// finish that step (K2: before W2; latent: before W_up).
enum Part { kPartDown, kPartShared, kPartRouted, kPartShOut, kPartW2, kPartShOutLat, kPartUp, kParts };

// The costs of the selected experts' features, by one warp.  An expert of many tokens has less of a
// slot for its weights: more pieces for the same bytes, and a CTA that gets such experts by their
// bytes alone finishes last (16 tokens over 96 experts, bf16: 744 us after a mean of 604; the whole
// layer took 960 us instead of 1075 with this).  A feature counts a quarter by its bytes and the rest
// by its pieces, in eighths of one with one token.
template <int WD, int NT>
__device__ __forceinline__ void split_by_cost(const FewParams& p, Selection& sel, int lane) {
  const int K = p.L ? p.L : p.d, planes = p.L ? 2 : 1;
  const int n = lane % kMaxT + 1;
  const int step = slot_cols<WD, NT>(K, n * planes);
  const int pieces = (K + step - 1) / step;
  const int one = __shfl_sync(0xffffffffu, pieces, 0);
  const int mine = min(2 + 6 * pieces / one, 64);
  int sum = 0;
  for (int a0 = 0; a0 < sel.n_active; a0 += 32) {
    const int a = a0 + lane;
    const uint32_t m = a < sel.n_active ? sel.active_mask[a] : 1u;
    int c = __shfl_sync(0xffffffffu, mine, __popc(m) - 1);
    if (a >= sel.n_active) c = 0;
    int incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (a < sel.n_active) {
      sel.cost[a] = (uint16_t)c;
      sel.before[a] = (uint16_t)(sum + incl - c);
    }
    sum += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) sel.before[sel.n_active] = (uint16_t)sum;
  __syncwarp();  // before lane 0 announces the selection
}

// Where CTA `cta`'s share of the selected experts' features begins: place * I + feature.
template <int G>
__device__ __forceinline__ int routed_begin(const FewParams& p, const Selection& sel, int cta,
                                            int lane) {
  const int64_t at = (int64_t)sel.before[sel.n_active] * p.I * cta / gridDim.x;
  int a = 0;  // the last place that begins at or before it
  for (int a0 = 0; a0 < sel.n_active; a0 += 32) {
    const int i = a0 + lane;
    const uint32_t in = __ballot_sync(0xffffffffu, i < sel.n_active && (int64_t)sel.before[i] * p.I <= at);
    if (in) a = a0 + 31 - __clz(in);
  }
  if (cta == (int)gridDim.x) return sel.n_active * p.I;
  const int f = (int)((at - (int64_t)sel.before[a] * p.I) / sel.cost[a]);
  return a * p.I + min(f, p.I) / G * G;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// A producer warp; warp i fills slot i with every kSlots-th piece of the stream.  (A copy instruction
// takes its addresses from uniform registers, so a warp issues the 16 and more copies of a slot one
// after another, about 60 clocks each: one warp for all slots held the stream to 4.2 TB/s.)
template <int WD, int NT>
struct Producer {
  const FewParams& p;
  StreamHead& hd;
  uint8_t* base;         // this warp's slot
  int slot, lane;
  int turn = 0;          // slot of the stream's next piece (pieces go round the slots)
  uint32_t filled = 0;   // times this warp has filled its slot
  uint32_t tile = 0;     // tiles begun
  uint32_t complete = 0; // counters known to be complete
  bool failed = false;

  // Waits until the consumers have left the slot.
  __device__ __forceinline__ bool slot_free() {
    if (failed) return false;
    const bool ok = mbar_wait_sleep(&hd.empty[slot], (filled & 1u) ^ 1u, &hd.abort, p.err);
    if (__any_sync(0xffffffffu, !ok)) failed = true;
    return !failed;
  }
  // Waits until a step is complete; the copies after it see what it published.
  __device__ __forceinline__ void step_complete(int dep) {
    if (dep == kNoDep || (complete >> dep & 1u)) return;
    int ok = 1;
    if (lane == 0) ok = counter_wait(p.bar + dep, gridDim.x, &hd.abort, p.err);
    if (!__shfl_sync(0xffffffffu, ok, 0)) failed = true;  // the copies bring what is there
    complete |= 1u << dep;
    asm volatile("fence.proxy.async;" ::: "memory");
  }
  __device__ __forceinline__ void next_tile(int kind, int f0, int cnt, int row0, uint32_t mask,
                                            int gated) {
    if (failed) return;  // no longer paced by the slot: the consumers still read what is there
    if (lane == 0)
      hd.tile[slot][tile % kTiles] = Tile{f0,           (uint16_t)row0, (uint16_t)mask, (uint8_t)kind,
                                          (uint8_t)cnt, (uint8_t)gated, 0};
    ++tile;
  }

  // Matrices [R][K] (one, or one of each expert) and the activation rows that they meet.
  struct Source {
    const uint8_t* w;
    const void* s;             // scales
    int R, K;
    int u_off;                 // > 0: pairs of rows, the W3 rows at + u_off
    const __nv_bfloat16* act;  // plane 0; plane 1 at + plane elements unless plane is 0
    int64_t plane;
    bool tokens;               // activation rows are the tokens of the mask, else row0 ...
    int dep;                   // part that must be complete before the activations are read
    bool scaled;               // multiply by the tokens' 1 / rms
    int lane_cols;             // lane n - 1: slot_cols() for n tokens and, above bit 20, the pieces
    int64_t w_step, s_step;    // bytes from one expert's matrix and scales to the next

    __device__ __forceinline__ void fit(int lane) {
      const int c = slot_cols<WD, NT>(K, (lane % kMaxT + 1) * (plane ? 2 : 1));
      lane_cols = c | (K + c - 1) / c << 20;
      w_step = (int64_t)R * Wt<WD>::bytes(K);
      s_step = WD == MOE_FP8_E4M3 ? (int64_t)(R >> 7) * (K >> 7) * 4 : (int64_t)(K >> 5) * R * 2;
    }
  };

  // The segment of matrix e (-1: the only one) for features f0 .. f0 + cnt and the tokens of mask:
  // this warp's pieces of it.
  __device__ __forceinline__ void seg(const Source& g, int e, int f0, int cnt, uint32_t mask,
                                      int row0) {
    const int n = __popc(mask);
    const int fit = __shfl_sync(0xffffffffu, g.lane_cols, n - 1);
    const int step = fit & 0xfffff, pieces = fit >> 20;
    const int first = (slot - turn) & (kSlots - 1);  // the first that falls to this warp
    turn = (turn + pieces) & (kSlots - 1);
    if (first >= pieces) return;
    int c0 = first * step;
    const uint8_t* w = g.w;
    const void* sc = g.s;
    if (e >= 0) {
      w += e * g.w_step;
      if constexpr (WD != MOE_BF16) sc = static_cast<const uint8_t*>(sc) + e * g.s_step;
    }
    const int wpitch = slot_pitch(Wt<WD>::bytes(step), 64);
    const int apitch = slot_pitch(step * 2, WD == MOE_BF16 ? 64 : 16);
    const int soff = 16 * wpitch, aoff = soff + (WD == MOE_INT4 ? step : 0);
    const int rows = n * (g.plane ? 2 : 1);
    // this lane's weight row
    const int r = g.u_off ? lane & 7 : lane;
    const bool has = lane < 16 && r < cnt;
    const uint8_t* w_row =
        w + (int64_t)(f0 + r + (g.u_off && lane >= 8 ? g.u_off : 0)) * g.K * Wt<WD>::kBits / 8;
    // this lane's activation row (rows <= 32)
    const int pl = lane >= n, j = lane - pl * n;
    const int a_src = lane < rows ? (g.tokens ? nth_token(mask, j) : row0 + j) : 0;
    const __nv_bfloat16* a_row = g.act + pl * g.plane + (int64_t)a_src * g.K;
    uint64_t* full = &hd.full[slot];
    for (; c0 < g.K; c0 += kSlots * step) {
      if (!slot_free()) return;
      const int cols = min(step, g.K - c0);
      const uint32_t nb = Wt<WD>::bytes(cols);
      if (lane == 0) {
        int4* i = reinterpret_cast<int4*>(&hd.info[slot]);
        const uint64_t sp = WD == MOE_FP8_E4M3
                                ? reinterpret_cast<uint64_t>(static_cast<const float*>(sc) + (c0 >> 7))
                                : 0;
        i[0] = make_int4(cols, wpitch, apitch, aoff);
        i[1] = make_int4(soff, g.plane ? n * apitch : 0, (int)(g.tokens ? (1u << n) - 1u : mask),
                         g.scaled ? kScaled : 0);
        i[2] = make_int4(f0, cnt, (int)(uint32_t)sp, (int)(sp >> 32));
        i[3] = make_int4(g.K >> 7, g.u_off, (int)(tile - 1), 0);
        mbar_arrive(&hd.info_bar[slot]);
        mbar_arrive_expect_tx(full, (g.u_off ? 2 * cnt : cnt) * nb);
      }
      __syncwarp();
      if (has) bulk_load(base + lane * wpitch, w_row + Wt<WD>::bytes(c0), nb, full);
      if constexpr (WD == MOE_INT4) {
        // scales [K / 32][R]: eight rows of a group a copy, into [group][16]
        const int q = lane & 1, grp = lane >> 1;
        if (g.u_off || q * 8 < cnt) {
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(sc) +
                                     (int64_t)((c0 >> 5) + grp) * g.R + f0 +
                                     (g.u_off ? q * g.u_off : q * 8);
          uint32_t dst = smem_u32(base + soff + grp * 32 + q * 16);
          for (int i = grp; i < cols >> 5; i += 16, src += 16 * (int64_t)g.R, dst += 512)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src)
                         : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full))
                     : "memory");
      }
      step_complete(g.dep);
      if (lane == 0) mbar_arrive_expect_tx(full, rows * cols * 2);
      __syncwarp();
      if (lane < rows) bulk_load(base + aoff + lane * apitch, a_row + c0, cols * 2, full);
      ++filled;
    }
  }

  // The CTA's share of the layer.
  __device__ void run() {
    constexpr int G = WD == MOE_INT4 ? 8 : 1;  // 16-byte copies of the bf16 scales of eight rows
    // the stream starts behind the router's loads (see Consumer::router)
    if (!mbar_wait_sleep(&hd.start_bar, 0, &hd.abort, p.err)) failed = true;
    failed = __any_sync(0xffffffffu, failed);
    const Selection& sel = hd.sel;
    const uint32_t all = (1u << p.T) - 1u;
    const int P = p.T * p.k, de = p.L ? p.L : p.d;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
    const __nv_bfloat16* x13 =
        WD == MOE_FP8_E4M3 ? reinterpret_cast<const __nv_bfloat16*>(p.x16) : x;
    const int dep13 = WD == MOE_FP8_E4M3 ? kCntX : kNoDep;
    auto u8 = [](const void* q) { return static_cast<const uint8_t*>(q); };
#pragma unroll 1
    for (int part = 0; part < kParts && !failed; ++part) {
      if ((part == kPartDown || part == kPartUp) && !p.L) continue;
      if (part == kPartShared && !p.n_shared) continue;
      if ((part == kPartShOut || part == kPartShOutLat) &&
          (!p.n_shared || (part == kPartShOutLat) != (p.L != 0)))
        continue;
      if (part == kPartRouted) {
        const bool ok = mbar_wait_sleep(&hd.sel_bar, 0, &hd.abort, p.err);
        if (__any_sync(0xffffffffu, !ok)) {
          failed = true;
          break;
        }
      }
      Source src;
      const bool pair = part == kPartShared || part == kPartRouted;
      int total, kind = kOut;
      if (part == kPartDown) {
        src = Source{u8(p.W_down), nullptr, p.L, p.d, 0, x, 0, true, kNoDep, false, 0, 0, 0};
        total = p.L;
        kind = kDown;
      } else if (part == kPartShared) {
        src = Source{u8(p.Ws13), p.ss13, 2 * p.I, p.d, p.I, x13, 0, true, dep13, false, 0, 0, 0};
        total = p.I;
        kind = kHid;
      } else if (part == kPartRouted) {
        src = Source{u8(p.W13), p.s13, 2 * p.I, de, p.I, x13, 0, true, dep13, false, 0, 0, 0};
        if (p.L) {
          src.act = p.x_lat2;
          src.plane = (int64_t)p.T * p.L;
          src.dep = kCntDown;
        }
        total = sel.n_active * p.I;
        kind = kHid;
      } else if (part == kPartW2) {
        src = Source{u8(p.W2), p.s2, de, p.I, 0, p.h2, (int64_t)(P + p.T) * p.I, false, kCntH,
                     false, 0, 0, 0};
        total = de;
        if (p.L) kind = kLat;
      } else if (part == kPartUp) {
        src = Source{u8(p.W_up), nullptr, p.d, p.L, 0, p.y_lat2, (int64_t)p.T * p.L, false, kCntLat,
                     true, 0, 0, 0};
        total = p.d;
      } else {
        src = Source{u8(p.Ws2), p.ss2, p.d, p.I, 0, p.h2, (int64_t)(P + p.T) * p.I, false,
                     kCntShared, false, 0, 0, 0};
        total = p.d;
        kind = kShOut;
      }
      src.fit(lane);
      const bool routed = part == kPartRouted;
      int u0, u1;
      if (routed) {
        u0 = routed_begin<G>(p, sel, blockIdx.x, lane);
        u1 = routed_begin<G>(p, sel, blockIdx.x + 1, lane);
      } else {
        u0 = (int)((int64_t)(total / G) * blockIdx.x / gridDim.x) * G;
        u1 = (int)((int64_t)(total / G) * (blockIdx.x + 1) / gridDim.x) * G;
      }
      int a = routed ? u0 / p.I : 0, f = u0 - a * p.I * (routed ? 1 : 0), left = u1 - u0;
#pragma unroll 1
      while (left > 0) {  // spans of one matrix (routed: of one expert), in tiles of nearly one size
        const int len = routed ? min(left, p.I - f) : left;
        const int n = (len + (pair ? 7 : 15)) >> (pair ? 3 : 4);
        const int size = len / G / n, more = len / G - size * n;
        const int e = routed ? sel.active[a] : -1;
        const uint32_t mask = routed ? sel.active_mask[a] : all;
        const int h_row = routed ? sel.row0[a] : P;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int cnt = (size + (i < more)) * G;
          next_tile(kind, f, cnt, h_row, (1u << __popc(mask)) - 1u, routed);
          if (part == kPartW2) {
#pragma unroll 1
            for (int j = 0; j < sel.n_active; ++j)
              seg(src, sel.active[j], f, cnt, sel.active_mask[j], sel.row0[j]);
          } else {
            seg(src, e, f, cnt, mask, part == kPartUp ? 0 : P);
          }
          f += cnt;
        }
        left -= len;
        ++a;
        if (routed) f = 0;
      }
      if (part == kPartDown) next_tile(kPublish, kCntDown, 0, 0, 0, 0);
      if (part == kPartShared) next_tile(kPublish, kCntShared, 0, 0, 0, 0);
      if (part == kPartRouted) next_tile(kPublish, kCntH, 0, 0, 0, 0);
      if (part == kPartW2 && p.L) next_tile(kPublish, kCntLat, 0, 0, 0, 0);
    }
    next_tile(kEnd, 0, 0, 0, 0, 0);
    if (slot_free() && lane == 0) {
      hd.info[slot].flags = kStop;
      hd.info[slot].tile = tile;
      mbar_arrive(&hd.info_bar[slot]);
    }
    // after a failure the copies in flight still have to land before the CTA ends
    if (filled) mbar_wait(&hd.full[slot], (filled - 1) & 1u, nullptr, nullptr, kDrainLimitNs);
  }
};

// Shared-memory loads and products without side effects, which the compiler may schedule freely: the
// addresses come from settle() after the wait for the slot, and the sums pass through settle()
// before the slot is given back, so none leaves the time in which the slot is the consumers'.
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds16_or_zero(uint32_t addr, bool on) {
  uint4 v;
  asm("{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "r"(addr), "r"((int)on));
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t addr) {
  uint16_t v;
  asm("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t settle(uint32_t v) {
  asm volatile("" : "+r"(v)::"memory");
  return v;
}
__device__ __forceinline__ void settle_sum(float& v) { asm volatile("" : "+f"(v)::"memory"); }

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as fp16, in order (exact, NaN included).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& p01, uint32_t& p23) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(p01), "=r"(p23)
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a),
                             *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  __nv_bfloat162 r = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&a),
                             *reinterpret_cast<__nv_bfloat162*>(&b),
                             *reinterpret_cast<__nv_bfloat162*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                             *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// Four e4m3 codes as bf16, in order (exact, NaN included).
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t& p01, uint32_t& p23) {
  uint32_t h[2];
  e4m3x4_to_f16(w, h[0], h[1]);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&h[0]));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&h[1]));
  const __nv_bfloat162 l = __float22bfloat162_rn(a), u = __float22bfloat162_rn(b);
  p01 = *reinterpret_cast<const uint32_t*>(&l);
  p23 = *reinterpret_cast<const uint32_t*>(&u);
}

// Eight 4-bit codes (nibbles j and j + 4 are channels 2j and 2j + 1) times their scale, rounded once.
// 0x00 to 0xff are bf16's multiples of 2^-133 without a gap (the subnormals and the first binade), so a
// nibble at bit 0 or 4 is u * 2^-133 or u * 2^-129 as it stands, and one fma with the scale times
// 2^133 or 2^129 and -8 times the scale, both exact, gives (u - 8) * scale.  Scales of 2^-5 and more,
// whose multiples end past the largest bf16, take the other form: 128 + u is 0x4300 | u, minus 136
// exact.  (15 operations a word there, 9 here and 4 a scale.)
struct Int4Scale {
  uint32_t low, high, minus8;
  __device__ __forceinline__ static bool fits(uint32_t sc) { return (sc & 0x7fffu) < 0x3d00u; }
  __device__ __forceinline__ void set(uint32_t sc) {  // two copies of the scale
    high = mul_bf16x2(mul_bf16x2(sc, 0x60006000u), 0x5f805f80u);  // 2^65, 2^64
    low = mul_bf16x2(high, 0x41804180u);                           // 2^4
    minus8 = mul_bf16x2(sc, 0xc100c100u);
  }
};
__device__ __forceinline__ void int4x8_to_bf16(uint32_t w, const Int4Scale& sc, uint32_t (&v)[4]) {
  const uint32_t w8 = w >> 8;
  v[0] = fma_bf16x2(w & 0x000f000fu, sc.low, sc.minus8);
  v[1] = fma_bf16x2(w & 0x00f000f0u, sc.high, sc.minus8);
  v[2] = fma_bf16x2(w8 & 0x000f000fu, sc.low, sc.minus8);
  v[3] = fma_bf16x2(w8 & 0x00f000f0u, sc.high, sc.minus8);
}
__device__ __forceinline__ void int4x8_to_bf16(uint32_t w, uint32_t sc, uint32_t (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = mul_bf16x2(sub_bf16x2(((w >> (4 * j)) & 0x000f000fu) | 0x43004300u, 0x43084308u), sc);
}

__device__ __forceinline__ void split_planes(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float f = __bfloat162float(hi);
  lo = __float2bfloat16_rn(isinf(f) ? 0.0f : v - f);
}

// The sixteen consumer warps: four to a lane of the stream, so that the latencies of a slot's few
// products and of its bookkeeping overlap with three other lanes', while the lane's other slot fills.
// A warp adds its channels of a tile's segments up over the pieces its lane gets; the tile's end brings
// the sixteen sums together.  NT: groups of
// 8 tokens.  Every wait gives up once the CTA's abort flag is set, so the warps may leave one by one.
template <int WD, int NT>
struct Consumer {
  const FewParams& p;
  StreamHead& hd;
  const uint8_t* slots;
  float* red;  // [kCons][NT][16 rows][8 tokens]
  int warp, lane;

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return mbar_wait_sleep(bar, parity, &hd.abort, p.err);
  }

  // Hands this warp's sums of tile number t to the reducers.
  __device__ __forceinline__ bool hand_over(const float (&acc)[NT][4], uint32_t t, const Tile& ti) {
    const int gr = lane >> 2, t4 = lane & 3;
    if (!wait(&hd.red_empty[t % kRed], (t / kRed & 1u) ^ 1u)) return false;
    if (warp == 0 && lane == 0) hd.red_tile[t % kRed] = ti;
    if (ti.kind < kPublish) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float* r = red + ((t % kRed * kCons + warp) * NT + n) * 128 + gr * 8 + t4 * 2;
        *reinterpret_cast<float2*>(r) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(r + 64) = make_float2(acc[n][2], acc[n][3]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&hd.red_full[t % kRed]);
    return true;
  }

  // Router logits: the CTA takes every gridDim-th expert, kExp at a time; the warps split the input
  // channels, so that a CTA reads the tokens once for them.  The stream starts when the first
  // kExp experts' loads are in: in the wake of a full ring they took 7 us instead of 4.
  __device__ void router() {
    constexpr int kExp = 3, kMost = 2, kTok = 4;  // loads in flight, in registers
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
    const int part = ((p.d + kCons - 1) / kCons + 31) / 32 * 32;
    const int end = min(p.d, (warp + 1) * part);
    if ((int)blockIdx.x >= p.E && lane == 0) mbar_arrive(&hd.start_bar);
    for (int e0 = blockIdx.x; e0 < p.E; e0 += kExp * (int)gridDim.x) {
#pragma unroll 1
      for (int n = 0; n < p.T; n += kTok) {
        float z[kExp][kTok];
#pragma unroll
        for (int j = 0; j < kExp; ++j)
#pragma unroll
          for (int t = 0; t < kTok; ++t) z[j][t] = 0.0f;
#pragma unroll 1
        for (int c0 = warp * part + lane * 4; c0 < end; c0 += 128 * kMost) {
          float4 wv[kMost][kExp];
          uint2 xv[kMost][kTok];
#pragma unroll
          for (int i = 0; i < kMost; ++i) {
            const int c = c0 + i * 128;
#pragma unroll
            for (int j = 0; j < kExp; ++j) {
              const int e = e0 + j * (int)gridDim.x;
              wv[i][j] = c < end && e < p.E
                             ? __ldg(reinterpret_cast<const float4*>(p.W_r + (int64_t)e * p.d + c))
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int t = 0; t < kTok; ++t)
              xv[i][t] = c < end && n + t < p.T
                             ? __ldg(reinterpret_cast<const uint2*>(x + (int64_t)(n + t) * p.d + c))
                             : make_uint2(0, 0);
          }
#pragma unroll
          for (int i = 0; i < kMost; ++i)
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
              const float x0 = __uint_as_float(xv[i][t].x << 16),
                          x1 = __uint_as_float(xv[i][t].x & 0xffff0000u),
                          x2 = __uint_as_float(xv[i][t].y << 16),
                          x3 = __uint_as_float(xv[i][t].y & 0xffff0000u);
#pragma unroll
              for (int j = 0; j < kExp; ++j) {
                z[j][t] = fmaf(wv[i][j].x, x0, z[j][t]);
                z[j][t] = fmaf(wv[i][j].y, x1, z[j][t]);
                z[j][t] = fmaf(wv[i][j].z, x2, z[j][t]);
                z[j][t] = fmaf(wv[i][j].w, x3, z[j][t]);
              }
            }
        }
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
          if (n + t >= p.T) break;
#pragma unroll
          for (int j = 0; j < kExp; ++j) {
            const float v = warp_sum(z[j][t]);
            if (lane == 0) red[(warp * kExp + j) * kMaxT + n + t] = v;
          }
        }
      }
      if (e0 == (int)blockIdx.x && lane == 0) mbar_arrive(&hd.start_bar);
      named_barrier(1, kCons * 32);
      for (int i = warp * 32 + lane; i < kExp * p.T; i += kCons * 32) {
        const int j = i / p.T, t = i - j * p.T, e = e0 + j * (int)gridDim.x;
        if (e >= p.E) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kCons; ++w) v += red[(w * kExp + j) * kMaxT + t];
        p.scores[(int64_t)t * p.E + e] = stored_score(v);
      }
      named_barrier(1, kCons * 32);  // red has been read
    }
  }

  // How a product takes the activations' planes: the only one; both in turn; or, with up to four
  // tokens, the first in columns 0 to 3 and the second in 4 to 7, which saves half of the products and
  // loads, and adds the columns up at the end.
  enum Planes { kOne, kInTurn, kSideBySide };

  // A slot's 16 rows times its tokens (NG groups of 8), this warp's channels: added to d.
  template <Planes PLANES, int NG>
  __device__ __forceinline__ void multiply(const SlotInfo& si, uint32_t base, int part,
                                           float (&d)[NT][4]) {
    using W = Wt<WD>;
    const int gr = lane >> 2, t4 = lane & 3;
    const int cols = si.cols;
    const int n_act = __popc(si.mask);
    const uint32_t wa_row = base + gr * si.wpitch, wb_row = wa_row + 8 * si.wpitch;
    const uint32_t sc_row = base + si.soff + gr * 2;
    constexpr bool kZeros = WD == MOE_INT4;
    const uint32_t zeros = settle(smem_u32(hd.zeros));
    // a column of a product is a token's place among the segment's: 8 tokens to a group of columns
    uint32_t arow[NG];
    bool on[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int col = PLANES == kSideBySide ? gr & 3 : n * 8 + gr;
      on[n] = col < n_act;
      arow[n] = base + si.aoff + col * si.apitch;
      if (PLANES == kSideBySide && gr >= 4) arow[n] += si.plane;
    }
    const float *s0p = nullptr, *s1p = nullptr;
    if constexpr (WD == MOE_FP8_E4M3) {
      const int r0 = si.f0 + min(gr, si.cnt - 1);
      const int r1 = si.u_off ? r0 + si.u_off : si.f0 + min(gr + 8, si.cnt - 1);
      s0p = si.s + (r0 >> 7) * si.s_ld;
      s1p = si.s + (r1 >> 7) * si.s_ld;
    }
    const uint32_t plane = PLANES == kInTurn ? si.plane : 0;
    // two bf16 units at a time, with sums of their own, so that their products overlap
    constexpr int kPar = WD == MOE_BF16 ? 2 : 1;
    constexpr int kSteps = WD == MOE_BF16 ? kPar : W::kUnit / W::kStep;
    float o[kPar][NG][4];
#pragma unroll
    for (int i = 0; i < kPar; ++i) zero_sums(o[i]);
#pragma unroll 1
    for (int u0 = part * W::kUnit; u0 < cols; u0 += kPar * 4 * W::kUnit) {
      float s0 = 0.0f, s1 = 0.0f;
      if constexpr (WD == MOE_FP8_E4M3) {  // one scale block: its own sum
        s0 = __ldg(s0p + (u0 >> 7));
        s1 = __ldg(s1p + (u0 >> 7));
        zero_sums(o[0]);
      }
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        constexpr int stride = WD == MOE_BF16 ? 4 * W::kUnit : W::kStep;
        if (WD == MOE_BF16 && u0 + st * stride >= cols) break;
        const int col = u0 + st * stride + t4 * W::kChunk;
        const uint4 ra = lds16(wa_row + W::bytes(col)), rb = lds16(wb_row + W::bytes(col));
        // 4-bit: the channels past the end of K (some lanes of the last unit) count as zeros
        const bool valid = WD != MOE_INT4 || col < cols;
        uint32_t sa = 0, sb = 0;
        if constexpr (WD == MOE_INT4) {
          sa = valid ? lds2(sc_row + col) * 0x10001u : 0u;  // 32 bytes a group of 32 channels
          sb = valid ? lds2(sc_row + 16 + col) * 0x10001u : 0u;
        }
        const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
        uint32_t q[NG], q2[NG];  // this lane's channels of its tokens, plane by plane
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          q[n] = arow[n] + col * 2;
          q2[n] = q[n] + plane;
          if (kZeros && !(on[n] && valid)) q[n] = q2[n] = zeros;
        }
        // A column without a token is zeros: not loaded, which spares the shared-memory pipe (e4m3,
        // 16 tokens over 96 experts: 773 -> 741 us), or loaded from a place of zeros, which spares
        // instructions (4-bit weights, of which these are the bound: 593 us, not loaded 620).
        auto token = [&](uint32_t at, int n) {
          return kZeros ? lds16(at) : lds16_or_zero(at, on[n]);
        };
        auto products = [&](const auto& fa, const auto& fb) {
#pragma unroll
          for (int h = 0; h < W::kChunk / 8; ++h) {  // 8 channels: two products
            uint32_t a[4], b[4];
            if constexpr (WD == MOE_BF16) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a[i] = wa[i];
                b[i] = wb[i];
              }
            } else if constexpr (WD == MOE_FP8_E4M3) {
              if constexpr (PLANES != kOne) {
                e4m3x4_to_bf16(wa[2 * h], a[0], a[1]);
                e4m3x4_to_bf16(wa[2 * h + 1], a[2], a[3]);
                e4m3x4_to_bf16(wb[2 * h], b[0], b[1]);
                e4m3x4_to_bf16(wb[2 * h + 1], b[2], b[3]);
              } else {
                e4m3x4_to_f16(wa[2 * h], a[0], a[1]);
                e4m3x4_to_f16(wa[2 * h + 1], a[2], a[3]);
                e4m3x4_to_f16(wb[2 * h], b[0], b[1]);
                e4m3x4_to_f16(wb[2 * h + 1], b[2], b[3]);
              }
            } else {
              int4x8_to_bf16(wa[h], fa, a);
              int4x8_to_bf16(wb[h], fb, b);
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              float(&sum)[4] = o[WD == MOE_BF16 ? st : 0][n];
              const uint4 v = token(q[n] + h * 16, n);
              if constexpr (WD == MOE_FP8_E4M3 && PLANES == kOne) {
                mma16816_f16(sum, a[0], b[0], a[1], b[1], v.x, v.y);
                mma16816_f16(sum, a[2], b[2], a[3], b[3], v.z, v.w);
              } else {
                mma16816(sum, a[0], b[0], a[1], b[1], v.x, v.y);
                mma16816(sum, a[2], b[2], a[3], b[3], v.z, v.w);
              }
              if (PLANES == kInTurn) {
                const uint4 v2 = token(q2[n] + h * 16, n);
                mma16816(sum, a[0], b[0], a[1], b[1], v2.x, v2.y);
                mma16816(sum, a[2], b[2], a[3], b[3], v2.z, v2.w);
              }
            }
          }
        };
        if constexpr (WD == MOE_INT4) {
          if (__all_sync(0xffffffffu, Int4Scale::fits(sa) && Int4Scale::fits(sb))) {
            Int4Scale fa, fb;
            fa.set(sa);
            fb.set(sb);
            products(fa, fb);
          } else {
            products(sa, sb);
          }
        } else {
          products(0, 0);
        }
      }
      if constexpr (WD == MOE_FP8_E4M3) {
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[n][i] = fmaf(i < 2 ? s0 : s1, o[0][n][i], d[n][i]);
      }
    }
    if constexpr (WD != MOE_FP8_E4M3) {
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < kPar; ++j) d[n][i] = j ? d[n][i] + o[j][n][i] : o[0][n][i];
    }
  }

  template <int N>
  __device__ __forceinline__ static void zero_sums(float (&v)[N][4]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[n][i] = 0.0f;
  }

  __device__ void run() {
    const int line = warp >> 2, part = warp & 3, t4 = lane & 3;
    float acc[NT][4];
    zero_sums(acc);
    uint32_t tile = 0;
    for (uint32_t piece = 0;; ++piece) {
      const int at = line + piece % kBufs * kLanes;  // pieces go round the slots, kLanes apart here
      const uint32_t parity = piece / kBufs & 1u;
      if (!wait(&hd.info_bar[at], parity)) return;
      SlotInfo si;  // in four loads
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<int4*>(&si)[i] = reinterpret_cast<const int4*>(&hd.info[at])[i];
      for (const uint32_t now = si.tile; tile != now; ++tile) {  // tiles that ended before it
        if (!hand_over(acc, tile, hd.tile[at][tile % kTiles])) return;
        zero_sums(acc);
      }
      const int flags = si.flags;
      if (flags & kStop) return;
      if (!wait(&hd.full[at], parity)) return;
      float d[NT][4];
      zero_sums(d);
      const uint32_t addr = settle(smem_u32(slots) + at * slot_bytes(NT));
      const int n_act = __popc(si.mask);
      const bool side = si.plane && n_act <= 4;
      if (side)
        multiply<kSideBySide, 1>(si, addr, part, d);
      else if (NT > 1 && n_act > 8)
        si.plane ? multiply<kInTurn, NT>(si, addr, part, d) : multiply<kOne, NT>(si, addr, part, d);
      else
        si.plane ? multiply<kInTurn, 1>(si, addr, part, d) : multiply<kOne, 1>(si, addr, part, d);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) settle_sum(d[n][i]);
      const uint32_t mask = si.mask;
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd.empty[at]);
      if (side) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[0][i] += __shfl_xor_sync(0xffffffffu, d[0][i], 2);
      }
      const bool scaled = flags & kScaled;
      if (scaled && !wait(&hd.inv_bar, 0)) return;
      if ((mask & (mask + 1u)) == 0) {  // places are tokens, or those of the tile's only segment
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // not the columns past the last: their zeros times an infinite weight are NaN
            const int tok = n * 8 + t4 * 2 + (i & 1);
            const float v = scaled ? d[n][i] * hd.inv[tok] : d[n][i];
            acc[n][i] += mask >> tok & 1u ? v : 0.0f;
          }
      } else {  // each place's sums to the lanes that hold its token's
        uint32_t m = mask;
        for (int j = 0; m; ++j, m &= m - 1) {
          const int tok = __ffs(m) - 1, src = (lane & ~3) | (j & 7) >> 1;
          float lo = j & 1 ? d[0][1] : d[0][0], hi = j & 1 ? d[0][3] : d[0][2];
          if (NT > 1 && j >= 8) {
            lo = j & 1 ? d[NT - 1][1] : d[NT - 1][0];
            hi = j & 1 ? d[NT - 1][3] : d[NT - 1][2];
          }
          lo = __shfl_sync(0xffffffffu, lo, src);
          hi = __shfl_sync(0xffffffffu, hi, src);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (tok == n * 8 + t4 * 2 + i) {
                acc[n][i] += lo;
                acc[n][2 + i] += hi;
              }
        }
      }
    }
  }
};

// The reducer warps: sum the consumer warps' partial tiles in warp order, store the tiles' features
// and publish the parts.
template <int WD, int NT>
struct Reducer {
  const FewParams& p;
  StreamHead& hd;
  const float* red;
  int tid, lane;  // of kRedWarps warps
  float ssq[2 * NT] = {};  // squares of the latent features of this thread's tokens

  __device__ void run() {
    if constexpr (WD == MOE_FP8_E4M3) {
      if ((int)blockIdx.x < p.T) token_to_f16(blockIdx.x);
      publish(kCntX);
    }
    for (uint32_t t = 0;; ++t) {
      if (!mbar_wait_sleep(&hd.red_full[t % kRed], t / kRed & 1u, &hd.abort, p.err)) return;
      const Tile ti = hd.red_tile[t % kRed];
      if (ti.kind == kEnd) return;
      if (ti.kind == kPublish) {
        publish(ti.f0);
      } else if (ti.kind == kHid) {
        hidden(ti, red + (t % kRed) * kCons * NT * 128);
      } else {
        rows(ti, red + (t % kRed) * kCons * NT * 128);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd.red_empty[t % kRed]);
    }
  }
  static __device__ __forceinline__ float sum(const float* r) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kCons; ++w) v += r[w * NT * 128];
    return v;
  }
  // 8 pairs of W1 and W3 features times 8 NT tokens, one a thread and turn
  __device__ __forceinline__ void hidden(const Tile& ti, const float* r) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = tid & 7, tok = n * 8 + (tid >> 3);
      const float* q = r + n * 128 + row * 8 + (tid >> 3);
      const float g = sum(q), u = sum(q + 64);
      if (row >= ti.cnt || !(ti.mask >> tok & 1u)) continue;
      const int hr = ti.row0 + __popc(ti.mask & ((1u << tok) - 1u));
      float v;
      if constexpr (WD == MOE_FP8_E4M3) {
        const float xs = __ldcg(p.x_scale + (ti.gated ? hd.sel.row_token[hr] : tok));
        v = silu_accurate(g * xs) * (u * xs);
      } else {
        v = silu_accurate(g) * u;
      }
      if (ti.gated) v *= hd.sel.row_gate[hr];
      store_planes(p.h2 + (int64_t)hr * p.I + ti.f0 + row, (int64_t)p.T * (p.k + 1) * p.I, v);
    }
  }
  // 16 features times 8 NT tokens, two a thread and token group
  __device__ __forceinline__ void rows(const Tile& ti, const float* r) {
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const int row = tid & 15, tok = i * 4 + (tid >> 4);
      const float v = sum(r + (tok >> 3) * 128 + row * 8 + (tok & 7));
      const bool live = row < ti.cnt && tok < p.T;
      if (ti.kind == kLat) {  // 16 consecutive lanes hold one token's features
        float q = live ? v * v : 0.0f;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
        ssq[i] += q;
      }
      if (!live) continue;
      const int f = ti.f0 + row;
      if (ti.kind == kShOut)  // for this very thread: the features' tiles are the same
        p.y_sh[(int64_t)tok * p.d + f] = v;
      else if (ti.kind == kOut)
        static_cast<__nv_bfloat16*>(p.out)[(int64_t)tok * p.d + f] =
            __float2bfloat16_rn(p.n_shared ? v + p.y_sh[(int64_t)tok * p.d + f] : v);
      else
        store_planes((ti.kind == kDown ? p.x_lat2 : p.y_lat2) + (int64_t)tok * p.L + f,
                     (int64_t)p.T * p.L, v);
    }
  }
  // The token for the products with e4m3 weights, which convert to fp16 in a fifth of the
  // instructions that bf16 takes: divided by the power of two that brings its largest magnitude to
  // 2^13 .. 2^14, so that nothing overflows and what is lost of small values is below 2^-38 of the
  // largest.  A row with an infinity or a NaN is taken as it is.
  __device__ void token_to_f16(int t) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + (int64_t)t * p.d;
    uint32_t top = 0;  // bits of the largest magnitude
    for (int c = tid * 8; c < p.d; c += kRedWarps * 256) {
      float v[8];
      load8(x + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&hd.x_top, top);
    named_barrier(3, kRedWarps * 32);
    top = *(volatile uint32_t*)&hd.x_top;
    int e = top == 0 || top >= 0x7f800000u ? 0 : (int)(top >> 23) - 127 - 13;
    e = max(e, -110);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    for (int c = tid * 8; c < p.d; c += kRedWarps * 256) {
      float v[8];
      load8(x + c, v);
      uint4 h;
      uint32_t* w = &h.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 q = __floats2half2_rn(v[2 * i] * down, v[2 * i + 1] * down);
        w[i] = *reinterpret_cast<const uint32_t*>(&q);
      }
      *reinterpret_cast<uint4*>(p.x16 + (int64_t)t * p.d + c) = h;
    }
    if (tid == 0) p.x_scale[t] = __uint_as_float((uint32_t)(127 + e) << 23);
  }
  static __device__ __forceinline__ void store_planes(__nv_bfloat16* at, int64_t plane, float v) {
    __nv_bfloat16 hi, lo;
    split_planes(v, hi, lo);
    at[0] = hi;
    at[plane] = lo;
  }
  // Publishes what the CTA has stored so far to the other CTAs' loads and bulk copies.
  __device__ void publish(int counter) {
    if (counter == kCntLat && (tid & 15) == 0) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i)
        p.ssq[blockIdx.x * kMaxT + i * 4 + (tid >> 4)] = ssq[i];
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    __threadfence();
    __syncwarp();
    // the last of the warps to come adds the CTA to the counter
    if (lane == 0 && atomicAdd(&hd.done[counter], 1u) == kRedWarps - 1) {
      __threadfence();
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.bar + counter) : "memory");
    }
    if (counter == kCntLat) inverse_rms();
  }
  // 1 / rms of the tokens' latent sums, once every CTA has published its squares.
  __device__ void inverse_rms() {
    int ok = 1;
    if (lane == 0) ok = counter_wait(p.bar + kCntLat, gridDim.x, &hd.abort, p.err);
    if (!__shfl_sync(0xffffffffu, ok, 0)) return;
    for (int t = tid >> 5; t < p.T; t += kRedWarps) {
      float ss = 0.0f;
      for (int c = lane; c < (int)gridDim.x; c += 32) ss += __ldcg(p.ssq + c * kMaxT + t);
      ss = warp_sum(ss);
      if (lane == 0) hd.inv[t] = p.latent_norm ? 1.0f / sqrtf(ss / (float)p.L + p.eps) : 1.0f;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&hd.inv_bar);
  }
};

template <int WD, int NT>
__global__ void __launch_bounds__(kStreamThreads, 1) few_stream_kernel(const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~uintptr_t(127));
  StreamHead& hd = *reinterpret_cast<StreamHead*>(smem);
  float* red = reinterpret_cast<float*>(smem + head_bytes());
  uint8_t* slots = smem + head_bytes() + (size_t)kRed * kCons * NT * 512;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&hd.full[i], 2 + (WD == MOE_INT4 ? 32 : 0));  // weights, activations (+ scales)
      mbar_init(&hd.info_bar[i], 1);
      mbar_init(&hd.empty[i], kCons / kLanes);
    }
    mbar_init(&hd.sel_bar, kCons);
    mbar_init(&hd.inv_bar, kRedWarps);
    mbar_init(&hd.start_bar, kCons);
    for (int i = 0; i < kRed; ++i) {
      mbar_init(&hd.red_full[i], kCons);
      mbar_init(&hd.red_empty[i], kRedWarps);
    }
    hd.abort = 0;
    hd.x_top = 0;
    for (int i = 0; i < 4; ++i) hd.zeros[i] = make_uint4(0, 0, 0, 0);
    for (int i = 0; i < kCounters; ++i) hd.done[i] = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp < kSlots) {
    Producer<WD, NT> v{p, hd, slots + (size_t)warp * slot_bytes(NT), warp, lane};
    v.run();
  } else if (warp < kFirstCons) {
    Reducer<WD, NT> v{p, hd, red, (int)threadIdx.x - 32 * kSlots, lane};
    v.run();
  } else {
    Consumer<WD, NT> v{p, hd, slots, red, warp - kFirstCons, lane};
    v.router();
    if (!build_selection(p, hd.sel, threadIdx.x - 32 * kFirstCons, &hd.abort)) return;
    if (warp == kFirstCons) split_by_cost<WD, NT>(p, hd.sel, lane);
    if (lane == 0) mbar_arrive(&hd.sel_bar);
    v.run();
  }
}

struct FewLayout {
  size_t scores, x_lat, h, y_lat, y_sh, x16, x_scale, ssq, total;
};

constexpr int kMaxCtas = 256;  // the grid is one CTA per SM, at most this many

FewLayout few_layout(const moe_config_t* c) {
  FewLayout l;
  size_t off = 256;  // status word and barrier counters
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~size_t(255);
    return at;
  };
  const size_t T = (size_t)c->T;
  l.scores = take(T * c->E * 4);  // follows the status word: cleared with it
  // 4 bytes a value: one fp32, or two bf16 planes
  l.x_lat = take(T * c->d_latent * 4);
  l.h = take((T * c->k + T) * c->I * 4);
  l.y_lat = take(T * c->d_latent * 4);
  l.y_sh = take(c->act_dtype == MOE_BF16 && c->n_shared ? T * c->d * 4 : 0);
  l.x16 = take(c->w_dtype == MOE_FP8_E4M3 ? T * c->d * 2 : 0);
  l.x_scale = take(c->w_dtype == MOE_FP8_E4M3 ? kMaxT * 4 : 0);
  l.ssq = take(c->d_latent ? (size_t)kMaxCtas * kMaxT * 4 : 0);
  l.total = off;
  return l;
}

moe_status_t validate_few(const moe_config_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->d <= 0 || c->E < 1 || c->k < 1 || c->k > c->E || c->I <= 0)
    return MOE_ERR_INVALID_ARG;
  if (c->n_shared != 0 && c->n_shared != 1) return MOE_ERR_INVALID_ARG;
  if (c->d_latent < 0 || c->reserved_ != 0) return MOE_ERR_INVALID_ARG;
  if (c->act_dtype != MOE_F32 && c->act_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->w_dtype != MOE_F32 && c->w_dtype != MOE_BF16 && c->w_dtype != MOE_FP8_E4M3 &&
      c->w_dtype != MOE_INT4)
    return MOE_ERR_INVALID_ARG;
  if (c->flags) return MOE_ERR_UNSUPPORTED;
  if (c->T > kMaxT || c->k > 32 || c->E > kMaxE) return MOE_ERR_UNSUPPORTED;
  if (c->d > 65536 || c->I > 65536 || c->d_latent > 65536) return MOE_ERR_UNSUPPORTED;
  if (c->n_shared && c->I_shared != c->I) return MOE_ERR_UNSUPPORTED;
  const bool quantised = c->w_dtype == MOE_FP8_E4M3 || c->w_dtype == MOE_INT4;
  if (quantised ? c->act_dtype != MOE_BF16 || c->d_latent > 0 : c->w_dtype != c->act_dtype)
    return MOE_ERR_UNSUPPORTED;
  if (c->w_dtype == MOE_FP8_E4M3 && c->quant_block != 128) return MOE_ERR_UNSUPPORTED;
  if (c->w_dtype == MOE_INT4 && c->quant_block != 32) return MOE_ERR_UNSUPPORTED;
  const int step = c->w_dtype == MOE_FP8_E4M3 ? 128 : c->w_dtype == MOE_F32 ? 16 : 32;
  if (c->d % step || c->I % step || c->d_latent % step) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

cudaError_t start(const void* kernel, FewParams& p, int threads, size_t smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int sms = num_sms();
  cfg.gridDim = dim3(sms < kMaxCtas ? sms : kMaxCtas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident at once: they wait for others
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&p};
  LaunchScope ls("few_layer", st);
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int WD>
cudaError_t start_stream(FewParams& p, cudaStream_t st) {
  // 8 or 16 tokens: the second group of columns costs registers and shared memory
  const int nt = p.T <= 8 ? 1 : 2;
  const void* kernel = nt == 1 ? (const void*)few_stream_kernel<WD, 1>
                               : (const void*)few_stream_kernel<WD, 2>;
  static std::atomic<uint64_t> ready[2];  // devices whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready[nt - 1].load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)stream_smem(nt));
    if (e != cudaSuccess) return e;
    ready[nt - 1].fetch_or(bit, std::memory_order_relaxed);
  }
  return start(kernel, p, kStreamThreads, stream_smem(nt), st);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_few_workspace_size(const moe_config_t* cfg) {
  return moe::validate_few(cfg) == MOE_OK ? moe::few_layout(cfg).total : 0;
}

extern "C" moe_status_t moe_forward_few(const moe_config_t* cfg, const void* x, const float* W_r,
                                        const float* b, const void* W13, const void* W2,
                                        const float* W13_scale, const float* W2_scale,
                                        const void* Ws13, const void* Ws2,
                                        const float* Ws13_scale, const float* Ws2_scale,
                                        const void* W_down, const void* W_up, void* out, void* ws,
                                        size_t ws_bytes, void* stream) {
  using namespace moe;
  moe_status_t s = validate_few(cfg);
  if (s != MOE_OK) return s;
  const FewLayout l = few_layout(cfg);
  if (!ws || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
  auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  if (!aligned(ws)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!x || !W_r || !b || !W13 || !W2 || !out) return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared && (!Ws13 || !Ws2)) return MOE_ERR_INVALID_ARG;
  const bool quantised = cfg->w_dtype == MOE_FP8_E4M3 || cfg->w_dtype == MOE_INT4;
  if (quantised && (!W13_scale || !W2_scale || (cfg->n_shared && (!Ws13_scale || !Ws2_scale))))
    return MOE_ERR_INVALID_ARG;
  if (cfg->d_latent > 0 && (!W_down || !W_up)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, (const void*)W_r, W13, W2, Ws13, Ws2, W_down, W_up, (const void*)out,
                        (const void*)W13_scale, (const void*)W2_scale, (const void*)Ws13_scale,
                        (const void*)Ws2_scale})
    if (!aligned(q)) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(b) & 3u) return MOE_ERR_INVALID_ARG;

  uint8_t* base = static_cast<uint8_t*>(ws);
  FewParams p = {};
  p.T = (int)cfg->T;
  p.d = cfg->d;
  p.E = cfg->E;
  p.k = cfg->k;
  p.I = cfg->I;
  p.L = cfg->d_latent;
  p.n_shared = cfg->n_shared;
  p.latent_norm = cfg->latent_norm;
  p.gate_scale = cfg->gate_scale;
  p.eps = cfg->rms_eps;
  p.x = x;
  p.W_r = W_r;
  p.b = b;
  p.W13 = W13;
  p.W2 = W2;
  p.Ws13 = Ws13;
  p.Ws2 = Ws2;
  p.W_down = W_down;
  p.W_up = W_up;
  p.s13 = W13_scale;
  p.s2 = W2_scale;
  p.ss13 = Ws13_scale;
  p.ss2 = Ws2_scale;
  p.out = out;
  p.err = reinterpret_cast<uint32_t*>(base);
  p.bar = reinterpret_cast<uint32_t*>(base + 128);
  p.scores = reinterpret_cast<float*>(base + l.scores);
  p.x_lat = reinterpret_cast<float*>(base + l.x_lat);
  p.h = reinterpret_cast<float*>(base + l.h);
  p.y_lat = reinterpret_cast<float*>(base + l.y_lat);
  p.x_lat2 = reinterpret_cast<__nv_bfloat16*>(base + l.x_lat);
  p.h2 = reinterpret_cast<__nv_bfloat16*>(base + l.h);
  p.y_lat2 = reinterpret_cast<__nv_bfloat16*>(base + l.y_lat);
  p.y_sh = reinterpret_cast<float*>(base + l.y_sh);
  p.x16 = reinterpret_cast<__half*>(base + l.x16);
  p.x_scale = reinterpret_cast<float*>(base + l.x_scale);
  p.ssq = reinterpret_cast<float*>(base + l.ssq);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();  // start from a clean launch-error state
  // status word, barrier counters and the scores' places
  cudaError_t e = cudaMemsetAsync(ws, 0, l.scores + (size_t)p.T * p.E * 4, st);
  if (e != cudaSuccess) return status_from_cuda(e);
  switch (cfg->w_dtype) {
    case MOE_F32: e = start((const void*)few_kernel, p, kThreads, 0, st); break;
    case MOE_BF16: e = start_stream<MOE_BF16>(p, st); break;
    case MOE_FP8_E4M3: e = start_stream<MOE_FP8_E4M3>(p, st); break;
    default: e = start_stream<MOE_INT4>(p, st); break;
  }
  return status_from_cuda(e);
}
