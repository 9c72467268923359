// few.cu -- the whole MoE layer for at most 16 tokens in one cooperative launch (moe_forward_few).
//
//   z = x W_r ; s = sigma(z) ; selected = top_k(s + b) ; G_i = gate_scale * s_i / sum_sel s_j
//   E_i(x) = (SiLU(x W1_i) * (x W3_i)) W2_i ;  y = sum_sel G_i E_i(x) + E_shared(x)
//   latent: experts on x W_down; y = RMSNorm(sum_sel G_i E_i) W_up + E_shared(x)
//
// Steps, with a grid barrier between them (each reads what every CTA of the step before wrote):
//   A  router logits; W_down rows; the shared expert's W1|W3 rows
//   B  every CTA repeats the selection, then W1|W3 rows of the distinct selected experts, each
//      read once for all of its tokens; h = G SiLU(g) u per (expert, token) row
//   C  W2: each output feature's sum over every selected expert (and the shared one)
//   D  (latent) the norm of the latent sum, W_up rows and the shared expert's W2 rows
// One warp computes one feature: lanes stride over its weight row(s), fp32 sums, a shuffle at the
// end, so equal calls give equal bits.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxT = MOE_FEW_MAX_TOKENS;
constexpr int kMaxE = 1023;
constexpr int kMaxPairs = kMaxT * 32;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

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
  float* logits;   // [T][E]
  float* x_lat;    // [T][L]
  float* h;        // [T * k + T][I]: routed rows expert by expert, then the shared rows
  float* y_lat;    // [T][L]
};

struct Selection {
  uint16_t mask[kMaxE + 1];      // tokens of each expert
  int16_t active[kMaxPairs];     // distinct selected experts, ascending
  int16_t row0[kMaxPairs + 1];   // first h row of each
  int16_t pair_e[kMaxPairs];
  float pair_g[kMaxPairs];
  float row_gate[kMaxPairs];
  int n_active;
};

// Arrive and wait until every CTA of the (cooperative) grid has; false once the wait expires.
__device__ bool grid_barrier(uint32_t* counter, uint32_t* err) {
  __shared__ int ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1u);
    const uint64_t t0 = globaltimer_ns();
    ok = 1;
    while (true) {
      uint32_t v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= gridDim.x) break;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        raise_flag(err, kErrTimeout);
        ok = 0;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
  const bool r = ok != 0;
  __syncthreads();
  return r;
}

// One warp selects the experts of token t: k rounds of the largest key, ties to the lower index;
// NaN keys count as -infinity.
__device__ void select_token(const FewParams& p, int t, Selection& sel) {
  const int lane = threadIdx.x & 31;
  uint32_t taken = 0;
  float my_s = 0.0f, den = 0.0f;
  int my_e = 0;
  for (int slot = 0; slot < p.k; ++slot) {
    float bk = -INFINITY, bs = 0.0f;
    int be = 0x7fffffff;
    for (int j = 0; lane + 32 * j < p.E; ++j) {
      const int e = lane + 32 * j;
      if ((taken >> j) & 1u) continue;
      const float s = 1.0f / (1.0f + expf(-__ldcg(p.logits + (int64_t)t * p.E + e)));
      float key = s + p.b[e];
      if (isnan(key)) key = -INFINITY;
      if (key > bk || (key == bk && e < be)) {
        bk = key;
        be = e;
        bs = s;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float ok = __shfl_xor_sync(0xffffffffu, bk, off);
      const int oe = __shfl_xor_sync(0xffffffffu, be, off);
      const float os = __shfl_xor_sync(0xffffffffu, bs, off);
      if (ok > bk || (ok == bk && oe < be)) {
        bk = ok;
        be = oe;
        bs = os;
      }
    }
    if (lane == slot) {
      my_e = be;
      my_s = bs;
    }
    den += bs;
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
  }
  if (lane < p.k) {
    sel.pair_e[t * p.k + lane] = (int16_t)my_e;
    sel.pair_g[t * p.k + lane] = p.gate_scale * my_s / den;
  }
}

// The CTA's copy of the selection: per-expert token masks, the distinct experts in index order,
// the first h row of each and each row's gate.
__device__ void build_selection(const FewParams& p, Selection& sel) {
  const int warp = threadIdx.x >> 5;
  for (int t = warp; t < p.T; t += kWarps) select_token(p, t, sel);
  for (int e = threadIdx.x; e < p.E; e += kThreads) sel.mask[e] = 0;
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    uint32_t m = 0;
    for (int i = 0; i < p.T * p.k; ++i)
      if (sel.pair_e[i] == e) m |= 1u << (i / p.k);
    sel.mask[e] = (uint16_t)m;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0, row = 0;
    for (int e = 0; e < p.E; ++e) {
      if (!sel.mask[e]) continue;
      sel.active[n] = (int16_t)e;
      sel.row0[n++] = (int16_t)row;
      row += __popc(sel.mask[e]);
    }
    sel.row0[n] = (int16_t)row;
    sel.n_active = n;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.k; i += kThreads) {
    const int e = sel.pair_e[i], t = i / p.k;
    int a = 0;
    while (sel.active[a] != e) ++a;
    sel.row_gate[sel.row0[a] + __popc(sel.mask[e] & ((1u << t) - 1u))] = sel.pair_g[i];
  }
  __syncthreads();
}

__device__ __forceinline__ void decode_bf16x8(uint4 raw, float (&v)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// e4m3 to fp32: the bits moved to fp32's exponent and mantissa give value * 2^-120, subnormals
// included (the product below is exact).
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  if ((b & 0x7fu) == 0x7fu) return __uint_as_float(0x7fffffffu);
  return __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7fu) << 20)) * 0x1p120f;
}

// 8 consecutive weights (row `row` of matrix `e`, columns c..c+7) of stacked [n][R][K] matrices.
template <int WD>
__device__ __forceinline__ void weights8(const void* w, const void* s, int64_t e, int R, int K,
                                         int row, int c, float (&v)[8]) {
  const int64_t at = (e * R + row) * K + c;
  if constexpr (WD == MOE_F32) {
    load8(static_cast<const float*>(w) + at, v);
  } else if constexpr (WD == MOE_BF16) {
    load8(static_cast<const __nv_bfloat16*>(w) + at, v);
  } else if constexpr (WD == MOE_FP8_E4M3) {
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(w) + at));
    const float sc = __ldg(static_cast<const float*>(s) +
                           (e * (R / 128) + row / 128) * (K / 128) + c / 128);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = e4m3_to_f32(raw.x >> (8 * i) & 0xffu) * sc;
      v[4 + i] = e4m3_to_f32(raw.y >> (8 * i) & 0xffu) * sc;
    }
  } else {
    const uint32_t raw =
        __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(w) + at / 2));
    const float sc = __bfloat162float(
        static_cast<const __nv_bfloat16*>(s)[(e * (K / 32) + c / 32) * (int64_t)R + row]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int code = (int)(raw >> (4 * (i / 2 + 4 * (i % 2))) & 15u) - 8;
      v[i] = __bfloat162float(__float2bfloat16_rn((float)code * sc));
    }
  }
}

// 8 values that an earlier step of this kernel wrote (past L1).
__device__ __forceinline__ void load8_cg(const float* p, float (&v)[8]) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// acc[n] += dot(weight row, activation row n) over this lane's columns; act(n, c, v) loads 8.
template <int WD, typename Act>
__device__ __forceinline__ void dot_rows(float (&acc)[kMaxT], int n, const void* w, const void* s,
                                         int64_t e, int R, int K, int row, Act act) {
  for (int c = (threadIdx.x & 31) * 8; c < K; c += 256) {
    float v[8];
    weights8<WD>(w, s, e, R, K, row, c, v);
#pragma unroll
    for (int i = 0; i < kMaxT; ++i) {
      if (i < n) {
        float a[8];
        act(i, c, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i] = fmaf(v[j], a[j], acc[i]);
      }
    }
  }
}

__device__ __forceinline__ void zero(float (&acc)[kMaxT]) {
#pragma unroll
  for (int i = 0; i < kMaxT; ++i) acc[i] = 0.0f;
}

template <typename TA>
__device__ __forceinline__ void store_act(void* out, int64_t i, float v);
template <>
__device__ __forceinline__ void store_act<float>(void* out, int64_t i, float v) {
  static_cast<float*>(out)[i] = v;
}
template <>
__device__ __forceinline__ void store_act<__nv_bfloat16>(void* out, int64_t i, float v) {
  static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// The n-th token of a mask.
__device__ __forceinline__ int nth_token(uint32_t mask, int n) { return __fns(mask, 0, n + 1); }

template <typename TA, int WD>
__global__ void __launch_bounds__(kThreads) few_kernel(const FewParams p) {
  __shared__ Selection sel;
  __shared__ float inv_rms[kMaxT];
  constexpr int AD = WD == MOE_F32 ? MOE_F32 : MOE_BF16;  // W_down, W_up: the activations' type
  const int lane = threadIdx.x & 31;
  const int gw = blockIdx.x * kWarps + (threadIdx.x >> 5), nw = gridDim.x * kWarps;
  const int de = p.L ? p.L : p.d;
  const int P = p.T * p.k;
  const TA* x = static_cast<const TA*>(p.x);
  float acc[kMaxT], acu[kMaxT];

  // A
  const int nA = p.E + p.L + (p.n_shared ? p.I : 0);
  auto act_x = [&](int n, int c, float(&a)[8]) { load8(x + (int64_t)n * p.d + c, a); };
  for (int u = gw; u < nA; u += nw) {
    zero(acc);
    if (u < p.E) {
      dot_rows<MOE_F32>(acc, p.T, p.W_r, nullptr, 0, p.E, p.d, u, act_x);
#pragma unroll
      for (int n = 0; n < kMaxT; ++n)
        if (n < p.T) {
          const float z = warp_sum(acc[n]);
          if (lane == 0) p.logits[(int64_t)n * p.E + u] = z;
        }
    } else if (u < p.E + p.L) {
      const int f = u - p.E;
      dot_rows<AD>(acc, p.T, p.W_down, nullptr, 0, p.L, p.d, f, act_x);
#pragma unroll
      for (int n = 0; n < kMaxT; ++n)
        if (n < p.T) {
          const float v = warp_sum(acc[n]);
          if (lane == 0) p.x_lat[(int64_t)n * p.L + f] = v;
        }
    } else {
      const int f = u - p.E - p.L;
      zero(acu);
      dot_rows<WD>(acc, p.T, p.Ws13, p.ss13, 0, 2 * p.I, p.d, f, act_x);
      dot_rows<WD>(acu, p.T, p.Ws13, p.ss13, 0, 2 * p.I, p.d, p.I + f, act_x);
#pragma unroll
      for (int n = 0; n < kMaxT; ++n)
        if (n < p.T) {
          const float g = warp_sum(acc[n]), q = warp_sum(acu[n]);
          if (lane == 0) p.h[(int64_t)(P + n) * p.I + f] = silu_accurate(g) * q;
        }
    }
  }
  if (!grid_barrier(p.bar, p.err)) return;

  // B
  build_selection(p, sel);
  for (int64_t u = gw; u < (int64_t)sel.n_active * p.I; u += nw) {
    const int a = (int)(u / p.I), f = (int)(u - (int64_t)a * p.I);
    const int e = sel.active[a], row0 = sel.row0[a], n_e = sel.row0[a + 1] - row0;
    const uint32_t mask = sel.mask[e];
    zero(acc);
    zero(acu);
    auto act = [&](int n, int c, float(&v)[8]) {
      const int t = nth_token(mask, n);
      if (p.L)
        load8_cg(p.x_lat + (int64_t)t * p.L + c, v);
      else
        load8(x + (int64_t)t * p.d + c, v);
    };
    dot_rows<WD>(acc, n_e, p.W13, p.s13, e, 2 * p.I, de, f, act);
    dot_rows<WD>(acu, n_e, p.W13, p.s13, e, 2 * p.I, de, p.I + f, act);
#pragma unroll
    for (int n = 0; n < kMaxT; ++n)
      if (n < n_e) {
        const float g = warp_sum(acc[n]), q = warp_sum(acu[n]);
        if (lane == 0)
          p.h[(int64_t)(row0 + n) * p.I + f] = sel.row_gate[row0 + n] * (silu_accurate(g) * q);
      }
  }
  if (!grid_barrier(p.bar + 1, p.err)) return;

  // C: per token the sum over its experts, in expert order (K2: then the shared expert)
  auto act_sh = [&](int n, int c, float(&v)[8]) {
    load8_cg(p.h + (int64_t)(P + n) * p.I + c, v);
  };
  for (int f = gw; f < de; f += nw) {
    zero(acc);
    for (int a = 0; a < sel.n_active; ++a) {
      const int e = sel.active[a], row0 = sel.row0[a], n_e = sel.row0[a + 1] - row0;
      const uint32_t mask = sel.mask[e];
      float part[kMaxT];
      zero(part);
      auto act = [&](int n, int c, float(&v)[8]) {
        load8_cg(p.h + (int64_t)(row0 + n) * p.I + c, v);
      };
      dot_rows<WD>(part, n_e, p.W2, p.s2, e, de, p.I, f, act);
#pragma unroll
      for (int t = 0; t < kMaxT; ++t) {
        const int n = __popc(mask & ((1u << t) - 1u));
#pragma unroll
        for (int i = 0; i < kMaxT; ++i)
          if ((mask >> t & 1u) && i == n) acc[t] += part[i];
      }
    }
    if (!p.L && p.n_shared) dot_rows<WD>(acc, p.T, p.Ws2, p.ss2, 0, p.d, p.I, f, act_sh);
#pragma unroll
    for (int t = 0; t < kMaxT; ++t)
      if (t < p.T) {
        const float v = warp_sum(acc[t]);
        if (lane == 0) {
          if (p.L)
            p.y_lat[(int64_t)t * p.L + f] = v;
          else
            store_act<TA>(p.out, (int64_t)t * p.d + f, v);
        }
      }
  }
  if (!p.L) return;
  if (!grid_barrier(p.bar + 2, p.err)) return;

  // D
  for (int t = threadIdx.x >> 5; t < p.T; t += kWarps) {
    float ss = 0.0f;
    for (int c = lane; c < p.L; c += 32) {
      const float v = __ldcg(p.y_lat + (int64_t)t * p.L + c);
      ss = fmaf(v, v, ss);
    }
    ss = warp_sum(ss);
    if (lane == 0) inv_rms[t] = p.latent_norm ? 1.0f / sqrtf(ss / (float)p.L + p.eps) : 1.0f;
  }
  __syncthreads();
  auto act_u = [&](int n, int c, float(&v)[8]) {
    load8_cg(p.y_lat + (int64_t)n * p.L + c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv_rms[n];
  };
  for (int f = gw; f < p.d; f += nw) {
    zero(acc);
    dot_rows<AD>(acc, p.T, p.W_up, nullptr, 0, p.d, p.L, f, act_u);
    if (p.n_shared) dot_rows<WD>(acc, p.T, p.Ws2, p.ss2, 0, p.d, p.I, f, act_sh);
#pragma unroll
    for (int t = 0; t < kMaxT; ++t)
      if (t < p.T) {
        const float v = warp_sum(acc[t]);
        if (lane == 0) store_act<TA>(p.out, (int64_t)t * p.d + f, v);
      }
  }
}

struct FewLayout {
  size_t logits, x_lat, h, y_lat, total;
};

FewLayout few_layout(const moe_config_t* c) {
  FewLayout l;
  size_t off = 256;  // status word and barrier counters
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~size_t(255);
    return at;
  };
  const size_t T = (size_t)c->T;
  l.logits = take(T * c->E * 4);
  l.x_lat = take(T * c->d_latent * 4);
  l.h = take((T * c->k + T) * c->I * 4);
  l.y_lat = take(T * c->d_latent * 4);
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

template <typename TA, int WD>
cudaError_t launch(FewParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident at once: they wait for others
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchScope ls("few_layer", st);
  return cudaLaunchKernelEx(&cfg, few_kernel<TA, WD>, (const FewParams)p);
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
  p.logits = reinterpret_cast<float*>(base + l.logits);
  p.x_lat = reinterpret_cast<float*>(base + l.x_lat);
  p.h = reinterpret_cast<float*>(base + l.h);
  p.y_lat = reinterpret_cast<float*>(base + l.y_lat);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();  // start from a clean launch-error state
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);  // status word and barrier counters
  if (e != cudaSuccess) return status_from_cuda(e);
  switch (cfg->w_dtype) {
    case MOE_F32: e = launch<float, MOE_F32>(p, st); break;
    case MOE_BF16: e = launch<__nv_bfloat16, MOE_BF16>(p, st); break;
    case MOE_FP8_E4M3: e = launch<__nv_bfloat16, MOE_FP8_E4M3>(p, st); break;
    default: e = launch<__nv_bfloat16, MOE_INT4>(p, st); break;
  }
  return status_from_cuda(e);
}
