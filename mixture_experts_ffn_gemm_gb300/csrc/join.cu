// join.cu -- what stands between two blocks: post-norm of the branch, gate, scales, residual sum and
// the next block's norm, one pass over the rows (moe_block_join).
//
//   v = y w_post / sqrt(mean(y^2) + eps) ;  r' = a r + b g v ;  n = r' w_pre / sqrt(mean(r'^2) + eps)
//
// Bound by memory: resid, branch (and an element gate) are read once and resid_out and normed written
// once, the row waiting in registers between the two norms.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

// Partial sums of a row's two norms, one float for each warp of a CTA.
constexpr int kRowSumBytes = 2 * 32 * sizeof(float);
constexpr int kRowsSmem = 100 * 1024;  // a row's operands in join_rows_kernel, two rows an SM at least

struct JoinParams {
  int64_t T;
  int d;
  int gate;
  bool sigmoid;
  float a, b, eps;
  int64_t ld_r, ld_y, ld_g, ld_ro, ld_n;
  const void *resid, *branch, *post_w, *g, *pre_w;
  void *resid_out, *normed;
};

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Streamed operands: read once, so they leave L1 to the per-channel vectors that every row reads.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// V consecutive elements as they are stored: 16-byte words for V = 8, one element for V = 1.
template <typename T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 q;
  __device__ __forceinline__ void stream(const __nv_bfloat16* p) { q = ld_stream16(p); }
  __device__ __forceinline__ void cached(const __nv_bfloat16* p) {
    q = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float, 8> {
  uint4 q[2];
  __device__ __forceinline__ void stream(const float* p) {
    q[0] = ld_stream16(p);
    q[1] = ld_stream16(p + 4);
  }
  __device__ __forceinline__ void cached(const float* p) {
    q[0] = __ldg(reinterpret_cast<const uint4*>(p));
    q[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(q[i].x);
      v[4 * i + 1] = __uint_as_float(q[i].y);
      v[4 * i + 2] = __uint_as_float(q[i].z);
      v[4 * i + 3] = __uint_as_float(q[i].w);
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T q;
  __device__ __forceinline__ void stream(const T* p) { q = *p; }
  __device__ __forceinline__ void cached(const T* p) { q = __ldg(p); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32<T>(q); }
};
template <typename T>
__device__ __forceinline__ void put(T* p, const float (&v)[8]) { store8(p, v); }
template <typename T>
__device__ __forceinline__ void put(T* p, const float (&v)[1]) { *p = from_f32<T>(v[0]); }

// Sum over the `lanes` threads of a row: a power of two of one warp's lanes, or the whole CTA
// through red (one float per warp; the caller uses another array for its next sum, so one barrier
// is enough).  The same order, hence the same bits, on every thread.
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float v, int lanes, float* red) {
  if constexpr (!BLOCK) {
    for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  } else {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    float s = lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
  }
}

// A row on `lanes` threads, NC chunks of V columns each, held in registers from the only read to
// the only write: chunk i of thread j covers columns (j + i * lanes) * V ...  BLOCK: the row takes
// the whole CTA; else lanes (a power of two <= 32) of a warp, several rows to a CTA.
template <typename TA, typename TR, int V, int NC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 256) join_kernel(const JoinParams p, int lanes) {
  __shared__ float red[2][32];
  const int j = BLOCK ? (int)threadIdx.x : (int)threadIdx.x & (lanes - 1);
  const int64_t t = BLOCK ? (int64_t)blockIdx.x
                          : blockIdx.x * (int64_t)(256 / lanes) + threadIdx.x / lanes;
  const bool live = t < p.T;  // BLOCK: always; idle threads still take part in the shuffles
  const TA* pw = static_cast<const TA*>(p.post_w);
  const TA* qw = static_cast<const TA*>(p.pre_w);
  const TA* gp = static_cast<const TA*>(p.g);
  const TA* y = static_cast<const TA*>(p.branch) + t * p.ld_y;
  const TR* r = static_cast<const TR*>(p.resid) + t * p.ld_r;
  Raw<TA, V> yr[NC], gr[NC];
  Raw<TR, V> rr[NC];
  bool on[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (j + i * lanes) * V;
    on[i] = live && c < p.d;
    if (on[i]) {
      yr[i].stream(y + c);
      rr[i].stream(r + c);
      if (p.gate == MOE_GATE_ELEMENT) gr[i].stream(gp + t * p.ld_g + c);
    }
  }
  float tg = 1.0f;
  if (p.gate == MOE_GATE_TOKEN && live) {
    tg = to_f32<TA>(gp[t]);
    if (p.sigmoid) tg = 1.0f / (1.0f + expf(-tg));
  }
  float inv = 1.0f;
  if (pw) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (on[i]) {
        float v[V];
        yr[i].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(v[e], v[e], ss);
      }
    inv = 1.0f / sqrtf(row_sum<BLOCK>(ss, lanes, red[0]) / (float)p.d + p.eps);
  }
  float s[NC][V];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!on[i]) continue;
    const int c = (j + i * lanes) * V;
    float rv[V];
    yr[i].get(s[i]);
    rr[i].get(rv);
    if (pw) {
      Raw<TA, V> wr;
      float w[V];
      wr.cached(pw + c);
      wr.get(w);
#pragma unroll
      for (int e = 0; e < V; ++e) s[i][e] = s[i][e] * inv * w[e];
    }
    if (p.gate == MOE_GATE_CHANNEL || p.gate == MOE_GATE_ELEMENT) {
      float g[V];
      if (p.gate == MOE_GATE_CHANNEL) gr[i].cached(gp + c);
      gr[i].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (p.sigmoid) g[e] = 1.0f / (1.0f + expf(-g[e]));
        s[i][e] *= g[e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s[i][e] = p.a * rv[e] + p.b * (s[i][e] * tg);
      ss = fmaf(s[i][e], s[i][e], ss);
    }
    if (live) put(static_cast<TR*>(p.resid_out) + t * p.ld_ro + c, s[i]);
  }
  if (!p.normed) return;
  const float ninv = 1.0f / sqrtf(row_sum<BLOCK>(ss, lanes, red[1]) / (float)p.d + p.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!on[i]) continue;
    const int c = (j + i * lanes) * V;
    Raw<TA, V> wr;
    float w[V];
    wr.cached(qw + c);
    wr.get(w);
#pragma unroll
    for (int e = 0; e < V; ++e) s[i][e] = s[i][e] * ninv * w[e];
    put(static_cast<TA*>(p.normed) + t * p.ld_n + c, s[i]);
  }
}

// Many wide rows: a row on a CTA of a quarter as many threads as it has chunks, and as many CTAs on
// an SM as its shared memory holds rows.  A row's operands arrive by asynchronous copies without a
// register, and r' takes their place between the norms; a thread reads only what it has copied, so
// that the sums' barriers are the only ones.  (Rows held in registers: at most four CTAs an SM, and
// 159 us where this takes 153 for 16384 x 7168 bf16 rows with a gate per channel, 6.1 TB/s.)
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// 8 elements to shared memory: 16-byte word i of chunk c at word i * chunks + c of the array.
template <typename T>
__device__ __forceinline__ void copy8(uint4* dst, int chunks, int c, const T* src) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    copy16(dst + i * chunks + c, reinterpret_cast<const uint4*>(src) + i);
}
template <typename T>
__device__ __forceinline__ void read8(const uint4* src, int chunks, int c, float (&v)[8]) {
  Raw<T, 8> w;
  if constexpr (sizeof(T) == 2) {
    w.q = src[c];
  } else {
    w.q[0] = src[c];
    w.q[1] = src[chunks + c];
  }
  w.get(v);
}

// Two fp32 operations an instruction, each rounded as the single one: the kernel below issues more
// instructions than its memory traffic has time for otherwise.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() = default;
  __device__ __forceinline__ F2(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ void pairs(const float (&x)[8], F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = F2(x[2 * i], x[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void put2(T* p, const F2 (&v)[4]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i].get(x[2 * i], x[2 * i + 1]);
  store8(p, x);
}
__device__ __forceinline__ float total(F2 s) {
  float a, b;
  s.get(a, b);
  return a + b;
}

template <typename TA, typename TR>
__global__ void __launch_bounds__(1024) join_rows_kernel(const JoinParams p) {
  extern __shared__ uint4 row4[];
  __shared__ float red[2][32];
  static_assert(sizeof(red) == kRowSumBytes, "counted when the launch sets its limit");
  const int chunks = p.d >> 3;
  const int64_t t = blockIdx.x;
  const bool el = p.gate == MOE_GATE_ELEMENT, gated = el || p.gate == MOE_GATE_CHANNEL;
  uint4* ys = row4;
  uint4* rs = ys + chunks * (int)(sizeof(TA) / 2);
  uint4* gs = rs + chunks * (int)(sizeof(TR) / 2);
  const TA* y = static_cast<const TA*>(p.branch) + t * p.ld_y;
  const TR* r = static_cast<const TR*>(p.resid) + t * p.ld_r;
  const TA* pw = static_cast<const TA*>(p.post_w);
  const TA* qw = static_cast<const TA*>(p.pre_w);
  const TA* gp = static_cast<const TA*>(p.g);
  TR* ro = static_cast<TR*>(p.resid_out) + t * p.ld_ro;
  TA* no = static_cast<TA*>(p.normed) + t * p.ld_n;
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    copy8(ys, chunks, c, y + c * 8);
    copy8(rs, chunks, c, r + c * 8);
    if (el) copy8(gs, chunks, c, gp + t * p.ld_g + c * 8);
  }
  float scale = p.b;  // of the branch: b, the token's gate, 1 / rms
  if (p.gate == MOE_GATE_TOKEN) {
    const float v = to_f32<TA>(gp[t]);
    scale *= p.sigmoid ? 1.0f / (1.0f + expf(-v)) : v;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  float x[8];
  F2 v[4], w[4];
  if (pw) {
    F2 ss(0.0f);
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      read8<TA>(ys, chunks, c, x);
      pairs(x, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fma2(v[e], v[e], ss);
    }
    scale *= 1.0f / sqrtf(row_sum<true>(total(ss), 0, red[0]) / (float)p.d + p.eps);
  }
  const F2 scale2(scale), a2(p.a);
  F2 ss(0.0f);
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    read8<TA>(ys, chunks, c, x);
    pairs(x, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] * scale2;
    if (pw) {
      load8(pw + c * 8, x);
      pairs(x, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * w[e];
    }
    if (gated) {
      if (el)
        read8<TA>(gs, chunks, c, x);
      else
        load8(gp + c * 8, x);
      if (p.sigmoid) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 1.0f / (1.0f + expf(-x[e]));
      }
      pairs(x, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * w[e];
    }
    read8<TR>(rs, chunks, c, x);
    pairs(x, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = fma2(a2, w[e], v[e]);
      ss = fma2(v[e], v[e], ss);
    }
    put2(ro + c * 8, v);
    if (p.normed) {
      ys[c] = *reinterpret_cast<const uint4*>(v);
      rs[c] = *reinterpret_cast<const uint4*>(v + 2);
    }
  }
  if (!p.normed) return;
  const F2 ninv(1.0f / sqrtf(row_sum<true>(total(ss), 0, red[1]) / (float)p.d + p.eps));
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    *reinterpret_cast<uint4*>(v) = ys[c];
    *reinterpret_cast<uint4*>(v + 2) = rs[c];
    load8(qw + c * 8, x);
    pairs(x, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] * ninv * w[e];
    put2(no + c * 8, v);
  }
}

// Rows too wide for registers without wide loads: r' waits in shared memory between the norms, each
// thread reading back its own columns.
template <typename TA, typename TR>
__global__ void __launch_bounds__(1024) join_wide_kernel(const JoinParams p) {
  extern __shared__ float row[];
  __shared__ float red[2][32];
  const TA* pw = static_cast<const TA*>(p.post_w);
  const TA* qw = static_cast<const TA*>(p.pre_w);
  const TA* gp = static_cast<const TA*>(p.g);
  const int64_t t = blockIdx.x;
  const TA* y = static_cast<const TA*>(p.branch) + t * p.ld_y;
  const TR* r = static_cast<const TR*>(p.resid) + t * p.ld_r;
  float inv = 1.0f;
  if (pw) {
    float ss = 0.0f;
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float v = to_f32<TA>(y[c]);
      ss = fmaf(v, v, ss);
    }
    inv = 1.0f / sqrtf(row_sum<true>(ss, 0, red[0]) / (float)p.d + p.eps);
  }
  float ss = 0.0f;
  for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
    float v = to_f32<TA>(y[c]);
    if (pw) v = v * inv * to_f32<TA>(pw[c]);
    if (p.gate != MOE_GATE_NONE) {
      float g = to_f32<TA>(gp[p.gate == MOE_GATE_CHANNEL ? c
                              : p.gate == MOE_GATE_TOKEN ? t : t * p.ld_g + c]);
      if (p.sigmoid) g = 1.0f / (1.0f + expf(-g));
      v *= g;
    }
    const float s = p.a * to_f32<TR>(r[c]) + p.b * v;
    row[c] = s;
    ss = fmaf(s, s, ss);
  }
  float ninv = 0.0f;
  if (p.normed) ninv = 1.0f / sqrtf(row_sum<true>(ss, 0, red[1]) / (float)p.d + p.eps);
  for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
    const float s = row[c];
    static_cast<TR*>(p.resid_out)[t * p.ld_ro + c] = from_f32<TR>(s);
    if (p.normed)
      static_cast<TA*>(p.normed)[t * p.ld_n + c] = from_f32<TA>(s * ninv * to_f32<TA>(qw[c]));
  }
}

template <typename TA, typename TR, int V, int NC>
void start_rows(const JoinParams& p, bool block, int lanes, cudaStream_t st) {
  if (block)
    join_kernel<TA, TR, V, NC, true><<<(unsigned)p.T, lanes, 0, st>>>(p, lanes);
  else if constexpr (NC <= 4)  // eight chunks a thread only for rows of more than 4096 of them
    join_kernel<TA, TR, V, NC, false>
        <<<(unsigned)((p.T + 256 / lanes - 1) / (256 / lanes)), 256, 0, st>>>(p, lanes);
}

template <typename TA, typename TR, int V>
cudaError_t launch_rows(const JoinParams& p, int chunks, cudaStream_t st) {
  // Chunks per thread: four keep 4 x 16 bytes of each operand in flight per thread, so few threads
  // hold a row and several rows share an SM; with fewer rows than SMs that only lengthens the one
  // row's chain, and the row takes as many threads as it has chunks.
  const bool few = p.T <= num_sms();
  int nc = few ? 1 : 4;
  bool block;
  int lanes;
  if (chunks <= 32 * nc) {
    block = false;
    lanes = 1;
    while (lanes * nc < chunks) lanes *= 2;
  } else {
    block = true;
    if (chunks > 1024 * nc) nc = 4;
    if (chunks > 1024 * nc) nc = 8;  // V = 1 only
    lanes = ((chunks + nc - 1) / nc + 31) / 32 * 32;
  }
  if (nc == 1)
    start_rows<TA, TR, V, 1>(p, block, lanes, st);
  else if (V == 8 || nc == 4)
    start_rows<TA, TR, V, 4>(p, block, lanes, st);
  else
    start_rows<TA, TR, 1, 8>(p, block, lanes, st);
  return cudaGetLastError();
}

template <typename TA, typename TR>
cudaError_t launch(const JoinParams& p, bool wide_loads, cudaStream_t st) {
  LaunchScope ls("block_join", st);
  const size_t row_bytes =
      (size_t)p.d * (sizeof(TA) * (p.gate == MOE_GATE_ELEMENT ? 2 : 1) + sizeof(TR));
  if (wide_loads && p.T > num_sms() && p.d > 1024 && row_bytes <= kRowsSmem) {
    // 48 KB without the attribute: the kernel's own arrays and the launch's together
    if (row_bytes + kRowSumBytes > 48 * 1024) {
      cudaError_t e = cudaFuncSetAttribute(join_rows_kernel<TA, TR>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
      if (e != cudaSuccess) return e;
    }
    int threads = (p.d / 32 + 31) / 32 * 32;
    if (threads > 1024) threads = 1024;
    join_rows_kernel<TA, TR><<<(unsigned)p.T, threads, row_bytes, st>>>(p);
    return cudaGetLastError();
  }
  if (wide_loads) return launch_rows<TA, TR, 8>(p, p.d / 8, st);  // d <= 32768: 4096 chunks
  if (p.d <= 8192) return launch_rows<TA, TR, 1>(p, p.d, st);
  // the widest row's, whatever this one takes: a limit of the call's own would be lowered by another
  // host thread's narrower row between here and the launch
  cudaError_t e = cudaFuncSetAttribute(join_wide_kernel<TA, TR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       MOE_JOIN_MAX_D * (int)sizeof(float));
  if (e != cudaSuccess) return e;
  join_wide_kernel<TA, TR><<<(unsigned)p.T, 1024, (size_t)p.d * sizeof(float), st>>>(p);
  return cudaGetLastError();
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_block_join(const moe_join_config_t* cfg, const void* resid,
                                       const void* branch, const void* post_w, const void* gate,
                                       const void* pre_w, void* resid_out, void* normed,
                                       void* stream) {
  using namespace moe;
  if (!cfg) return MOE_ERR_INVALID_ARG;
  if (cfg->T < 0 || cfg->d < 1) return MOE_ERR_INVALID_ARG;
  if (cfg->act_dtype != MOE_F32 && cfg->act_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (cfg->resid_dtype != MOE_F32 && cfg->resid_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (cfg->gate < MOE_GATE_NONE || cfg->gate > MOE_GATE_ELEMENT) return MOE_ERR_INVALID_ARG;
  if (cfg->flags & ~MOE_JOIN_GATE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (cfg->d > MOE_JOIN_MAX_D || cfg->T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (cfg->act_dtype == MOE_F32 && cfg->resid_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  // Offsets are 64-bit: the last row's, in bytes, stays below 2^62.
  const int64_t d = cfg->d, max_ld = ((int64_t)1 << 60) / (cfg->T > 0 ? cfg->T : 1);
  for (int64_t ld : {cfg->ld_resid, cfg->ld_branch, cfg->ld_gate, cfg->ld_resid_out})
    if (ld != 0 && (ld < d || ld > max_ld)) return MOE_ERR_INVALID_ARG;
  if (cfg->ld_normed != 0 && (cfg->ld_normed < d || cfg->ld_normed > MOE_JOIN_MAX_LD_NORMED))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!resid || !branch || !resid_out) return MOE_ERR_INVALID_ARG;
  if ((cfg->gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((pre_w != nullptr) != (normed != nullptr)) return MOE_ERR_INVALID_ARG;
  const size_t ab = cfg->act_dtype == MOE_F32 ? 4 : 2, rb = cfg->resid_dtype == MOE_F32 ? 4 : 2;
  if (!aligned_to(resid, rb) || !aligned_to(resid_out, rb)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {branch, post_w, gate, pre_w, (const void*)normed})
    if (!aligned_to(q, ab)) return MOE_ERR_INVALID_ARG;

  JoinParams p;
  p.T = cfg->T;
  p.d = cfg->d;
  p.gate = cfg->gate;
  p.sigmoid = (cfg->flags & MOE_JOIN_GATE_SIGMOID) != 0;
  p.a = cfg->resid_scale;
  p.b = cfg->branch_scale;
  p.eps = cfg->rms_eps;
  auto pitch = [&](int64_t ld) { return ld ? ld : d; };
  p.ld_r = pitch(cfg->ld_resid);
  p.ld_y = pitch(cfg->ld_branch);
  p.ld_g = pitch(cfg->ld_gate);
  p.ld_ro = pitch(cfg->ld_resid_out);
  p.ld_n = pitch(cfg->ld_normed);
  p.resid = resid;
  p.branch = branch;
  p.post_w = post_w;
  p.g = gate;
  p.pre_w = pre_w;
  p.resid_out = resid_out;
  p.normed = normed;
  // 8-column chunks: whole chunks only, every row and operand on 16 bytes (ld in elements of 2 or 4)
  bool wide = d % 8 == 0;
  for (const void* q : {resid, branch, post_w, cfg->gate == MOE_GATE_TOKEN ? nullptr : gate, pre_w,
                        (const void*)resid_out, (const void*)normed})
    wide = wide && aligned_to(q, 16);
  const size_t ga = cfg->gate == MOE_GATE_ELEMENT ? (size_t)p.ld_g * ab : 0;
  wide = wide && (p.ld_r * rb) % 16 == 0 && (p.ld_ro * rb) % 16 == 0 && (p.ld_y * ab) % 16 == 0 &&
         (p.ld_n * ab) % 16 == 0 && ga % 16 == 0;
  (void)cudaGetLastError();  // start from a clean launch-error state
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cfg->act_dtype == MOE_F32)
    e = launch<float, float>(p, wide, st);
  else if (cfg->resid_dtype == MOE_F32)
    e = launch<__nv_bfloat16, float>(p, wide, st);
  else
    e = launch<__nv_bfloat16, __nv_bfloat16>(p, wide, st);
  return status_from_cuda(e);
}
