// join.cu -- what stands between two blocks: post-norm of the branch, gate, scales, residual sum and
// the next block's norm, one pass over the rows (moe_block_join).
//
//   v = y w_post / sqrt(mean(y^2) + eps) ;  r' = a r + b g v ;  n = r' w_pre / sqrt(mean(r'^2) + eps)
//
// One CTA per row (grid-stride); the row's r' stays in shared memory between the two norms.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

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

// Sum over the CTA, the same value on every thread; red holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();  // red of the previous sum has been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += red[i];
  return s;
}

template <typename TA, typename TR>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  extern __shared__ float row[];
  __shared__ float red[32];
  const TA* pw = static_cast<const TA*>(p.post_w);
  const TA* qw = static_cast<const TA*>(p.pre_w);
  const TA* gp = static_cast<const TA*>(p.g);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const TA* y = static_cast<const TA*>(p.branch) + t * p.ld_y;
    const TR* r = static_cast<const TR*>(p.resid) + t * p.ld_r;
    float inv = 1.0f;
    if (pw) {
      float ss = 0.0f;
      for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
        const float v = to_f32<TA>(y[c]);
        ss = fmaf(v, v, ss);
      }
      inv = 1.0f / sqrtf(block_sum(ss, red) / (float)p.d + p.eps);
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
    if (p.normed) ninv = 1.0f / sqrtf(block_sum(ss, red) / (float)p.d + p.eps);
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) {  // each thread reads back its own columns
      const float s = row[c];
      static_cast<TR*>(p.resid_out)[t * p.ld_ro + c] = from_f32<TR>(s);
      if (p.normed)
        static_cast<TA*>(p.normed)[t * p.ld_n + c] = from_f32<TA>(s * ninv * to_f32<TA>(qw[c]));
    }
  }
}

template <typename TA, typename TR>
cudaError_t launch(const JoinParams& p, cudaStream_t st) {
  const size_t smem = (size_t)p.d * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(join_kernel<TA, TR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t cap = (int64_t)num_sms() * 8;
  LaunchScope ls("block_join", st);
  join_kernel<TA, TR><<<(unsigned)(p.T < cap ? p.T : cap), 256, smem, st>>>(p);
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
  if (cfg->d > MOE_JOIN_MAX_D || cfg->T > ((int64_t)1 << 40)) return MOE_ERR_UNSUPPORTED;
  if (cfg->act_dtype == MOE_F32 && cfg->resid_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  const int64_t d = cfg->d, max_ld = (int64_t)1 << 20;
  const int64_t lds[] = {cfg->ld_resid, cfg->ld_branch, cfg->ld_gate, cfg->ld_resid_out,
                         cfg->ld_normed};
  for (int64_t ld : lds)
    if (ld != 0 && (ld < d || ld > max_ld)) return MOE_ERR_INVALID_ARG;
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
  (void)cudaGetLastError();  // start from a clean launch-error state
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cfg->act_dtype == MOE_F32)
    e = launch<float, float>(p, st);
  else if (cfg->resid_dtype == MOE_F32)
    e = launch<__nv_bfloat16, float>(p, st);
  else
    e = launch<__nv_bfloat16, __nv_bfloat16>(p, st);
  return status_from_cuda(e);
}
