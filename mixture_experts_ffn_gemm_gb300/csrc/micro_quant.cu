// micro_quant.cu -- microscaled 4-bit floating point: rows to codes and scales, and back.
//
// A row is cut into blocks of B channels.  A block has a scale S and a 4-bit code c per channel (e2m1: a
// sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6); the value is c S.
//   MOE_MICRO_MX  B = 32, S = 2^(floor(log2 amax) - 2): the exponent's field less two, exact.
//   MOE_MICRO_NV  B = 16, S = s g, s = e4m3(amax / (6 g)) rounded to nearest, g a factor of the tensor.
// c is x / S rounded to nearest, ties to the even code, at most 6.  Both roundings are those of the
// exact quotient: MX divides by a power of two, which is exact.  NV rounds the quotient's fp32
// approximation (relative error below 2^-22: S, 1 / S and the product round by 2^-24 each) moved by
// 2^-21 either way; where both moved values give one code it is the exact quotient's too, and where
// they do not, the sign of |x| - m s g decides, m the midpoint between the two codes: m s has at most
// seven bits and is exact, and one fma keeps the sign of the difference.
//
// Bound by memory: a row is read once and its codes (K / 2 bytes) and scales (K / B) are written to
// each row that takes it, so the experts' copies of a token are quantised once and written k times.
// A warp takes a row (or a part of one, when there are few), a lane 16 channels at a time.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxCopies = 32;

struct MicroParams {
  const void* x;             // quantise: [src_rows][ld]; dequantise: out [rows][ld]
  const int32_t* dest;       // [src_rows][copies] or null
  const int32_t* offsets;    // [G + 1] or null: groups of group_rows rows
  const float* factor;       // g, or null: 1
  uint8_t* codes;
  uint8_t* scales;
  uint32_t* err;
  int64_t ld;
  int64_t src_rows, rows;
  int32_t K, G, group_rows, copies, parts, ktiles;
};

// Where a row's scales start: its group's first tile is (first row) / 128 + group, the row's place in
// a tile of 128 rows x 4 columns (r % 32) * 16 + (r / 32) * 4.  The whole warp calls this for one row;
// -1 (and kErrIndex) for a row outside the groups.  Two rounds of 32 loads find the group.
__device__ __forceinline__ int64_t scale_base(const MicroParams& p, int64_t row, int lane) {
  int64_t g, start;
  if (row < 0 || row >= p.rows) {
    if (lane == 0) raise_flag(p.err, kErrIndex);
    return -1;
  }
  if (!p.offsets) {
    g = row / p.group_rows;
    start = g * p.group_rows;
  } else {
    const int stride = (p.G + 31) / 32;
    const int i1 = lane * stride;
    const bool le = i1 < p.G && __ldg(p.offsets + i1) <= row;
    const int seg = __popc(__ballot_sync(~0u, le)) - 1;
    const int i2 = max(seg, 0) * stride + lane;
    const bool in = lane < stride && i2 < p.G;
    const int o2 = in ? __ldg(p.offsets + i2) : 0;
    const int cnt = __popc(__ballot_sync(~0u, in && o2 <= row));
    start = __shfl_sync(~0u, o2, max(cnt - 1, 0));
    g = max(seg, 0) * stride + cnt - 1;
    bool ok = seg >= 0 && cnt > 0 && start >= 0 && start <= row;
    if (ok && g == p.G - 1) ok = row < __ldg(p.offsets + p.G);
    if (!ok) {
      if (lane == 0) raise_flag(p.err, kErrIndex);
      return -1;
    }
  }
  const int64_t lr = row - start;
  return ((start >> 7) + g + (lr >> 7)) * p.ktiles * 512 + (lr & 31) * 16 + ((lr & 127) >> 5) * 4;
}

__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Two e4m3 codes of two values, rounded to nearest, at most 448 (low byte: lo).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

constexpr float kLess = 1.0f - 4.76837158203125e-7f;  // 1 - 2^-21
constexpr float kMore = 1.0f + 4.76837158203125e-7f;

// e4m3 code of amax / (6 g), rounded as the exact quotient.
__device__ __forceinline__ uint32_t nv_scale(float amax, float g) {
  const float q = amax / (6.0f * g);
  const uint32_t pair = e4m3x2(q * kLess, q * kMore);
  const uint32_t lo = pair & 0xffu, hi = pair >> 8;
  if (lo == hi) return lo;
  const float m6 = 3.0f * (e4m3_value(lo) + e4m3_value(hi));  // six times the midpoint
  const float r = fmaf(-m6, g, amax);
  return r > 0.0f || (r == 0.0f && (lo & 1u)) ? hi : lo;
}

// A magnitude's code between a and a + 1 (which both moved quotients gave), by the exact difference.
__device__ __forceinline__ uint32_t settle(uint32_t a, uint32_t b, float ax, float s, float g) {
  const float lut[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
  const float m = 0.5f * (lut[a] + lut[b]);
  const float r = fmaf(-(m * s), g, ax);
  return r > 0.0f || (r == 0.0f && (a & 1u)) ? b : a;
}

template <bool kNv, bool kF32>
__global__ void __launch_bounds__(kThreads) micro_quantize_kernel(const MicroParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / p.parts;
  if (t >= p.src_rows) return;
  const int part = (int)(w - t * p.parts);
  float g = 1.0f;
  bool bad_factor = false;
  if (kNv && p.factor) {
    g = __ldg(p.factor);
    bad_factor = !(g >= 0x1p-100f && g <= 0x1p100f);
    if (bad_factor && lane == 0) raise_flag(p.err, kErrIndex);
  }
  // lane j: the row that the j-th copy goes to, and where its scales start
  int64_t my_row = -1, my_scale = -1;
  for (int j = 0; j < p.copies; ++j) {
    const int64_t row = p.dest ? (int64_t)__ldg(p.dest + t * p.copies + j) : t;
    const int64_t sb = scale_base(p, row, lane);
    if (lane == j) {
      my_row = sb < 0 ? -1 : row;
      my_scale = sb;
    }
  }
  const int chunks = p.K / 16;
  for (int c0 = part * 32; c0 < chunks; c0 += p.parts * 32) {
    const int c = c0 + lane;
    const bool in = c < chunks;
    float v[16];
    uint32_t amax = 0;  // as an integer: NaN and infinities compare above every finite value
    if (in) {
      if (kF32) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(p.x) + t * p.ld) +
                           (int64_t)c * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 r = __ldg(src + q);
          const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[4 * q + i] = __uint_as_float(u[i]);
            amax = max(amax, u[i] & 0x7fffffffu);
          }
        }
      } else {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) +
                                                          t * p.ld) +
                           (int64_t)c * 2;
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint4 r = __ldg(src + q);
          const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[8 * q + 2 * i] = __uint_as_float(u[i] << 16);
            v[8 * q + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            m = __vmaxu2(m, u[i] & 0x7fff7fffu);
          }
        }
        amax = max(m << 16, m & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    uint32_t code0, code1, scale;
    bool nan;
    if (!kNv) {
      amax = max(amax, __shfl_xor_sync(~0u, amax, 1));
      const uint32_t e = amax >> 23;
      nan = e == 255u;
      scale = nan ? 255u : amax == 0 ? 127u : e > 2u ? e - 2u : 0u;
      const float inv = __uint_as_float((254u - min(scale, 253u)) << 23);  // 2^(127 - scale)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= inv;
      code0 = e2m1x8(v);
      code1 = e2m1x8(v + 8);
    } else {
      nan = bad_factor || (amax >> 23) == 255u;
      scale = nan ? 0x7fu : nv_scale(__uint_as_float(amax), g);
      const float s = nan ? 0.0f : e4m3_value(scale);
      const float inv = s > 0.0f ? 1.0f / (s * g) : 0.0f;
      const float il = inv * kLess, ih = inv * kMore;
      float a[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] = v[i] * il;
      code0 = e2m1x8(a);
      code1 = e2m1x8(a + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] = v[i] * ih;
      const uint32_t d0 = code0 ^ e2m1x8(a), d1 = code1 ^ e2m1x8(a + 8);
      if (d0 | d1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t& code = i < 8 ? code0 : code1;
          const uint32_t d = ((i < 8 ? d0 : d1) >> (4 * (i & 7))) & 7u;
          if (d) {
            const uint32_t lo = (code >> (4 * (i & 7))) & 7u;
            const uint32_t pick = settle(lo, lo ^ d, fabsf(v[i]), s, g);
            code ^= (pick ^ lo) << (4 * (i & 7));
          }
        }
      }
    }
    if (nan) code0 = code1 = 0;
    // four (NV) or two (MX) neighbouring scales leave in one store: 64 channels
    uint32_t packed;
    if (kNv) {
      packed = scale | __shfl_down_sync(~0u, scale, 1) << 8;
      packed |= __shfl_down_sync(~0u, packed, 2) << 16;
    } else {
      packed = scale | __shfl_down_sync(~0u, scale, 2) << 8;
    }
    const int col = kNv ? c : c >> 1;
    const int64_t scale_off = (int64_t)(col >> 2) * 512 + (col & 3);
    for (int j = 0; j < p.copies; ++j) {
      const int64_t row = __shfl_sync(~0u, my_row, j);
      const int64_t sb = __shfl_sync(~0u, my_scale, j);
      if (row < 0 || !in) continue;
      *reinterpret_cast<uint2*>(p.codes + row * (p.K / 2) + (int64_t)c * 8) =
          make_uint2(code0, code1);
      if ((lane & 3) == 0) {
        if (kNv)
          *reinterpret_cast<uint32_t*>(p.scales + sb + scale_off) = packed;
        else
          *reinterpret_cast<uint16_t*>(p.scales + sb + scale_off) = (uint16_t)packed;
      }
    }
  }
}

template <bool kNv, bool kF32>
__global__ void __launch_bounds__(kThreads) micro_dequantize_kernel(const MicroParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = w / p.parts;
  const int64_t end = p.offsets ? min(p.rows, (int64_t)max(__ldg(p.offsets + p.G), 0)) : p.rows;
  if (row >= end) return;  // rows behind the last group are left as they are
  const int part = (int)(w - row * p.parts);
  const float g = kNv && p.factor ? __ldg(p.factor) : 1.0f;
  const int64_t sb = scale_base(p, row, lane);
  if (sb < 0) return;
  const int chunks = p.K / 16;
  for (int c = part * 32 + lane; c < chunks; c += p.parts * 32) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(p.codes + row * (p.K / 2)) + c);
    const int col = kNv ? c : c >> 1;
    const uint32_t sc = __ldg(p.scales + sb + (int64_t)(col >> 2) * 512 + (col & 3));
    float s;
    if (kNv)
      s = e4m3_value(sc);
    else  // 2^(sc - 127); 2^-127 is a subnormal number, 255 stands for NaN
      s = sc == 255u ? __uint_as_float(0x7fffffffu) : sc == 0u ? 0x1p-127f : __uint_as_float(sc << 23);
    float v[16];
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t by = ((b < 4 ? q.x : q.y) >> (8 * (b & 3))) & 0xffu;
      uint32_t h;
      asm("{\n\t.reg .b8 t;\n\t.reg .b16 u;\n\tcvt.u16.u32 u, %1;\n\tcvt.u8.u16 t, u;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
          : "=r"(h)
          : "r"(by));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      // code times scale is exact (at most six bits); times g rounds once
      v[2 * b] = f.x * s;
      v[2 * b + 1] = f.y * s;
      if (kNv) {
        v[2 * b] *= g;
        v[2 * b + 1] *= g;
      }
    }
    if (kF32) {
      float* dst = static_cast<float*>(const_cast<void*>(p.x)) + row * p.ld + (int64_t)c * 16;
      store8(dst, reinterpret_cast<const float(&)[8]>(v[0]));
      store8(dst + 8, reinterpret_cast<const float(&)[8]>(v[8]));
    } else {
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(const_cast<void*>(p.x)) + row * p.ld + (int64_t)c * 16;
      store8(dst, reinterpret_cast<const float(&)[8]>(v[0]));
      store8(dst + 8, reinterpret_cast<const float(&)[8]>(v[8]));
    }
  }
}

MicroParams params(const MicroOp& m) {
  MicroParams p;
  p.x = m.x;
  p.dest = m.dest;
  p.offsets = m.offsets;
  p.factor = m.factor;
  p.codes = m.codes;
  p.scales = m.scales;
  p.err = m.err;
  p.ld = m.ld;
  p.src_rows = m.src_rows;
  p.rows = m.rows;
  p.K = m.K;
  p.G = m.groups;
  p.group_rows = (int32_t)(m.rows / m.groups);
  p.copies = m.copies;
  p.ktiles = m.ktiles;
  return p;
}

// Warps for a row: one, or as many as fill the GPU when there are few rows.
int row_parts(int64_t rows, int K, int sms) {
  const int64_t most = (K / 16 + 31) / 32;
  int64_t n = (int64_t)sms * 16 / (rows > 0 ? rows : 1);
  return (int)(n < 1 ? 1 : n > most ? most : n);
}

}  // namespace

cudaError_t launch_micro_quantize(const MicroOp& m, int sms, cudaStream_t st) {
  MicroParams p = params(m);
  p.parts = row_parts(m.src_rows, m.K, sms);
  const unsigned grid = (unsigned)((m.src_rows * p.parts + kThreads / 32 - 1) / (kThreads / 32));
  LaunchScope ls("micro_quantize", st);
  const bool f32 = m.dtype == MOE_F32;
  if (m.format == MOE_MICRO_NV) {
    if (f32)
      micro_quantize_kernel<true, true><<<grid, kThreads, 0, st>>>(p);
    else
      micro_quantize_kernel<true, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (f32)
      micro_quantize_kernel<false, true><<<grid, kThreads, 0, st>>>(p);
    else
      micro_quantize_kernel<false, false><<<grid, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_micro_dequantize(const MicroOp& m, int sms, cudaStream_t st) {
  MicroParams p = params(m);
  p.parts = row_parts(m.rows, m.K, sms);
  const unsigned grid = (unsigned)((m.rows * p.parts + kThreads / 32 - 1) / (kThreads / 32));
  LaunchScope ls("micro_dequantize", st);
  const bool f32 = m.dtype == MOE_F32;
  if (m.format == MOE_MICRO_NV) {
    if (f32)
      micro_dequantize_kernel<true, true><<<grid, kThreads, 0, st>>>(p);
    else
      micro_dequantize_kernel<true, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (f32)
      micro_dequantize_kernel<false, true><<<grid, kThreads, 0, st>>>(p);
    else
      micro_dequantize_kernel<false, false><<<grid, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace moe
