// micro_quant.cu -- microscaled 4-bit floating point: rows to codes and scales, and back.
//
// A row is cut into blocks of B channels.  A block has a scale S and a 4-bit code c per channel (e2m1: a
// sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6); the value is c S.
//   MOE_MICRO_MX  B = 32, S = 2^(floor(log2 amax) - 2): the exponent's field less two, exact.
//   MOE_MICRO_NV  B = 16, S = s g, s = e4m3(amax / (6 g)) rounded to nearest, g a factor of the tensor.
// c is x / S rounded to nearest, ties to the even code, at most 6.  Both roundings are those of the
// exact quotient: MX divides by a power of two, which is exact.  NV rounds the quotient's fp32
// approximation (1 / g rounds by 2^-24, the approximate division by s by at most two steps of 2^-23, the
// products by 2^-24 each: below 2^-21 together) moved by 2^-20 either way; where both moved values give one
// code it is the exact quotient's too, and where they do not, the sign of |x| - m s g decides, m the midpoint
// between the two codes: m s has at most seven bits and is exact, and one fma keeps the sign of the
// difference.
//
// Bound by memory: a row is read once and its codes (K / 2 bytes) and scales (K / B) are written to
// each row that takes it, so the experts' copies of a token are quantised once and written k times.
// A warp takes a row (or a part of one, when there are few), a lane 32 channels at a time (16 going back).
//
// Measured (GB300, rows of 7168 bf16): 4096 rows to 8 rows each nv 54 us (of 28 for the bytes), mx 42; 32768 rows to
// one each 135 and 105 us (of 89, 88); back 99 us (of 89).  Copies are bound by their scales, four bytes in each
// 512-byte tile: without those stores 8192 rows nv take 73 us instead of 112.  One row: 3.5 us.
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "launch_order.cuh"

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
  int32_t wide;              // x or the values: rows at multiples of 32 bytes, which one access takes
};

// Operands are what a kernel before this one may have written: read by volatile loads, which stay behind the
// wait for it (__ldg may be moved in front: its data is constant).  Ordinary loads would stay too, but later than
// need be among the shuffles and stores (one row 3.3 -> 3.7 us; back, 32768 rows nv, 99 -> 103).
__device__ __forceinline__ int32_t ld_int(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_float(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_16(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Where the scales of `n` rows (lane j's `row`, j < n <= kMaxCopies) start, in lane j: a group's first
// tile is (first row) / 128 + group, a row's place in a tile of 128 rows x 4 columns (r % 32) * 16 + (r / 32) * 4.
// -1 for a row outside the groups, with kErrIndex but for rows of the buffer behind the last one where those are
// `allowed` (rows without destinations in a buffer with room; asked here, where the bound is read anyway: in front of
// the row's loads 8 to 1024 rows took 0.1-0.2 us longer).  The whole warp finds each row's group in two rounds of
// 32 loads, the second round's in flight for kBatch rows at once.
constexpr int kBatch = 8;
__device__ __forceinline__ int64_t scale_base(const MicroParams& p, int row, int n, int lane,
                                              bool allowed) {
  int g, start;
  bool ok = row >= 0 && row < p.rows, behind = false;
  if (!p.offsets) {
    g = ok ? row / p.group_rows : 0;
    start = g * p.group_rows;
  } else {
    const int stride = (p.G + 31) / 32;
    const int i1 = lane * stride;
    const int first = i1 < p.G ? ld_int(p.offsets + i1) : INT32_MAX;
    const int last = ld_int(p.offsets + p.G);
    g = -1;
    start = 0;
    for (int j0 = 0; j0 < n; j0 += kBatch) {
      int o2[kBatch], i2[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = __shfl_sync(~0u, row, j0 + b);
        i2[b] = max(__popc(__ballot_sync(~0u, i1 < p.G && first <= r)) - 1, 0) * stride;
        o2[b] = lane < stride && i2[b] + lane < p.G ? ld_int(p.offsets + i2[b] + lane) : INT32_MAX;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = __shfl_sync(~0u, row, j0 + b);
        const int cnt = __popc(__ballot_sync(~0u, o2[b] <= r && o2[b] != INT32_MAX));
        const int o = __shfl_sync(~0u, o2[b], max(cnt - 1, 0));
        if (lane == j0 + b) {
          g = cnt > 0 ? i2[b] + cnt - 1 : -1;
          start = o;
        }
      }
    }
    behind = ok && row >= last;
    ok = ok && g >= 0 && start >= 0 && start <= row && row < last;
  }
  if (lane >= n) return -1;
  if (!ok) {
    if (!(behind && allowed)) raise_flag(p.err, kErrIndex);
    return -1;
  }
  const int lr = row - start;
  return (int64_t)((start >> 7) + g + (lr >> 7)) * p.ktiles * 512 + (lr & 31) * 16 + ((lr & 127) >> 5) * 4;
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

constexpr float kLess = 1.0f - 0x1p-20f;
constexpr float kMore = 1.0f + 0x1p-20f;

// e4m3 code of amax / (6 g), rounded as the exact quotient; per6g = RN(1 / RN(6 g)).
__device__ __forceinline__ uint32_t nv_scale(float amax, float g, float per6g) {
  const float q = amax * per6g;
  const uint32_t pair = e4m3x2(q * kLess, q * kMore);
  const uint32_t lo = pair & 0xffu, hi = pair >> 8;
  if (lo == hi) return lo;
  const float m6 = 3.0f * (e4m3_value(lo) + e4m3_value(hi));  // six times the midpoint
  const float r = fmaf(-m6, g, amax);
  return r > 0.0f || (r == 0.0f && (lo & 1u)) ? hi : lo;
}

// The magnitude of a code: 0, 0.5, then two to a power of two.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  return code < 2u ? 0.5f * (float)code : __uint_as_float(((code >> 1) + 126u) << 23 | (code & 1u) << 22);
}

// A magnitude's code between a and a + 1 (which both moved quotients gave), by the exact difference.
__device__ __forceinline__ uint32_t settle(uint32_t a, uint32_t b, float ax, float s, float g) {
  const float m = 0.5f * (e2m1_value(a) + e2m1_value(b));
  const float r = fmaf(-(m * s), g, ax);
  return r > 0.0f || (r == 0.0f && (a & 1u)) ? b : a;
}

__device__ __forceinline__ void load32(const uint4* p, bool wide, uint4& a, uint4& b) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = ld_16(p);
    b = ld_16(p + 1);
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// 16 channels: their magnitude's largest as an integer (NaN and infinities compare above every finite
// value) and the values.
template <bool kF32>
__device__ __forceinline__ uint32_t unpack16(const uint4* raw, float (&v)[16]) {
  uint32_t top = 0;
  if constexpr (kF32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t u[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[4 * q + i] = __uint_as_float(u[i]);
        top = max(top, u[i] & 0x7fffffffu);
      }
    }
    return top;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t u[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * q + 2 * i] = __uint_as_float(u[i] << 16);
      v[8 * q + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      top = __vmaxu2(top, u[i] & 0x7fff7fffu);
    }
  }
  return max(top << 16, top & 0xffff0000u);
}

__device__ __forceinline__ uint2 codes_mx(float (&v)[16], float inv) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= inv;
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

// Codes of a block of 16 with the scale s g (all zero for s = 0): by both moved quotients, and by the exact
// difference where they disagree.
__device__ __forceinline__ uint2 codes_nv(const float (&v)[16], float s, float g, float per_g) {
  const float inv = s > 0.0f ? __fdividef(per_g, s) : 0.0f;
  const float il = inv * kLess, ih = inv * kMore;
  float a[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = v[i] * il;
  uint32_t c[2] = {e2m1x8(a), e2m1x8(a + 8)};
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = v[i] * ih;
  const uint32_t d[2] = {c[0] ^ e2m1x8(a), c[1] ^ e2m1x8(a + 8)};
  if (d[0] | d[1]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = (d[i >> 3] >> (4 * (i & 7))) & 7u;
      if (x) {
        const uint32_t lo = (c[i >> 3] >> (4 * (i & 7))) & 7u;
        c[i >> 3] ^= (settle(lo, lo ^ x, fabsf(v[i]), s, g) ^ lo) << (4 * (i & 7));
      }
    }
  }
  return make_uint2(c[0], c[1]);
}

struct CopyTo {  // where a copy of the row starts
  uint8_t* codes;
  uint8_t* scales;
};

template <bool kNv, bool kF32>
__global__ void __launch_bounds__(kThreads, kF32 ? 2 : 3) micro_quantize_kernel(const MicroParams p) {
  __shared__ CopyTo to_all[kThreads / 32][kMaxCopies];
  allow_next_kernel();
  wait_for_prior_kernel();
  const int lane = threadIdx.x & 31;
  CopyTo* to = to_all[threadIdx.x >> 5];
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / p.parts;
  if (t >= p.src_rows) return;
  const int part = (int)(w - t * p.parts);
  // a lane has 32 channels: one block of MX, two of NV
  constexpr int kRaw = kF32 ? 8 : 4;
  const int chunks = p.K / 32;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) +
                                                    t * p.ld * (kF32 ? 4 : 2));
  uint4 raw[kRaw];
  int c = part * 32 + lane;
  if (c < chunks) {  // the first loads are under way while the rows' groups are found
#pragma unroll
    for (int q = 0; q < kRaw; q += 2) load32(src + (int64_t)c * kRaw + q, p.wide, raw[q], raw[q + 1]);
  }
  float g = 1.0f;
  bool bad_factor = false;
  if (kNv && p.factor) {
    g = ld_float(p.factor);
    bad_factor = !(g >= 0x1p-100f && g <= 0x1p100f);
    if (bad_factor && lane == 0) raise_flag(p.err, kErrIndex);
  }
  const float per_g = 1.0f / g, per6g = 1.0f / (6.0f * g);
  int copies;
  {
    int row = -1;
    if (lane < p.copies) row = p.dest ? ld_int(p.dest + t * p.copies + lane) : (int)t;
    const int64_t sb = scale_base(p, row, p.copies, lane, !p.dest);
    const uint32_t good = __ballot_sync(~0u, sb >= 0);  // the others are skipped
    if (sb >= 0)
      to[__popc(good & ((1u << lane) - 1u))] = {p.codes + (int64_t)row * (p.K / 2), p.scales + sb};
    copies = __popc(good);
    __syncwarp();
    if (copies == 0) return;
  }
  for (int c0 = part * 32; c0 < chunks; c0 += p.parts * 32) {
    const bool in = c < chunks;
    uint32_t code[4], scale;
    if (!in) {
#pragma unroll
      for (int q = 0; q < kRaw; ++q) raw[q] = make_uint4(0, 0, 0, 0);
    }
    uint4 now[kRaw];
#pragma unroll
    for (int q = 0; q < kRaw; ++q) now[q] = raw[q];
    c += p.parts * 32;
    if (c < chunks) {
#pragma unroll
      for (int q = 0; q < kRaw; q += 2) load32(src + (int64_t)c * kRaw + q, p.wide, raw[q], raw[q + 1]);
    }
    if constexpr (!kNv) {
      float v0[16], v1[16];
      const uint32_t t0 = unpack16<kF32>(now, v0), t1 = unpack16<kF32>(now + kRaw / 2, v1);
      const uint32_t top = max(t0, t1), e = top >> 23;
      const bool nan = e == 255u;
      scale = nan ? 255u : top == 0 ? 127u : e > 2u ? e - 2u : 0u;
      const float inv = __uint_as_float((254u - min(scale, 253u)) << 23);  // 2^(127 - scale)
      const uint2 a = codes_mx(v0, inv), b = codes_mx(v1, inv);
      code[0] = nan ? 0u : a.x;
      code[1] = nan ? 0u : a.y;
      code[2] = nan ? 0u : b.x;
      code[3] = nan ? 0u : b.y;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[16];
        const uint32_t top = unpack16<kF32>(now + h * (kRaw / 2), v);
        const bool nan = bad_factor || (top >> 23) == 255u;
        const uint32_t sc = nan ? 0x7fu : nv_scale(__uint_as_float(top), g, per6g);
        const uint2 a = codes_nv(v, nan ? 0.0f : e4m3_value(sc), g, per_g);
        code[2 * h] = nan ? 0u : a.x;
        code[2 * h + 1] = nan ? 0u : a.y;
        scale = h ? scale | sc << 8 : sc;
      }
    }
    // a tile's four columns leave in one store: two lanes' scales (NV), or four lanes' (MX; of the last tile
    // two may lie behind K)
    uint32_t packed = scale | __shfl_down_sync(~0u, scale, 1) << (kNv ? 16 : 8);
    if (!kNv) packed |= __shfl_down_sync(~0u, packed, 2) << 16;
    const int at = c - p.parts * 32;           // this chunk
    const int64_t code_off = (int64_t)at * 16, scale_off = (int64_t)(at >> (kNv ? 1 : 2)) * 512;
    if (in) {
      for (int j = 0; j < copies; ++j) {
        const CopyTo d = to[j];
        *reinterpret_cast<uint4*>(d.codes + code_off) = make_uint4(code[0], code[1], code[2], code[3]);
        if ((lane & (kNv ? 1 : 3)) == 0) *reinterpret_cast<uint32_t*>(d.scales + scale_off) = packed;
      }
    }
  }
}

template <bool kNv, bool kF32>
__global__ void __launch_bounds__(kThreads) micro_dequantize_kernel(const MicroParams p) {
  wait_for_prior_kernel();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = w / p.parts;
  const int64_t end = p.offsets ? min(p.rows, (int64_t)max(ld_int(p.offsets + p.G), 0)) : p.rows;
  if (row >= end) return;  // rows behind the last group are left as they are
  const int part = (int)(w - row * p.parts);
  const float g = kNv && p.factor ? ld_float(p.factor) : 1.0f;
  const int64_t sb = __shfl_sync(~0u, scale_base(p, (int)row, 1, lane, false), 0);
  if (sb < 0) return;
  const int chunks = p.K / 16;
  const auto fetch = [&](int c, uint2& q, uint32_t& sc) {
    const int col = kNv ? c : c >> 1;
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];"
                 : "=r"(q.x), "=r"(q.y)
                 : "l"(p.codes + row * (p.K / 2) + (int64_t)c * 8));
    asm volatile("ld.global.u8 %0, [%1];"
                 : "=r"(sc)
                 : "l"(p.scales + sb + (int64_t)(col >> 2) * 512 + (col & 3)));
  };
  uint2 next;
  uint32_t next_sc;
  int c = part * 32 + lane;
  if (c < chunks) fetch(c, next, next_sc);
  while (c < chunks) {
    const uint2 q = next;
    const uint32_t sc = next_sc;
    const int here = c;
    c += p.parts * 32;
    if (c < chunks) fetch(c, next, next_sc);
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
    uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(p.x)) +
                   (row * p.ld + (int64_t)here * 16) * (kF32 ? 4 : 2);
    uint32_t u[kF32 ? 16 : 8];
    if constexpr (kF32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i]);
      store32(dst + 32, p.wide, reinterpret_cast<const uint32_t(&)[8]>(u[8]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    store32(dst, p.wide, reinterpret_cast<const uint32_t(&)[8]>(u[0]));
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
  p.wide = ((reinterpret_cast<uintptr_t>(m.x) | (uint64_t)m.ld * (m.dtype == MOE_F32 ? 4 : 2)) & 31) == 0;
  return p;
}

// Warps for a row: as many as give the GPU 64 warps an SM (a few waves of them, whose ends then overlap),
// at most one for each 32 lanes' channels.
int row_parts(int64_t rows, int K, int lane_channels, int sms) {
  const int64_t most = (K / lane_channels + 31) / 32;
  int64_t n = (int64_t)sms * 64 / (rows > 0 ? rows : 1);
  return (int)(n < 1 ? 1 : n > most ? most : n);
}

}  // namespace

// Both kernels start as the one before them ends (programmatic launch) and wait for it by themselves.
template <typename Kernel>
static cudaError_t launch_rows(Kernel kern, unsigned grid, cudaStream_t st, const MicroParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_micro_quantize(const MicroOp& m, int sms, cudaStream_t st) {
  MicroParams p = params(m);
  p.parts = row_parts(m.src_rows, m.K, 32, sms);
  const unsigned grid = (unsigned)((m.src_rows * p.parts + kThreads / 32 - 1) / (kThreads / 32));
  LaunchScope ls("micro_quantize", st);
  const bool f32 = m.dtype == MOE_F32;
  if (m.format == MOE_MICRO_NV)
    return f32 ? launch_rows(micro_quantize_kernel<true, true>, grid, st, p)
               : launch_rows(micro_quantize_kernel<true, false>, grid, st, p);
  return f32 ? launch_rows(micro_quantize_kernel<false, true>, grid, st, p)
             : launch_rows(micro_quantize_kernel<false, false>, grid, st, p);
}

cudaError_t launch_micro_dequantize(const MicroOp& m, int sms, cudaStream_t st) {
  MicroParams p = params(m);
  p.parts = row_parts(m.rows, m.K, 16, sms);
  const unsigned grid = (unsigned)((m.rows * p.parts + kThreads / 32 - 1) / (kThreads / 32));
  LaunchScope ls("micro_dequantize", st);
  const bool f32 = m.dtype == MOE_F32;
  if (m.format == MOE_MICRO_NV)
    return f32 ? launch_rows(micro_dequantize_kernel<true, true>, grid, st, p)
               : launch_rows(micro_dequantize_kernel<true, false>, grid, st, p);
  return f32 ? launch_rows(micro_dequantize_kernel<false, true>, grid, st, p)
             : launch_rows(micro_dequantize_kernel<false, false>, grid, st, p);
}

}  // namespace moe
