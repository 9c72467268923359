// product_api.cu -- the C ABI of the products grouped by expert and of the microscaled 4-bit operators:
// host validation, tensor maps, launches.  No allocation and no host synchronisation.
#include <cstdint>
#include <mutex>

#include "internal.h"

namespace moe {

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(ptr);
  });
  return fn;
}

bool make_map(CUtensorMap* m, int el, const void* base, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint32_t ones[3] = {1, 1, 1};
  return enc(m,
             el == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
             : el == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                       : CU_TENSOR_MAP_DATA_TYPE_UINT8,
             (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             box[0] * el == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 26;
constexpr int32_t kMaxWidth = 131072;
constexpr int32_t kMaxGroups = 1023;
constexpr int64_t kMaxPitch = (int64_t)1 << 32;  // a buffer's bytes stay within 2^60
constexpr size_t kStatusBytes = 256;

moe_status_t check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
  return aligned(ws) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// 0: the width itself; -1: not a pitch.
int64_t pitch(int64_t ld, int64_t width) {
  if (ld == 0) return width;
  return ld < width || ld % 8 || ld > kMaxPitch ? -1 : ld;
}

moe_status_t validate(const moe_product_config_t* c) {
  if (!c || c->rows < 0 || c->E < 1 || c->N < 1 || c->K < 1) return MOE_ERR_INVALID_ARG;
  if (c->kind < MOE_PRODUCT_FORWARD || c->kind > MOE_PRODUCT_GRAD_W) return MOE_ERR_INVALID_ARG;
  if (c->out_dtype != MOE_BF16 && c->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->flags & ~(MOE_PRODUCT_ACCUMULATE | MOE_PRODUCT_TEST_STALL | MOE_PRODUCT_TEST_SHORT_WAITS))
    return MOE_ERR_INVALID_ARG;
  if ((c->flags & MOE_PRODUCT_ACCUMULATE) &&
      (c->kind != MOE_PRODUCT_GRAD_W || c->out_dtype != MOE_F32))
    return MOE_ERR_UNSUPPORTED;
  if (c->rows > kMaxRows || c->E > kMaxGroups || c->N > kMaxWidth || c->K > kMaxWidth || c->N % 8 ||
      c->K % 8)
    return MOE_ERR_UNSUPPORTED;
  if (pitch(c->ld_x, c->K) < 0 || pitch(c->ld_y, c->N) < 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int scale_columns(int format) { return format == MOE_MICRO_NV ? 64 : 128; }  // channels of a tile

moe_status_t validate(const moe_micro_config_t* c) {
  if (!c || c->rows < 0 || c->src_rows < 0 || c->K < 1 || c->groups < 1 || c->copies < 1 || c->flags)
    return MOE_ERR_INVALID_ARG;
  if (c->format != MOE_MICRO_MX && c->format != MOE_MICRO_NV) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16 && c->dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->rows > kMaxRows || c->src_rows > kMaxRows || c->K > kMaxWidth || c->K % 64 ||
      c->groups > kMaxGroups || c->copies > MOE_MICRO_MAX_COPIES)
    return MOE_ERR_UNSUPPORTED;
  if (pitch(c->ld, c->K) < 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status_t validate(const moe_micro_product_config_t* c) {
  if (!c || c->rows < 0 || c->E < 1 || c->N < 1 || c->K < 1 || (c->flags & ~MOE_MICRO_SWIGLU))
    return MOE_ERR_INVALID_ARG;
  if (c->format != MOE_MICRO_MX && c->format != MOE_MICRO_NV) return MOE_ERR_INVALID_ARG;
  if (c->out_dtype != MOE_BF16 && c->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->rows > kMaxRows || c->E > kMaxGroups || c->N > kMaxWidth || c->K > kMaxWidth || c->N % 8 ||
      c->K % 64 || ((c->flags & MOE_MICRO_SWIGLU) && c->N % 128))
    return MOE_ERR_UNSUPPORTED;
  // scale tiles are counted in 31 bits, with room for a row of tiles behind the last
  const int64_t kt = (c->K + 63) / 64, per = (int64_t)c->N * (c->flags & MOE_MICRO_SWIGLU ? 2 : 1);
  constexpr int64_t kMost = (int64_t)1 << 30;
  if ((c->E * per / 128 + c->E) * kt > kMost || (c->rows / 128 + c->E) * kt > kMost)
    return MOE_ERR_UNSUPPORTED;
  if (pitch(c->ld_out, c->N) < 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

MicroOp micro_op(const moe_micro_config_t* c, const int32_t* offsets, const float* factor, void* ws) {
  MicroOp m;
  m.offsets = offsets;
  m.factor = c->format == MOE_MICRO_NV ? factor : nullptr;
  m.err = static_cast<uint32_t*>(ws);
  m.ld = pitch(c->ld, c->K);
  m.rows = c->rows;
  m.K = c->K;
  m.groups = c->groups;
  m.ktiles = (c->K + scale_columns(c->format) - 1) / scale_columns(c->format);
  m.format = c->format;
  m.dtype = c->dtype;
  return m;
}

}  // namespace

bool make_map_2d(CUtensorMap* m, int el, const void* base, uint64_t cols, uint64_t rows, uint64_t ld,
                 uint32_t box_cols, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * el};
  const cuuint32_t box[2] = {box_cols, box_rows};
  return make_map(m, el, base, 2, dims, strides, box);
}

bool make_map_3d(CUtensorMap* m, int el, const void* base, uint64_t cols, uint64_t rows,
                 uint64_t depth, uint32_t box_cols, uint32_t box_rows) {
  const cuuint64_t dims[3] = {cols, rows, depth}, strides[2] = {cols * el, cols * rows * el};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  return make_map(m, el, base, 3, dims, strides, box);
}

bool make_map_tiles(CUtensorMap* m, const void* base, uint64_t tiles, uint32_t box_tiles) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {128, tiles}, strides[1] = {512};
  const cuuint32_t box[2] = {128, box_tiles}, ones[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t set_smem_once(const void* kern, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_product_workspace_size(const moe_product_config_t* cfg) {
  return validate(cfg) == MOE_OK ? kStatusBytes : 0;
}

moe_status_t moe_grouped_product(const moe_product_config_t* cfg, const int32_t* offsets,
                                 const void* a, const void* b, void* out, void* ws,
                                 size_t ws_bytes, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_ws(ws, ws_bytes, moe_product_workspace_size(cfg))) != MOE_OK) return s;
  const bool grad_w = cfg->kind == MOE_PRODUCT_GRAD_W;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cfg->rows == 0) {
    if (!grad_w || (cfg->flags & MOE_PRODUCT_ACCUMULATE)) return MOE_OK;
    if (!aligned(out)) return MOE_ERR_INVALID_ARG;
    return status_from_cuda(cudaMemsetAsync(
        out, 0, (size_t)cfg->E * cfg->N * cfg->K * (cfg->out_dtype == MOE_F32 ? 4 : 2), st));
  }
  if (!offsets || !aligned(a) || !aligned(b) || !aligned(out)) return MOE_ERR_INVALID_ARG;
  GroupedProduct g;
  const int64_t ldx = pitch(cfg->ld_x, cfg->K), ldy = pitch(cfg->ld_y, cfg->N);
  g.kind = cfg->kind;
  g.offsets = offsets;
  g.E = cfg->E;
  g.N = cfg->N;
  g.K = cfg->K;
  g.rows = cfg->rows;
  g.a = a;
  g.ld_a = cfg->kind == MOE_PRODUCT_FORWARD ? ldx : ldy;
  g.b = b;
  g.ld_b = grad_w ? ldx : 0;
  g.out = out;
  g.ldo = cfg->kind == MOE_PRODUCT_FORWARD ? ldy : cfg->kind == MOE_PRODUCT_GRAD_X ? ldx : cfg->K;
  g.out_dtype = cfg->out_dtype;
  g.accumulate = (cfg->flags & MOE_PRODUCT_ACCUMULATE) != 0;
  g.test_stall = (cfg->flags & MOE_PRODUCT_TEST_STALL) != 0;
  g.test_short_waits = (cfg->flags & MOE_PRODUCT_TEST_SHORT_WAITS) != 0;
  g.err = static_cast<uint32_t*>(ws);
  const int sms = num_sms();
  (void)cudaGetLastError();
  return status_from_cuda(launch_grouped_product(g, sms, st));
}

size_t moe_micro_scales_size(const moe_micro_config_t* cfg) {
  if (validate(cfg) != MOE_OK) return 0;
  const int per = scale_columns(cfg->format);
  return (size_t)(cfg->rows / 128 + cfg->groups) * ((cfg->K + per - 1) / per) * 512;
}

moe_status_t moe_micro_quantize(const moe_micro_config_t* cfg, const void* x, const int32_t* dest,
                                const int32_t* offsets, const float* factor, void* codes,
                                void* scales, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_ws(ws, ws_bytes, kStatusBytes)) != MOE_OK) return s;
  if (!offsets && cfg->rows % cfg->groups) return MOE_ERR_INVALID_ARG;
  if (!dest && (cfg->copies != 1 || cfg->src_rows != cfg->rows)) return MOE_ERR_INVALID_ARG;
  if (cfg->src_rows == 0 || cfg->rows == 0) return MOE_OK;
  if (!aligned(x) || !aligned(codes) || !aligned(scales)) return MOE_ERR_INVALID_ARG;
  MicroOp m = micro_op(cfg, offsets, factor, ws);
  m.x = x;
  m.dest = dest;
  m.codes = static_cast<uint8_t*>(codes);
  m.scales = static_cast<uint8_t*>(scales);
  m.src_rows = cfg->src_rows;
  m.copies = cfg->copies;
  const int sms = num_sms();
  (void)cudaGetLastError();
  return status_from_cuda(launch_micro_quantize(m, sms, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_micro_dequantize(const moe_micro_config_t* cfg, const void* codes,
                                  const void* scales, const int32_t* offsets, const float* factor,
                                  void* out, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_ws(ws, ws_bytes, kStatusBytes)) != MOE_OK) return s;
  if (!offsets && cfg->rows % cfg->groups) return MOE_ERR_INVALID_ARG;
  if (cfg->rows == 0) return MOE_OK;
  if (!aligned(codes) || !aligned(scales) || !aligned(out)) return MOE_ERR_INVALID_ARG;
  MicroOp m = micro_op(cfg, offsets, factor, ws);
  m.x = out;
  m.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  m.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  const int sms = num_sms();
  (void)cudaGetLastError();
  return status_from_cuda(launch_micro_dequantize(m, sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_micro_product_workspace_size(const moe_micro_product_config_t* cfg) {
  return validate(cfg) == MOE_OK ? kStatusBytes : 0;
}

moe_status_t moe_micro_product(const moe_micro_product_config_t* cfg, const int32_t* offsets,
                               const void* a, const void* a_scales, const float* a_factor,
                               const void* w, const void* w_scales, const float* w_factor,
                               void* out, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_ws(ws, ws_bytes, moe_micro_product_workspace_size(cfg))) != MOE_OK) return s;
  if (cfg->rows == 0) return MOE_OK;
  if (!offsets || !aligned(a) || !aligned(a_scales) || !aligned(w) || !aligned(w_scales) ||
      !aligned(out))
    return MOE_ERR_INVALID_ARG;
  MicroProduct g;
  g.offsets = offsets;
  g.E = cfg->E;
  g.N = cfg->N;
  g.K = cfg->K;
  g.format = cfg->format;
  g.rows = cfg->rows;
  g.swiglu = (cfg->flags & MOE_MICRO_SWIGLU) != 0;
  g.a = static_cast<const uint8_t*>(a);
  g.a_scales = static_cast<const uint8_t*>(a_scales);
  g.a_factor = a_factor;
  g.w = static_cast<const uint8_t*>(w);
  g.w_scales = static_cast<const uint8_t*>(w_scales);
  g.w_factor = w_factor;
  g.out = out;
  g.ldo = pitch(cfg->ld_out, cfg->N);
  g.out_dtype = cfg->out_dtype;
  g.err = static_cast<uint32_t*>(ws);
  const int sms = num_sms();
  (void)cudaGetLastError();
  return status_from_cuda(launch_micro_product(g, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
