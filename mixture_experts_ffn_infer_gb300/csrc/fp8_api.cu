// C ABI of the FP8 operators (moe_fp8.h): argument checks and launches.
#include <cuda_runtime.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kMaxExpertsFp8 = 1024, kMaxCols = 65536;
constexpr int kMaxRowCols = 16384;  // moe_fp8_quantise: a row in one CTA's registers
constexpr int kMaxPositions = 1024;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 4096;
constexpr int64_t kMaxUnits = (int64_t(1) << 31) - 4096;  // a CTA counts one round past them in 32 bits

bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool weights_dims_ok(const moe_fp8_weights* w) {
  return w->num_experts >= 1 && w->num_experts <= kMaxExpertsFp8 && w->n_out >= 1 && w->n_out <= kMaxCols &&
         w->k >= 16 && w->k <= kMaxCols && w->k % 16 == 0;
}

bool overlaps(const void* p, size_t pn, const void* q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + qn && b < a + pn;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_fp8_scale_pitch(int64_t cols) {
  if (cols <= 0 || cols % 16 != 0) return 0;
  return (fp8_blocks(cols) + 3) / 4 * 4;
}

moe_status moe_fp8_quantise(int64_t n, int32_t k, int32_t d, const void* x, int64_t x_ld, const int32_t* positions,
                            int64_t out_rows, void* codes, float* scales, cudaStream_t s) {
  if (n < 0 || k < 1 || out_rows < 0) return MOE_ERR_INVALID_ARG;
  if (d < 16 || d > kMaxRowCols || d % 16 != 0 || k > kMaxPositions || n > kMaxRows / k || out_rows > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!x || !codes || !scales || !is_aligned(x, 16) || !is_aligned(codes, 16) || !is_aligned(scales, 16) || x_ld < d ||
      x_ld % 8 != 0 || (!positions && k != 1) || !is_aligned(positions, 4))
    return MOE_ERR_INVALID_ARG;
  const Fp8RowsLaunch a{n, k, d, static_cast<const uint16_t*>(x), x_ld, positions, out_rows,
                        static_cast<uint8_t*>(codes), scales};
  return launch_fp8_rows(a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp8_dequantise(int64_t rows, int32_t d, const void* codes, const float* scales, void* out,
                              int64_t out_ld, cudaStream_t s) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (d < 16 || d > kMaxCols || d % 16 != 0 || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !out || !is_aligned(codes, 16) || !is_aligned(scales, 16) || !is_aligned(out, 16) ||
      out_ld < d || out_ld % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  return launch_fp8_dequantise(rows, d, static_cast<const uint8_t*>(codes), scales, static_cast<uint16_t*>(out), out_ld,
                               s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

size_t moe_fp8_packed_bytes(const moe_fp8_weights* w) {
  if (!w || !weights_dims_ok(w)) return 0;
  return static_cast<size_t>(w->num_experts * fp8_units(w) * fp8_blocks(w->k)) * kFp8Block;
}

moe_status moe_fp8_pack_weights(const moe_fp8_weights* w, const void* codes, const float* scales, int32_t transpose,
                                void* packed, float* scales_out, cudaStream_t s) {
  if (!w) return MOE_ERR_INVALID_ARG;
  if (!weights_dims_ok(w) || (transpose && w->n_out % 16 != 0)) return MOE_ERR_UNSUPPORTED;
  const size_t bytes = static_cast<size_t>(w->num_experts) * w->n_out * w->k;
  const size_t scale_bytes = 4 * static_cast<size_t>(w->num_experts * fp8_blocks(w->n_out) * fp8_blocks(w->k));
  if (!codes || !packed || !is_aligned(codes, 16) || !is_aligned(packed, 16) ||
      overlaps(codes, bytes, packed, moe_fp8_packed_bytes(w)))
    return MOE_ERR_INVALID_ARG;
  if (transpose && (!scales || !scales_out || !is_aligned(scales, 4) || !is_aligned(scales_out, 4) ||
                    overlaps(scales, scale_bytes, scales_out, scale_bytes)))
    return MOE_ERR_INVALID_ARG;
  return launch_fp8_pack(w, static_cast<const uint8_t*>(codes), scales, transpose != 0, static_cast<uint8_t*>(packed),
                         scales_out, s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_fp8_grouped_product(const moe_fp8_weights* w, int64_t rows, const void* x_codes, const float* x_scales,
                                   const int32_t* expert_offsets, void* out, int32_t out_type, int64_t out_rows,
                                   int64_t out_ld, const int32_t* out_pos, const float* row_weight, void* ws,
                                   size_t ws_bytes, cudaStream_t s) {
  if (!w || rows < 0) return MOE_ERR_INVALID_ARG;
  if (!weights_dims_ok(w) || rows > kMaxRows ||
      (rows / 128 + w->num_experts) * fp8_blocks(w->n_out) >= kMaxUnits)
    return MOE_ERR_UNSUPPORTED;
  if (out_rows < 0 || out_type < MOE_FP8_OUT_BF16 || out_type > MOE_FP8_OUT_F32) return MOE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256) || ws_bytes < MOE_FP8_PRODUCT_WORKSPACE) return MOE_ERR_WORKSPACE;
  if (rows == 0) return MOE_OK;
  if (!w->packed || !w->scales || !is_aligned(w->packed, 16) || !is_aligned(w->scales, 4) || !x_codes || !x_scales ||
      !is_aligned(x_codes, 16) || !is_aligned(x_scales, 16) || (!expert_offsets && w->num_experts != 1) ||
      !is_aligned(expert_offsets, 4) || !out || !is_aligned(out, out_type == MOE_FP8_OUT_F32 ? 4 : 2) ||
      out_ld < w->n_out || !is_aligned(out_pos, 4) || !is_aligned(row_weight, 4))
    return MOE_ERR_INVALID_ARG;
  Fp8ProductLaunch g{};
  g.w = w;
  g.rows = static_cast<int32_t>(rows);
  g.x_codes = static_cast<const uint8_t*>(x_codes);
  g.x_scales = x_scales;
  g.offsets = expert_offsets;
  g.out = out;
  g.out_type = out_type;
  g.out_rows = out_rows;
  g.out_ld = out_ld;
  g.out_pos = out_pos;
  g.row_weight = row_weight;
  g.err = static_cast<uint32_t*>(ws);
  g.num_sms = device_sms();
  if (g.num_sms <= 0) return MOE_ERR_CUDA;
  return launch_fp8_product(g, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
