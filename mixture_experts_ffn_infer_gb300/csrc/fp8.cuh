// Rows and weights in the FP8 bank's form (moe_fp8.h): the launchers of fp8_rows.cu
// and fp8_gemm.cu.
#pragma once
#include "common.cuh"
#include "moe_fp8.h"

namespace moe {

constexpr int kFp8UnitRows = 256;                 // weight rows of a packed block
constexpr int kFp8Block = kFp8UnitRows * 128;     // its bytes
inline int64_t fp8_blocks(int64_t cols) { return (cols + 127) / 128; }
inline int64_t fp8_units(const moe_fp8_weights* w) { return (w->n_out + kFp8UnitRows - 1) / kFp8UnitRows; }

struct Fp8RowsLaunch {
  int64_t n;
  int32_t k, d;
  const uint16_t* x;
  int64_t x_ld;
  const int32_t* positions;
  int64_t out_rows;
  uint8_t* codes;
  float* scales;
};
cudaError_t launch_fp8_rows(const Fp8RowsLaunch& a, cudaStream_t s);
cudaError_t launch_fp8_dequantise(int64_t rows, int32_t d, const uint8_t* codes, const float* scales, uint16_t* out,
                                  int64_t out_ld, cudaStream_t s);
cudaError_t launch_fp8_pack(const moe_fp8_weights* w, const uint8_t* codes, const float* scales, bool transpose,
                            uint8_t* packed, float* scales_out, cudaStream_t s);

struct Fp8ProductLaunch {
  const moe_fp8_weights* w;
  int32_t rows;
  const uint8_t* x_codes;
  const float* x_scales;
  const int32_t* offsets;  // null: one expert, all rows
  void* out;
  int32_t out_type;
  int64_t out_rows, out_ld;
  const int32_t* out_pos;
  const float* row_weight;
  uint32_t* err;
  int num_sms;
};
cudaError_t launch_fp8_product(const Fp8ProductLaunch& g, cudaStream_t s);

}  // namespace moe
