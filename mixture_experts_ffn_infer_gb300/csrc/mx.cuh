// Microscaled formats: their sizes, the quantisation of a group, and the
// launchers of mx_rows.cu and mx_gemm.cu.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "moe_mx.h"

namespace moe {

// cols: columns in 128 bytes of codes; group: columns of a scale (0: none);
// words: 4-byte words of scales that go with 128 bytes of codes.
template <int FMT>
struct Mx;
template <>
struct Mx<MOE_MX_BF16> {
  static constexpr int cols = 64, group = 0, words = 0;
};
template <>
struct Mx<MOE_MX_MXFP8> {
  static constexpr int cols = 128, group = 32, words = 1;
};
template <>
struct Mx<MOE_MX_MXFP4> {
  static constexpr int cols = 256, group = 32, words = 2;
};
template <>
struct Mx<MOE_MX_NVFP4> {
  static constexpr int cols = 256, group = 16, words = 4;
};

inline int mx_cols(int fmt) { return fmt == MOE_MX_BF16 ? 64 : fmt == MOE_MX_MXFP8 ? 128 : 256; }
inline int mx_group(int fmt) { return fmt == MOE_MX_BF16 ? 0 : fmt == MOE_MX_NVFP4 ? 16 : 32; }
inline int mx_words(int fmt) { return fmt == MOE_MX_BF16 ? 0 : fmt == MOE_MX_MXFP8 ? 1 : fmt == MOE_MX_MXFP4 ? 2 : 4; }
constexpr int kMxUnitRows = 256;               // weight rows of a packed block
constexpr int kMxCodeBlock = kMxUnitRows * 128;  // its bytes of codes
inline int64_t mx_block_bytes(int fmt) { return kMxCodeBlock + 1024 * mx_words(fmt); }
inline int64_t mx_unit_rows(const moe_mx_weights* w) {  // packed blocks along n_out
  const int tall = w->swiglu ? 128 : 256;
  return (w->n_out + tall - 1) / tall;
}
inline int64_t mx_chunks(const moe_mx_weights* w) { return (w->k + mx_cols(w->format) - 1) / mx_cols(w->format); }

// ---------------------------------------------------------------- quantisation

// What a group's codes are divided by.
struct GroupScale {
  uint32_t byte;  // the stored scale
  float div;      // NVFP4: the divisor; MX formats: unused
  float mul;      // its reciprocal, exact for the MX formats; 0: all codes zero
};

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// a / b, correctly rounded, from b's correctly rounded reciprocal r: the quotient
// a * r corrected by its own remainder (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990: q' = q + r (a - q b)).  b lies
// within 2^-72 .. 2^72 here, and where a is so small that the remainder is not exact
// the quotient rounds to zero in every format.  From `top` on, where the result
// saturates, the quotient is left alone (it may be infinite).  Five instructions
// against a division's twenty and a branch.
__device__ __forceinline__ float quotient(float a, float b, float r, float top) {
  const float q = a * r;
  return fabsf(q) < top ? fmaf(fmaf(-q, b, a), r, q) : q;
}

// What all groups of an NVFP4 tensor share: its factor, six times it and that one's reciprocal.
struct GroupFactor {
  float g, six, inv;
};
template <int FMT>
__device__ __forceinline__ GroupFactor group_factor(float g) {
  if constexpr (FMT != MOE_MX_NVFP4) return GroupFactor{1.f, 6.f, 0.f};
  return GroupFactor{g, 6.0f * g, __frcp_rn(6.0f * g)};
}

// amax: the largest of the group's |v|, NaN where one is (abs_max).
template <int FMT>
__device__ __forceinline__ GroupScale group_scale(float amax, const GroupFactor& f) {
  const uint32_t abs_bits = __float_as_uint(amax);
  const bool bad = abs_bits >= 0x7f800000u;
  if constexpr (FMT == MOE_MX_NVFP4) {
    const float t = quotient(amax, f.six, f.inv, 1024.f);
    const uint32_t byte = bad ? 0x7fu : __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    const float div = e4m3_value(byte) * f.g;
    return GroupScale{byte, div, !bad && div > 0.f ? __frcp_rn(div) : 0.f};
  } else {
    // The smallest k with a <= M 2^k: M = 1.75 2^8 or 1.5 2^2, so a = 1.m 2^e takes
    // k = e - 8 (e - 2) while 1.m is at most 1.75 (1.5), one more above that.
    constexpr uint32_t kTop = FMT == MOE_MX_MXFP8 ? 0x600000u : 0x400000u;
    constexpr int kExp = FMT == MOE_MX_MXFP8 ? 8 : 2;
    const int k127 = max(1, static_cast<int>(abs_bits >> 23) - kExp + ((abs_bits & 0x7fffffu) > kTop ? 1 : 0));
    return bad ? GroupScale{0xffu, 0.f, 0.f}
               : GroupScale{static_cast<uint32_t>(k127), 0.f, __uint_as_float(static_cast<uint32_t>(254 - k127) << 23)};
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes of N quotients into N / 8 (e2m1) or N / 4 (e4m3) words; all zero with `none` (a zero
// divisor, or a group that is not finite).
template <int FMT, int N>
__device__ __forceinline__ void pack_codes(const float* t, bool none, uint32_t* w) {
  if constexpr (FMT == MOE_MX_MXFP8) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * i], t[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * i + 2], t[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = none ? 0u : lo | (hi << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        word |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(t[8 * i + 2 * j], t[8 * i + 2 * j + 1]),
                                                               __NV_E2M1, cudaRoundNearest))
                << (8 * j);
      w[i] = none ? 0u : word;
    }
  }
}

template <int FMT>
__device__ __forceinline__ float over_scale(float v, const GroupScale& s) {
  return FMT == MOE_MX_NVFP4 ? quotient(v, s.div, s.mul, 8.f) : v * s.mul;
}

// Codes of N consecutive columns, all of one group.
template <int FMT, int N>
__device__ __forceinline__ void codes_of(const float* v, const GroupScale& s, uint32_t* w) {
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = over_scale<FMT>(v[i], s);
  pack_codes<FMT, N>(t, s.mul == 0.f, w);
}

// The larger magnitude, NaN if either is: as bits it is above every finite value's.
__device__ __forceinline__ float abs_max(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// ---------------------------------------------------------------- launchers
struct MxRowsLaunch {
  int64_t n;
  int32_t k, d;
  const uint16_t* x;
  int64_t x_ld;
  const uint16_t* residual;
  int64_t r_ld;
  const uint16_t* gain;  // null: no norm
  float eps;
  const int32_t* positions;
  const float* global;
  int64_t out_rows;
  uint16_t* sum;
  uint8_t* codes;
  uint8_t* scales;
  // x, residual, gain and global were complete before the kernel in front began (positions are that one's):
  // they are read while it still runs
  int32_t late;
  int32_t wide_x, wide_r, wide_gain, wide_out;  // set by the launcher: rows on 32-byte boundaries
};
cudaError_t launch_mx_rows(int32_t fmt, const MxRowsLaunch& a, cudaStream_t s);
cudaError_t launch_mx_dequantise(int32_t fmt, int64_t rows, int32_t d, const uint8_t* codes, const uint8_t* scales,
                                 const float* global, uint16_t* out, int64_t out_ld, cudaStream_t s);
cudaError_t launch_mx_pack(const moe_mx_weights* w, const uint8_t* codes, const uint8_t* scales,
                           const uint8_t* codes_up, const uint8_t* scales_up, uint8_t* packed, cudaStream_t s);

struct MxProductLaunch {
  const moe_mx_weights* w;
  int32_t rows;
  const uint8_t* x_codes;
  const uint8_t* x_scales;
  const float* x_global;
  const int32_t* offsets;
  // rows out
  void* out;
  int32_t out_f16;
  int64_t out_rows, out_ld;
  const int32_t* out_pos;
  const float* row_weight;
  // swiglu out
  const float* h_global;
  uint8_t* h_codes;
  uint8_t* h_scales;
  uint32_t* err;
  int num_sms;
  // the offsets and weights were complete before the kernel in front began: they are read, and
  // weights streamed, while that one still runs
  bool early;
  const moe_mx_weights* next;  // swiglu: the product that follows on the same rows, or null
};
cudaError_t launch_mx_product(const MxProductLaunch& a, cudaStream_t s);

// api.cu
bool encode_rows_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows);
int device_sms();

}  // namespace moe
