// Rows into and out of the microscaled formats (moe_mx.h), and the packed
// weight layout.  All four kernels move bytes: HBM bounds them.  Rows in and out
// are dependent launches that wait before they read anything, so that in a
// sequence of short calls one's launch overlaps the other's end.
//
// mx_rows_kernel       - [add the residual, RMS norm,] quantise, write to each
//                        position of the token.  One CTA per token; a thread
//                        holds eight consecutive columns in registers (one
//                        16-byte load) from the first read to the codes, so x
//                        is read once.  A group is two (16 columns) or four (32)
//                        neighbouring lanes: its maximum takes one or two
//                        shuffles.
// mx_dequantise_kernel - codes and scales to bf16, eight columns a thread.
// mx_pack_kernel       - one CTA per packed block.
#include "mx.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

template <int FMT>
__device__ __forceinline__ int64_t code_pitch(int d) {
  return FMT == MOE_MX_BF16 ? 2 * static_cast<int64_t>(d) : FMT == MOE_MX_MXFP8 ? d : d / 2;
}
template <int FMT>
__device__ __forceinline__ int64_t scale_pitch(int d) {
  if constexpr (FMT == MOE_MX_BF16) return 0;
  else return (d / Mx<FMT>::group + 15) & ~15;
}

constexpr int kRowsMaxThreads = 1024;
constexpr int kRowsSplitThreads = 256;

// ITER passes of blockDim.x * 8 columns cover the row, held as the bf16 pairs they
// are read as (the stored sum is bf16 too).  The sum of squares is taken per thread
// in column order, then by shuffles, then over the warps.
template <int FMT, bool NORM, int ITER>
__global__ void __launch_bounds__(ITER <= 2 ? kRowsMaxThreads : kRowsSplitThreads)
mx_rows_kernel(const MxRowsLaunch a) {
  __shared__ float part[32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int d = a.d, nc = d / 8;
  uint4 raw[ITER];
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int c = it * blockDim.x + threadIdx.x;
    raw[it] = make_uint4(0u, 0u, 0u, 0u);
    if (c < nc) raw[it] = *(reinterpret_cast<const uint4*>(a.x + t * a.x_ld) + c);
  }
  float rs = 1.f;
  if constexpr (NORM) {
    float ss = 0.f;
    if (a.residual) {
      uint4 res[ITER];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int c = it * blockDim.x + threadIdx.x;
        res[it] = make_uint4(0u, 0u, 0u, 0u);
        if (c < nc) res[it] = *(reinterpret_cast<const uint4*>(a.residual + t * a.r_ld) + c);
      }
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        float v[8], r[8];
        unpack8(raw[it], v);
        unpack8(res[it], r);
        raw[it] = make_uint4(pack_bf16(v[0] + r[0], v[1] + r[1]), pack_bf16(v[2] + r[2], v[3] + r[3]),
                             pack_bf16(v[4] + r[4], v[5] + r[5]), pack_bf16(v[6] + r[6], v[7] + r[7]));
      }
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int c = it * blockDim.x + threadIdx.x;
      if (a.sum && c < nc) *(reinterpret_cast<uint4*>(a.sum + t * a.r_ld) + c) = raw[it];
      float v[8];
      unpack8(raw[it], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (warps > 1) {
      if (lane == 0) part[warp] = ss;
      __syncthreads();
      ss = lane < warps ? part[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    rs = rsqrtf(ss / static_cast<float>(d) + a.eps);
  }
  const GroupFactor factor = group_factor<FMT>(a.global);
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int c = it * blockDim.x + threadIdx.x;
    float v[8];
    unpack8(raw[it], v);
    if constexpr (NORM) {
      if (c < nc) {
        float g[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.gain) + c), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * rs * g[i];
      }
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    GroupScale sc{};
    if constexpr (FMT == MOE_MX_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      if constexpr (Mx<FMT>::group == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      sc = group_scale<FMT>(m, factor);
      uint32_t cw[2];
      codes8<FMT>(v, sc, cw);
      w[0] = cw[0];
      w[1] = cw[1];
    }
    if (c >= nc) continue;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      int32_t at[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        at[j] = j0 + j >= a.k ? -1 : a.positions ? __ldg(a.positions + t * a.k + j0 + j) : static_cast<int32_t>(t);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (at[j] < 0 || at[j] >= a.out_rows) continue;
        uint8_t* row = a.codes + at[j] * code_pitch<FMT>(d);
        if constexpr (FMT == MOE_MX_BF16) {
          reinterpret_cast<uint4*>(row)[c] = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          if constexpr (FMT == MOE_MX_MXFP8) reinterpret_cast<uint2*>(row)[c] = make_uint2(w[0], w[1]);
          else reinterpret_cast<uint32_t*>(row)[c] = w[0];
          constexpr int kLanes = Mx<FMT>::group / 8;
          if (c % kLanes == 0) a.scales[at[j] * scale_pitch<FMT>(d) + c / kLanes] = static_cast<uint8_t>(sc.byte);
        }
      }
    }
  }
}

template <int FMT, bool NORM>
cudaError_t launch_rows(const MxRowsLaunch& a, cudaStream_t s) {
  const int nc = a.d / 8;
  // Few rows: as many threads as the row has pieces, for the shortest way through one row.  More rows
  // than SMs: 256 threads with several pieces each, so that an SM holds more rows in different phases.
  const int most = a.n > 2 * device_sms() ? kRowsSplitThreads : kRowsMaxThreads;
  int iters = 1;
  while (iters * most < nc) iters *= 2;
  const int threads = ((nc + iters - 1) / iters + 31) / 32 * 32;
  auto kern = iters == 1   ? mx_rows_kernel<FMT, NORM, 1>
              : iters == 2 ? mx_rows_kernel<FMT, NORM, 2>
              : iters == 4 ? mx_rows_kernel<FMT, NORM, 4>
                           : mx_rows_kernel<FMT, NORM, 8>;
  return launch_maybe_overlapped(kern, static_cast<int>(a.n), threads, 0, s, true, a);
}

// A CTA covers 1024 pieces of eight columns, of as many rows as fit or of one row's
// part, four pieces a thread: their loads are all under way before the first is used.
constexpr int kDeqPieces = 1024;

template <int FMT>
__global__ void __launch_bounds__(256)
mx_dequantise_kernel(int64_t rows, int32_t d, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                     const float* __restrict__ global_p, uint16_t* __restrict__ out, int64_t out_ld) {
  pdl_launch_dependents();
  pdl_wait();
  const int nc = d / 8;
  const int segs = (nc + kDeqPieces - 1) / kDeqPieces, rpb = nc < kDeqPieces ? kDeqPieces / nc : 1;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / segs) * rpb;
  const int c0 = static_cast<int>(blockIdx.x % segs) * kDeqPieces;
  const float global = FMT == MOE_MX_NVFP4 && global_p ? __ldg(global_p) : 1.f;
  int64_t r[4];
  int c[4];
  uint4 w[4];
  uint32_t sb[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 256 * u + threadIdx.x;
    const int rl = nc < kDeqPieces ? i / nc : 0;
    c[u] = nc < kDeqPieces ? i - rl * nc : c0 + i;
    r[u] = rl < rpb && c[u] < nc && row0 + rl < rows ? row0 + rl : -1;
    if (r[u] >= 0) {
      const uint8_t* row = codes + r[u] * code_pitch<FMT>(d);
      if constexpr (FMT == MOE_MX_BF16) {
        w[u] = __ldg(reinterpret_cast<const uint4*>(row) + c[u]);
      } else {
        if constexpr (FMT == MOE_MX_MXFP8) {
          const uint2 q = __ldg(reinterpret_cast<const uint2*>(row) + c[u]);
          w[u].x = q.x;
          w[u].y = q.y;
        } else {
          w[u].x = __ldg(reinterpret_cast<const uint32_t*>(row) + c[u]);
        }
        sb[u] = __ldg(scales + r[u] * scale_pitch<FMT>(d) + c[u] / (Mx<FMT>::group / 8));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (r[u] < 0) continue;
    uint4 o = w[u];
    if constexpr (FMT != MOE_MX_BF16) {
      float sc;
      if constexpr (FMT == MOE_MX_NVFP4) sc = e4m3_value(sb[u]) * global;
      else if (sb[u] == 255u) sc = __uint_as_float(0x7fc00000u);
      else sc = sb[u] == 0u ? 0x1p-127f : __uint_as_float(sb[u] << 23);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __half2 h;
        if constexpr (FMT == MOE_MX_MXFP8) {
          const uint32_t pair = ((j < 2 ? w[u].x : w[u].y) >> (16 * (j & 1))) & 0xffffu;
          h = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3));
        } else {
          h = __half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((w[u].x >> (8 * j)) & 0xffu),
                                                 __NV_E2M1));
        }
        v[2 * j] = __low2float(h) * sc;
        v[2 * j + 1] = __high2float(h) * sc;
      }
      o = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
    *(reinterpret_cast<uint4*>(out + r[u] * out_ld) + c[u]) = o;
  }
}

// Block (e, u, c): 2048 pieces of 16 bytes of codes, then 256 * words words of scales.
__global__ void __launch_bounds__(256)
mx_pack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
               const uint8_t* __restrict__ codes_up, const uint8_t* __restrict__ scales_up, uint8_t* __restrict__ dst,
               int32_t n_out, int32_t swiglu, int64_t row_bytes, int64_t pitch, int32_t groups, int32_t words,
               int32_t units, int32_t chunks) {
  const int64_t b = blockIdx.x;
  const int c = static_cast<int>(b % chunks);
  const int64_t eu = b / chunks;
  const int u = static_cast<int>(eu % units);
  const int64_t e = eu / units;
  uint8_t* d = dst + b * (kMxCodeBlock + 1024 * words);
  // matrix row of block row r, or -1
  auto row_of = [&](int r, bool& up) {
    up = swiglu && r >= 128;
    const int n = swiglu ? 128 * u + (r & 127) : 256 * u + r;
    return n < n_out ? e * n_out + n : static_cast<int64_t>(-1);
  };
  for (int i = threadIdx.x; i < 2048; i += 256) {
    const int r = i >> 3, j = i & 7;
    bool up;
    const int64_t row = row_of(r, up);
    const int64_t at = static_cast<int64_t>(c) * 128 + j * 16;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0 && at < row_bytes) v = __ldg(reinterpret_cast<const uint4*>((up ? codes_up : codes) + row * row_bytes + at));
    *reinterpret_cast<uint4*>(d + r * 128 + ((j ^ (r & 7)) << 4)) = v;
  }
  for (int i = threadIdx.x; i < 256 * words; i += 256) {
    const int r = i / words, w = i % words;
    bool up;
    const int64_t row = row_of(r, up);
    const int g0 = (c * words + w) * 4;
    uint32_t v = 0;
    if (row >= 0 && g0 < groups) {
      v = __ldg(reinterpret_cast<const uint32_t*>((up ? scales_up : scales) + row * pitch + g0));
      const int left = groups - g0;  // bytes past the last group are padding
      if (left < 4) v &= (1u << (8 * left)) - 1u;
    }
    *reinterpret_cast<uint32_t*>(d + kMxCodeBlock + w * 1024 + (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4) = v;
  }
}

}  // namespace

cudaError_t launch_mx_rows(int32_t fmt, const MxRowsLaunch& a, cudaStream_t s) {
  const bool norm = a.gain != nullptr;
  switch (fmt) {
    case MOE_MX_BF16: return norm ? launch_rows<MOE_MX_BF16, true>(a, s) : launch_rows<MOE_MX_BF16, false>(a, s);
    case MOE_MX_MXFP8: return norm ? launch_rows<MOE_MX_MXFP8, true>(a, s) : launch_rows<MOE_MX_MXFP8, false>(a, s);
    case MOE_MX_MXFP4: return norm ? launch_rows<MOE_MX_MXFP4, true>(a, s) : launch_rows<MOE_MX_MXFP4, false>(a, s);
    case MOE_MX_NVFP4: return norm ? launch_rows<MOE_MX_NVFP4, true>(a, s) : launch_rows<MOE_MX_NVFP4, false>(a, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx_dequantise(int32_t fmt, int64_t rows, int32_t d, const uint8_t* codes, const uint8_t* scales,
                                 const float* global, uint16_t* out, int64_t out_ld, cudaStream_t s) {
  const int nc = d / 8;
  const int64_t segs = (nc + kDeqPieces - 1) / kDeqPieces, rpb = nc < kDeqPieces ? kDeqPieces / nc : 1;
  const int64_t blocks = (rows + rpb - 1) / rpb * segs;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kern = fmt == MOE_MX_BF16    ? mx_dequantise_kernel<MOE_MX_BF16>
              : fmt == MOE_MX_MXFP8 ? mx_dequantise_kernel<MOE_MX_MXFP8>
              : fmt == MOE_MX_MXFP4 ? mx_dequantise_kernel<MOE_MX_MXFP4>
                                    : mx_dequantise_kernel<MOE_MX_NVFP4>;
  return launch_maybe_overlapped(kern, static_cast<int>(blocks), 256, 0, s, true, rows, d, codes, scales, global, out,
                                 out_ld);
}

cudaError_t launch_mx_pack(const moe_mx_weights* w, const uint8_t* codes, const uint8_t* scales,
                           const uint8_t* codes_up, const uint8_t* scales_up, uint8_t* packed, cudaStream_t s) {
  const int64_t units = mx_unit_rows(w), chunks = mx_chunks(w), blocks = w->num_experts * units * chunks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int g = mx_group(w->format);
  mx_pack_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(
      codes, scales, codes_up, scales_up, packed, w->n_out, w->swiglu, moe_mx_code_bytes(w->format, w->k),
      moe_mx_scale_pitch(w->format, w->k), g ? w->k / g : 0, mx_words(w->format), static_cast<int32_t>(units),
      static_cast<int32_t>(chunks));
  return cudaGetLastError();
}

}  // namespace moe
