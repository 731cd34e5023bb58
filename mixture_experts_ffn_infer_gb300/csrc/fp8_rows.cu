// Rows into and out of e4m3 with a scale per 128 columns, and the packed weight
// layout (moe_fp8.h).  All of them move bytes: HBM bounds them.
//
// fp8_rows_kernel       - quantise, write to each position of the row.  A thread holds
//                         16 consecutive columns (32 bytes read, 16 written) from the read
//                         to the codes, eight threads a block of 128: its largest
//                         magnitude takes three exchanges.  A CTA a row, several where few
//                         come, or a warp where many narrow ones do.
// fp8_dequantise_kernel - codes and scales to bf16, 16 columns at a time, four a thread
//                         under way at once.
// fp8_pack_kernel       - a CTA a packed block.
// fp8_transpose_kernel  - the same from the transposed matrix: a CTA a 128 x 128 tile, turned
//                         in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kPiece = 16;  // columns a thread holds together
constexpr int kFewThreads = 64, kSplitThreads = 256;

__device__ __forceinline__ void load_piece(const uint16_t* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// The larger magnitude, NaN if either is.
__device__ __forceinline__ float abs_max_nan(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

struct BlockScale {
  float scale;  // what is stored
  float inv;    // its correctly rounded reciprocal, 0 where the quotient takes the division
  bool none;    // not finite: codes of zero
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale b;
  b.none = !(amax <= 3.4028234663852886e38f);
  b.scale = b.none ? __uint_as_float(0x7fc00000u) : amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  if (b.scale == 0.f) b.scale = 1.f;  // (amax below 448 of the smallest float)
  b.inv = b.scale > 0x1p-60f && b.scale < 0x1p60f ? __frcp_rn(b.scale) : 0.f;
  return b;
}
// v / scale, correctly rounded: the quotient by the reciprocal corrected by its own remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  Blocks whose scale lies
// outside 2^-60 .. 2^60, where a remainder could be inexact, divide.
__device__ __forceinline__ float over(float v, const BlockScale& b) {
  if (b.inv == 0.f) return __fdiv_rn(v, b.scale);
  const float q = v * b.inv;
  return fmaf(fmaf(-q, b.scale, v), b.inv, q);
}

__device__ __forceinline__ void codes_of(const uint32_t (&raw)[8], const BlockScale& b, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t[2 * j] = over(__uint_as_float(raw[2 * i + j] << 16), b);
      t[2 * j + 1] = over(__uint_as_float(raw[2 * i + j] & 0xffff0000u), b);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = b.none ? 0u : lo | (hi << 16);
  }
}

// ITER passes of `width` pieces cover the row.
template <int ITER, bool WARP>
__global__ void __launch_bounds__(kSplitThreads)
fp8_rows_kernel(const Fp8RowsLaunch a, int32_t pitch, int32_t wide, int32_t parts) {
  pdl_wait();
  pdl_launch_dependents();
  const int width = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5) : blockIdx.x / parts;
  const int first = WARP ? 0 : (blockIdx.x % parts) * (ITER * width);
  if (WARP && t >= a.n) return;
  const int np = a.d / kPiece;
  uint32_t raw[ITER][8];
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int c = first + it * width + tid;
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[it][i] = 0u;
    if (c < np) load_piece(a.x + t * a.x_ld + kPiece * c, wide != 0, raw[it]);
  }
  int32_t at[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    at[j] = j >= a.k ? -1 : a.positions ? __ldg(a.positions + t * a.k + j) : 0;
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int c = first + it * width + tid;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = abs_max_nan(m, __uint_as_float(raw[it][i] << 16));
      m = abs_max_nan(m, __uint_as_float(raw[it][i] & 0xffff0000u));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = abs_max_nan(m, __shfl_xor_sync(kAll, m, o));
    const BlockScale b = block_scale(m);
    uint32_t w[4];
    codes_of(raw[it], b, w);
    if (c >= np) continue;
    auto store = [&](int64_t pos) {
      if (pos < 0 || pos >= a.out_rows) return;
      reinterpret_cast<uint4*>(a.codes + pos * a.d)[c] = make_uint4(w[0], w[1], w[2], w[3]);
      if (c % 8 == 0) a.scales[pos * pitch + c / 8] = b.scale;
    };
    if (!a.positions) {
      store(t);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) store(at[j]);
      for (int j = 8; j < a.k; ++j) store(__ldg(a.positions + t * a.k + j));
    }
  }
}

bool aligned32(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && ld % 16 == 0; }

// 1024 pieces to a CTA, four to a thread, of as many rows as fit or of a part of one.
constexpr int kDeqPieces = 1024;

__global__ void __launch_bounds__(256)
fp8_dequantise_kernel(int64_t rows, int32_t d, const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                      uint16_t* __restrict__ out, int64_t out_ld, int32_t pitch, uint32_t magic, int32_t segs,
                      int32_t rpb, int32_t wide) {
  pdl_wait();
  pdl_launch_dependents();
  const int np = d / kPiece;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / segs) * rpb;
  const int c0 = static_cast<int>(blockIdx.x % segs) * kDeqPieces;
  int r[4], c[4];
  uint4 w[4];
  float sc[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 256 * u + threadIdx.x;
    // magic: ceil(2^32 / np), by which i / np is one multiplication for i < 1024 (np 1: the row is i)
    const int rl = np >= kDeqPieces ? 0 : np == 1 ? i : static_cast<int>(__umulhi(i, magic));
    c[u] = np < kDeqPieces ? i - rl * np : c0 + i;
    r[u] = rl < rpb && c[u] < np && row0 + rl < rows ? rl : -1;
    if (r[u] < 0) continue;
    w[u] = __ldg(reinterpret_cast<const uint4*>(codes + (row0 + rl) * d) + c[u]);
    sc[u] = __ldg(scales + (row0 + rl) * pitch + c[u] / 8);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (r[u] < 0) continue;
    const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>((q[j >> 1] >> (16 * (j & 1))) & 0xffffu), __NV_E4M3));
      const __nv_bfloat162 v = __floats2bfloat162_rn(__low2float(h) * sc[u], __high2float(h) * sc[u]);
      o[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint16_t* p = out + (row0 + r[u]) * out_ld + kPiece * c[u];
    if (wide) {
      stg256(p, o);
    } else {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// Block (e, u, c): 256 rows of eight 16-byte pieces.
__global__ void __launch_bounds__(256)
fp8_pack_kernel(const uint8_t* __restrict__ codes, uint8_t* __restrict__ packed, int32_t n_out, int32_t k,
                int32_t units, int32_t chunks) {
  const int64_t b = blockIdx.x;
  const int c = static_cast<int>(b % chunks), u = static_cast<int>(b / chunks % units);
  const int64_t e = b / chunks / units;
  uint8_t* d = packed + b * kFp8Block;
  for (int i = threadIdx.x; i < 2048; i += 256) {
    const int r = i >> 3, j = i & 7, n = kFp8UnitRows * u + r, at = 128 * c + 16 * j;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n < n_out && at < k) v = __ldg(reinterpret_cast<const uint4*>(codes + (e * n_out + n) * k + at));
    *reinterpret_cast<uint4*>(d + r * 128 + ((j ^ (r & 7)) << 4)) = v;
  }
}

// The half (128 rows) h of block (e, u, c) from codes [E][k][n_out]; the tile's scale is turned with it.
__global__ void __launch_bounds__(256)
fp8_transpose_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, uint8_t* __restrict__ packed,
                     float* __restrict__ scales_out, int32_t n_out, int32_t k, int32_t units, int32_t chunks) {
  __shared__ uint8_t tile[128][132];  // [column of the result][its rows]; the pitch spreads a column over the banks
  const int64_t b = blockIdx.x >> 1;
  const int h = blockIdx.x & 1;
  const int c = static_cast<int>(b % chunks), u = static_cast<int>(b / chunks % units);
  const int64_t e = b / chunks / units;
  const int n0 = kFp8UnitRows * u + 128 * h, k0 = 128 * c;
  uint8_t* d = packed + b * kFp8Block + 128 * 128 * h;
  for (int i = threadIdx.x; i < 1024; i += 256) {
    const int r = i >> 3, j = i & 7;  // row k0 + r of the source, its columns n0 + 16 j ..
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (k0 + r < k && n0 + 16 * j < n_out)
      v = __ldg(reinterpret_cast<const uint4*>(codes + (e * k + k0 + r) * n_out + n0 + 16 * j));
    uint32_t* p = reinterpret_cast<uint32_t*>(&tile[r][16 * j]);
    p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 1024; i += 256) {
    const int r = i & 127, j = i >> 7;  // row r of the result, its columns 16 j ..
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) w[q] |= static_cast<uint32_t>(tile[16 * j + 4 * q + x][r]) << (8 * x);
    }
    *reinterpret_cast<uint4*>(d + r * 128 + ((j ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int nb = (n_out + 127) / 128, at = n0 / 128;
  if (threadIdx.x == 0 && at < nb)
    scales_out[(e * nb + at) * chunks + c] = __ldg(scales + (e * chunks + c) * nb + at);
}

}  // namespace

cudaError_t launch_fp8_rows(const Fp8RowsLaunch& a, cudaStream_t s) {
  const int np = a.d / kPiece;
  // Few rows: a piece a thread, 64 threads to a CTA, so that a row's stores to its positions are on several SMs (16 rows of
  // 16,384 columns to 8 positions on one GB300: 6.1 us, 8.2 by a CTA a row).  More rows than the SMs hold at once: two pieces a thread, and
  // rows of up to 64 pieces one to a warp, eight to a CTA.
  const bool many = a.n > 2 * device_sms(), by_warp = many && np <= 64;
  int iters = many && !by_warp ? 2 : 1;
  while (many && iters * (by_warp ? 32 : kSplitThreads) < np) iters *= 2;
  const int threads = by_warp ? 256 : many ? ((np + iters - 1) / iters + 31) / 32 * 32 : kFewThreads;
  const int parts = many ? 1 : (np + kFewThreads - 1) / kFewThreads;
  const int64_t grid = by_warp ? (a.n + 7) / 8 : a.n * parts;
  auto kern = by_warp      ? iters == 1 ? fp8_rows_kernel<1, true> : fp8_rows_kernel<2, true>
              : iters == 1 ? fp8_rows_kernel<1, false>
              : iters == 2 ? fp8_rows_kernel<2, false>
                           : fp8_rows_kernel<4, false>;
  return launch_maybe_overlapped(kern, static_cast<int>(grid), threads, 0, s, true, a,
                                 static_cast<int32_t>(moe_fp8_scale_pitch(a.d)),
                                 static_cast<int32_t>(aligned32(a.x, a.x_ld)), parts);
}

cudaError_t launch_fp8_dequantise(int64_t rows, int32_t d, const uint8_t* codes, const float* scales, uint16_t* out,
                                  int64_t out_ld, cudaStream_t s) {
  const int np = d / kPiece;
  const int segs = (np + kDeqPieces - 1) / kDeqPieces, rpb = np < kDeqPieces ? kDeqPieces / np : 1;
  const uint32_t magic = np > 1 ? static_cast<uint32_t>(((1ull << 32) + np - 1) / np) : 0u;
  const int64_t blocks = (rows + rpb - 1) / rpb * segs;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_maybe_overlapped(fp8_dequantise_kernel, static_cast<int>(blocks), 256, 0, s, true, rows, d, codes, scales,
                                 out, out_ld, static_cast<int32_t>(moe_fp8_scale_pitch(d)), magic, segs, rpb,
                                 static_cast<int32_t>(aligned32(out, out_ld)));
}

cudaError_t launch_fp8_pack(const moe_fp8_weights* w, const uint8_t* codes, const float* scales, bool transpose,
                            uint8_t* packed, float* scales_out, cudaStream_t s) {
  const int64_t units = fp8_units(w), chunks = fp8_blocks(w->k), blocks = w->num_experts * units * chunks;  // below 2^28
  if (transpose)
    fp8_transpose_kernel<<<static_cast<unsigned>(2 * blocks), 256, 0, s>>>(
        codes, scales, packed, scales_out, w->n_out, w->k, static_cast<int32_t>(units), static_cast<int32_t>(chunks));
  else
    fp8_pack_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(codes, packed, w->n_out, w->k,
                                                                 static_cast<int32_t>(units), static_cast<int32_t>(chunks));
  return cudaGetLastError();
}

}  // namespace moe
