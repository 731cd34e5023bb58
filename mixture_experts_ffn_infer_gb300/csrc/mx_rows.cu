// Rows into and out of the microscaled formats (moe_mx.h), and the packed
// weight layout.  All three kernels move bytes: HBM bounds them.  Rows in and out
// are dependent launches, so that in a sequence of short calls one's launch
// overlaps the other's end; they wait before they read anything (in the layer,
// before the positions: MxRowsLaunch::late).
//
// mx_rows_kernel       - [add the residual, RMS norm,] quantise, write to each
//                        position of the token.  One CTA per token, or one
//                        warp where many narrow rows come; a thread holds
//                        16 consecutive columns at a time (32 bytes) in
//                        registers from the first read to the codes, so x is
//                        read once, and a group is the thread's own columns
//                        (16) or its and its neighbour's (32).  With eight
//                        columns and fp32 sums the kernel took 37
//                        instructions a column and the issue slots bounded it
//                        (67 % busy, DRAM 58 %).
// mx_dequantise_kernel - codes and scales to bf16, 16 columns at a time.
// mx_pack_kernel       - one CTA per packed block.
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kPiece = 16;  // columns a thread holds together

__device__ __forceinline__ void unpack(const uint32_t (&w)[8], float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 16 bf16: one 32-byte access where rows are aligned for it, else two of 16.
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
__device__ __forceinline__ void store_piece(void* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    stg256(p, w);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
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

// One piece's codes (and its group's scale) to row `pos`.
template <int FMT>
__device__ __forceinline__ void store_codes(const MxRowsLaunch& a, int64_t pos, int c, const uint32_t (&w)[8],
                                            uint32_t scale) {
  if (pos < 0 || pos >= a.out_rows) return;
  uint8_t* row = a.codes + pos * code_pitch<FMT>(a.d);
  if constexpr (FMT == MOE_MX_BF16) {
    store_piece(row + 32 * c, a.wide_out != 0, w);
  } else {
    if constexpr (FMT == MOE_MX_MXFP8) reinterpret_cast<uint4*>(row)[c] = make_uint4(w[0], w[1], w[2], w[3]);
    else reinterpret_cast<uint2*>(row)[c] = make_uint2(w[0], w[1]);
    constexpr int kLanes = Mx<FMT>::group / kPiece;
    if (c % kLanes == 0) a.scales[pos * scale_pitch<FMT>(a.d) + c / kLanes] = static_cast<uint8_t>(scale);
  }
}

// ---------------------------------------------------------------- the sum of squares
// A code of 2 to 4 bits turns a difference in y's last bit into a step of a quarter where y
// lies on a rounding border, and the norm's factor moves a whole row's.  The 16 squares of a piece
// are summed in fp32, always in the same order (four sums of every fourth); the pieces' sums are
// joined over a thread's pieces, lanes and warps as sums of two floats.  Those carry some 47 bits,
// so the rounded sum, and with it a token's rows, does not depend on how many tokens come with it
// (which decides the pieces a thread holds), unless it lies within 2^-44 of the middle between two
// floats.

struct Pair {
  float hi, lo;
};
// a + b with what the rounded sum leaves out (D. Knuth's two-sum).
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = a + b, bb = s - a;
  return Pair{s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}
__device__ __forceinline__ Pair warp_sum_pair(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}
// ITER passes of blockDim.x pieces cover the row, held as the bf16 pairs they are
// read as (the stored sum is bf16 too).
template <int FMT, bool NORM, int ITER, bool WARP>
// (Two passes: five CTAs an SM, at 48 registers, were faster than four, 355 us against 369 for 32,768 rows of 7168
// to MXFP8 and back, which take 338 now.)
__global__ void __launch_bounds__(ITER == 1 ? kRowsMaxThreads : kRowsSplitThreads, ITER == 1 ? 1 : ITER == 2 ? 5 : 2)
mx_rows_kernel(const MxRowsLaunch a) {
  __shared__ Pair part[32];
  // A dependent kernel may read what the kernel in front of this one wrote without waiting
  // (MxProductLaunch::early), so it is let in only after this wait.
  if (!a.late) {
    pdl_wait();
    pdl_launch_dependents();
  }
  // the row, and this thread's place among those that share it
  const int width = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && t >= a.n) return;
  const int d = a.d, np = d / kPiece;
  uint32_t raw[ITER][8];
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int c = it * width + tid;
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[it][i] = 0u;
    if (c < np) load_piece(a.x + t * a.x_ld + kPiece * c, a.wide_x != 0, raw[it]);
  }
  // A row in one pass is a matter of latency: all that it reads is under way before anything waits (behind
  // it, the next kernel's weights may already queue for HBM).
  constexpr bool kEarly = ITER == 1;
  uint32_t gain_early[8] = {};
  const int cols_early = min(tid, np - 1);
  if constexpr (kEarly && NORM) load_piece(a.gain + kPiece * cols_early, a.wide_gain != 0, gain_early);
  int32_t at_early[8];
  auto load_positions = [&]() {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      at_early[j] = j >= a.k ? -1 : a.positions ? __ldcg(a.positions + t * a.k + j) : static_cast<int32_t>(t);
  };
  if (kEarly && !a.late) load_positions();
  const float* gp = FMT == MOE_MX_NVFP4 ? a.global : nullptr;
  const float global_early = gp ? __ldg(gp) : 1.f;
  float rs = 1.f;
  if constexpr (NORM) {
    Pair mine{0.f, 0.f};
    if (a.residual) {
      uint32_t res[ITER][8];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int c = it * width + tid;
#pragma unroll
        for (int i = 0; i < 8; ++i) res[it][i] = 0u;
        if (c < np) load_piece(a.residual + t * a.r_ld + kPiece * c, a.wide_r != 0, res[it]);
      }
      // bf16 + bf16 rounded once to bf16, which is what is stored and what is normalised
#pragma unroll
      for (int it = 0; it < ITER; ++it)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 sum = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&raw[it][i]),
                                             *reinterpret_cast<const __nv_bfloat162*>(&res[it][i]));
          raw[it][i] = *reinterpret_cast<const uint32_t*>(&sum);
        }
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int c = it * width + tid;
      if (a.sum && c < np) store_piece(a.sum + t * a.r_ld + kPiece * c, a.wide_r != 0, raw[it]);
      float v[16];
      unpack(raw[it], v);
      float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) sq[i & 3] = fmaf(v[i], v[i], sq[i & 3]);
      const Pair piece{(sq[0] + sq[1]) + (sq[2] + sq[3]), 0.f};
      mine = it == 0 ? piece : add(mine, piece);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = WARP ? 1 : blockDim.x >> 5;
    Pair ss = warp_sum_pair(mine);
    if (!WARP && warps > 1) {
      if (lane == 0) part[warp] = ss;
      __syncthreads();
      ss = warp_sum_pair(lane < warps ? part[lane] : Pair{0.f, 0.f});
    }
    const float sum = ss.hi + ss.lo;  // (an infinite sum's low part is NaN)
    rs = rsqrtf((sum == sum ? sum : ss.hi) / static_cast<float>(d) + a.eps);
  }
  const GroupFactor factor = group_factor<FMT>(global_early);
  if (a.late) {  // the positions are the kernel's in front, which may still run until here
    pdl_wait();
    pdl_launch_dependents();
    if (kEarly) load_positions();
  }
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int c = it * width + tid;
    float v[16];
    unpack(raw[it], v);
    if constexpr (NORM) {
      if (c < np) {
        uint32_t gw[8];
        if constexpr (kEarly) {
#pragma unroll
          for (int i = 0; i < 8; ++i) gw[i] = gain_early[i];
        } else {
          load_piece(a.gain + kPiece * c, a.wide_gain != 0, gw);
        }
        float g[16];
        unpack(gw, g);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * rs * g[i];
      }
    }
    uint32_t w[8];
    uint32_t scale = 0;
    if constexpr (FMT == MOE_MX_BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = abs_max(m, v[i]);
      if constexpr (Mx<FMT>::group == 32) m = abs_max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const GroupScale sc = group_scale<FMT>(m, factor);
      codes_of<FMT, 16>(v, sc, w);
      scale = sc.byte;
    }
    if (c >= np) continue;
    if constexpr (kEarly) {
#pragma unroll
      for (int j = 0; j < 8; ++j) store_codes<FMT>(a, at_early[j], c, w, scale);
      for (int j = 8; j < a.k; ++j) store_codes<FMT>(a, __ldcg(a.positions + t * a.k + j), c, w, scale);
    } else if (a.k == 1) {
      store_codes<FMT>(a, a.positions ? __ldcg(a.positions + t) : t, c, w, scale);
    } else {
      for (int j0 = 0; j0 < a.k; j0 += 4) {
        int32_t at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = j0 + j < a.k ? __ldcg(a.positions + t * a.k + j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) store_codes<FMT>(a, at[j], c, w, scale);
      }
    }
  }
}

bool aligned32(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && ld % 16 == 0; }

template <int FMT, bool NORM>
cudaError_t launch_rows(MxRowsLaunch a, cudaStream_t s) {
  const int np = a.d / kPiece;
  // Few rows: as many threads as the row has pieces, for the shortest way through one row.  More rows than
  // SMs: two pieces a thread, so that an SM holds more rows in different phases; and rows of up to 64 pieces
  // one to a warp, eight to a CTA (a CTA each, the launch of the CTAs bounded them: 32,768 rows to MXFP8
  // took 37 us at 128 columns as at 1024; so they take 14 and 22).  At 4096 columns two pieces a thread take 65 us
  // and one 74; the norm 141 and 164.
  const bool many = a.n > 2 * device_sms(), by_warp = many && np <= 64;
  int iters = 1;
  while (iters * (by_warp ? 32 : many ? kRowsSplitThreads : kRowsMaxThreads) < np) iters *= 2;
  if (many && !by_warp && iters == 1) iters = 2;
  const int threads = by_warp ? 256 : ((np + iters - 1) / iters + 31) / 32 * 32;
  const int64_t grid = by_warp ? (a.n + 7) / 8 : a.n;
  a.wide_x = aligned32(a.x, a.x_ld);
  a.wide_r = aligned32(a.residual, a.r_ld) && aligned32(a.sum, a.r_ld);
  a.wide_gain = aligned32(a.gain, 0);
  a.wide_out = aligned32(a.codes, 0);
  auto kern = by_warp      ? iters == 1 ? mx_rows_kernel<FMT, NORM, 1, true> : mx_rows_kernel<FMT, NORM, 2, true>
              : iters == 1 ? mx_rows_kernel<FMT, NORM, 1, false>
              : iters == 2 ? mx_rows_kernel<FMT, NORM, 2, false>
                           : mx_rows_kernel<FMT, NORM, 4, false>;
  return launch_maybe_overlapped(kern, static_cast<int>(grid), threads, 0, s, true, a);
}

// A CTA covers 1024 pieces, of as many rows as fit or of one row's part, four a
// thread: their loads are all under way before the first is used.
constexpr int kDeqPieces = 1024;

// magic: ceil(2^32 / np) for rows of np < 1024 pieces (i / np = umulhi(i, magic) for i < 1024).
template <int FMT>
__global__ void __launch_bounds__(256)
mx_dequantise_kernel(int64_t rows, int32_t d, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                     const float* __restrict__ global_p, uint16_t* __restrict__ out, int64_t out_ld, uint32_t magic,
                     int32_t segs, int32_t rpb, int32_t wide) {
  pdl_wait();
  pdl_launch_dependents();
  const int np = d / kPiece;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / segs) * rpb;
  const int c0 = static_cast<int>(blockIdx.x % segs) * kDeqPieces;
  const float global = FMT == MOE_MX_NVFP4 && global_p ? __ldg(global_p) : 1.f;
  constexpr int kWords = FMT == MOE_MX_BF16 ? 8 : FMT == MOE_MX_MXFP8 ? 4 : 2;
  int r[4], c[4];
  uint32_t w[4][kWords];
  uint32_t sb[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 256 * u + threadIdx.x;
    const int rl = np < kDeqPieces ? static_cast<int>(__umulhi(i, magic)) : 0;
    c[u] = np < kDeqPieces ? i - rl * np : c0 + i;
    r[u] = rl < rpb && c[u] < np && row0 + rl < rows ? rl : -1;
    if (r[u] >= 0) {
      const uint8_t* row = codes + (row0 + rl) * code_pitch<FMT>(d);
      if constexpr (FMT == MOE_MX_BF16) {
        load_piece(reinterpret_cast<const uint16_t*>(row) + kPiece * c[u], false, w[u]);
      } else if constexpr (FMT == MOE_MX_MXFP8) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(row) + c[u]);
        w[u][0] = q.x, w[u][1] = q.y, w[u][2] = q.z, w[u][3] = q.w;
      } else {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(row) + c[u]);
        w[u][0] = q.x, w[u][1] = q.y;
      }
      if constexpr (FMT != MOE_MX_BF16)
        sb[u] = __ldg(scales + (row0 + rl) * scale_pitch<FMT>(d) + c[u] / (Mx<FMT>::group / kPiece));
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (r[u] < 0) continue;
    uint32_t o[8];
    if constexpr (FMT == MOE_MX_BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = w[u][i];
    } else {
      float sc;
      if constexpr (FMT == MOE_MX_NVFP4) sc = e4m3_value(sb[u]) * global;
      else if (sb[u] == 255u) sc = __uint_as_float(0x7fc00000u);
      else sc = sb[u] == 0u ? 0x1p-127f : __uint_as_float(sb[u] << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        __half2 h;
        if constexpr (FMT == MOE_MX_MXFP8)
          h = __half2(__nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>((w[u][j >> 1] >> (16 * (j & 1))) & 0xffffu), __NV_E4M3));
        else
          h = __half2(__nv_cvt_fp4x2_to_halfraw2(
              static_cast<__nv_fp4x2_storage_t>((w[u][j >> 2] >> (8 * (j & 3))) & 0xffu), __NV_E2M1));
        o[j] = pack_bf16(__low2float(h) * sc, __high2float(h) * sc);
      }
    }
    store_piece(out + (row0 + r[u]) * out_ld + kPiece * c[u], wide != 0, o);
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
  const int np = d / kPiece;
  const int segs = (np + kDeqPieces - 1) / kDeqPieces, rpb = np < kDeqPieces ? kDeqPieces / np : 1;
  const uint32_t magic = np > 1 ? static_cast<uint32_t>(((1ull << 32) + np - 1) / np) : 0u;
  const int64_t blocks = (rows + rpb - 1) / rpb * segs;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kern = fmt == MOE_MX_BF16    ? mx_dequantise_kernel<MOE_MX_BF16>
              : fmt == MOE_MX_MXFP8 ? mx_dequantise_kernel<MOE_MX_MXFP8>
              : fmt == MOE_MX_MXFP4 ? mx_dequantise_kernel<MOE_MX_MXFP4>
                                    : mx_dequantise_kernel<MOE_MX_NVFP4>;
  return launch_maybe_overlapped(kern, static_cast<int>(blocks), 256, 0, s, true, rows, d, codes, scales, global, out,
                                 out_ld, magic, segs, rpb, static_cast<int>(aligned32(out, out_ld)));
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
