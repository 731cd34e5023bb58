// Products grouped by expert on e4m3 rows (a scale per 128 columns) and e4m3 weights (a
// scale per 128 x 128 block), moe_fp8.h:
//
//   D[r][n] = sum_b sx[r][b] sw[n / 128][b] sum_{c in block b} X[r][c] W[n][c]
//
// The tensor core sums the codes' products of one block of K (tcgen05.mma kind::f8f6f4, fp32
// accumulators); every block has a factor of its own for each row, so each block's sums
// are read from tensor memory and added to fp32 registers times that factor.
//
//  * Unit = a tile of up to 128 rows of one expert x NB blocks of 128 weight rows: M = 128,
//    N = 128 NB.  A chunk is one block of K: one bulk copy brings its weights, one TMA box
//    the tile's rows.
//  * Tensor memory holds 4 / NB chunks' sums, so that the MMAs of the next chunks run while
//    one is read.
//  * An epilogue thread owns a row and 64 weight rows of each block; a warp whose rows do not
//    exist only frees the buffers.
//
// Warps (384 threads, one CTA per SM, persistent over units):
//   0 weight copies   1 MMA issue   2 row copies   3 idle   4-11 epilogue
//
// Within an expert up to eight tiles run a weight block one after another, so that they
// take place at the same time and share it through L2.  Every wait is bounded (common.cuh);
// after one gives up all roles drain and the kernel ends.
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kMaxExperts = 1024;
constexpr int kChunkTiles = 8;
constexpr int kRowBytes = kTile * 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kWarpWeights = 0, kWarpIssue = 1, kWarpRows = 2, kWarpEpi = 4;
// Registers a thread after the split (the epilogue holds 64 NB accumulators): the launch's own
// number times its threads has to cover it.
constexpr int kRegsLow = 56, kRegsEpi = 224;
constexpr int kRegsLaunch = 128 * kRegsLow + 256 * kRegsEpi;

template <int NB>
struct Cfg {
  static constexpr int kStages = NB == 2 ? 4 : 6;
  static constexpr int kBuffers = 4 / NB;
  static constexpr int kWBytes = NB * 128 * 128;
  static constexpr int kStage = kWBytes + kRowBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 1;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kPlanOff = kBarOff + kNumBars * 8 + 16;  // tile prefix, warp sums
  static constexpr int kTurnOff = (kPlanOff + (kMaxExperts + 1) * 4 + 32 * 4 + 15) / 16 * 16;
  static constexpr int kTurn = 1024;  // an epilogue warp's
  static constexpr int kSmem = 1024 + kTurnOff + 8 * kTurn;
  static_assert(kStage % 1024 == 0, "operand tiles stay 1024-byte aligned");
  static_assert(kSmem <= 232448, "shared memory per CTA");
  static_assert(kBuffers * NB * 128 <= static_cast<int>(kTmemCols), "tensor memory");
};

struct Args {
  const uint8_t* packed;
  const float* w_scales;  // [E][nblocks][chunks]
  int32_t experts, n_out, upt, chunks, units256, nblocks;  // upt: units of a tile
  uint64_t upt_inv;
  int32_t rows;
  const float* x_scales;
  int32_t x_pitch;
  const int32_t* offsets;
  void* out;
  int32_t out_vec;
  int64_t out_rows, out_ld;
  const int32_t* out_pos;
  const float* row_weight;
  uint32_t* err;
};

// Rows' maps with boxes of 16, 32, 64 and 128 rows: a tile's copy brings its own rows and few others.
struct RowMaps {
  CUtensorMap box[4];
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&p)[32]) {
  tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(&p[0]));
  tmem_ld16(taddr + 16, *reinterpret_cast<uint32_t(*)[16]>(&p[16]));
}

// acc += f * p, two at a time (each rounded as fmaf's).
__device__ __forceinline__ void add_scaled(float2 (&acc)[16], const uint32_t (&p)[32], float f) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 v = make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<unsigned long long&>(acc[i]))
        : "l"(reinterpret_cast<const unsigned long long&>(v)), "l"(reinterpret_cast<const unsigned long long&>(ff)));
  }
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) return;
}

struct Unit {
  int e, row0, nv, u;
};

__device__ __forceinline__ int first_row(const Args& a, int e) {
  return a.offsets ? __ldg(a.offsets + e) : e == 0 ? 0 : a.rows;
}

// Unit number x.  Expert e's units are consecutive, T tiles x upt: its tiles in chunks of eight, weight block after
// weight block within a chunk, tile after tile within a weight block.
// (upt_inv: ceil(2^64 / upt), by which a 32-bit quotient is one multiplication.)
__device__ __forceinline__ Unit unit_of(const Args& a, const int32_t* first_tile, int x) {
  const int upt = a.upt;
  const int t = upt == 1 ? x : static_cast<int>(__umul64hi(static_cast<uint64_t>(x), a.upt_inv));
  int lo = 0, hi = a.experts;  // first_tile[lo] <= t < first_tile[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first_tile[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int l = x - first_tile[lo] * upt, tiles = first_tile[lo + 1] - first_tile[lo];
  const int chunk = tiles <= kChunkTiles ? 0 : l / (kChunkTiles * upt), in = l - chunk * kChunkTiles * upt;
  const int nc = min(kChunkTiles, tiles - chunk * kChunkTiles);
  const int u = nc == 1 ? in : in / nc, tile = chunk * kChunkTiles + in - u * nc;
  Unit un;
  un.e = lo;
  un.u = u;
  un.row0 = first_row(a, lo) + tile * kTile;
  un.nv = min(kTile, first_row(a, lo + 1) - un.row0);
  return un;
}

// Where a row's results go and how they are stored.
template <int OUT>
struct Out {
  static constexpr int kSize = OUT == MOE_FP8_OUT_F32 ? 4 : 2;
  static constexpr int kCols = 32 / kSize;  // columns of a 32-byte piece
  static __device__ __forceinline__ void piece(const float* v, uint32_t (&w)[8], float& top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (OUT == MOE_FP8_OUT_F32) {
        w[i] = __float_as_uint(v[i]);
      } else if constexpr (OUT == MOE_FP8_OUT_F16) {
        top = fmaxf(top, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};

// 64 columns from `at` on of this thread's row `to` (-1: none), times f; all lanes of a warp together.
template <int OUT>
__device__ __forceinline__ void store_columns(const Args& a, float2 (&acc)[32], float f, int to, int at, uint8_t* turn,
                                              float& top) {
  using O = Out<OUT>;
  const int lane = threadIdx.x & 31;
  uint8_t* base = static_cast<uint8_t*>(a.out);
  const int64_t pitch = a.out_ld * O::kSize;
  float* v = reinterpret_cast<float*>(acc);
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] *= f;
  float mine = 0.f;
  if (a.out_vec) {
    // Four lanes exchange their rows' four 32-byte pieces, so that a store covers whole 128-byte lines of eight rows
    // instead of a piece of each of 32.
    const int j = lane & 3;
    uint8_t* row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = __shfl_sync(kAll, to, (lane & ~3) + i);
      row[i] = r >= 0 ? base + r * pitch : nullptr;
    }
#pragma unroll
    for (int g = 0; g < 64 / (4 * O::kCols); ++g) {
      uint32_t w[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) O::piece(v + (4 * g + i) * O::kCols, w[i], mine);
#pragma unroll
      for (int step = 1; step <= 2; step *= 2) {
        const bool up = (lane & step) != 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (p & step) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t got = __shfl_xor_sync(kAll, up ? w[p][i] : w[p + step][i], step);
            if (up) w[p][i] = got;
            else w[p + step][i] = got;
          }
        }
      }
      const int col = at + (4 * g + j) * O::kCols;  // w[i]: these columns of the i-th row
      if (col + O::kCols <= a.n_out) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row[i]) stg256(row[i] + static_cast<int64_t>(col) * O::kSize, w[i]);
      } else if (col < a.n_out) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!row[i]) continue;
#pragma unroll
          for (int c = 0; c < O::kCols - 1; ++c) {
            if (col + c >= a.n_out) continue;
            if constexpr (O::kSize == 4) reinterpret_cast<uint32_t*>(row[i])[col + c] = w[i][c];
            else reinterpret_cast<uint16_t*>(row[i])[col + c] = static_cast<uint16_t>(w[i][c >> 1] >> (16 * (c & 1)));
          }
        }
      }
    }
  } else {
    // Rows that are not aligned: a piece of each of the 32 rows at a time, turned through shared memory so that
    // neighbouring lanes write one row's columns.
#pragma unroll
    for (int p = 0; p < 64 / O::kCols; ++p) {
      uint32_t w[8];
      O::piece(v + p * O::kCols, w, mine);
      const int col0 = at + p * O::kCols;
      if (col0 >= a.n_out) continue;
      __syncwarp();
      reinterpret_cast<uint4*>(turn)[2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(turn)[2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
      __syncwarp();
#pragma unroll 4
      for (int i = 0; i < O::kCols; ++i) {
        const int at_el = 32 * i + lane, col = col0 + at_el % O::kCols;
        const int r = __shfl_sync(kAll, to, at_el / O::kCols);
        if (r < 0 || col >= a.n_out) continue;
        if constexpr (O::kSize == 4)
          reinterpret_cast<uint32_t*>(base + r * pitch)[col] = reinterpret_cast<const uint32_t*>(turn)[at_el];
        else
          reinterpret_cast<uint16_t*>(base + r * pitch)[col] = reinterpret_cast<const uint16_t*>(turn)[at_el];
      }
    }
  }
  if (to >= 0) top = fmaxf(top, mine);
}

template <int NB, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
fp8_product_kernel(const __grid_constant__ RowMaps maps, const Args a) {
  using C = Cfg<NB>;
  constexpr int kStages = C::kStages, kBuffers = C::kBuffers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBarOff;
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (kStages + i); };
  auto acc_full = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
  auto acc_empty = [&](int i) { return bar0 + 8u * (2 * kStages + kBuffers + i); };
  const uint32_t drain_bar = bar0 + 8u * (C::kNumBars - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + C::kNumBars * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int32_t* first_tile = reinterpret_cast<int32_t*>(smem + C::kPlanOff);
  int32_t* warp_sum = first_tile + kMaxExperts + 1;

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 2);  // weights, rows
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), 8);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kWarpRows && lane < 4) prefetch_tmap(&maps.box[lane]);
  if (warp == kWarpIssue) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  // The tile plan: thread i counts the tiles of experts 4 i to 4 i + 3.
  {
    int n[4] = {0, 0, 0, 0};
    bool bad = false;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * threadIdx.x + j;
      if (e < a.experts) {
        const int lo = first_row(a, e), hi = first_row(a, e + 1);
        bad |= lo < 0 || hi < lo || hi > a.rows;
        n[j] = bad ? 0 : (hi - lo + kTile - 1) / kTile;
        mine += n[j];
      }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    bad = __syncthreads_or(bad);
    int at = __reduce_add_sync(kAll, lane < warp ? warp_sum[lane] : 0) + incl - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * threadIdx.x + j;
      at += n[j];
      if (e < a.experts) first_tile[e + 1] = bad ? 0 : at;
    }
    if (threadIdx.x == 0) first_tile[0] = 0;
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, DEV_ERR_ROUTING);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int chunks = a.chunks, total = first_tile[a.experts] * a.upt, stride = gridDim.x;

  if (warp < kWarpEpi) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == kWarpWeights) {
      if (lane == 0) {
        const uint64_t pol = policy_evict_normal();
        uint32_t it = 0;
        bool ok = true;
        for (int x = blockIdx.x; ok && x < total; x += stride) {
          const Unit un = unit_of(a, first_tile, x);
          const int blk = NB == 2 ? un.u : un.u >> 1;
          const uint8_t* src = a.packed + (static_cast<int64_t>(un.e) * a.units256 + blk) * chunks * kFp8Block +
                               (NB == 1 ? (un.u & 1) * (128 * 128) : 0);
          for (int c = 0; c < chunks; ++c, ++it) {
            const int s = it % kStages;
            if (!wait_bounded(empty(s), ((it / kStages) & 1) ^ 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(full(s), C::kWBytes);
            bulk_load(sbase + s * C::kStage, src + static_cast<int64_t>(c) * kFp8Block, C::kWBytes, full(s), pol);
          }
        }
        if (!ok)
          for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) wait_drain(full(i % kStages), (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == kWarpRows) {
      if (lane == 0) {
        const uint64_t pol = policy_evict_last();
        uint32_t it = 0;
        bool ok = true;
        for (int x = blockIdx.x; ok && x < total; x += stride) {
          const Unit un = unit_of(a, first_tile, x);
          const int b = un.nv <= 16 ? 0 : un.nv <= 32 ? 1 : un.nv <= 64 ? 2 : 3;
          const uint32_t bytes = (16u << b) * 128u;
          for (int c = 0; c < chunks; ++c, ++it) {
            const int s = it % kStages;
            if (!wait_bounded(empty(s), ((it / kStages) & 1) ^ 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(full(s), bytes);
            tma_load_2d(sbase + s * C::kStage + C::kWBytes, &maps.box[b], full(s), c * 128, un.row0, pol);
          }
        }
        if (!ok)
          for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) wait_drain(full(i % kStages), (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == kWarpIssue) {
      if (elect_one()) {
        // kind::f8f6f4 with e4m3 operands: format code 0, the same bits as f16
        constexpr uint32_t idesc = idesc_f16_f32(128, 128 * NB);
        uint32_t it = 0;
        bool ok = true;
        for (int x = blockIdx.x; ok && x < total; x += stride) {
          for (int c = 0; c < chunks; ++c, ++it) {
            const int s = it % kStages, b = it % kBuffers;
            if (!wait_bounded(acc_empty(b), ((it / kBuffers) & 1) ^ 1, abort_flag, a.err) ||
                !wait_bounded(full(s), (it / kStages) & 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t w = sbase + s * C::kStage;
            const uint64_t ad = desc_kmajor_sw128(w + C::kWBytes), bd = desc_kmajor_sw128(w);
            const uint32_t d = tmem + static_cast<uint32_t>(b) * (128 * NB);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f8(d, desc_advance(ad, 32 * kk), desc_advance(bd, 32 * kk), idesc, kk > 0);
            tc_commit(empty(s));
            tc_commit(acc_full(b));
          }
        }
        tc_commit(drain_bar);  // every MMA issued above has completed once this arrives
        wait_drain(drain_bar, 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const int q = warp & 3, hf = (warp - kWarpEpi) >> 2;
    const int tok = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint8_t* turn = smem + C::kTurnOff + (warp - kWarpEpi) * C::kTurn;
    uint32_t it = 0;
    bool ok = true;
    for (int x = blockIdx.x; ok && x < total; x += stride) {
      const Unit un = unit_of(a, first_tile, x);
      const bool any = q * 32 < un.nv, valid = tok < un.nv;
      const int64_t row = static_cast<int64_t>(un.row0) + tok;
      int to = -1;
      float f = 1.f;
      if (valid) {
        to = a.out_pos ? __ldg(a.out_pos + row) : static_cast<int>(row);
        if (to >= a.out_rows) to = -1;
        if (a.row_weight && to >= 0) f = __ldg(a.row_weight + to);
      }
      const float* xs = a.x_scales + row * a.x_pitch;
      const float* ws[NB];
#pragma unroll
      for (int m = 0; m < NB; ++m)
        ws[m] = a.w_scales + (static_cast<int64_t>(un.e) * a.nblocks + min(NB * un.u + m, a.nblocks - 1)) * chunks;
      float2 acc[NB][2][16];
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[m][i >> 4][i & 15] = make_float2(0.f, 0.f);
      // this chunk's factors; each iteration loads the next one's
      float sx = valid ? __ldg(xs) : 0.f, sw[NB];
#pragma unroll
      for (int m = 0; m < NB; ++m) sw[m] = __ldg(ws[m]);
      for (int c = 0; c < chunks; ++c, ++it) {
        const int b = it % kBuffers;
        float nsx = 0.f, nsw[NB] = {};
        if (c + 1 < chunks) {
          nsx = valid ? __ldg(xs + c + 1) : 0.f;
#pragma unroll
          for (int m = 0; m < NB; ++m) nsw[m] = __ldg(ws[m] + c + 1);
        }
        ok = __all_sync(kAll, wait_bounded(acc_full(b), (it / kBuffers) & 1, abort_flag, a.err));
        if (!ok) break;
        tc_fence_after();
        if (any) {
          const uint32_t tcol = tmem + lane_base + static_cast<uint32_t>(b) * (128 * NB) + 64 * hf;
          // 32 columns are read while the 32 before them are added
          uint32_t p[2][32];
          tmem_ld32(tcol, p[0]);
#pragma unroll
          for (int i = 0; i < 2 * NB; ++i) {
            tmem_ld_wait();
            if (i + 1 < 2 * NB) tmem_ld32(tcol + 128 * ((i + 1) >> 1) + 32 * ((i + 1) & 1), p[(i + 1) & 1]);
            if (i + 1 == 2 * NB) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(acc_empty(b));
            }
            add_scaled(acc[i >> 1][i & 1], p[i & 1], sw[i >> 1] * sx);
          }
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(b));
        }
        sx = nsx;
#pragma unroll
        for (int m = 0; m < NB; ++m) sw[m] = nsw[m];
      }
      if (!ok) break;
      if (!any) continue;
      float top = 0.f;  // largest magnitude, for f16's range
#pragma unroll
      for (int m = 0; m < NB; ++m) {
        const int at = 128 * (NB * un.u + m) + 64 * hf;
        if (at < a.n_out)
          store_columns<OUT>(a, reinterpret_cast<float2(&)[32]>(acc[m]), f, to, at, turn, top);
      }
      if (OUT == MOE_FP8_OUT_F16 && __any_sync(kAll, top >= 65520.f) && lane == 0) atomicOr(a.err, DEV_ERR_RANGE);
    }
  }
  __syncthreads();
  if (warp == kWarpIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int NB, int OUT>
cudaError_t launch(const Fp8ProductLaunch& g, cudaStream_t s) {
  using C = Cfg<NB>;
  auto kern = fp8_product_kernel<NB, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // An increase of the register split that cannot be met never returns: launch only if the kernel's own
  // count covers it (a property of the binary, looked up until it is known).
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) * kThreads < kRegsLaunch) return cudaErrorInvalidConfiguration;
  const moe_fp8_weights* w = g.w;
  Args a{};
  a.packed = static_cast<const uint8_t*>(w->packed);
  a.w_scales = w->scales;
  a.experts = w->num_experts;
  a.n_out = w->n_out;
  a.nblocks = static_cast<int32_t>(fp8_blocks(w->n_out));
  a.units256 = static_cast<int32_t>(fp8_units(w));
  a.upt = NB == 2 ? a.units256 : a.nblocks;
  a.upt_inv = a.upt > 1 ? ~0ull / static_cast<uint64_t>(a.upt) + 1 : 0ull;
  a.chunks = static_cast<int32_t>(fp8_blocks(w->k));
  a.rows = g.rows;
  a.x_scales = g.x_scales;
  a.x_pitch = static_cast<int32_t>(moe_fp8_scale_pitch(w->k));
  a.offsets = g.offsets;
  a.out = g.out;
  const int size = OUT == MOE_FP8_OUT_F32 ? 4 : 2;
  a.out_vec = reinterpret_cast<uintptr_t>(g.out) % 32 == 0 && g.out_ld * size % 32 == 0;
  a.out_rows = g.out_rows;
  a.out_ld = g.out_ld;
  a.out_pos = g.out_pos;
  a.row_weight = g.row_weight;
  a.err = g.err;
  RowMaps maps;
  for (int i = 0; i < 4; ++i)
    if (!encode_rows_map(&maps.box[i], g.x_codes, static_cast<uint64_t>(w->k), g.rows, 16u << i))
      return cudaErrorInvalidValue;
  // The most units there can be: an expert's last tile may be short.
  const int64_t tiles = static_cast<int64_t>(g.rows) / kTile + (g.rows < w->num_experts ? g.rows : w->num_experts);
  const int64_t units = tiles * a.upt;
  return launch_maybe_overlapped(kern, static_cast<int>(units < g.num_sms ? units : g.num_sms), kThreads, C::kSmem, s, true,
                                 maps, a);
}

template <int OUT>
cudaError_t launch_out(const Fp8ProductLaunch& g, cudaStream_t s) {
  return launch<2, OUT>(g, s);
}

}  // namespace

cudaError_t launch_fp8_product(const Fp8ProductLaunch& g, cudaStream_t s) {
  switch (g.out_type) {
    case MOE_FP8_OUT_BF16: return launch_out<MOE_FP8_OUT_BF16>(g, s);
    case MOE_FP8_OUT_F16: return launch_out<MOE_FP8_OUT_F16>(g, s);
    case MOE_FP8_OUT_F32: return launch_out<MOE_FP8_OUT_F32>(g, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
