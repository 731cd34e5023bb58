// Products grouped by expert on e4m3 rows (a scale per 128 columns) and e4m3 weights (a
// scale per 128 x 128 block), moe_fp8.h:
//
//   D[r][n] = sum_b sx[r][b] sw[n / 128][b] sum_{c in block b} X[r][c] W[n][c]
//
// The tensor core sums the codes' products of one block of K (tcgen05.mma kind::f8f6f4, fp32
// accumulators); every block has a factor of its own for each row, so each block's sums
// are read from tensor memory and added to fp32 registers times that factor.
//
//  * Unit = a tile of rows of one expert x blocks of 128 weight rows.  A chunk is one block of K:
//    one bulk copy brings its weights, one TMA box the tile's rows.  Four kinds:
//      few   32 rows x one block, the weights as the MMA's M = 128 and the rows as its N = 16 or
//            32: an epilogue thread has a weight row and 16 of the tile's
//      one   128 rows x one block, M = N = 128
//      two   128 rows x two blocks, N = 256
//      pair  256 rows x two blocks by a pair of CTAs (M = 256, tcgen05 cta_group::2): each brings
//            its own 128 rows and half of the weights, 32 KB a chunk instead of 48, and sums
//            its rows' part
//    An epilogue thread of the last three owns a row and 64 weight rows of each block; a warp
//    whose rows do not exist only frees the buffers.
//  * Tensor memory holds 2 to 8 chunks' sums, so that the MMAs of the next chunks run while one
//    is read.
//  * A warp of its own lays the chunks' factors out in shared memory, four chunks at a time:
//    the rows' scales times the weights'.  (Global loads in the epilogue, even four chunks
//    ahead, held up its reads of tensor memory.)
//
// Warps (384 threads, one CTA per SM, persistent over units):
//   0 weight copies   1 MMA issue   2 row copies   3 factors   4-11 epilogue
//
// What bounds the kernel where HBM does not is the way around a buffer of sums: the MMAs (512
// cycles at N = 256), the barrier's flip, the reads and the additions (the 64 packed FMAs of two
// warps take 280 cycles), the release, the next MMAs.  The MMAs' operands take most of shared
// memory's cycles, and whatever else goes there waits: a test of a barrier that is complete
// already takes 180 cycles beside MMAs of N = 128.  So barriers are tested ahead where that
// can be (the issuing thread's two together: one row of 7168 x 7168 20.0 -> 16.2 us), and
// nothing on that way may come from local memory: see `fresh`.  8192 x 7168 x 7168 on one
// GB300: 318 us in a row on one set of operands, 348 in turn with others (2.42 PFLOP/s), some
// 850 cycles a chunk (a loop of the same steps without units, 690).
//
// Within an expert up to eight tiles run a weight block one after another, so that they
// take place at the same time and share it through L2.  Every wait is bounded; after one
// gives up all roles drain and the kernel ends.
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kTile = 128;  // rows of a CTA's tile
constexpr int kMaxExperts = 1024;
constexpr int kChunkTiles = 8;
constexpr int kFewTile = 32;  // where few rows come
constexpr uint32_t kTmemCols = 512;
constexpr int kWarpWeights = 0, kWarpIssue = 1, kWarpRows = 2, kWarpScales = 3, kWarpEpi = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (kWarpEpi + kEpiWarps);
constexpr int kSlots = 4;  // groups of four chunks' factors
// Registers a thread after the split where the epilogue holds 128 sums: the launch's own number times its threads has to
// cover it.
constexpr int kRegsLow = 72, kRegsEpi = 216;
constexpr int kRegsLaunch = 32 * kWarpEpi * kRegsLow + 32 * kEpiWarps * kRegsEpi;

enum Kind { kOne, kTwo, kPair, kFew };

template <Kind KIND>
struct Cfg {
  static constexpr bool kIsPair = KIND == kPair, kIsFew = KIND == kFew;
  static constexpr int NB = KIND == kTwo || KIND == kPair ? 2 : 1;  // weight blocks of a unit
  static constexpr int kRows = kIsFew ? kFewTile : kTile;           // of this CTA's tile
  static constexpr int kTileRows = kIsPair ? 2 * kTile : kRows;
  static constexpr int kRowBytes = kRows * 128;
  static constexpr int kWBytes = (kIsPair ? 1 : NB) * 128 * 128;  // of this CTA
  static constexpr int kStage = kWBytes + kRowBytes;
  static constexpr int kStages = kIsFew ? 10 : KIND == kTwo ? 4 : 5;
  static constexpr int kColumns = kIsFew ? kFewTile : 128 * NB;  // of a buffer
  static constexpr int kBuffers = kIsFew ? 8 : 4 / NB;
  static constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 2 * kSlots + 1;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kSlotOff = kBarOff + kNumBars * 8;  // tensor memory's address, the abort flag
  static constexpr int kPlanOff = kSlotOff + 16;  // tile prefix, warp sums
  static constexpr int kTurnOff = (kPlanOff + (kMaxExperts + 1) * 4 + 32 * 4 + 15) / 16 * 16;
  static constexpr int kTurn = 1024;  // an epilogue warp's
  // a group's factors: four chunks' of each row and block
  static constexpr int kScaleOff = kTurnOff + kEpiWarps * kTurn;
  static constexpr int kScales = NB * kRows * 16;
  static constexpr int kSmem = 1024 + kScaleOff + kSlots * kScales;
  static_assert(kStage % 1024 == 0, "operand tiles stay 1024-byte aligned");
  static_assert(kSmem <= 232448, "shared memory per CTA");
  static_assert(kBuffers * kColumns <= static_cast<int>(kTmemCols), "tensor memory");
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

// Rows' maps with boxes of 16, 32, 64 and 128 rows: a tile's copy brings its own rows and few others.  (A pair takes
// whole boxes, and its weights through a map too, of the packed buffer as rows of 128 bytes.)
struct Maps {
  CUtensorMap box[4];
  CUtensorMap weights;
};

template <bool PAIR>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
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

// ---------------------------------------------------------------- a pair of CTAs
__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address in the pair's first CTA, which issues the MMAs, of what is at `addr` here.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// (Relaxed: what it orders is reads of tensor memory, complete and fenced by tcgen05.fence; as a release it cost a
// membar a chunk and warp, 1500 of 2300 cycles.)
__device__ __forceinline__ void leader_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
// A box to this CTA's memory, its bytes counted by the leader's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}
// tc_commit; of a pair to the barriers at this place in both CTAs.
template <bool PAIR>
__device__ __forceinline__ void commit_to(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}
// acc += f * p, two at a time (each rounded as fmaf's).
__device__ __forceinline__ void add_scaled(float2 (&acc)[8], const uint32_t (&p)[16], float f) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<unsigned long long&>(acc[i]))
        : "l"(reinterpret_cast<const unsigned long long&>(v)), "l"(reinterpret_cast<const unsigned long long&>(ff)));
  }
}

// acc += f * p
__device__ __forceinline__ void add_product(float2& acc, uint32_t p0, uint32_t p1, uint32_t f0, uint32_t f1) {
  asm("{\n\t.reg .b64 p, f;\n\tmov.b64 p, {%1, %2};\n\tmov.b64 f, {%3, %4};\n\tfma.rn.f32x2 %0, p, f, %0;\n\t}"
      : "+l"(reinterpret_cast<unsigned long long&>(acc))
      : "r"(p0), "r"(p1), "r"(f0), "r"(f1));
}

// wait_bounded with a shorter way through: the clock (of the GPU, in 2^20 ns) is looked at every 1024 tries, and the wait
// gives up about a second after the first look.
__device__ __forceinline__ uint32_t millis() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return static_cast<uint32_t>(t >> 20);
}
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* err) {
  uint32_t tries = 0, since = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if ((++tries & 1023u) != 0) continue;
    if (*abort_flag) return false;
    if (tries == 1024u) {
      since = millis();
    } else if (millis() - since > 1000u) {
      *abort_flag = 1u;
      atomicOr(err, DEV_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// A copy that the compiler takes for another value.  Values of the whole kernel that the epilogue has no registers for
// are put into local memory, for every role: the thread that issues the MMAs then reloaded them chunk for chunk, 290 of
// 1010 cycles.  With copies of its own a role's loop is in registers.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ int fresh(int v) { return static_cast<int>(fresh(static_cast<uint32_t>(v))); }
template <typename T>
__device__ __forceinline__ T* fresh(T* v) {
  T* r;
  asm volatile("mov.b64 %0, %1;" : "=l"(r) : "l"(v));
  return r;
}
// Whether a phase is complete; does not wait for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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
// TILE: rows of a tile, ROWS of them a CTA's (a pair's second CTA has the second half).
template <int TILE, int ROWS>
__device__ __forceinline__ Unit unit_of(const Args& a, const int32_t* first_tile, int x, int rank) {
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
  un.row0 = first_row(a, lo) + tile * TILE + rank * ROWS;
  un.nv = min(ROWS, first_row(a, lo + 1) - un.row0);  // (not above 0: no rows)
  return un;
}

// What every role of a CTA works with.
template <Kind KIND>
struct Role {
  using C = Cfg<KIND>;
  uint8_t* smem;
  uint32_t* err;
  uint32_t base, tmem;  // shared and tensor memory
  int rank;             // of a pair's CTAs
  int chunks, total, first, stride;  // of a unit; units, and this CTA's
  // A role's own copy: see the function `fresh`.
  __device__ __forceinline__ Role fresh() const {
    Role r;
    r.smem = moe::fresh(smem);
    r.err = moe::fresh(err);
    r.base = moe::fresh(base);
    r.tmem = moe::fresh(tmem);
    r.rank = moe::fresh(rank);
    r.chunks = moe::fresh(chunks);
    r.total = moe::fresh(total);
    r.first = moe::fresh(first);
    r.stride = moe::fresh(stride);
    return r;
  }
  __device__ __forceinline__ uint32_t bar(int i) const { return base + C::kBarOff + 8u * i; }
  __device__ __forceinline__ uint32_t full(int i) const { return bar(i); }  // a pair's: in the leader
  __device__ __forceinline__ uint32_t empty(int i) const { return bar(C::kStages + i); }
  __device__ __forceinline__ uint32_t acc_full(int i) const { return bar(2 * C::kStages + i); }
  __device__ __forceinline__ uint32_t acc_empty(int i) const { return bar(2 * C::kStages + C::kBuffers + i); }  // likewise
  __device__ __forceinline__ uint32_t scales_full(int i) const { return bar(2 * C::kStages + 2 * C::kBuffers + i); }
  __device__ __forceinline__ uint32_t scales_empty(int i) const {
    return bar(2 * C::kStages + 2 * C::kBuffers + kSlots + i);
  }
  __device__ __forceinline__ uint32_t drain() const { return bar(C::kNumBars - 1); }
  __device__ __forceinline__ bool wait(uint32_t at, uint32_t parity) const {
    return wait_on(at, parity, reinterpret_cast<volatile uint32_t*>(smem + C::kSlotOff) + 1, err);
  }
  __device__ __forceinline__ Unit unit(const Args& a, int x) const {
    return unit_of<C::kTileRows, C::kRows>(a, reinterpret_cast<const int32_t*>(smem + C::kPlanOff), x, rank);
  }
};

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

template <Kind KIND, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
fp8_product_kernel(const __grid_constant__ Maps maps, const Args a) {
  using C = Cfg<KIND>;
  constexpr int NB = C::NB, kStages = C::kStages, kBuffers = C::kBuffers, kTileRows = C::kTileRows;
  constexpr bool PAIR = C::kIsPair, FEW = C::kIsFew;
  extern __shared__ uint8_t smem_raw[];
  Role<KIND> r0;
  r0.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  r0.base = smem_u32(r0.smem);
  r0.err = a.err;
  int32_t* first_tile = reinterpret_cast<int32_t*>(r0.smem + C::kPlanOff);
  int32_t* warp_sum = first_tile + kMaxExperts + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(r0.smem + C::kSlotOff);

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  r0.rank = PAIR ? static_cast<int>(pair_rank()) : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(r0.full(i), 2);  // weights, rows
      mbar_init(r0.empty(i), 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(r0.acc_full(i), 1);
      mbar_init(r0.acc_empty(i), PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(r0.scales_full(i), 1);
      mbar_init(r0.scales_empty(i), kEpiWarps);
    }
    mbar_init(r0.drain(), 1);
    tmem_slot[1] = 0u;  // the abort flag
    fence_mbar_init();
  }
  if (warp == kWarpRows && lane < 4) prefetch_tmap(&maps.box[lane]);
  if (PAIR && warp == kWarpWeights && lane == 0) prefetch_tmap(&maps.weights);
  if (warp == kWarpIssue) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish();
    }
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
        n[j] = bad ? 0 : (hi - lo + kTileRows - 1) / kTileRows;
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
  if constexpr (PAIR) pair_sync();  // the other CTA's barriers are initialised
  tc_fence_after();
  r0.tmem = *tmem_slot;
  r0.chunks = a.chunks;
  r0.total = first_tile[a.experts] * a.upt;
  r0.first = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  r0.stride = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp < kWarpEpi) {
    if constexpr (NB == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == kWarpWeights) {
      const auto r = r0.fresh();
      if (lane == 0) {
        const uint64_t pol = policy_evict_normal();
        uint32_t it = 0;
        bool ok = true;
        for (int x = r.first; ok && x < r.total; x += r.stride) {
          const Unit un = r.unit(a, x);
          const int blk = NB == 2 ? un.u : un.u >> 1;
          const int64_t block0 = (static_cast<int64_t>(un.e) * a.units256 + blk) * r.chunks;
          const uint8_t* src = a.packed + block0 * kFp8Block + (NB == 1 ? (un.u & 1) * (128 * 128) : 0);
          for (int c = 0; c < r.chunks; ++c, ++it) {
            const int s = it % kStages;
            if (!r.wait(r.empty(s), ((it / kStages) & 1) ^ 1)) {
              ok = false;
              break;
            }
            if constexpr (PAIR) {
              if (r.rank == 0) mbar_arrive_expect_tx(r.full(s), 2 * C::kWBytes);
              tma_load_pair(r.base + s * C::kStage, &maps.weights, leader_addr(r.full(s)), 0,
                            static_cast<int32_t>((block0 + c) * kFp8UnitRows) + 128 * r.rank, pol);
            } else {
              mbar_arrive_expect_tx(r.full(s), C::kWBytes);
              bulk_load(r.base + s * C::kStage, src + static_cast<int64_t>(c) * kFp8Block, C::kWBytes, r.full(s), pol);
            }
          }
        }
        if (!ok && r.rank == 0)
          for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) wait_drain(r.full(i % kStages), (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == kWarpRows) {
      const auto r = r0.fresh();
      if (lane == 0) {
        const uint64_t pol = policy_evict_last();
        uint32_t it = 0;
        bool ok = true;
        for (int x = r.first; ok && x < r.total; x += r.stride) {
          const Unit un = r.unit(a, x);
          const int b = PAIR ? 3 : un.nv <= 16 ? 0 : un.nv <= 32 ? 1 : un.nv <= 64 ? 2 : 3;
          const uint32_t bytes = (16u << b) * 128u;
          for (int c = 0; c < r.chunks; ++c, ++it) {
            const int s = it % kStages;
            if (!r.wait(r.empty(s), ((it / kStages) & 1) ^ 1)) {
              ok = false;
              break;
            }
            if constexpr (PAIR) {
              if (r.rank == 0) mbar_arrive_expect_tx(r.full(s), 2 * bytes);
              tma_load_pair(r.base + s * C::kStage + C::kWBytes, &maps.box[3], leader_addr(r.full(s)), c * 128, un.row0, pol);
            } else {
              mbar_arrive_expect_tx(r.full(s), bytes);
              tma_load_2d(r.base + s * C::kStage + C::kWBytes, &maps.box[b], r.full(s), c * 128, un.row0, pol);
            }
          }
        }
        if (!ok && r.rank == 0)
          for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) wait_drain(r.full(i % kStages), (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == kWarpIssue && r0.rank == 0) {
      if (elect_one()) {
        const auto r = r0.fresh();
        // kind::f8f6f4 with e4m3 operands: format code 0, the same bits as f16
        uint32_t idesc = idesc_f16_f32(FEW ? 128 : kTileRows, C::kColumns);
        uint32_t s = 0, sp = 0, b = 0, bp = 1;
        bool ok = true, there = false, empty = false;
        for (int x = r.first; ok && x < r.total; x += r.stride) {
          if constexpr (FEW) idesc = idesc_f16_f32(128, r.unit(a, x).nv <= 16 ? 16 : 32);
          for (int c = 0; c < r.chunks; ++c) {
            const uint32_t w = r.base + s * C::kStage;
            const uint64_t rows = desc_kmajor_sw128(w + C::kWBytes), weights = desc_kmajor_sw128(w);
            const uint64_t ad = FEW ? weights : rows, bd = FEW ? rows : weights;
            const uint32_t d = r.tmem + b * C::kColumns;
            if ((!there && !r.wait(r.full(s), sp)) || (!empty && !r.wait(r.acc_empty(b), bp))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8<PAIR>(d, desc_advance(ad, 32 * kk), desc_advance(bd, 32 * kk), idesc, kk > 0);
            commit_to<PAIR>(r.acc_full(b));
            commit_to<PAIR>(r.empty(s));
            if (++s == kStages) s = 0, sp ^= 1;
            if (++b == kBuffers) b = 0, bp ^= 1;
            // looked at ahead, so that one answer does not wait for the other (of two buffers none is free so early)
            there = mbar_test(r.full(s), sp);
            if constexpr (kBuffers > 2) empty = mbar_test(r.acc_empty(b), bp);
          }
        }
        // every MMA issued above has completed once this arrives
        if constexpr (PAIR)
          asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(r.drain())
                       : "memory");
        else
          tc_commit(r.drain());
        wait_drain(r.drain(), 0);
      }
      __syncwarp();
    } else if (warp == kWarpScales) {
      const auto r = r0.fresh();
      // Rows lane, lane + 32, ..: four chunks of each at a time, read a group ahead.
      uint32_t g = 0;
      bool ok = true;
      for (int x = r.first; ok && x < r.total; x += r.stride) {
        const Unit un = r.unit(a, x);
        const float* ws = a.w_scales + (static_cast<int64_t>(un.e) * a.nblocks + NB * un.u) * r.chunks;
        const int other = NB == 2 && 2 * un.u + 1 < a.nblocks ? r.chunks : 0;  // to the second block's
        constexpr int kMine = C::kRows / 32;
        float4 next[kMine];
        float next_w[NB][4];
        auto read = [&](int c0) {
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (32 * i + lane < un.nv && c0 < r.chunks)
              next[i] = __ldg(reinterpret_cast<const float4*>(
                                  a.x_scales + (static_cast<int64_t>(un.row0) + 32 * i + lane) * a.x_pitch) + (c0 >> 2));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int m = 0; m < NB; ++m) next_w[m][i] = c0 + i < r.chunks ? __ldg(ws + m * other + c0 + i) : 0.f;
          }
        };
        read(0);
        for (int c0 = 0; c0 < r.chunks; c0 += 4, ++g) {
          const int s = g % kSlots;
          ok = __all_sync(kAll, r.wait(r.scales_empty(s), ((g / kSlots) & 1) ^ 1));
          if (!ok) break;
          float4* to = reinterpret_cast<float4*>(r.smem + C::kScaleOff + s * C::kScales);
          if constexpr (FEW) {  // of each chunk all rows' together
            float* at = reinterpret_cast<float*>(to) + lane;
            at[0] = next_w[0][0] * next[0].x, at[32] = next_w[0][1] * next[0].y;
            at[64] = next_w[0][2] * next[0].z, at[96] = next_w[0][3] * next[0].w;
          } else {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
#pragma unroll
              for (int m = 0; m < NB; ++m)
                to[kTile * m + 32 * i + lane] = make_float4(next_w[m][0] * next[i].x, next_w[m][1] * next[i].y,
                                                           next_w[m][2] * next[i].z, next_w[m][3] * next[i].w);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(r.scales_full(s));
          read(c0 + 4);
        }
      }
    }
  } else {
    if constexpr (NB == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const auto r = r0.fresh();
    // lane quarter; half of each block's columns
    const int q = warp & 3, hf = (warp - kWarpEpi) >> 2;
    const int tok = q * 32 + lane;
    const uint32_t tcol0 = r.tmem + (static_cast<uint32_t>(q * 32) << 16) + (FEW ? 16u : 64u) * hf;
    uint8_t* turn = r.smem + C::kTurnOff + (warp - kWarpEpi) * C::kTurn;
    uint32_t it = 0, g = 0;
    bool ok = true, there = false, scales_there = false;
    auto release = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) leader_arrive(r.acc_empty(b));
        else mbar_arrive(r.acc_empty(b));
      }
    };
    if constexpr (FEW) {
      // Lanes are weight rows here, columns the tile's rows: the first 16 of them of warps 4 to 7, the others of 8 to 11.
      for (int x = r.first; ok && x < r.total; x += r.stride) {
        const Unit un = r.unit(a, x);
        const bool any = 16 * hf < un.nv;
        float2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c0 = 0; c0 < r.chunks; c0 += 4, ++g) {
          if (!__all_sync(kAll, scales_there)) {
            ok = __all_sync(kAll, r.wait(r.scales_full(g % kSlots), (g / kSlots) & 1));
            if (!ok) break;
          }
          const uint32_t from = r.base + C::kScaleOff + (g % kSlots) * C::kScales + 64 * hf;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (c0 + j >= r.chunks) break;
            uint4 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = lds128(from + 128 * j + 16 * i);
            const int b = it % kBuffers;
            if (!__all_sync(kAll, there)) {
              ok = __all_sync(kAll, r.wait(r.acc_full(b), (it / kBuffers) & 1));
              if (!ok) break;
            }
            ++it;
            tc_fence_after();
            uint32_t p[16];
            if (any) {
              tmem_ld16(tcol0 + static_cast<uint32_t>(b) * C::kColumns, p);
              tmem_ld_wait();
            }
            release(b);
            there = mbar_test(r.acc_full(it % kBuffers), (it / kBuffers) & 1);
            if (j == 3 || c0 + j + 1 >= r.chunks)
              scales_there = mbar_test(r.scales_full((g + 1) % kSlots), ((g + 1) / kSlots) & 1);
            if (any) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                add_product(acc[2 * i], p[4 * i], p[4 * i + 1], f[i].x, f[i].y);
                add_product(acc[2 * i + 1], p[4 * i + 2], p[4 * i + 3], f[i].z, f[i].w);
              }
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(r.scales_empty(g % kSlots));
        }
        if (!ok) break;
        if (!any) continue;
        // of row 16 hf + lane
        int to = -1;
        float f = 1.f;
        if (lane < 16 && 16 * hf + lane < un.nv) {
          const int64_t row = static_cast<int64_t>(un.row0) + 16 * hf + lane;
          to = a.out_pos ? __ldg(a.out_pos + row) : static_cast<int>(row);
          if (to >= a.out_rows) to = -1;
          if (a.row_weight && to >= 0) f = __ldg(a.row_weight + to);
        }
        const int n = 128 * un.u + tok;  // this lane's weight row
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = __shfl_sync(kAll, to, i);
          const float v = (i & 1 ? acc[i >> 1].y : acc[i >> 1].x) * __shfl_sync(kAll, f, i);
          if (t < 0 || n >= a.n_out) continue;
          const int64_t at = t * a.out_ld + n;
          if constexpr (OUT == MOE_FP8_OUT_F32) {
            static_cast<float*>(a.out)[at] = v;
          } else if constexpr (OUT == MOE_FP8_OUT_F16) {
            top = fmaxf(top, fabsf(v));
            static_cast<__half*>(a.out)[at] = __float2half_rn(v);
          } else {
            static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
          }
        }
        if (OUT == MOE_FP8_OUT_F16 && __any_sync(kAll, top >= 65520.f) && lane == 0) atomicOr(r.err, DEV_ERR_RANGE);
      }
    } else {
      for (int x = r.first; ok && x < r.total; x += r.stride) {
        const Unit un = r.unit(a, x);
        const bool any = q * 32 < un.nv, valid = tok < un.nv;
        const int64_t row = static_cast<int64_t>(un.row0) + tok;
        float2 acc[NB][4][8];
#pragma unroll
        for (int m = 0; m < NB; ++m)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[m][i >> 3][i & 7] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c0 = 0; c0 < r.chunks; c0 += 4, ++g) {
          if (!__all_sync(kAll, scales_there)) {
            ok = __all_sync(kAll, r.wait(r.scales_full(g % kSlots), (g / kSlots) & 1));
            if (!ok) break;
          }
          const uint32_t from = r.base + C::kScaleOff + (g % kSlots) * C::kScales;
          float factor[NB][4];
#pragma unroll
          for (int m = 0; m < NB; ++m) {
            const uint4 w = lds128(from + 16 * (kTile * m + tok));
            factor[m][0] = __uint_as_float(w.x), factor[m][1] = __uint_as_float(w.y), factor[m][2] = __uint_as_float(w.z),
            factor[m][3] = __uint_as_float(w.w);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (c0 + j >= r.chunks) break;
            const int b = it % kBuffers;
            if (!__all_sync(kAll, there)) {
              ok = __all_sync(kAll, r.wait(r.acc_full(b), (it / kBuffers) & 1));
              if (!ok) break;
            }
            ++it;
            tc_fence_after();
            if (any) {
              const uint32_t tcol = tcol0 + static_cast<uint32_t>(b) * (128 * NB);
              constexpr int kPieces = 4 * NB;
              // 16 columns are read while the 16 before them are added
              uint32_t p[2][16];
              tmem_ld16(tcol, p[0]);
#pragma unroll
              for (int i = 0; i < kPieces; ++i) {
                tmem_ld_wait();
                if (i + 1 < kPieces) {
                  tmem_ld16(tcol + 128 * ((i + 1) >> 2) + 16 * ((i + 1) & 3), p[(i + 1) & 1]);
                } else {
                  release(b);
                  there = mbar_test(r.acc_full(it % kBuffers), (it / kBuffers) & 1);
                  if (j == 3 || c0 + j + 1 >= r.chunks)
                    scales_there = mbar_test(r.scales_full((g + 1) % kSlots), ((g + 1) / kSlots) & 1);
                }
                add_scaled(acc[i >> 2][i & 3], p[i & 1], factor[i >> 2][j]);
              }
            } else {
              release(b);
              there = scales_there = false;
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(r.scales_empty(g % kSlots));
        }
        if (!ok) break;
        if (!any) continue;
        int to = -1;
        float f = 1.f;
        if (valid) {
          to = a.out_pos ? __ldg(a.out_pos + row) : static_cast<int>(row);
          if (to >= a.out_rows) to = -1;
          if (a.row_weight && to >= 0) f = __ldg(a.row_weight + to);
        }
        float top = 0.f;  // largest magnitude, for f16's range
#pragma unroll
        for (int m = 0; m < NB; ++m) {
          const int at = 128 * (NB * un.u + m) + 64 * hf;
          if (at < a.n_out) store_columns<OUT>(a, reinterpret_cast<float2(&)[32]>(acc[m]), f, to, at, turn, top);
        }
        if (OUT == MOE_FP8_OUT_F16 && __any_sync(kAll, top >= 65520.f) && lane == 0) atomicOr(r.err, DEV_ERR_RANGE);
      }
    }
  }
  __syncthreads();
  if constexpr (PAIR) pair_sync();  // neither CTA's memory goes while the other may still use it
  if (warp == kWarpIssue) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(r0.tmem), "r"(kTmemCols) : "memory");
    else
      tmem_dealloc(r0.tmem, kTmemCols);
  }
  if constexpr (PAIR) pair_sync();
}

template <Kind KIND, int OUT>
cudaError_t launch(const Fp8ProductLaunch& g, cudaStream_t s) {
  using C = Cfg<KIND>;
  constexpr int NB = C::NB;
  constexpr bool PAIR = C::kIsPair;
  auto kern = fp8_product_kernel<KIND, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if constexpr (NB == 2) {
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
  }
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
  Maps maps{};
  for (int i = 0; i < 4; ++i)
    if (!encode_rows_map(&maps.box[i], g.x_codes, static_cast<uint64_t>(w->k), g.rows, 16u << i))
      return cudaErrorInvalidValue;
  if (PAIR && !encode_dense_map(&maps.weights, w->packed, moe_fp8_packed_bytes(w) / 128)) return cudaErrorInvalidValue;
  // The most units there can be: an expert's last tile may be short.
  const int64_t tiles = static_cast<int64_t>(g.rows) / C::kTileRows + (g.rows < w->num_experts ? g.rows : w->num_experts);
  const int64_t units = tiles * a.upt, most = PAIR ? g.num_sms / 2 : g.num_sms, at_once = units < most ? units : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? 2 * at_once : at_once));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

// Which of the four kinds: the one with the least estimate of its time, in units of 25 ns: rounds of units over the SMs
// (the pairs) x chunks x the time of a chunk measured (300 ns with one block, 500 with two, 475 of a pair, and a pair's
// 0.8 us more to start), the experts' last tiles being half full where the rows are not known to the host.  Where weights
// are read for few rows each, a chunk's time is that of its bytes: 375 ns with one block, a little more by tiles of 128
// rows than by those of 32, and 700 with two.  Measured, in us on one GB300 (rows x n_out x k: few | one | two | pair):
//   1 x 7168 x 7168: 16.2 | 18.2 | 26.7 | 32.6             256: 41.8 | 20.1 | 29.2 | 30.5      512: 80 | 35.5 | 31.4 | 31.3
//   1024 x 7168 x 7168: 155 | 52.2 | 57.4 | 57.5           2048: 305 | 102 | 85.8 | 83.5       8192: 1187 | 393 | 330 | 317
//   64 experts x 2048 x 2048, 8 rows each: 45.0 | 47.4 | 51.3 | 68.5     64: 79 | 50.1 | 55.6 | 72.6     1024: 967 | 332 | 287 | 302
//   256 experts x 4096 x 7168, 16 rows each: 1064 | 1080 | 1034 | 1386   32 experts, 2048 each: 5565 | 1784 | 1530 | 1499
// Who has the rows is not known here.  Where one expert has them all, tiles of 32 rows are the wrong ones: 1024 rows of 64
// experts x 2048 x 2048 take 60 us evenly, 27 all of one expert, which by itself takes 15 (32 experts x 4096 x 7168, 512
// rows: 163, 60, 25; all but one row each: 72 and 191).
template <int OUT>
cudaError_t launch_out(const Fp8ProductLaunch& g, cudaStream_t s) {
  const int64_t experts = g.rows < g.w->num_experts ? g.rows : g.w->num_experts, k = fp8_blocks(g.w->k);
  const auto rounds = [&](int64_t tile, int64_t units, int64_t at_once) {
    const int64_t half_full = (g.rows + tile / 2 * (experts - 1) + tile - 1) / tile;
    return ((half_full > experts ? half_full : experts) * units + at_once - 1) / at_once;
  };
  const int64_t sms = g.num_sms, blocks = fp8_blocks(g.w->n_out), units = fp8_units(g.w);
  const int64_t one = rounds(kTile, blocks, sms), two = rounds(kTile, units, sms);
  if (g.rows <= 64 * experts) {
    const int64_t few = rounds(kFewTile, blocks, sms);
    if (few * 15 < one * 16 && few * 15 < two * 28) return launch<kFew, OUT>(g, s);
    return one * 16 <= two * 28 ? launch<kOne, OUT>(g, s) : launch<kTwo, OUT>(g, s);
  }
  const int64_t pair = rounds(2 * kTile, units, sms / 2) * k * 19 + 30;
  const bool mapped = moe_fp8_packed_bytes(g.w) / 128 <= 0x7fffffffu;  // a map's rows are counted in 32 bits
  if (mapped && pair < one * k * 12 && pair < two * k * 20) return launch<kPair, OUT>(g, s);
  return one * 12 <= two * 20 ? launch<kOne, OUT>(g, s) : launch<kTwo, OUT>(g, s);
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
