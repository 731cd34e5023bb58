// Products grouped by expert on microscaled operands (moe_mx.h).
//
//   D[r][n] = sum_k X[r][k] W_e[n][k],  X = codes * scales, W = codes * scales
//
// The tensor core multiplies the codes and applies both operands' scales inside
// the product (tcgen05.mma block_scale, fp32 accumulators), so nothing is widened
// on chip: a byte of weights read from HBM is a byte the tensor core consumes.
//
//  * Unit = a tile of up to 128 rows of one expert x one packed block row (256
//    weight rows, or 128 gate + 128 up): M = 128 rows, N = 256.  Rows are the M
//    side whatever their number: padding one token to 128 costs tensor time only,
//    and at these rates (the four MMAs of a 32 KB weight block: 590 to 690 cycles
//    with their scales' copies) less than half of what its bytes take from HBM.
//  * A chunk is 128 bytes of codes along K: one bulk copy brings the packed weight
//    block with its scales (33 to 36 KB), one TMA box the tile's rows.  Four stages.
//  * Scales go from shared to tensor memory by tcgen05.cp.  The packed weights hold
//    theirs in the order it wants; a tile's row scales start at any row, so warps 4-7
//    read them from global memory, 32 rows each and four chunks ahead, and lay them out
//    in the stage.  (With each warp storing all 128 rows to its own quarter of tensor
//    memory the same loads ran four times, and bounded a dense product: NVFP4 8192 x
//    7168 x 7168 203 us against 164 us without them.)  Each stage has its own scale
//    columns, so a stage's barriers cover them.
//  * One accumulator of 256 columns beside the scales (bf16: two, no scales).  For rows
//    out the epilogue empties it into registers, 128 columns a thread, and releases it
//    before it computes, so the next unit's products wait for the read alone; for SwiGLU
//    it takes 32 features at a time and releases it with the second half's read.
//  * An epilogue thread owns a row and 64 + 64 weight rows: gate and up of the same
//    64 features, whose groups of 16 or 32 lie within the thread.
//
// Warps (512 threads, one CTA per SM, persistent over units):
//   0 weight copies   1 MMA issue   2 row copies   3 idle   4-7 row scales   8-15 epilogue
// Measured on one GB300: the down projection of 32,768 K2 rows over 384 experts (MXFP4) 489
// us (its bytes at the rate of a plain copy: 517); dense 8192 x 7168 x 7168 NVFP4 5.0,
// MXFP4 5.4, MXFP8 3.0, bf16 1.7 PFLOP/s, bounded by the 50 to 55 KB that a chunk brings
// from L2 (about 55 bytes a cycle and SM; bf16 by the MMAs).
//
// Few units with a long K leave most SMs idle, and each of the others bound by the latency
// of its own four stages.  Then a cluster of 2, 4 or 8 CTAs takes one unit, each a part of
// K; every CTA finishes a slice of the columns, for which the others write their partial
// sums into its stage memory (added in the CTAs' order, so the result does not depend on
// which is first).  One expert, K 7168: NVFP4 4096 outputs, 16 rows 14.2 -> 9.9 us, bf16 512
// outputs, 100 rows 36 -> 14 us.
//
// Within an expert up to eight tiles run a weight block one after another, so that
// they take place at the same time and share it through L2.  Every wait is bounded
// (common.cuh); after one gives up all roles drain and the kernel ends.
#include <atomic>

#include "mx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kStages = 4;
constexpr int kTile = 128;
constexpr int kMaxExperts = 1024;
constexpr int kChunkTiles = 8;
// Chunks of a CTA from which units go to clusters.  Without / with them, us, one expert, weights that no call before has
// read, by K: NVFP4 4096 outputs, 16 rows: 3584 (seven chunks a CTA of two) 9.3 / 9.4, 4096 10.0 / 9.7, 5120 11.4 /
// 10.5, 7168 (seven of four) 14.3 / 10.1; MXFP8: 1536 (six of two) 8.4 / 9.0, 2048 9.7 / 9.6, 3584 (seven of four) 13.8 /
// 10.0; bf16 2048 outputs: 1024 (eight of two) 9.2 / 9.1, 2048 (eight of four) 14.4 / 9.2, 7168 (14 of eight) 40 / 12.4;
// 512 outputs, 100 rows: 1024 (eight of two) 8.5 / 9.3, 1536 (six of four) 12.2 / 10.2.  Two CTAs break even at seven or
// eight chunks each, four gain from about four on (NVFP4 4096 outputs, K 4096: 8.7; 1024 outputs, K 5120: 8.4, two 10.2):
// one number for all loses up to 0.8 us at the first and leaves up to 1.9 at the second.
constexpr int kSplitChunks = 6;
constexpr int kEarlyChunks = 8;  // 152 x 8 x 36 KB: 45 MB of the 129 MB L2, 6.6 us of HBM time
// The weights' lines are the first to leave L2 ("stream") where little else moves, up to kStreamRows rows an expert on
// average, or where an expert's tiles run at the same time (kChunkTiles) and the weights are few.  Stream / normal, us,
// weights that no call before has read: K2 layer (NVFP4, 384 experts x 7168 x 2048) of 1 token 50.8 / 57.2, of 8 226 /
// 237, 64 962 / 967, 128 (2.7 rows an expert) 1230 / 1218, 192 1328 / 1293, 256 1350 / 1320, 4096 1649 / 1610; layer of
// 64 experts x 4096 x 1024 of 8 tokens 69.5 / 80.1, of 128 95.8 / 106, of 512 112 / 121; NVFP4 16 experts x 7168 x 2048,
// 80 rows 24.2 / 24.7, 2048 rows 32.8 / 34.4; one bf16 expert x 4096 x 4096, 1000 rows 26.1 / 28.4.  Elsewhere later
// tiles read them again, or outputs push lines that are to leave first out before all their readers came (one bf16
// expert x 6093 x 480, 25,414 rows, 142 / 125).  The rule loses where few weights meet outputs of L2's size: the 16
// experts with 8192 rows 76.5 / 72.4.
constexpr int kStreamRows = 2;
constexpr int64_t kStreamBytes = int64_t(512) << 20;
constexpr int kABytes = kTile * 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kWarpWeights = 0, kWarpIssue = 1, kWarpRows = 2, kWarpScales = 4, kWarpEpi = 8;
// Registers a thread after the split: the epilogue's two warpgroups hold 128 accumulators (rows out, with
// their pieces) or 64 and the features made of them (SwiGLU).
template <int OUT>
struct Regs {
  static constexpr int low = OUT == 2 ? 80 : 56, epi = 256 - low;
};
constexpr int kRegsLaunch = 256 * 256;  // of the block: two warpgroups of each

constexpr int kOutBf16 = 0, kOutF16 = 1, kOutSwiglu = 2;

template <int FMT>
struct Cfg {
  static constexpr int kWords = Mx<FMT>::words;
  static constexpr int kWBytes = kMxCodeBlock + 1024 * kWords;
  static constexpr int kSBytes = (512 * kWords + 1023) / 1024 * 1024;  // row scales, after the rows
  static constexpr int kStage = kWBytes + kABytes + kSBytes;
  static constexpr int kAcc = FMT == MOE_MX_BF16 ? 2 : 1;
  static constexpr uint32_t kScaleCols = 12 * kWords;  // 4 words columns of row scales, 8 of weight scales
  static constexpr int kNumBars = 2 * kStages + 2 * kAcc + 3;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kPlanOff = kBarOff + kNumBars * 8 + 16;  // tile prefix, warp sums
  static constexpr int kTurnOff = (kPlanOff + (kMaxExperts + 1) * 4 + 32 * 4 + 15) / 16 * 16;
  static constexpr int kTurn = 512;  // an epilogue warp's
  static constexpr int kSmem = 1024 + kTurnOff + 8 * kTurn;
  static_assert(kStages * kStage >= kTile * 256 * 4, "the other CTAs' partial sums");
  static_assert(kStage % 1024 == 0, "operand tiles stay 1024-byte aligned");
  static_assert(kSmem <= 232448, "shared memory per CTA");
  static_assert(256 * kAcc + kStages * kScaleCols <= kTmemCols, "tensor memory");
};

struct Args {
  const uint8_t* packed;
  const float* alpha;
  const float* alpha_up;
  int32_t experts, n_out, upt, chunks, groups;  // upt: packed block rows; groups: scales of a row
  uint64_t upt_inv, next_upt_inv;
  int32_t split;                                // CTAs (a cluster) of a unit
  int32_t rows;
  const uint8_t* x_scales;
  int64_t x_pitch;
  const float* x_global;
  const int32_t* offsets;
  void* out;
  int32_t out_vec;
  int64_t out_rows, out_ld;
  const int32_t* out_pos;
  const float* row_weight;
  const float* h_global;
  uint8_t* h_codes;
  uint8_t* h_scales;
  int64_t h_row_bytes, h_pitch;
  uint32_t* err;
  int32_t early;
  int32_t stream;  // the weights' lines leave L2 first (kStreamRows)
  const uint8_t* next_packed;  // the product that follows on the same rows (may be null)
  int32_t next_upt, next_chunks, next_units;  // its units that run first
};

// Rows' maps with boxes of 16, 32, 64 and 128 rows: a tile's copy brings its own
// rows and few others.
struct RowMaps {
  CUtensorMap box[4];
};

__device__ __forceinline__ void mma_block_scaled_nv(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                                    uint32_t sb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_block_scaled_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                                     uint32_t sb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_block_scaled_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                                     uint32_t sb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// 32 rows x 16 bytes of shared memory to four tensor-memory columns, in all four lane quarters.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Descriptor of 512 contiguous bytes as 32 rows of 16: no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

// Instruction descriptors, M = 128, N = 256, both operands K-major.  Block-scaled
// kinds: formats at bits 7 and 10 (e4m3 0; e2m1 1), N / 8 at 17, the scales' type at
// 23 (e4m3 0, e8m0 1), M / 16 at 24, and which byte (1X) or half (2X) of the 4-byte
// scale column an MMA reads at 4 (B) and 29 (A).
template <int FMT>
__device__ __forceinline__ constexpr uint32_t idesc_of(int kk) {
  constexpr uint32_t mn = (static_cast<uint32_t>(256 >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
  if constexpr (FMT == MOE_MX_BF16) return mn | (1u << 4) | (1u << 7) | (1u << 10);
  else if constexpr (FMT == MOE_MX_MXFP8)
    return mn | (1u << 23) | (static_cast<uint32_t>(kk) << 4) | (static_cast<uint32_t>(kk) << 29);
  else if constexpr (FMT == MOE_MX_MXFP4)
    return mn | (1u << 23) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(2 * (kk & 1)) << 4) |
           (static_cast<uint32_t>(2 * (kk & 1)) << 29);
  else return mn | (1u << 7) | (1u << 10);
}

template <int FMT>
__device__ __forceinline__ void issue_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t sa, uint32_t sb, int kk,
                                          uint32_t acc) {
  if constexpr (FMT == MOE_MX_BF16) mma_bf16(d, a, b, idesc_of<FMT>(kk), acc);
  else if constexpr (FMT == MOE_MX_MXFP8) mma_block_scaled_mx8(d, a, b, idesc_of<FMT>(kk), sa, sb, acc);
  else if constexpr (FMT == MOE_MX_MXFP4)
    mma_block_scaled_mx4(d, a, b, idesc_of<FMT>(kk), sa + 4 * (kk >> 1), sb + 8 * (kk >> 1), acc);
  else mma_block_scaled_nv(d, a, b, idesc_of<FMT>(kk), sa + 4 * kk, sb + 8 * kk, acc);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address in CTA `rank` of the cluster of what is at `addr` here.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// wait_bounded for what other CTAs of the cluster wrote before they arrived.
__device__ __forceinline__ bool wait_peers(uint32_t bar, volatile uint32_t* abort_flag, uint32_t* err) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort_flag = 1u;
      atomicOr(err, DEV_ERR_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) return;
}

// silu(g) = g / (1 + e^-g).  By the documented bounds of the two fast functions within (5 + 1.2 |g|) 2^-23 of its
// value; below -87 the denominator passes 2^126 and the result is 0.  (A correctly rounded division here, inlined 64
// times, cost a single row 7.4 us of instruction fetches.)
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

struct Unit {
  int e, row0, nv, u;
};

// Unit number x.  Expert e's units are consecutive, T tiles x upt block rows: its
// tiles in chunks of eight, block row after block row within a chunk, tile after
// tile within a block row.
// (upt_inv: ceil(2^64 / upt), by which a 32-bit quotient is one multiplication; every role waits for this.)
__device__ __forceinline__ Unit unit_of(const int32_t* first_tile, const int32_t* offsets, int experts, int upt,
                                        uint64_t upt_inv, int x) {
  const int t = upt == 1 ? x : static_cast<int>(__umul64hi(static_cast<uint64_t>(x), upt_inv));
  int lo = 0, hi = experts;  // first_tile[lo] <= t < first_tile[hi]
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
  un.row0 = __ldg(offsets + lo) + tile * kTile;
  un.nv = min(kTile, __ldg(offsets + lo + 1) - un.row0);
  return un;
}

// 32 features of h from column `at` on, in the format, to their row's codes and scales (where `on`).
template <int FMT>
__device__ __forceinline__ void store_h(bool on, uint8_t* hc, uint8_t* hs, int at, const float (&h)[32],
                                        const GroupFactor& hf_factor) {
  if constexpr (FMT == MOE_MX_BF16) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16(h[2 * i], h[2 * i + 1]);
    if (!on) return;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<uint4*>(hc + 2 * at + 16 * v) = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
  } else {
    constexpr int G = Mx<FMT>::group;
    uint32_t out[8];
    uint32_t sbytes = 0;
#pragma unroll
    for (int g = 0; g < 32 / G; ++g) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) m = abs_max(m, h[G * g + i]);
      const GroupScale sc = group_scale<FMT>(m, hf_factor);
      sbytes |= sc.byte << (8 * g);
      codes_of<FMT, G>(h + G * g, sc, out + (FMT == MOE_MX_MXFP8 ? 8 : G / 8) * g);
    }
    if (!on) return;
    if constexpr (FMT == MOE_MX_MXFP8) {
      *reinterpret_cast<uint4*>(hc + at) = make_uint4(out[0], out[1], out[2], out[3]);
      *reinterpret_cast<uint4*>(hc + at + 16) = make_uint4(out[4], out[5], out[6], out[7]);
    } else {
      *reinterpret_cast<uint4*>(hc + at / 2) = make_uint4(out[0], out[1], out[2], out[3]);
    }
    if constexpr (G == 16) *reinterpret_cast<uint16_t*>(hs + at / 16) = static_cast<uint16_t>(sbytes);
    else hs[at / 32] = static_cast<uint8_t>(sbytes);
  }
}

// The epilogue of a cluster's unit: column c of a 128-column half is CTA c / width's.  What the
// others own of this thread's row goes to them; what they have of this CTA's columns is added
// to its own.
template <int FMT, int OUT>
__device__ __forceinline__ void finish_split(const Args& a, uint32_t sbase, uint32_t tcol, int rank, int hf, int tok,
                                             bool speaker, int u, int row, int to, float f0, float f1,
                                             uint32_t ready_bar, uint32_t parts_bar, volatile uint32_t* abort_flag) {
  // (split is a power of two: its divisions as shifts; as divisions they took most of the epilogue)
  const int lane = threadIdx.x & 31, split = a.split, log_width = 7 - (31 - __clz(split)), width = 1 << log_width;
  const int half_split = split >> 1, my_half = rank * width >= 64;
  const bool rows_on = __any_sync(0xffffffffu, to >= 0);
  // this CTA's stages are free: the others may write to them
  if (speaker && lane < split && lane != rank) peer_arrive(peer_addr(ready_bar, lane));
  if (!__all_sync(0xffffffffu, wait_peers(ready_bar, abort_flag, a.err))) return;
  // where CTA s's partial sums of columns col + 4 i .. of half m of this row are: float4s, rows innermost
  auto part_at = [&](int s, int m, int col, int i) {
    const uint32_t at = ((2 * s + m) << (log_width - 2)) + ((col & (width - 1)) >> 2) + i;
    return sbase + 16u * (at * kTile + tok);
  };
  if (rows_on) {
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int col = 64 * hf + 16 * k, owner = col >> log_width;
      if (owner == rank) continue;
      uint32_t p[2][16];
      tmem_ld16(tcol + 16 * k, p[0]);
      tmem_ld16(tcol + 128 + 16 * k, p[1]);
      tmem_ld_wait();
      if (to >= 0)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t dst = peer_addr(part_at(rank, m, col, 0), owner);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            peer_store(dst + 16 * kTile * i, p[m][4 * i], p[m][4 * i + 1], p[m][4 * i + 2], p[m][4 * i + 3]);
        }
    }
  }
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  __syncwarp();
  if (lane < half_split && half_split * hf + lane != rank) peer_arrive(peer_addr(parts_bar, half_split * hf + lane));
  if (my_half != hf || !__all_sync(0xffffffffu, wait_peers(parts_bar, abort_flag, a.err)) || !rows_on) return;

  // 16 columns of both halves, summed in the CTAs' order
  auto summed = [&](int col, float* x0, float* x1) {
    uint32_t p[2][16];
    tmem_ld16(tcol + col - 64 * hf, p[0]);
    tmem_ld16(tcol + 128 + col - 64 * hf, p[1]);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) x0[i] = x1[i] = 0.f;
#pragma unroll 1
    for (int s = 0; s < split; ++s) {
      uint4 v[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (the CTA's own place holds nothing that is used)
          v[m][i] = lds128(part_at(s, m, col, i));
      if (s == rank) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[m][i] = make_uint4(p[m][4 * i], p[m][4 * i + 1], p[m][4 * i + 2], p[m][4 * i + 3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x0[4 * i] += __uint_as_float(v[0][i].x);
        x0[4 * i + 1] += __uint_as_float(v[0][i].y);
        x0[4 * i + 2] += __uint_as_float(v[0][i].z);
        x0[4 * i + 3] += __uint_as_float(v[0][i].w);
        x1[4 * i] += __uint_as_float(v[1][i].x);
        x1[4 * i + 1] += __uint_as_float(v[1][i].y);
        x1[4 * i + 2] += __uint_as_float(v[1][i].z);
        x1[4 * i + 3] += __uint_as_float(v[1][i].w);
      }
    }
  };
  const int first = width * rank;
  if constexpr (OUT == kOutSwiglu) {
    const GroupFactor hf_factor = group_factor<FMT>(a.h_global ? __ldg(a.h_global) : 1.f);
    uint8_t* hc = a.h_codes + static_cast<int64_t>(row) * a.h_row_bytes;
    uint8_t* hs = a.h_scales + static_cast<int64_t>(row) * a.h_pitch;
#pragma unroll 1
    for (int col = first; col < first + width; col += 32) {
      const int at = 128 * u + col;
      float g[32], up[32];
      summed(col, g, up);
      summed(col + 16, g + 16, up + 16);
#pragma unroll
      for (int i = 0; i < 32; ++i) g[i] = silu(g[i] * f0) * (up[i] * f1);
      store_h<FMT>(to >= 0 && at < a.n_out, hc, hs, at, g, hf_factor);
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(max(to, 0)) * a.out_ld;
    float top = 0.f;  // largest magnitude, for f16's range
#pragma unroll 1
    for (int col = first; col < first + width; col += 16) {
      float x[2][16];
      summed(col, x[0], x[1]);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int at = 256 * u + 128 * m + col;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y0 = x[m][2 * i] * f0, y1 = x[m][2 * i + 1] * f0;
          if constexpr (OUT == kOutF16) {
            top = fmaxf(top, fmaxf(fabsf(y0), fabsf(y1)));
            const __half2 h2 = __floats2half2_rn(y0, y1);
            w[i] = *reinterpret_cast<const uint32_t*>(&h2);
          } else {
            w[i] = pack_bf16(y0, y1);
          }
        }
        if (a.out_vec && at + 16 <= a.n_out) {
          if (to >= 0) stg256(o + at, w);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (to >= 0 && at + c < a.n_out) o[at + c] = static_cast<uint16_t>(w[c >> 1] >> (16 * (c & 1)));
        }
      }
    }
    if (OUT == kOutF16 && __any_sync(0xffffffffu, to >= 0 && top >= 65520.f) && lane == 0) atomicOr(a.err, DEV_ERR_RANGE);
  }
}

template <int FMT, int OUT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mx_product_kernel(const __grid_constant__ RowMaps maps, const Args a) {
  using C = Cfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBarOff;
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (kStages + i); };
  auto acc_full = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
  auto acc_empty = [&](int i) { return bar0 + 8u * (2 * kStages + C::kAcc + i); };
  const uint32_t drain_bar = bar0 + 8u * (C::kNumBars - 1);
  const uint32_t ready_bar = bar0 + 8u * (C::kNumBars - 2);  // the peers' stages are free
  const uint32_t parts_bar = bar0 + 8u * (C::kNumBars - 3);  // the peers' partial sums are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + C::kNumBars * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int32_t* first_tile = reinterpret_cast<int32_t*>(smem + C::kPlanOff);
  int32_t* warp_sum = first_tile + kMaxExperts + 1;

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), FMT == MOE_MX_BF16 ? 2 : 6);  // weights, rows (and the four scale warps)
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < C::kAcc; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), 8);
    }
    mbar_init(drain_bar, 1);
    mbar_init(ready_bar, SPLIT ? a.split - 1 : 1);
    mbar_init(parts_bar, SPLIT ? 4 * (a.split - 1) : 1);  // four warps of each peer
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kWarpRows && lane < 4) prefetch_tmap(&maps.box[lane]);
  if (warp == kWarpIssue) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (!a.early) pdl_wait();  // else only what the kernel in front writes is waited for, by its readers
  // The tile plan: thread i counts the tiles of experts 2 i and 2 i + 1.
  {
    int n[2] = {0, 0};
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * threadIdx.x + j;
      if (e < a.experts) {
        const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
        bad |= lo < 0 || hi < lo || hi > a.rows;
        n[j] = bad ? 0 : (hi - lo + kTile - 1) / kTile;
      }
    }
    const int mine = n[0] + n[1];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    bad = __syncthreads_or(bad);
    const int base = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
    const int excl = base + incl - mine;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * threadIdx.x + j;
      if (e < a.experts) {
        first_tile[e + 1] = bad ? 0 : excl + n[0] + (j ? n[1] : 0);
        if (e == 0) first_tile[0] = 0;
      }
    }
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, DEV_ERR_ROUTING);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (SPLIT) cluster_sync();  // the peers' barriers are initialised
  const int upt = a.upt, chunks = a.chunks;
  const int total = first_tile[a.experts] * upt;
  // This CTA's units (one at most with a cluster to each), and its part of their chunks.
  const int stride = gridDim.x;
  const int split = SPLIT ? a.split : 1;
  const int rank = SPLIT ? static_cast<int>(blockIdx.x) % split : 0, first = static_cast<int>(blockIdx.x) / split;
  const int c0 = SPLIT ? chunks * rank / split : 0, c1 = SPLIT ? chunks * (rank + 1) / split : chunks;
  auto unit_at = [&](int x) { return unit_of(first_tile, a.offsets, a.experts, upt, a.upt_inv, x); };

  if (warp < kWarpScales) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<OUT>::low));
    if (warp == kWarpWeights) {
      if (lane == 0) {
        const uint64_t pol = a.stream ? policy_evict_first() : policy_evict_normal();
        uint32_t it = 0;
        bool ok = true;
        for (int x = first; ok && x < total; x += stride) {
          const Unit un = unit_at(x);
          const uint8_t* src = a.packed + (static_cast<int64_t>(un.e) * upt + un.u) * chunks * C::kWBytes;
          for (int c = c0; c < c1; ++c, ++it) {
            const int s = it % kStages;
            if (!wait_bounded(empty(s), ((it / kStages) & 1) ^ 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(full(s), C::kWBytes);
            bulk_load(sbase + s * C::kStage, src + static_cast<int64_t>(c) * C::kWBytes, C::kWBytes, full(s), pol);
            // The rows are not there yet: keep HBM busy beyond the stages that the copies fill.
            if (a.early && it == kStages - 1)
              for (int f = c + 1; f < min(c1, c + 1 + kEarlyChunks); ++f)
                bulk_prefetch_l2(src + static_cast<int64_t>(f) * C::kWBytes, C::kWBytes);
          }
        }
        if (!ok)
          for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) wait_drain(full(i % kStages), (i / kStages) & 1);
        // HBM would idle from this CTA's last copy to the next product's first: bring that one's first
        // blocks into L2 (152 units' first six blocks, 33 MB at most).
        if (OUT == kOutSwiglu && ok && a.next_packed) {
          const int next_total = min(first_tile[a.experts] * a.next_upt, a.next_units);
          for (int x = blockIdx.x; x < next_total; x += stride) {
            const Unit un = unit_of(first_tile, a.offsets, a.experts, a.next_upt, a.next_upt_inv, x);
            const uint8_t* src = a.next_packed + (static_cast<int64_t>(un.e) * a.next_upt + un.u) * a.next_chunks * C::kWBytes;
            for (int c = 0; c < min(a.next_chunks, 6); ++c)
              bulk_prefetch_l2(src + static_cast<int64_t>(c) * C::kWBytes, C::kWBytes);
          }
        }
      }
      __syncwarp();
    } else if (warp == kWarpRows) {
      if (a.early) pdl_wait();
      if (lane == 0) {
        const uint64_t pol = policy_evict_last();
        uint32_t it = 0;
        bool ok = true;
        for (int x = first; ok && x < total; x += stride) {
          const Unit un = unit_at(x);
          const int b = un.nv <= 16 ? 0 : un.nv <= 32 ? 1 : un.nv <= 64 ? 2 : 3;
          const uint32_t bytes = (16u << b) * 128u;
          for (int c = c0; c < c1; ++c, ++it) {
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
        uint32_t it = 0, ui = 0;
        bool ok = true;
        for (int x = first; ok && x < total; x += stride, ++ui) {
          const int ab = ui % C::kAcc;
          if (!wait_bounded(acc_empty(ab), ((ui / C::kAcc) & 1) ^ 1, abort_flag, a.err)) break;
          const uint32_t d = tmem + 256u * ab;
          for (int c = c0; c < c1; ++c, ++it) {
            const int s = it % kStages;
            if (!wait_bounded(full(s), (it / kStages) & 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t w = sbase + s * C::kStage;
            const uint32_t sa = tmem + 256u * C::kAcc + s * C::kScaleCols, sb = sa + 4u * C::kWords;
            if constexpr (FMT != MOE_MX_BF16) {
              const uint64_t wd = desc_scales(w + kMxCodeBlock), rd = desc_scales(w + C::kWBytes + kABytes);
#pragma unroll
              for (int i = 0; i < 2 * C::kWords; ++i) tmem_copy_scales(sb + 4 * i, desc_advance(wd, 512 * i));
#pragma unroll
              for (int i = 0; i < C::kWords; ++i) tmem_copy_scales(sa + 4 * i, desc_advance(rd, 512 * i));
            }
            const uint64_t ad = desc_kmajor_sw128(w + C::kWBytes), bd = desc_kmajor_sw128(w);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              issue_mma<FMT>(d, desc_advance(ad, 32 * kk), desc_advance(bd, 32 * kk), sa, sb, kk, c > c0 || kk > 0);
            tc_commit(empty(s));
          }
          if (ok) tc_commit(acc_full(ab));
        }
        tc_commit(drain_bar);  // every MMA issued above has completed once this arrives
        wait_drain(drain_bar, 0);
      }
      __syncwarp();
    }
  } else if (warp < kWarpEpi) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<OUT>::low));
    if constexpr (FMT != MOE_MX_BF16) {
      pdl_wait();
      constexpr int W = C::kWords;
      const int row = 32 * (warp & 3) + lane;  // this thread's row of the tile
      // word i of row r at 512 i + 16 (r % 32) + 4 (r / 32), as in the packed weights
      const uint32_t at = sbase + C::kWBytes + kABytes + 16 * lane + 4 * (warp & 3);
      // what is loaded runs four chunks ahead of what is stored
      int lx = first, lc = c0;
      const uint8_t* src = nullptr;
      uint32_t buf[kStages][W];
      auto load = [&](uint32_t (&w)[W]) {
        if (lx >= total) return;
        if (lc == c0) {
          const Unit un = unit_at(lx);
          src = row < un.nv ? a.x_scales + (static_cast<int64_t>(un.row0) + row) * a.x_pitch : nullptr;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
        if (src) {
          const uint8_t* p = src + lc * 4 * W;
          if constexpr (W == 4) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
          } else if constexpr (W == 2) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = q.x, w[1] = q.y;
          } else {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
          }
        }
        const int left = a.groups - lc * 4 * W;  // scales of this chunk that exist
        if (left < 4 * W) {                      // the last chunk: bytes past them are padding
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const int k = left - 4 * i;
            w[i] &= k >= 4 ? 0xffffffffu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
          }
        }
        if (++lc == c1) {
          lc = c0;
          lx += stride;
        }
      };
      const int64_t mine = first < total ? (total - 1 - first) / stride + 1 : 0;
      const int64_t iters = mine * (c1 - c0);
      bool ok = true;
#pragma unroll
      for (int j = 0; j < kStages; ++j) load(buf[j]);
      for (int64_t it = 0; ok && it < iters; it += kStages) {
#pragma unroll
        for (int j = 0; j < kStages; ++j) {
          if (ok && it + j < iters) {
            ok = __all_sync(0xffffffffu, wait_bounded(empty(j), ((it / kStages) & 1) ^ 1, abort_flag, a.err));
            if (ok) {
#pragma unroll
              for (int i = 0; i < W; ++i)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + j * C::kStage + 512 * i), "r"(buf[j][i]) : "memory");
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copies to tensor memory read it
              __syncwarp();
              if (lane == 0) mbar_arrive(full(j));
              load(buf[j]);
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<OUT>::epi));
    if (a.early) pdl_wait();
    const int q = warp & 3, hf = (warp - kWarpEpi) >> 2;
    const int tok = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const float xg = a.x_global ? __ldg(a.x_global) : 1.f;
    // What this thread needs for a unit besides the accumulators, fetched a unit ahead.
    struct Mine {
      int u, row, to;  // packed block row; the thread's row, and where it goes (-1: nowhere)
      float f0, f1;    // factors of the two 128-column halves
    };
    auto mine_of = [&](int x) {
      Mine m{0, 0, -1, 0.f, 0.f};
      if (x >= total) return m;
      const Unit un = unit_at(x);
      m.u = un.u;
      m.row = un.row0 + tok;
      m.f0 = xg * (a.alpha ? __ldg(a.alpha + un.e) : 1.f);
      if constexpr (OUT == kOutSwiglu) m.f1 = xg * (a.alpha_up ? __ldg(a.alpha_up + un.e) : 1.f);
      if (tok < un.nv) {
        m.to = OUT != kOutSwiglu && a.out_pos ? __ldg(a.out_pos + m.row) : m.row;
        if (OUT != kOutSwiglu && m.to >= a.out_rows) m.to = -1;
        if (OUT != kOutSwiglu && a.row_weight && m.to >= 0) m.f0 *= __ldg(a.row_weight + m.to);
      }
      return m;
    };
    uint32_t ui = 0;
    Mine me = mine_of(first);
    for (int x = first; x < total; x += stride, ++ui) {
      const int ab = ui % C::kAcc;
      if (!__all_sync(0xffffffffu, wait_bounded(acc_full(ab), (ui / C::kAcc) & 1, abort_flag, a.err))) break;
      tc_fence_after();
      const uint32_t rows_on = __ballot_sync(0xffffffffu, me.to >= 0);
      const uint32_t tcol = tmem + lane_base + 256u * ab + 64u * hf;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(ab));
      };
      if constexpr (SPLIT) {
        finish_split<FMT, OUT>(a, sbase, tcol, rank, hf, tok, warp == kWarpEpi, me.u, me.row, me.to, me.f0, me.f1, ready_bar,
                               parts_bar, abort_flag);
        break;  // a cluster has one unit
      }
      Mine next;
      if constexpr (OUT == kOutSwiglu) {
        // 32 features at a time: half the registers, and no slower than with all 128 accumulators read first
        const GroupFactor hf_factor = group_factor<FMT>(a.h_global ? __ldg(a.h_global) : 1.f);
        uint8_t* hc = a.h_codes + static_cast<int64_t>(me.row) * a.h_row_bytes;
        uint8_t* hs = a.h_scales + static_cast<int64_t>(me.row) * a.h_pitch;
        if (rows_on == 0) release();
#pragma unroll 1
        for (int half = 0; half < 2 && rows_on != 0; ++half) {
          const int at = 128 * me.u + 64 * hf + 32 * half;
          float h[32];
          {
            uint32_t g[32], u[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              tmem_ld16(tcol + 32 * half + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(&g[16 * i]));
              tmem_ld16(tcol + 128 + 32 * half + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(&u[16 * i]));
            }
            tmem_ld_wait();
            if (half == 1) release();
#pragma unroll
            for (int i = 0; i < 32; ++i) h[i] = silu(__uint_as_float(g[i]) * me.f0) * (__uint_as_float(u[i]) * me.f1);
          }
          store_h<FMT>(me.to >= 0 && at < a.n_out, hc, hs, at, h, hf_factor);
        }
        next = mine_of(x + stride);
      } else {
        uint16_t* o = static_cast<uint16_t*>(a.out);
        float top = 0.f;  // largest magnitude, for f16's range
        auto pack2 = [&](uint32_t r0, uint32_t r1) {
          const float y0 = __uint_as_float(r0) * me.f0, y1 = __uint_as_float(r1) * me.f0;
          if constexpr (OUT == kOutF16) {
            top = fmaxf(top, fmaxf(fabsf(y0), fabsf(y1)));
            const __half2 h2 = __floats2half2_rn(y0, y1);
            return *reinterpret_cast<const uint32_t*>(&h2);
          } else {
            return pack_bf16(y0, y1);
          }
        };
        if (rows_on == 0) {
          release();
          next = mine_of(x + stride);
        } else if (a.out_vec) {
          uint32_t p[2][64];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tmem_ld16(tcol + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(&p[0][16 * i]));
            tmem_ld16(tcol + 128 + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(&p[1][16 * i]));
          }
          tmem_ld_wait();
          release();
          next = mine_of(x + stride);
          // Four lanes exchange their rows' four 32-byte pieces, so that a store covers whole 128-byte
          // lines of eight rows instead of a piece of each of 32 (which the load/store unit takes one
          // line at a time).
          const int j = lane & 3;
          uint16_t* to[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = __shfl_sync(0xffffffffu, me.to, (lane & ~3) + i);
            to[i] = r >= 0 ? o + static_cast<int64_t>(r) * a.out_ld : nullptr;
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t w[4][8];
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
              for (int i = 0; i < 8; ++i) w[v][i] = pack2(p[m][16 * v + 2 * i], p[m][16 * v + 2 * i + 1]);
#pragma unroll
            for (int step = 1; step <= 2; step *= 2) {
              const bool up = (lane & step) != 0;
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                if (v & step) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[v][i] : w[v + step][i], step);
                  if (up) w[v][i] = got;
                  else w[v + step][i] = got;
                }
              }
            }
            const int at = 256 * me.u + 128 * m + 64 * hf + 16 * j;  // w[i]: these 16 columns of the i-th row
            if (at + 16 <= a.n_out) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (to[i]) stg256(to[i] + at, w[i]);
            } else if (at < a.n_out) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (!to[i]) continue;
#pragma unroll
                for (int c = 0; c < 15; ++c)
                  if (at + c < a.n_out) to[i][at + c] = static_cast<uint16_t>(w[i][c >> 1] >> (16 * (c & 1)));
              }
            }
          }
        } else {
          // Rows that are not aligned: 16 columns of 16 rows at a time, turned through shared memory so
          // that eight lanes write the 16 columns of one row.  What a lane writes is always of the same
          // eight rows.
          uint8_t* turn = smem + C::kTurnOff + (warp - kWarpEpi) * C::kTurn;
          uint16_t* to[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = __shfl_sync(0xffffffffu, me.to, 4 * i + (lane >> 3));
            to[i] = r >= 0 ? o + r * a.out_ld + 2 * (lane & 7) : nullptr;
          }
#pragma unroll 1
          for (int v = 0; v < 8; ++v) {
            uint32_t p[16], w[8];
            tmem_ld16(tcol + 128 * (v >> 2) + 16 * (v & 3), p);
            tmem_ld_wait();
            const int at = 256 * me.u + 128 * (v >> 2) + 64 * hf + 16 * (v & 3);
            if (at >= a.n_out) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack2(p[2 * i], p[2 * i + 1]);
            const int left = a.n_out - at - 2 * (lane & 7);  // columns from this lane's first on
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if ((rows_on >> (16 * half) & 0xffffu) == 0) continue;
              __syncwarp();
              if (lane >> 4 == half) {
                reinterpret_cast<uint4*>(turn)[2 * (lane & 15)] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(turn)[2 * (lane & 15) + 1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
              __syncwarp();
              uint32_t two[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                two[i] = *reinterpret_cast<const uint32_t*>(turn + 32 * (4 * i + (lane >> 3)) + 4 * (lane & 7));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint16_t* q = to[4 * half + i];
                if (q && left > 0) q[at] = static_cast<uint16_t>(two[i]);
                if (q && left > 1) q[at + 1] = static_cast<uint16_t>(two[i] >> 16);
              }
            }
          }
          release();
          next = mine_of(x + stride);
        }
        if (OUT == kOutF16) {
          const bool over = me.to >= 0 && top >= 65520.f;  // f16 rounds these to infinity
          if (__any_sync(0xffffffffu, over) && lane == 0) atomicOr(a.err, DEV_ERR_RANGE);
        }
      }
      me = next;
    }
  }
  __syncthreads();
  if constexpr (SPLIT) cluster_sync();  // no CTA's memory goes while another may still write to it
  if (warp == kWarpIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int FMT, int OUT, bool SPLIT>
cudaError_t launch(const MxProductLaunch& g, int64_t units, int split, cudaStream_t s) {
  using C = Cfg<FMT>;
  auto kern = mx_product_kernel<FMT, OUT, SPLIT>;
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
  if (regs.load(std::memory_order_relaxed) * kThreads < kRegsLaunch)
    return cudaErrorInvalidConfiguration;
  const moe_mx_weights* w = g.w;
  Args a{};
  a.packed = static_cast<const uint8_t*>(w->packed);
  a.alpha = w->alpha;
  a.alpha_up = w->alpha_up;
  a.experts = w->num_experts;
  a.n_out = w->n_out;
  auto inverse = [](int64_t d) { return d > 1 ? ~0ull / static_cast<uint64_t>(d) + 1 : 0ull; };  // ceil(2^64 / d)
  a.upt = static_cast<int32_t>(mx_unit_rows(w));
  a.upt_inv = inverse(a.upt);
  a.chunks = static_cast<int32_t>(mx_chunks(w));
  a.groups = Mx<FMT>::group ? w->k / (Mx<FMT>::group ? Mx<FMT>::group : 1) : 0;
  a.rows = g.rows;
  a.x_scales = g.x_scales;
  a.x_pitch = static_cast<int64_t>(moe_mx_scale_pitch(FMT, w->k));
  a.x_global = FMT == MOE_MX_NVFP4 ? g.x_global : nullptr;
  a.offsets = g.offsets;
  a.out = g.out;
  a.out_vec = reinterpret_cast<uintptr_t>(g.out) % 32 == 0 && g.out_ld % 16 == 0;
  a.out_rows = g.out_rows;
  a.out_ld = g.out_ld;
  a.out_pos = g.out_pos;
  a.row_weight = g.row_weight;
  a.h_global = FMT == MOE_MX_NVFP4 ? g.h_global : nullptr;
  a.h_codes = g.h_codes;
  a.h_scales = g.h_scales;
  a.h_row_bytes = static_cast<int64_t>(moe_mx_code_bytes(FMT, w->n_out));
  a.h_pitch = static_cast<int64_t>(moe_mx_scale_pitch(FMT, w->n_out));
  a.err = g.err;
  a.early = g.early ? 1 : 0;
  const int64_t touched = static_cast<int64_t>(g.rows < w->num_experts ? g.rows : w->num_experts) * a.upt * a.chunks * C::kWBytes;
  a.stream = g.rows <= static_cast<int64_t>(kStreamRows) * w->num_experts ||
             (g.rows <= static_cast<int64_t>(kChunkTiles * kTile) * w->num_experts && touched <= kStreamBytes);
  if (g.next) {
    a.next_packed = static_cast<const uint8_t*>(g.next->packed);
    a.next_upt = static_cast<int32_t>(mx_unit_rows(g.next));
    a.next_upt_inv = inverse(a.next_upt);
    a.next_chunks = static_cast<int32_t>(mx_chunks(g.next));
    a.next_units = g.num_sms;
  }
  RowMaps maps;
  for (int i = 0; i < 4; ++i)
    if (!encode_rows_map(&maps.box[i], g.x_codes, moe_mx_code_bytes(FMT, w->k), g.rows, 16u << i))
      return cudaErrorInvalidValue;
  a.split = split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(SPLIT ? units * split : units < g.num_sms ? units : g.num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

}  // namespace

// How many clusters of n CTAs run at once (looked up until it is known; 0 where it cannot be).
template <int FMT, int OUT>
static int max_clusters(int n) {
  using C = Cfg<FMT>;
  static std::atomic<int> known[9];  // one more than the number
  const int k = known[n].load(std::memory_order_relaxed);
  if (k > 0) return k - 1;
  auto kern = mx_product_kernel<FMT, OUT, true>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(n);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) return 0;
  known[n].store(clusters + 1, std::memory_order_relaxed);
  return clusters;
}

template <int FMT, int OUT>
static cudaError_t launch_out(const MxProductLaunch& g, cudaStream_t s) {
  // The most units there can be: an expert's last tile may be short.
  const int64_t tiles = static_cast<int64_t>(g.rows) / kTile + (g.rows < g.w->num_experts ? g.rows : g.w->num_experts);
  const int64_t units = tiles * mx_unit_rows(g.w), chunks = mx_chunks(g.w);
  // A cluster to each unit where all of them fit and each CTA keeps kSplitChunks chunks (SwiGLU: up to
  // four, so that a slice holds whole groups).
  // (A cluster of eight leaves SMs of its processing cluster over: 15 or so fit at once, not 19.)
  for (int n = OUT == kOutSwiglu ? 4 : 8; n > 1; n /= 2)
    if (units * n <= g.num_sms && chunks >= kSplitChunks * n && units <= max_clusters<FMT, OUT>(n))
      return launch<FMT, OUT, true>(g, units, n, s);
  return launch<FMT, OUT, false>(g, units, 1, s);
}

template <int FMT>
static cudaError_t launch_format(const MxProductLaunch& g, cudaStream_t s) {
  if (g.w->swiglu) return launch_out<FMT, kOutSwiglu>(g, s);
  return g.out_f16 ? launch_out<FMT, kOutF16>(g, s) : launch_out<FMT, kOutBf16>(g, s);
}

cudaError_t launch_mx_product(const MxProductLaunch& g, cudaStream_t s) {
  switch (g.w->format) {
    case MOE_MX_BF16: return launch_format<MOE_MX_BF16>(g, s);
    case MOE_MX_MXFP8: return launch_format<MOE_MX_MXFP8>(g, s);
    case MOE_MX_MXFP4: return launch_format<MOE_MX_MXFP4>(g, s);
    case MOE_MX_NVFP4: return launch_format<MOE_MX_NVFP4>(g, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
