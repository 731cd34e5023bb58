/*
 * moe_fp8.h - operators on rows and weights in the FP8 bank's own form, one by
 * one: rows quantised per 128 columns, and products grouped by expert.
 *
 * Rows: e4m3 codes [rows][cols], dense, and one fp32 scale per 128 columns,
 * [rows][moe_fp8_scale_pitch(cols)] (the last block may be short; entries past it
 * are not used and not written).  Value = code * scale.  cols is a multiple of
 * 16; both bases are 16-byte aligned.
 * Quantising a block with largest magnitude a, as MOE_ACT_FP8_DYNAMIC does:
 *   scale = a / 448 in fp32, 1 for a block of zeros
 *   code  = e4m3 nearest to the fp32 quotient v / scale (ties to even), saturating at 448
 * A block that holds a NaN or an infinity gets zero codes and the scale NaN, so
 * the block, and every product that reads it, is NaN and nothing else is.
 *
 * Weights: E matrices [n_out, k] of e4m3 codes with one fp32 scale per 128 x 128
 * block, [E][ceil(n_out / 128)][ceil(k / 128)] (moe_weights' w_* and s_*).
 *
 * All pointers except the struct are device pointers; every call is asynchronous
 * on `stream`, allocates nothing, does not synchronise and can be captured.  Calls
 * with the same workspace may overlap (it holds only an error word).  Sizes are
 * checked before anything is launched; n or rows of 0 is MOE_OK and does nothing.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_FP8_BLOCK 128

/* Workspace of the products: the error word (moe_get_error) and padding. */
#define MOE_FP8_PRODUCT_WORKSPACE ((size_t)256)

/* fp32 scales from one row's to the next's: ceil(cols / 128) rounded up to 4 (0 where cols is not a positive
 * multiple of 16). */
int64_t moe_fp8_scale_pitch(int64_t cols);

/* Rows quantised: row t of x to row positions[t * k + j] for each j.
 *   x          [n] rows of d bf16, x_ld elements apart (>= d, a multiple of 8); 16-byte aligned
 *   positions  [n, k] int32; NULL: k = 1 and row t.  Entries outside [0, out_rows) are skipped; a row that two
 *              entries name holds parts of either.
 *   codes, scales  [out_rows] rows
 * d a multiple of 16 up to 16384. */
moe_status moe_fp8_quantise(int64_t n, int32_t k, int32_t d, const void *x, int64_t x_ld, const int32_t *positions,
                            int64_t out_rows, void *codes, float *scales, cudaStream_t stream);

/* bf16 values of `rows` rows: code * scale rounded to fp32, as a product reads it, and that to bf16.  out rows out_ld elements
 * apart, a multiple of 8; 16-byte aligned. */
moe_status moe_fp8_dequantise(int64_t rows, int32_t d, const void *codes, const float *scales, void *out,
                              int64_t out_ld, cudaStream_t stream);

/* E matrices [n_out, k] in the packed layout that moe_fp8_pack_weights writes: out = x W^T. */
typedef struct {
    int32_t num_experts;    /* 1 to 1024 */
    int32_t n_out;          /* 1 to 65536 */
    int32_t k;              /* a multiple of 16, up to 65536 */
    const void *packed;     /* 16-byte aligned */
    const float *scales;    /* [E][ceil(n_out / 128)][ceil(k / 128)] */
} moe_fp8_weights;

/* The packed layout streams: blocks of 256 matrix rows by 128 columns (32 KB), block (e, u, c) at
 * ((e * ceil(n_out / 256) + u) * ceil(k / 128) + c) * 32768.  16-byte piece j of block row r is at
 * 128 r + 16 (j ^ (r % 8)): what a 128-byte-swizzled tile is in shared memory.  Rows and columns past the matrix are
 * zeros.  (Where n_out and k are multiples of 128 this is what moe_pack_weights makes of w_down.)
 *   codes      [E][n_out][k], or with transpose != 0 [E][k][n_out] (n_out then a multiple of 16 too), whose
 *              transposes are packed: the weights of the gradient dx = dy W of y = x W^T
 *   scales     with transpose the blocks' scales [E][ceil(k / 128)][ceil(n_out / 128)], else not read
 *   scales_out with transpose the transposed scales (what w->scales will be), else not written
 *   packed     moe_fp8_packed_bytes bytes */
moe_status moe_fp8_pack_weights(const moe_fp8_weights *w, const void *codes, const float *scales, int32_t transpose,
                                void *packed, float *scales_out, cudaStream_t stream);

/* Bytes of a packed buffer (0 for unsupported sizes; reads no pointer of w). */
size_t moe_fp8_packed_bytes(const moe_fp8_weights *w);

#define MOE_FP8_OUT_BF16 0
#define MOE_FP8_OUT_F16 1
#define MOE_FP8_OUT_F32 2

/* Products grouped by expert: rows expert_offsets[e] .. expert_offsets[e + 1] - 1 of x belong to expert e.
 *   out[p(r)] = row_weight[p(r)] * sum_b x_scale[r][b] w_scale[e][n / 128][b] * sum_{c in block b} X[r][c] W_e[n][c]
 * with p(r) = out_pos[r]; a block's products are summed in fp32 on the tensor cores, the two scales' product is fp32, the
 * blocks are summed in fp32 (a block's sum times its scales added with one rounding), the row weight multiplies in fp32,
 * and that is rounded to out_type.
 *   rows            rows of x, below 2^31; (rows / 128 + E) * ceil(n_out / 128) at most 2^31 - 4097
 *   expert_offsets  [E + 1] int32, ascending from >= 0 to <= rows; anything else computes nothing and raises
 *                   MOE_ERR_ROUTING.  Rows of no expert are left alone, empty experts cost nothing.  NULL, where
 *                   num_experts is 1: all rows.  The tiles' size is chosen by rows and num_experts, all that the host knows:
 *                   where one of many experts has most of a few rows, a call may take twice as long as for that
 *                   expert alone.
 *   out             [out_rows] rows of n_out (out_type), out_ld elements apart (>= n_out), aligned to their
 *                   elements (fastest with 32-byte aligned rows)
 *   out_pos         [rows] int32, NULL = r.  Rows sent outside [0, out_rows) are skipped; a row that two are sent to
 *                   holds parts of either.
 *   row_weight      [out_rows] fp32 or NULL = 1
 *   workspace       MOE_FP8_PRODUCT_WORKSPACE bytes, 256-byte aligned; its error word accumulates until
 *                   moe_get_error reads it (zero it once).  f16 results beyond its range raise MOE_ERR_RANGE. */
moe_status moe_fp8_grouped_product(const moe_fp8_weights *w, int64_t rows, const void *x_codes, const float *x_scales,
                                   const int32_t *expert_offsets, void *out, int32_t out_type, int64_t out_rows,
                                   int64_t out_ld, const int32_t *out_pos, const float *row_weight, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
