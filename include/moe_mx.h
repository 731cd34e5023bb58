/*
 * moe_mx.h - microscaled-format operators of the GB300 routed-expert library:
 * rows held in 4 or 8 bits with scales, products grouped by expert on them,
 * and the MoE block made of the two.
 *
 * The FP8 bank of moe_ffn.h stores one fp32 scale per 128 x 128 block.  The
 * formats here scale short groups along a row, weights and activations alike,
 * which the tensor core undoes inside the product (tcgen05 block_scale):
 *
 *   format          code            group  scale of a group      bytes per column
 *   MOE_MX_BF16     bf16            -      -                     2
 *   MOE_MX_MXFP8    e4m3            32     power of two (e8m0)   1 + 1/32
 *   MOE_MX_MXFP4    e2m1            32     power of two (e8m0)   1/2 + 1/32
 *   MOE_MX_NVFP4    e2m1            16     e4m3, times one fp32  1/2 + 1/16
 *                                          factor per tensor
 *
 * Quantising a group with largest magnitude a:
 *   MXFP8, MXFP4  scale 2^k, the smallest k >= -126 with a <= M 2^k (M = 448, 6);
 *                 nothing saturates.  Byte k + 127.
 *   NVFP4         scale s = e4m3(a / (6 g)), g the tensor's factor, saturating at
 *                 448; divisor s g (rounded to fp32).  A zero divisor gives zero codes.
 *   code          nearest (ties to even) of value / divisor, saturating.
 * A group that holds a NaN or an infinity gets zero codes and the NaN scale
 * (e8m0 255, e4m3 0x7f), so the group, and every product that reads it, is NaN
 * and nothing else is.
 *
 * Rows (activations): codes [rows][moe_mx_code_bytes] and scales
 * [rows][moe_mx_scale_pitch], both dense, both bases 16-byte aligned.  Two e2m1
 * codes share a byte, the even column in the low half.  Scale j of a row is byte
 * j; the bytes past the last group round the pitch up to 16, are never read for
 * their value and not written.  Columns are a multiple of 32.
 *
 * All pointers except the structs are device pointers; every call is
 * asynchronous on `stream`, allocates nothing, does not synchronise and can be
 * captured.  Calls with the same workspace must not overlap.  Sizes are checked
 * before anything is launched; n or rows of 0 is MOE_OK and does nothing.
 */
#ifndef MOE_MX_H
#define MOE_MX_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MX_BF16 0
#define MOE_MX_MXFP8 1
#define MOE_MX_MXFP4 2
#define MOE_MX_NVFP4 3

/* Workspace of the grouped products: the error word (moe_get_error) and padding. */
#define MOE_MX_PRODUCT_WORKSPACE ((size_t)256)

/* Bytes of codes of one row of `cols` columns; 0 for an unknown format or cols
 * not a positive multiple of 32. */
size_t moe_mx_code_bytes(int32_t format, int64_t cols);

/* Bytes from one row's scales to the next's (0 for MOE_MX_BF16 and where
 * moe_mx_code_bytes is 0). */
size_t moe_mx_scale_pitch(int32_t format, int64_t cols);

/* Rows into a format:  Q(x[t]) written to row positions[t * k + j] for each j.
 *   x          [n] rows of d bf16, x_ld elements apart (>= d, a multiple of 8); 16-byte aligned
 *   positions  [n, k] int32; NULL: k = 1 and row t.  Entries outside [0, out_rows) are skipped.
 *   global     [1] fp32, NVFP4's factor g, 2^-60 to 2^60 (NULL = 1); not read for other formats
 *   codes, scales  [out_rows] rows; scales not read for MOE_MX_BF16
 * d up to 16384. */
moe_status moe_mx_quantise(int32_t format, int64_t n, int32_t k, int32_t d, const void *x, int64_t x_ld,
                           const int32_t *positions, const float *global, int64_t out_rows, void *codes, void *scales,
                           cudaStream_t stream);

/* The decoder block's step in front of its feed-forward half, into a format:
 *   sum[t] = bf16(x[t] + residual[t])
 *   y[t]   = sum[t] / sqrt(mean(sum[t]^2) + eps) * gain     (fp32, not rounded)
 *   Q(y[t]) written as by moe_mx_quantise
 *   residual   as x with r_ld, or NULL (sum = x)
 *   gain       [d] bf16, 16-byte aligned;  eps >= 0
 *   sum        [n] rows, r_ld elements apart, or NULL; may be x or residual itself (same stride) */
moe_status moe_mx_add_rmsnorm(int32_t format, int64_t n, int32_t k, int32_t d, const void *x, int64_t x_ld,
                              const void *residual, int64_t r_ld, const void *gain, float eps,
                              const int32_t *positions, const float *global, int64_t out_rows, void *sum, void *codes,
                              void *scales, cudaStream_t stream);

/* bf16 values of `rows` rows (rounded once; exact for the MX formats and for
 * NVFP4 with a power-of-two factor, unless below bf16's range). */
moe_status moe_mx_dequantise(int32_t format, int64_t rows, int32_t d, const void *codes, const void *scales,
                             const float *global, void *out, int64_t out_ld, cudaStream_t stream);

/* Weights of a grouped product: E matrices [n_out, k], out = x W^T, in the
 * packed layout that moe_mx_pack_weights writes.  With swiglu != 0 each expert
 * has two, gate and up, of n_out rows each.
 *   alpha, alpha_up  [E] fp32: what expert e's product is multiplied by (its
 *                    matrix's factor g for NVFP4); NULL = 1.  alpha_up is up's
 *                    and only read with swiglu. */
typedef struct {
    int32_t format;
    int32_t num_experts;    /* 1 to 1024 */
    int32_t n_out;          /* rows of a matrix, 1 to 65536 (a multiple of 32 with swiglu) */
    int32_t k;              /* columns, a multiple of 32, up to 65536 */
    int32_t swiglu;
    const void *packed;     /* 16-byte aligned */
    const float *alpha, *alpha_up;
} moe_mx_weights;

/* The packed layout streams: blocks of 256 matrix rows by 128 bytes of codes
 * (C = 64, 128, 256, 256 columns) with their scales, block (e, u, c) at
 * ((e * U + u) * ceil(k / C) + c) * (32768 + S), S = 0, 1024, 2048, 4096.
 *   block row r is matrix row 256 u + r (U = ceil(n_out / 256)); with swiglu
 *   gate row 128 u + r for r < 128, else up row 128 u + r - 128 (U = ceil(n_out / 128))
 *   16-byte piece j of row r's codes at 128 r + 16 (j ^ (r % 8)): what a
 *   128-byte-swizzled tile is in shared memory
 *   scale bytes 4 w .. 4 w + 3 of row r at 32768 + 1024 w + 512 (r / 128)
 *   + 16 (r % 32) + 4 ((r / 32) % 4): the order in which the tensor core takes them
 * Rows and columns past the matrix are zeros.
 *   codes, scales        [E * n_out] rows of k columns, laid out as rows are
 *   codes_up, scales_up  the same for up, NULL without swiglu */
moe_status moe_mx_pack_weights(const moe_mx_weights *w, const void *codes, const void *scales, const void *codes_up,
                               const void *scales_up, void *packed, cudaStream_t stream);

/* Bytes of a packed buffer (0 for unsupported sizes; reads no pointer of w). */
size_t moe_mx_packed_bytes(const moe_mx_weights *w);

#define MOE_MX_OUT_BF16 0
#define MOE_MX_OUT_F16 1

/* Products grouped by expert: rows expert_offsets[e] .. expert_offsets[e + 1] - 1 of x belong to expert e.
 *   out[p(r)] = row_weight[p(r)] * (global * alpha[e]) * x[r] W_e^T,   p(r) = out_pos[r]
 * accumulated in fp32 and rounded once.
 *   rows            rows of x, below 2^31; (rows / 128 + E) * ceil(n_out / 256) at most 2^31 - 4097
 *   x_codes, x_scales  rows of w->k columns in w->format;  x_global  x's factor (NULL = 1)
 *   expert_offsets  [E + 1] int32, ascending from >= 0 to <= rows; anything else computes nothing
 *                   and raises MOE_ERR_ROUTING.  Rows of no expert are left alone, empty experts cost nothing.
 *   out             [out_rows] rows of n_out bf16 or f16 (out_type), out_ld elements apart (>= n_out);
 *                   2-byte aligned (fastest with 32-byte aligned rows)
 *   out_pos         [rows] int32, NULL = r.  Rows sent outside [0, out_rows) are skipped.
 *   row_weight      [out_rows] fp32 or NULL = 1
 *   workspace       MOE_MX_PRODUCT_WORKSPACE bytes, 256-byte aligned; its error word accumulates until
 *                   moe_get_error reads it (zero it once).  f16 results beyond its range raise MOE_ERR_RANGE. */
moe_status moe_mx_grouped_product(const moe_mx_weights *w, int64_t rows, const void *x_codes, const void *x_scales,
                                  const float *x_global, const int32_t *expert_offsets, void *out, int32_t out_type,
                                  int64_t out_rows, int64_t out_ld, const int32_t *out_pos, const float *row_weight,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* The gate/up half of a SwiGLU expert on grouped rows (w->swiglu != 0):
 *   h[r] = silu(g) * u,  g = (x_global alpha[e]) x[r] Wg_e^T,  u = (x_global alpha_up[e]) x[r] Wu_e^T
 * formed from the fp32 accumulators and quantised as by moe_mx_quantise, with
 * no rounding in between: h_codes, h_scales [rows] rows of n_out columns,
 * h_global its factor (NULL = 1). */
moe_status moe_mx_grouped_swiglu(const moe_mx_weights *w, int64_t rows, const void *x_codes, const void *x_scales,
                                 const float *x_global, const int32_t *expert_offsets, const float *h_global,
                                 void *h_codes, void *h_scales, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/* The MoE block on microscaled experts:
 *   sum = bf16(x + residual)
 *   out = sum + sum_j topk_weight[t][j] * E_{ids[t][j]}(Q(rmsnorm(sum)))
 *   E(v) = down(Q(silu(gate v) * up v))
 * i.e. moe_permute, moe_mx_add_rmsnorm to the sorted rows, moe_mx_grouped_swiglu,
 * moe_mx_grouped_product (f16 rows, weighted) and moe_combine.
 * The norm is moe_mx_add_rmsnorm's, in fp32 until Q.  moe_layer_forward's rounds
 * the normalised row and its product with the gain to bf16 each; on rows that are
 * normalised that way this call, with gain NULL, is that block's routed sum.
 * The weighted rows are f16 also where out is fp32: 2^-11 of each (2^-25 below
 * 2^-14), and MOE_ERR_RANGE beyond 65504.
 *   gate_up, down  one format; gate_up->swiglu = 1, n_out = d_ff, k = d; down n_out = d, k = d_ff;
 *                  d a multiple of 128
 *   x, residual    [n, d] bf16;  residual may be NULL.  With gain NULL there is no norm and no residual
 *                  stream: out = sum_j ..., E applied to Q(x) (residual and sum must be NULL).
 *   sum            [n, d] bf16 out
 *   out            [n, d] bf16, or fp32 when out_is_fp32
 * Errors as in moe_infer; the first kernel resets the workspace's error word. */
size_t moe_mx_layer_workspace_size(const moe_mx_weights *gate_up, const moe_mx_weights *down, int32_t top_k,
                                   int64_t n_tokens);
moe_status moe_mx_layer_forward(const moe_mx_weights *gate_up, const moe_mx_weights *down, int32_t top_k,
                                int64_t n_tokens, const void *x, const void *residual, const void *gain, float eps,
                                const int32_t *topk_ids, const float *topk_weight, const float *x_global,
                                const float *h_global, void *sum, void *out, int32_t out_is_fp32, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MX_H */
