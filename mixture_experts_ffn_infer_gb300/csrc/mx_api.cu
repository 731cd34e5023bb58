// C ABI of the microscaled-format operators (moe_mx.h): argument checks,
// workspace layout and the launch sequence of each entry point.
#include <cuda_runtime.h>

#include "mx.cuh"
#include "mx_default.h"

// Host code must not pass the symbol itself on: it only names a stand-in there (moe_mx_default_workspace).
static __device__ __align__(256) uint8_t mx_default_ws[MOE_MX_PRODUCT_WORKSPACE];

namespace moe {
namespace {

constexpr int kMaxExpertsMx = 1024;
constexpr int kMaxCols = 65536;
constexpr int kMaxRowCols = 16384;  // moe_mx_quantise, moe_mx_add_rmsnorm: a row in one CTA's registers
constexpr int kMaxPositions = 1024;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 4096;
constexpr int64_t kMaxUnits = (int64_t(1) << 31) - 4096;  // a CTA counts one round past them in 32 bits

bool format_ok(int32_t f) { return f >= MOE_MX_BF16 && f <= MOE_MX_NVFP4; }
bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool weights_dims_ok(const moe_mx_weights* w) {
  return format_ok(w->format) && w->num_experts >= 1 && w->num_experts <= kMaxExpertsMx && w->n_out >= 1 &&
         w->n_out <= kMaxCols && w->k >= 32 && w->k <= kMaxCols && w->k % 32 == 0 &&
         (!w->swiglu || w->n_out % 32 == 0);
}

bool overlaps(const void* p, size_t pn, const void* q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + qn && b < a + pn;
}

moe_status rows_check(int32_t format, int64_t n, int32_t k, int32_t d, int64_t out_rows) {
  if (n < 0 || k < 1 || out_rows < 0) return MOE_ERR_INVALID_ARG;
  if (!format_ok(format) || d < 32 || d > kMaxRowCols || d % 32 != 0 || k > kMaxPositions || n > kMaxRows / k ||
      out_rows > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Arguments that moe_mx_quantise and moe_mx_add_rmsnorm share.
bool rows_args_ok(const MxRowsLaunch& a, int32_t format, bool norm) {
  const bool mx = format != MOE_MX_BF16;
  if (!a.x || !a.codes || (mx && !a.scales) || !is_aligned(a.x, 16) || !is_aligned(a.codes, 16) ||
      (mx && !is_aligned(a.scales, 16)) || a.x_ld < a.d || a.x_ld % 8 != 0 || (!a.positions && a.k != 1))
    return false;
  if (!norm) return true;
  return a.gain && is_aligned(a.gain, 16) && a.eps >= 0.f && (!a.residual || is_aligned(a.residual, 16)) &&
         (!a.sum || is_aligned(a.sum, 16)) && ((!a.residual && !a.sum) || (a.r_ld >= a.d && a.r_ld % 8 == 0)) &&
         (!a.sum || a.sum != a.x || a.r_ld == a.x_ld);
}

moe_status product_check(const moe_mx_weights* w, int64_t rows) {
  if (!w || rows < 0) return MOE_ERR_INVALID_ARG;
  if (!weights_dims_ok(w) || rows > kMaxRows ||
      (rows / 128 + w->num_experts) * mx_unit_rows(w) >= kMaxUnits)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool operands_ok(const moe_mx_weights* w, const void* x_codes, const void* x_scales, const int32_t* offsets) {
  return w->packed && is_aligned(w->packed, 16) && x_codes && is_aligned(x_codes, 16) && offsets &&
         (w->format == MOE_MX_BF16 || (x_scales && is_aligned(x_scales, 16)));
}

// ---------------------------------------------------------------- the layer's workspace
struct LayerLayout {
  size_t route = 0, counts = 0, offsets = 0, sorted_pos = 0, inv_pos = 0, x_codes = 0, x_scales = 0, h_codes = 0,
         h_scales = 0, rows = 0, total = 0;
};

bool layer_layout(const moe_mx_weights* gu, const moe_mx_weights* dn, int32_t k, int64_t n, LayerLayout* L) {
  if (!gu || !dn || n < 0 || k < 1 || k > 32 || !weights_dims_ok(gu) || !weights_dims_ok(dn) || !gu->swiglu ||
      dn->swiglu || gu->format != dn->format || gu->num_experts != dn->num_experts || gu->n_out != dn->k ||
      gu->k != dn->n_out || gu->k % 128 != 0 || gu->k > kMaxRowCols || n > kMaxRows / k)
    return false;
  const int64_t R = n * k;
  if (product_check(gu, R) != MOE_OK || product_check(dn, R) != MOE_OK) return false;
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 1023) & ~size_t(1023);
    return at;
  };
  const int32_t f = gu->format;
  L->route = take(4 * static_cast<size_t>(route_scratch_ints(R, gu->num_experts)));
  L->counts = take(4 * static_cast<size_t>(gu->num_experts));
  L->offsets = take(4 * static_cast<size_t>(gu->num_experts + 1));
  L->sorted_pos = take(4 * static_cast<size_t>(R));
  L->inv_pos = take(4 * static_cast<size_t>(R));
  L->x_codes = take(R * moe_mx_code_bytes(f, gu->k));
  L->x_scales = take(R * moe_mx_scale_pitch(f, gu->k));
  L->h_codes = take(R * moe_mx_code_bytes(f, dn->k));
  L->h_scales = take(R * moe_mx_scale_pitch(f, dn->k));
  L->rows = take(2 * static_cast<size_t>(R) * gu->k);
  L->total = off;
  return true;
}

template <typename T>
T* ws_at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// moe_mx_layer_forward; the errors go to *err, or to the workspace's word, set back first, where it is null.
moe_status layer_forward(const moe_mx_weights* gu, const moe_mx_weights* dn, int32_t top_k, int64_t n, const void* x,
                         const void* residual, const void* gain, float eps, const int32_t* topk_ids,
                         const float* topk_weight, const float* x_global, const float* h_global, void* sum, void* out,
                         int32_t out_is_fp32, void* ws, size_t ws_bytes, uint32_t* err, cudaStream_t s) {
  if (!gu || !dn || n < 0) return MOE_ERR_INVALID_ARG;
  LayerLayout L;
  if (!layer_layout(gu, dn, top_k, n, &L)) return MOE_ERR_UNSUPPORTED;
  if (!ws || !is_aligned(ws, 256) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (n == 0) return MOE_OK;
  if (!x || !topk_ids || !topk_weight || !out || !is_aligned(x, 16) || !is_aligned(out, 16) || !gu->packed ||
      !dn->packed || !is_aligned(gu->packed, 16) || !is_aligned(dn->packed, 16))
    return MOE_ERR_INVALID_ARG;
  if (gain ? (!sum || !is_aligned(sum, 16) || !is_aligned(gain, 16) || !(eps >= 0.f) ||
              (residual && !is_aligned(residual, 16)))
           : (sum || residual))
    return MOE_ERR_INVALID_ARG;
  const int32_t f = gu->format, d = gu->k, R = static_cast<int32_t>(n * top_k);
  const bool reset = err == nullptr;
  if (reset) err = static_cast<uint32_t*>(ws);
  int32_t* offsets = ws_at<int32_t>(ws, L.offsets);
  int32_t* sorted_pos = ws_at<int32_t>(ws, L.sorted_pos);
  int32_t* inv_pos = ws_at<int32_t>(ws, L.inv_pos);
  if (launch_route_permute(topk_ids, static_cast<int32_t>(n), top_k, gu->num_experts, ws_at<int32_t>(ws, L.counts),
                           offsets, sorted_pos, inv_pos, 0, ws_at<int32_t>(ws, L.route), err, 0, nullptr, nullptr, s,
                           reset) != cudaSuccess)
    return MOE_ERR_CUDA;
  MxRowsLaunch a{};
  a.n = n;
  a.k = top_k;
  a.d = d;
  a.x = static_cast<const uint16_t*>(x);
  a.x_ld = d;
  a.residual = static_cast<const uint16_t*>(residual);
  a.r_ld = d;
  a.gain = static_cast<const uint16_t*>(gain);
  a.eps = eps;
  a.positions = inv_pos;
  a.global = x_global;
  a.out_rows = R;
  a.sum = static_cast<uint16_t*>(sum);
  a.codes = ws_at<uint8_t>(ws, L.x_codes);
  a.scales = ws_at<uint8_t>(ws, L.x_scales);
  a.late = 1;
  if (launch_mx_rows(f, a, s) != cudaSuccess) return MOE_ERR_CUDA;

  MxProductLaunch g{};
  g.w = gu;
  g.rows = R;
  g.x_codes = a.codes;
  g.x_scales = a.scales;
  g.x_global = x_global;
  g.offsets = offsets;
  g.h_global = h_global;
  g.h_codes = ws_at<uint8_t>(ws, L.h_codes);
  g.h_scales = ws_at<uint8_t>(ws, L.h_scales);
  g.err = err;
  g.num_sms = device_sms();
  g.next = dn;
  g.early = true;  // the routing plan was complete before the rows' kernel began
  if (g.num_sms <= 0 || launch_mx_product(g, s) != cudaSuccess) return MOE_ERR_CUDA;

  MxProductLaunch q{};
  q.w = dn;
  q.rows = R;
  q.x_codes = g.h_codes;
  q.x_scales = g.h_scales;
  q.x_global = h_global;
  q.offsets = offsets;
  // The experts' weighted rows are f16 until the combine's fp32 sum, as moe_infer's are: 11 bits, where a bf16
  // output keeps 8, in half the bytes of fp32 (4096 tokens of 8 experts x 7168: 470 MB written and read again, 140
  // of the block's 1620 us).  Below 2^-14 they lose last bits, 2^-25 at most; beyond 65504 they raise MOE_ERR_RANGE.
  q.out = ws_at<void>(ws, L.rows);
  q.out_f16 = 1;
  q.out_rows = R;
  q.out_ld = d;
  q.out_pos = sorted_pos;
  q.row_weight = topk_weight;
  q.err = err;
  q.num_sms = g.num_sms;
  q.early = true;
  if (launch_mx_product(q, s) != cudaSuccess) return MOE_ERR_CUDA;
  return launch_combine(static_cast<const uint16_t*>(q.out), nullptr, static_cast<const uint16_t*>(sum),
                        static_cast<int32_t>(n), top_k, d, out, out_is_fp32, s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mx_code_bytes(int32_t f, int64_t cols) {
  if (!format_ok(f) || cols <= 0 || cols % 32 != 0) return 0;
  return static_cast<size_t>(f == MOE_MX_BF16 ? 2 * cols : f == MOE_MX_MXFP8 ? cols : cols / 2);
}

size_t moe_mx_scale_pitch(int32_t f, int64_t cols) {
  if (f == MOE_MX_BF16 || moe_mx_code_bytes(f, cols) == 0) return 0;
  return static_cast<size_t>((cols / mx_group(f) + 15) / 16 * 16);
}

moe_status moe_mx_quantise(int32_t format, int64_t n, int32_t k, int32_t d, const void* x, int64_t x_ld,
                           const int32_t* positions, const float* global, int64_t out_rows, void* codes, void* scales,
                           cudaStream_t s) {
  const moe_status st = rows_check(format, n, k, d, out_rows);
  if (st != MOE_OK || n == 0) return st;
  MxRowsLaunch a{};
  a.n = n;
  a.k = k;
  a.d = d;
  a.x = static_cast<const uint16_t*>(x);
  a.x_ld = x_ld;
  a.positions = positions;
  a.global = global;
  a.out_rows = out_rows;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  if (!rows_args_ok(a, format, false)) return MOE_ERR_INVALID_ARG;
  return launch_mx_rows(format, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mx_add_rmsnorm(int32_t format, int64_t n, int32_t k, int32_t d, const void* x, int64_t x_ld,
                              const void* residual, int64_t r_ld, const void* gain, float eps,
                              const int32_t* positions, const float* global, int64_t out_rows, void* sum, void* codes,
                              void* scales, cudaStream_t s) {
  const moe_status st = rows_check(format, n, k, d, out_rows);
  if (st != MOE_OK || n == 0) return st;
  MxRowsLaunch a{};
  a.n = n;
  a.k = k;
  a.d = d;
  a.x = static_cast<const uint16_t*>(x);
  a.x_ld = x_ld;
  a.residual = static_cast<const uint16_t*>(residual);
  a.r_ld = r_ld;
  a.gain = static_cast<const uint16_t*>(gain);
  a.eps = eps;
  a.positions = positions;
  a.global = global;
  a.out_rows = out_rows;
  a.sum = static_cast<uint16_t*>(sum);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  if (!rows_args_ok(a, format, true)) return MOE_ERR_INVALID_ARG;
  return launch_mx_rows(format, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mx_dequantise(int32_t format, int64_t rows, int32_t d, const void* codes, const void* scales,
                             const float* global, void* out, int64_t out_ld, cudaStream_t s) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (!format_ok(format) || d < 32 || d > kMaxCols || d % 32 != 0 || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!codes || !out || (format != MOE_MX_BF16 && !scales) || !is_aligned(codes, 16) || !is_aligned(out, 16) ||
      (format != MOE_MX_BF16 && !is_aligned(scales, 16)) || out_ld < d || out_ld % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  return launch_mx_dequantise(format, rows, d, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                              global, static_cast<uint16_t*>(out), out_ld, s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

size_t moe_mx_packed_bytes(const moe_mx_weights* w) {
  if (!w || !weights_dims_ok(w)) return 0;
  return static_cast<size_t>(w->num_experts * mx_unit_rows(w) * mx_chunks(w) * mx_block_bytes(w->format));
}

moe_status moe_mx_pack_weights(const moe_mx_weights* w, const void* codes, const void* scales, const void* codes_up,
                               const void* scales_up, void* packed, cudaStream_t s) {
  if (!w) return MOE_ERR_INVALID_ARG;
  if (!weights_dims_ok(w) || w->num_experts * mx_unit_rows(w) * mx_chunks(w) >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  const bool mx = w->format != MOE_MX_BF16, sw = w->swiglu != 0;
  const size_t rows = static_cast<size_t>(w->num_experts) * w->n_out;
  const size_t cb = rows * moe_mx_code_bytes(w->format, w->k), sb = rows * moe_mx_scale_pitch(w->format, w->k);
  if (!packed || !is_aligned(packed, 16)) return MOE_ERR_INVALID_ARG;
  const void* src[4] = {codes, mx ? scales : nullptr, sw ? codes_up : nullptr, mx && sw ? scales_up : nullptr};
  const bool need[4] = {true, mx, sw, mx && sw};
  for (int i = 0; i < 4; ++i)
    if (need[i] && (!src[i] || !is_aligned(src[i], 16) ||
                    overlaps(src[i], i & 1 ? sb : cb, packed, moe_mx_packed_bytes(w))))
      return MOE_ERR_INVALID_ARG;
  return launch_mx_pack(w, static_cast<const uint8_t*>(src[0]), static_cast<const uint8_t*>(src[1]),
                        static_cast<const uint8_t*>(src[2]), static_cast<const uint8_t*>(src[3]),
                        static_cast<uint8_t*>(packed), s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_mx_grouped_product(const moe_mx_weights* w, int64_t rows, const void* x_codes, const void* x_scales,
                                  const float* x_global, const int32_t* expert_offsets, void* out, int32_t out_type,
                                  int64_t out_rows, int64_t out_ld, const int32_t* out_pos, const float* row_weight,
                                  void* ws, size_t ws_bytes, cudaStream_t s) {
  const moe_status st = product_check(w, rows);
  if (st != MOE_OK) return st;
  if (w->swiglu || out_rows < 0 || (out_type != MOE_MX_OUT_BF16 && out_type != MOE_MX_OUT_F16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256) || ws_bytes < MOE_MX_PRODUCT_WORKSPACE) return MOE_ERR_WORKSPACE;
  if (rows == 0) return MOE_OK;
  if (!operands_ok(w, x_codes, x_scales, expert_offsets) || !out || !is_aligned(out, 2) || out_ld < w->n_out)
    return MOE_ERR_INVALID_ARG;
  MxProductLaunch g{};
  g.w = w;
  g.rows = static_cast<int32_t>(rows);
  g.x_codes = static_cast<const uint8_t*>(x_codes);
  g.x_scales = static_cast<const uint8_t*>(x_scales);
  g.x_global = x_global;
  g.offsets = expert_offsets;
  g.out = out;
  g.out_f16 = out_type == MOE_MX_OUT_F16;
  g.out_rows = out_rows;
  g.out_ld = out_ld;
  g.out_pos = out_pos;
  g.row_weight = row_weight;
  g.err = static_cast<uint32_t*>(ws);
  g.num_sms = device_sms();
  if (g.num_sms <= 0) return MOE_ERR_CUDA;
  return launch_mx_product(g, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mx_grouped_swiglu(const moe_mx_weights* w, int64_t rows, const void* x_codes, const void* x_scales,
                                 const float* x_global, const int32_t* expert_offsets, const float* h_global,
                                 void* h_codes, void* h_scales, void* ws, size_t ws_bytes, cudaStream_t s) {
  const moe_status st = product_check(w, rows);
  if (st != MOE_OK) return st;
  if (!w->swiglu) return MOE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256) || ws_bytes < MOE_MX_PRODUCT_WORKSPACE) return MOE_ERR_WORKSPACE;
  if (rows == 0) return MOE_OK;
  if (!operands_ok(w, x_codes, x_scales, expert_offsets) || !h_codes || !is_aligned(h_codes, 16) ||
      (w->format != MOE_MX_BF16 && (!h_scales || !is_aligned(h_scales, 16))))
    return MOE_ERR_INVALID_ARG;
  MxProductLaunch g{};
  g.w = w;
  g.rows = static_cast<int32_t>(rows);
  g.x_codes = static_cast<const uint8_t*>(x_codes);
  g.x_scales = static_cast<const uint8_t*>(x_scales);
  g.x_global = x_global;
  g.offsets = expert_offsets;
  g.h_global = h_global;
  g.h_codes = static_cast<uint8_t*>(h_codes);
  g.h_scales = static_cast<uint8_t*>(h_scales);
  g.err = static_cast<uint32_t*>(ws);
  g.num_sms = device_sms();
  if (g.num_sms <= 0) return MOE_ERR_CUDA;
  return launch_mx_product(g, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_mx_layer_workspace_size(const moe_mx_weights* gate_up, const moe_mx_weights* down, int32_t top_k,
                                   int64_t n_tokens) {
  LayerLayout L;
  return layer_layout(gate_up, down, top_k, n_tokens, &L) ? L.total : 0;
}

moe_status moe_mx_layer_forward(const moe_mx_weights* gu, const moe_mx_weights* dn, int32_t top_k, int64_t n,
                                const void* x, const void* residual, const void* gain, float eps,
                                const int32_t* topk_ids, const float* topk_weight, const float* x_global,
                                const float* h_global, void* sum, void* out, int32_t out_is_fp32, void* ws,
                                size_t ws_bytes, cudaStream_t s) {
  return layer_forward(gu, dn, top_k, n, x, residual, gain, eps, topk_ids, topk_weight, x_global, h_global, sum, out,
                       out_is_fp32, ws, ws_bytes, nullptr, s);
}

// ---------------------------------------------------------------- calls without a workspace (mx_default.h)

void* moe_mx_default_workspace(void) {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, mx_default_ws) == cudaSuccess ? p : nullptr;
}

moe_status moe_mx_layer_forward_default(const moe_mx_weights* gu, const moe_mx_weights* dn, int32_t top_k, int64_t n,
                                        const void* x, const void* residual, const void* gain, float eps,
                                        const int32_t* topk_ids, const float* topk_weight, const float* x_global,
                                        const float* h_global, void* sum, void* out, int32_t out_is_fp32, void* ws,
                                        size_t ws_bytes, cudaStream_t s) {
  if (!gu || !dn || n < 0) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  uint32_t* err = static_cast<uint32_t*>(moe_mx_default_workspace());
  if (!err) return MOE_ERR_CUDA;
  return layer_forward(gu, dn, top_k, n, x, residual, gain, eps, topk_ids, topk_weight, x_global, h_global, sum, out,
                       out_is_fp32, ws, ws_bytes, err, s);
}

}  // extern "C"
