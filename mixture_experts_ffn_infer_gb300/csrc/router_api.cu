// C ABI of the router's operators (moe_router.h): argument checks, workspace
// layout and launches.
#include <cuda_runtime.h>

#include "router.cuh"

namespace moe {
namespace {

constexpr int kMaxRouterExperts = 1024, kMaxTopK = 32, kMaxGroups = 32;
constexpr int64_t kMaxSequences = 65536, kMaxRouterRows = (int64_t(1) << 31) - 4096;

bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t logit_bytes(const moe_router* r) { return r->logits_type == MOE_LOGITS_F32 ? 4 : 2; }

// The struct, and the number of rows.
moe_status router_check(const moe_router* r, int64_t n) {
  if (!r || n < 0) return MOE_ERR_INVALID_ARG;
  if (r->num_experts < 1 || r->num_experts > kMaxRouterExperts || r->top_k < 1 || r->top_k > kMaxTopK ||
      r->top_k > r->num_experts || (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) ||
      (r->logits_type != MOE_LOGITS_F32 && r->logits_type != MOE_LOGITS_BF16) || n > kMaxRouterRows / r->top_k)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool rows_ok(const moe_router* r, const void* p, int64_t ld) {
  return p && is_aligned(p, logit_bytes(r)) && ld >= r->num_experts;
}

// Where the workspace's arrays begin; total 0: unsupported.
struct BalanceLayout {
  size_t parts = 0, sums = 0, hist = 0, total = 0;
};
BalanceLayout balance_layout(const moe_router* r, int64_t n, int64_t sequences) {
  BalanceLayout L;
  const size_t pieces = static_cast<size_t>(balance_plan(n).chunks + sequences);
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) & ~size_t(255);
    return at;
  };
  L.parts = take(4 * static_cast<size_t>(sequences) * balance_parts(r->num_experts));
  L.sums = take(4 * pieces * r->num_experts);
  L.hist = take(4 * pieces * r->num_experts);
  L.total = off;
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route(const moe_router* r, int64_t n, const void* logits, int64_t logits_ld, const float* bias,
                     int32_t* topk_ids, float* topk_weight, cudaStream_t s) {
  const moe_status st = router_check(r, n);
  if (st != MOE_OK) return st;
  if (r->groups < 1 || r->groups > kMaxGroups || r->num_experts % r->groups != 0 || r->top_groups < 1 ||
      r->top_groups > r->groups || r->top_k > r->top_groups * (r->num_experts / r->groups))
    return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!rows_ok(r, logits, logits_ld) || !topk_ids || !topk_weight || !is_aligned(topk_ids, 4) ||
      !is_aligned(topk_weight, 4) || !is_aligned(bias, 4))
    return MOE_ERR_INVALID_ARG;
  RouteLaunch a{*r, n, logits, logits_ld, bias, topk_ids, topk_weight};
  return launch_route(a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_balance_workspace_size(const moe_router* r, int64_t n, int64_t sequences) {
  if (router_check(r, n) != MOE_OK || sequences < 1 || sequences > kMaxSequences) return 0;
  return balance_layout(r, n, sequences).total;
}

moe_status moe_balance_loss(const moe_router* r, int64_t n, const void* logits, int64_t logits_ld,
                            const int32_t* topk_ids, float coef, const int32_t* seq_offsets, int64_t sequences,
                            int32_t* counts, float* loss, void* ws, size_t ws_bytes, cudaStream_t s) {
  const moe_status st = router_check(r, n);
  if (st != MOE_OK) return st;
  if (sequences < 1 || (!seq_offsets && sequences != 1)) return MOE_ERR_INVALID_ARG;
  if (sequences > kMaxSequences) return MOE_ERR_UNSUPPORTED;
  const BalanceLayout L = balance_layout(r, n, sequences);
  if (!ws || !is_aligned(ws, 256) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (!counts || !loss || !is_aligned(counts, 4) || !is_aligned(loss, 4) || !is_aligned(seq_offsets, 4) ||
      !is_aligned(topk_ids, 4) || (n > 0 && (!rows_ok(r, logits, logits_ld) || !topk_ids)))
    return MOE_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  BalanceLaunch a{};
  a.r = *r;
  a.n = n;
  a.logits = logits;
  a.ld = logits_ld;
  a.ids = topk_ids;
  a.coef = coef;
  a.offsets = seq_offsets;
  a.sequences = static_cast<int32_t>(sequences);
  a.counts = counts;
  a.loss = loss;
  a.ticket = reinterpret_cast<uint32_t*>(base);
  a.parts = reinterpret_cast<float*>(base + L.parts);
  a.sums = reinterpret_cast<float*>(base + L.sums);
  a.hist = reinterpret_cast<int32_t*>(base + L.hist);
  return launch_balance(a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_route_backward(const moe_router* r, int64_t n, const void* logits, int64_t logits_ld,
                              const int32_t* topk_ids, const float* d_weight, float coef, const int32_t* counts,
                              const float* d_loss, const int32_t* seq_offsets, int64_t sequences, void* d_logits,
                              int64_t d_ld, cudaStream_t s) {
  const moe_status st = router_check(r, n);
  if (st != MOE_OK) return st;
  if (counts) {
    if (sequences < 1 || (!seq_offsets && sequences != 1)) return MOE_ERR_INVALID_ARG;
    if (sequences > kMaxSequences) return MOE_ERR_UNSUPPORTED;
  }
  if (n == 0) return MOE_OK;
  if (!rows_ok(r, logits, logits_ld) || !rows_ok(r, d_logits, d_ld) || (d_weight && !topk_ids) ||
      (d_logits == logits && d_ld != logits_ld) || !is_aligned(topk_ids, 4) || !is_aligned(d_weight, 4) ||
      !is_aligned(counts, 4) || !is_aligned(d_loss, 4) || !is_aligned(seq_offsets, 4))
    return MOE_ERR_INVALID_ARG;
  RouteGradLaunch a{};
  a.r = *r;
  a.n = n;
  a.logits = logits;
  a.ld = logits_ld;
  a.ids = topk_ids;
  a.d_weight = d_weight;
  a.coef = coef;
  a.counts = counts;
  a.d_loss = d_loss;
  a.offsets = seq_offsets;
  a.sequences = counts ? static_cast<int32_t>(sequences) : 0;
  a.d_logits = d_logits;
  a.d_ld = d_ld;
  return launch_route_grad(a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
