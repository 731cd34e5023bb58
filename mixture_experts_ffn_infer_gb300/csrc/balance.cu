// The router's balance loss and the gradient of its logits (moe_router.h).
//
// The loss needs sum_t q[t][e] per sequence and the counts, and multiplies them at the
// end, so one pass over the logits is enough, and the counts need not come first:
//  balance_rows_kernel  a CTA takes a run of rows; a warp adds its rows' shares in
//                       registers, E / 32 experts a lane.  Where a sequence ends inside the
//                       run, and at its end, the warps' sums are joined and written as one
//                       piece.  CTA c and sequence s meet at most once, and c + s names the
//                       pieces in order.
//  balance_loss_kernel  adds each sequence's pieces in that order, 32 experts to a CTA; the
//                       last CTA adds the sequences.
// No float is added atomically: the result does not depend on the order of the CTAs.
//
// route_grad_kernel      both parts of the gradient in one pass, read and write once:
//   ds = d_weight through the weights' normalisation, at the chosen experts
//   softmax   dl = s (ds + c - sum (ds + c) s)
//   sigmoid   dl = s (1 - s) (ds + (c - sum c q) / sum s)
// with c[e] = d_loss coef E / (S k T^2) count_e.  All three are bound by HBM.
#include "router.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRowWarps = 8;
constexpr float kTiny = 1e-20f;

// The shares q of a row (sum 1, or all 0 where every logit is -inf).
template <typename Row>
__device__ __forceinline__ void shares(bool sigmoid, const float (&l)[Row::width], float (&q)[Row::width]) {
  constexpr int V = Row::width;
  if (sigmoid) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q[i] = sigmoid_of(l[i]);
      sum += q[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);  // (a masked row's shares are 0)
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] *= inv;
  } else {
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
    softmax_row(l, warp_max_nan(top), q);
  }
}

// Row ranges of sequence s, held within [0, n] whatever the offsets say.
__device__ __forceinline__ int64_t offset_at(const int32_t* offsets, int64_t n, int s) {
  if (!offsets) return s == 0 ? 0 : n;
  const int64_t o = __ldg(offsets + s);
  return o < 0 ? 0 : o > n ? n : o;
}
// The first sequence that ends behind row t (the number of sequences: none).
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int sequences, int64_t n, int64_t t) {
  int lo = 0, hi = sequences;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offset_at(offsets, n, mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

template <typename Row>
__global__ void __launch_bounds__(32 * kRowWarps, Row::width <= 12 ? 4 : 1)
balance_rows_kernel(const BalanceLaunch a, const BalancePlan plan) {
  using T = typename Row::type;
  constexpr int V = Row::width;
  extern __shared__ float joined[];  // [warps][E], then the counts [E]
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.r.num_experts, k = a.r.top_k;
  const bool sigmoid = a.r.score == MOE_SCORE_SIGMOID;
  int32_t* hist = reinterpret_cast<int32_t*>(joined + kRowWarps * E);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  const int64_t r0 = blockIdx.x * plan.chunk, r1 = min(r0 + plan.chunk, a.n);
  __syncthreads();
  for (int s = sequence_of(a.offsets, a.sequences, a.n, r0); s < a.sequences; ++s) {
    const int64_t lo = max(r0, offset_at(a.offsets, a.n, s)), hi = min(r1, offset_at(a.offsets, a.n, s + 1));
    if (lo >= r1) break;
    if (lo >= hi) continue;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    const T* logits = static_cast<const T*>(a.logits);
    float l[V];
    if (lo + warp < hi) Row::load(logits + (lo + warp) * a.ld, E, lane, -kInf, l);
    for (int64_t t = lo + warp; t < hi; t += kRowWarps) {
      float q[V];
      shares<Row>(sigmoid, l, q);
      if (t + kRowWarps < hi) Row::load(logits + (t + kRowWarps) * a.ld, E, lane, -kInf, l);
      if (lane < k) {
        const int id = a.ids[t * k + lane];
        if (id >= 0 && id < E) atomicAdd(hist + id, 1);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += q[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (Row::expert(i, lane) < E) joined[warp * E + Row::expert(i, lane)] = sum[i];
    __syncthreads();
    const int64_t piece = static_cast<int64_t>(blockIdx.x) + s;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) v += joined[w * E + e];
      a.sums[piece * E + e] = v;
      a.hist[piece * E + e] = hist[e];
      hist[e] = 0;
    }
    __syncthreads();
  }
}

// Grid (parts, sequences): 32 experts of a sequence, a warp every eighth piece.
__global__ void __launch_bounds__(256)
balance_loss_kernel(const BalanceLaunch a, const BalancePlan plan) {
  __shared__ float psum[8][32];
  __shared__ int pcount[8][32];
  __shared__ double total[8];
  __shared__ int lives[8];
  __shared__ bool last;
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.r.num_experts, parts = gridDim.x;
  const int e = blockIdx.x * 32 + lane;
  for (int s = blockIdx.y; s < a.sequences; s += gridDim.y) {
    const int64_t lo = offset_at(a.offsets, a.n, s), hi = offset_at(a.offsets, a.n, s + 1);
    float sum = 0.f;
    int count = 0;
    if (lo < hi && e < E) {
      const int64_t c1 = (hi - 1) / plan.chunk;
#pragma unroll 4
      for (int64_t c = lo / plan.chunk + warp; c <= c1; c += 8) {
        sum += a.sums[(c + s) * E + e];
        count += a.hist[(c + s) * E + e];
      }
    }
    psum[warp][lane] = sum;
    pcount[warp][lane] = count;
    __syncthreads();
    if (warp == 0) {
      sum = 0.f;
      count = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) sum += psum[w][lane], count += pcount[w][lane];
      if (e < E) a.counts[static_cast<int64_t>(s) * E + e] = count;
      const float rows = static_cast<float>(hi - lo), part = warp_sum(static_cast<float>(count) * sum) / (rows * rows);
      if (lane == 0) a.parts[static_cast<int64_t>(s) * parts + blockIdx.x] = part;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0;
  int live = 0;
  bool bad = false;  // offsets that do not ascend within the rows
  for (int s = threadIdx.x; s < a.sequences; s += blockDim.x) {
    if (a.offsets) {
      const int64_t o0 = __ldg(a.offsets + s), o1 = __ldg(a.offsets + s + 1);
      bad |= o0 < 0 || o1 < o0 || o1 > a.n;
    }
    if (offset_at(a.offsets, a.n, s + 1) <= offset_at(a.offsets, a.n, s)) continue;
    ++live;
    float part = 0.f;
    for (int i = 0; i < parts; ++i) part += __ldcg(a.parts + static_cast<int64_t>(s) * parts + i);
    sum += part;
  }
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(kAll, sum, o);
    live += __shfl_xor_sync(kAll, live, o);
  }
  if (lane == 0) total[warp] = sum, lives[warp] = live;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    live = 0;
    for (int w = 0; w < 8; ++w) sum += total[w], live += lives[w];
    const double factor = static_cast<double>(a.coef) * E / a.r.top_k;
    *a.loss = bad ? kNaN : live ? static_cast<float>(sum * factor / live) : 0.f;
  }
}

// CTAs of the gradient that an SM holds.
template <typename Row>
constexpr int kGradResident = Row::width <= 12 ? 3 : Row::width <= 16 ? 2 : 1;

template <typename Row>
__global__ void __launch_bounds__(32 * kRowWarps, kGradResident<Row>)
route_grad_kernel(const RouteGradLaunch a, const int64_t run) {
  using T = typename Row::type;
  constexpr int V = Row::width;
  extern __shared__ float scatter[];  // [warps][E]: ds at the chosen experts, zeros elsewhere
  __shared__ int lives[kRowWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.r.num_experts, k = a.r.top_k;
  const bool sigmoid = a.r.score == MOE_SCORE_SIGMOID;
  float* ds = scatter + warp * E;
  for (int e = lane; e < E; e += 32) ds[e] = 0.f;
  float factor = 0.f;  // d_loss coef E / (S k)
  if (a.counts) {
    int live = 0;
    for (int s = threadIdx.x; s < a.sequences; s += blockDim.x)
      live += offset_at(a.offsets, a.n, s + 1) > offset_at(a.offsets, a.n, s) ? 1 : 0;
    live = __reduce_add_sync(kAll, live);
    if (lane == 0) lives[warp] = live;
    __syncthreads();
    live = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) live += lives[w];
    factor = (a.d_loss ? __ldg(a.d_loss) : 1.f) * (a.coef * static_cast<float>(E) / (static_cast<float>(k) * live));
  }
  __syncwarp();
  // a warp's rows follow one another, so that a sequence's counts stay in its registers
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp) * run, t1 = min(t0 + run, a.n);
  if (t0 >= t1) return;
  const T* logits = static_cast<const T*>(a.logits);
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 0.f;
  int seq = a.counts ? sequence_of(a.offsets, a.sequences, a.n, t0) : 0;
  int64_t until = t0;  // where c changes next
  for (int64_t t = t0; t < t1; ++t) {
    const T* p = logits + t * a.ld;
    float l[V];
    Row::load(p, E, lane, -kInf, l);
    int id = -1;
    float g = 0.f, lj = -kInf;
    if (a.d_weight && lane < k) {
      id = a.ids[t * k + lane];
      if (id < 0 || id >= E) id = -1;
      else g = a.d_weight[t * k + lane] * a.r.scale, lj = to_float(p[id]);
    }
    if (a.counts && t >= until) {
      // sequences that end at or in front of t are over; between two (and behind the last) there are none
      while (seq < a.sequences && offset_at(a.offsets, a.n, seq + 1) <= t) ++seq;
      const int64_t lo = seq < a.sequences ? offset_at(a.offsets, a.n, seq) : a.n,
                    hi = seq < a.sequences ? offset_at(a.offsets, a.n, seq + 1) : a.n;
      const bool in = lo <= t && t < hi;
      const float rows = static_cast<float>(hi - lo), f = in ? factor / (rows * rows) : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = Row::expert(i, lane);
        c[i] = in && e < E ? f * static_cast<float>(__ldg(a.counts + static_cast<int64_t>(seq) * E + e)) : 0.f;
      }
      until = in ? hi : lo > t ? lo : a.n;
    }
    float s[V], u[V];  // scores; sigmoid: e^-l s = 1 - s
    float dj;  // ds of the lane's chosen expert
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
    SoftmaxRow soft{0.f, 0.f};
    float total = 0.f;
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = sigmoid_of(l[i], u[i]);
        u[i] *= s[i];
        total += s[i];
      }
    } else {
      top = warp_max_nan(top);
      soft = softmax_row(l, top, s);
    }
    const bool bad = __any_sync(kAll, top != top || (!sigmoid && top == kInf));
    if (a.d_weight) {
      dj = g;
      if (a.r.normalise) {
        const float sj = id < 0 ? 0.f : sigmoid ? sigmoid_of(lj) : softmax_term(lj, soft.shift) * soft.inv;
        const float sum = warp_sum(sj) + kTiny, dot = warp_sum(g * sj);
        dj = __fdividef(g - __fdividef(dot, sum), sum);
      }
      const uint32_t same = __match_any_sync(kAll, id);
      if (__any_sync(kAll, id >= 0 && (same & (same - 1u)) != 0)) {
        // an expert named twice: its entries in order
        for (int j = 0; j < k; ++j) {
          if (lane == j && id >= 0) ds[id] += dj;
          __syncwarp();
        }
      } else if (id >= 0) {
        ds[id] = dj;
      }
      __syncwarp();
    }
    float d[V];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = Row::expert(i, lane);
      d[i] = a.d_weight && e < E ? ds[e] : 0.f;
    }
    if (a.d_weight) {
      __syncwarp();
      if (id >= 0) ds[id] = 0.f;
    }
    if (sigmoid) {
      if (a.counts) {
#pragma unroll
        for (int i = 0; i < V; ++i) dot = fmaf(c[i], s[i], dot);
        total = warp_sum(total);
        dot = warp_sum(dot);
        const float inv = total == 0.f ? 0.f : __frcp_rn(total);
        dot *= inv;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = fmaf(c[i] - dot, inv, d[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = d[i] * s[i] * u[i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] += c[i];
        dot = fmaf(d[i], s[i], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = s[i] * (d[i] - dot);
    }
    if (bad) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = kNaN;
    }
    Row::store(static_cast<T*>(a.d_logits) + t * a.d_ld, E, lane, d);
    __syncwarp();
  }
}

}  // namespace

BalancePlan balance_plan(int64_t n) {
  // Runs of eight rows a warp at least, four CTAs an SM at most.
  constexpr int64_t kMost = 608, kLeast = 64;
  int64_t chunk = (n + kMost - 1) / kMost;
  if (chunk < kLeast) chunk = kLeast;
  if (chunk > n) chunk = n < 1 ? 1 : n;
  const int64_t chunks = (n + chunk - 1) / chunk;
  return BalancePlan{chunk, static_cast<int32_t>(chunks < 1 ? 1 : chunks)};  // without rows one CTA, for the ticket
}

cudaError_t launch_balance(const BalanceLaunch& a, cudaStream_t s) {
  const BalancePlan plan = balance_plan(a.n);
  const size_t smem = (kRowWarps + 1) * sizeof(float) * a.r.num_experts;
  cudaError_t e = with_row(a.r, rows_by_four(a.r, a.logits, a.ld), [&](auto row) {
    return launch_maybe_overlapped(balance_rows_kernel<decltype(row)>, plan.chunks, 32 * kRowWarps, smem, s, true, a, plan);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(balance_parts(a.r.num_experts)),
                     static_cast<unsigned>(a.sequences < 4096 ? a.sequences : 4096));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, balance_loss_kernel, a, plan);
}

cudaError_t launch_route_grad(const RouteGradLaunch& a, cudaStream_t s) {
  const int64_t sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidValue;
  int warps = 1;
  while (warps < kRowWarps && a.n > sms * warps) warps *= 2;
  const size_t smem = sizeof(float) * static_cast<size_t>(warps) * a.r.num_experts;
  const bool vec = rows_by_four(a.r, a.logits, a.ld) && rows_by_four(a.r, a.d_logits, a.d_ld);
  return with_row(a.r, vec, [&](auto row) {
    // one round of the CTAs that the SMs hold
    const int64_t most = sms * kGradResident<decltype(row)> * kRowWarps, run = (a.n + most - 1) / most;
    const int64_t ctas = (a.n + run * warps - 1) / (run * warps);
    return launch_maybe_overlapped(route_grad_kernel<decltype(row)>, static_cast<int>(ctas), 32 * warps, smem, s, true, a,
                                   run);
  });
}

}  // namespace moe
