// The router's choice of experts (moe_route in moe_router.h).
//
// A warp takes a row: its scores, the k largest and their weights in one read of the
// row.  HBM would bound it; what has to be kept below that is the number of
// instructions, of which a plain "largest, k times" over E / 32 values a lane would
// take most.  So
//  1. each lane's largest value, and the (k + 1)-th largest of the 32 (k + 1 warp
//     maxima): no value of the k + 1 largest is below it;
//  2. the values from there up, some k + 3, one to a lane;
//  3. these in order, by warp maxima over one value a lane.
// Step 2 finds more than 32 only where many values are equal; such rows take the slow
// way, k maxima over all values.
//
// The choice is that of the exact scores.  With a bias (or groups) fp32 scores order two
// experts wrongly where they are closer than the scores' errors: adjacent ones of the
// k + 1 largest that are closer than `tolerance` and not equal by their inputs send the
// row (one in a thousand of random ones) to the comparison in 64 bits.
#include "router.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kTiny = 1e-20f;

// Floats as integers of the same order, above 0, which stands for "not to be chosen".
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 is +0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint32_t key_if(bool on, float x) { return on && x > -kInf ? key_of(x) : 0u; }

// Scores in 64 bits.
__device__ __forceinline__ double exact_sigmoid(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }
__device__ __forceinline__ double exact_softmax(float l, float shift, double total) {
  return total > 0.0 ? exp(static_cast<double>(l) - static_cast<double>(shift)) / total : 0.0;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The bound of |difference of two fp32 choices - the exact one|, doubled for safety.  Sigmoid: expf within 2 ulp, the
// sum and the reciprocal 1 ulp each: below 2^-21 of a score, twice, and the sums with the bias 2^-24 each.  Softmax:
// besides these l - shift rounds (|l - shift| 2^-24 of the score, at most 104 of them before it is 0) and the row's
// sum has (V + 5) 2^-24.
__device__ __forceinline__ float tolerance(bool sigmoid, float s, float x) {
  return fmaf(sigmoid ? 0x1p-19f : 0x1p-15f, s, 0x1p-21f * fabsf(x));
}

struct Best {
  double x;
  int e;
};
// The warp's largest x, of equal ones the lowest e; e < 0: none.
__device__ __forceinline__ Best warp_best(Best b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double x = __shfl_xor_sync(kAll, b.x, o);
    const int e = __shfl_xor_sync(kAll, b.e, o);
    if (e >= 0 && (b.e < 0 || x > b.x || (x == b.x && e < b.e))) b = Best{x, e};
  }
  return b;
}

// The slow way, in 64 bits: lane j gets the j-th expert or -1.
template <typename Row>
__device__ __noinline__ int exact_choice(const moe_router r, const typename Row::type* p, const float* bias, int group_inv, int lane) {
  constexpr int V = Row::width;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  float l[V];
  Row::load(p, r.num_experts, lane, -kInf, l);
  double x[V];
  float top = -kInf;
#pragma unroll
  for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
  top = warp_max_nan(top);
  const float shift = top == -kInf ? 0.f : top;
  double total = 0.0;
  if (!sigmoid) {
#pragma unroll 1
    for (int i = 0; i < V; ++i) total += exp(static_cast<double>(l[i]) - static_cast<double>(shift));
    total = warp_sum(total);
  }
  uint32_t on = 0;  // bit i: value i can be chosen
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const int e = Row::expert(i, lane);
    if (e >= r.num_experts || !(l[i] > -kInf)) continue;
    const float b = bias ? bias[e] : 0.f;
    // without a bias the logits are in the scores' order (and keep it where scores round to 0 or 1)
    x[i] = sigmoid ? exact_sigmoid(l[i]) : exact_softmax(l[i], shift, total);
    x[i] += static_cast<double>(b);
    if (b > -kInf) on |= 1u << i;
  }
  if (r.groups > 1) {
    double value = 0.0;  // lane g: group g's
    bool any = false;
    for (int g = 0; g < r.groups; ++g) {
      Best one{0.0, -1}, two{0.0, -1};
#pragma unroll 1
      for (int i = 0; i < V; ++i) {
        const int e = Row::expert(i, lane);
        if (!(on >> i & 1u) || (e * group_inv) >> 20 != g) continue;
        if (one.e < 0 || x[i] > one.x) two = one, one = Best{x[i], e};
        else if (two.e < 0 || x[i] > two.x) two = Best{x[i], e};
      }
      const Best first = warp_best(one);
      const Best second = warp_best(one.e == first.e ? two : one);
      if (lane == g) {
        any = first.e >= 0;
        value = first.x + (second.e >= 0 ? second.x : 0.0);
      }
    }
    uint32_t kept = 0;
    Best mine{value, any ? lane : -1};
    for (int j = 0; j < r.top_groups; ++j) {
      const Best b = warp_best(mine);
      if (b.e < 0) break;
      kept |= 1u << b.e;
      if (b.e == lane) mine.e = -1;
    }
#pragma unroll 1
    for (int i = 0; i < V; ++i)
      if (!(kept >> (((Row::expert(i, lane) * group_inv) >> 20) & 31) & 1u)) on &= ~(1u << i);
  }
  int id = -1;
  for (int j = 0; j < r.top_k; ++j) {
    Best mine{0.0, -1};
    int at = 0;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
      const double xi = bias ? x[i] : static_cast<double>(l[i]);
      if ((on >> i & 1u) && (mine.e < 0 || xi > mine.x)) mine = Best{xi, Row::expert(i, lane)}, at = i;
    }
    const Best b = warp_best(mine);
    if (lane == j) id = b.e;
    if (b.e >= 0 && b.e == mine.e) on &= ~(1u << at);
  }
  return id;
}

template <typename Row>
__global__ void __launch_bounds__(32 * kWarps)
route_kernel(const RouteLaunch a, const int group_inv) {
  using T = typename Row::type;
  constexpr int V = Row::width;
  __shared__ int list[kWarps][32];
  extern __shared__ float group_row[];  // with groups: [warps][E]
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const moe_router& r = a.r;
  const int E = r.num_experts, k = r.top_k;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  const bool by_logit = a.bias == nullptr;  // the choice within the groups is the logits' order
  const int64_t rows = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp; t < a.n; t += rows) {
    const T* p = static_cast<const T*>(a.logits) + t * a.ld;
    float l[V], s[V];
    Row::load(p, E, lane, -kInf, l);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
    SoftmaxRow soft{0.f, 0.f};
    if (!sigmoid) {
      top = warp_max_nan(top);
      soft = softmax_row(l, top, s);
    } else if (!by_logit || r.groups > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = sigmoid_of(l[i]);
    }
    int32_t* ids = a.ids + t * k;
    float* weight = a.weight + t * k;
    if (__any_sync(kAll, top != top || (!sigmoid && top == kInf))) {
      if (lane < k) ids[lane] = -1, weight[lane] = kNaN;
      continue;
    }
    const float most = sigmoid ? 1.f : soft.inv;  // no score is larger
    uint32_t key[V];
    uint32_t local = 0;
    bool slow = false;
    if (by_logit && r.groups == 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key_if(true, l[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = Row::expert(i, lane);
        key[i] = key_if(e < E && l[i] > -kInf, s[i] + (a.bias && e < E ? __ldg(a.bias + e) : 0.f));
      }
    }
    if (r.groups > 1) {
      // A group's two largest: its experts over 32 / groups lanes (rounded down to a power of two).
      float* row = group_row + warp * E;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = Row::expert(i, lane);
        if (e < E) row[e] = __uint_as_float(key[i]);
      }
      __syncwarp();
      const int share = 1 << (31 - __clz(32 / r.groups)), size = E / r.groups;
      const int g = lane / share, first = g * size;
      uint32_t one = 0, two = 0;
      if (g < r.groups)
        for (int i = lane % share; i < size; i += share) {
          const uint32_t v = __float_as_uint(row[first + i]);
          two = max(two, min(one, v));
          one = max(one, v);
        }
      for (int o = share >> 1; o > 0; o >>= 1) {
        const uint32_t q1 = __shfl_xor_sync(kAll, one, o), q2 = __shfl_xor_sync(kAll, two, o);
        two = max(max(two, q2), min(one, q1));
        one = max(one, q1);
      }
      // one value a group, on its first lane
      const bool mine = lane % share == 0 && one != 0;
      const float sum = mine ? value_of(one) + (two ? value_of(two) : 0.f) : 0.f;
      uint32_t gk = mine ? key_of(sum) : 0u, kept = 0, last = 0;
      for (int j = 0; j < r.top_groups; ++j) {
        const uint32_t best = __reduce_max_sync(kAll, gk);
        if (best == 0) break;
        const int at = __ffs(__ballot_sync(kAll, gk == best)) - 1;
        kept |= 1u << (at / share);
        last = best;
        if (lane == at) gk = 0;
      }
      const uint32_t next = __reduce_max_sync(kAll, gk);
      if (next != 0) {
        const float x = value_of(last), y = value_of(next);
        const float size_of = fabsf(x) + fabsf(y);
        slow = !(x - y > tolerance(sigmoid, 4.f * most, size_of));  // of four scores
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = Row::expert(i, lane);
        if (!(kept >> ((e * group_inv >> 20) & 31) & 1u)) key[i] = 0u;
        else if (by_logit) key[i] = key_if(e < E, l[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) local = max(local, key[i]);
    // the (k + 1)-th largest of the lanes' largest (by logits the k-th: their order needs no margin)
    const int deep = by_logit ? k : k + 1;
    uint32_t from = 0;
    if (deep <= 32) {
      uint32_t left = local;
      for (int j = 0; j < deep; ++j) {
        from = __reduce_max_sync(kAll, left);
        if (from == 0) break;
        if (left == from) left = 0;
      }
    }
    if (!by_logit && from != 0) {
      const float x = value_of(from);
      const float low = x - tolerance(sigmoid, most, x);
      from = low > -kInf ? key_of(low) : 1u;
    }
    from = max(from, 1u);
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mask |= key[i] >= from ? 1u << i : 0u;
    int found = 0;
    for (uint32_t who; (who = __ballot_sync(kAll, mask != 0)) != 0;) {
      if (mask != 0) {
        const int at = found + __popc(who & ((1u << lane) - 1u));
        if (at < 32) list[warp][at] = Row::expert(__ffs(mask) - 1, lane);
        mask &= mask - 1;
      }
      found += __popc(who);
    }
    __syncwarp();
    // one of them to a lane
    const int e = lane < min(found, 32) ? list[warp][lane] : -1;
    __syncwarp();
    float cl = -kInf, cb = 0.f, cs = 0.f, cx = 0.f;
    if (e >= 0) {
      cl = to_float(p[e]);
      cs = sigmoid ? sigmoid_of(cl) : expf(cl - soft.shift) * soft.inv;
      if (a.bias) cb = __ldg(a.bias + e);
      cx = by_logit ? cl : cs + cb;
    }
    int id = -1, src = 0;
    float w = 0.f;
    if (found > 32) slow = true;
    if (!slow) {
      uint32_t ck = e >= 0 ? key_of(cx) : 0u, got = 0;
      for (int j = 0; j < deep; ++j) {
        const uint32_t best = __reduce_max_sync(kAll, ck);
        if (best == 0) break;
        const int first = __reduce_min_sync(kAll, ck == best ? e : 0x7fffffff);
        const int at = __ffs(__ballot_sync(kAll, e == first)) - 1;
        if (lane == j) id = first, src = at, got = best;
        if (lane == at) ck = 0;
      }
      if (!by_logit) {
        // lane j against the one behind it (lane 32 is not asked: deep is at most 32 here)
        const float x = value_of(got), sj = __shfl_sync(kAll, cs, src), lj = __shfl_sync(kAll, cl, src),
                    bj = __shfl_sync(kAll, cb, src);
        const uint32_t got1 = __shfl_down_sync(kAll, got, 1);
        const float s1 = __shfl_down_sync(kAll, sj, 1), l1 = __shfl_down_sync(kAll, lj, 1),
                    b1 = __shfl_down_sync(kAll, bj, 1);
        const bool close = lane < k && lane < 31 && got != 0 && got1 != 0 && !(lj == l1 && bj == b1) &&
                           !(x - value_of(got1) > tolerance(sigmoid, fmaxf(sj, s1), fabsf(x) + fabsf(value_of(got1))));
        if (__any_sync(kAll, close)) {
          // the same values in 64 bits
          double total = 0.0;
          if (!sigmoid) {
#pragma unroll 1
            for (int i = 0; i < V; ++i) {
              const int at = Row::expert(i, lane);
              if (at < E) total += exp(static_cast<double>(to_float(p[at])) - static_cast<double>(soft.shift));
            }
            total = warp_sum(total);
          }
          Best mine{0.0, e};
          if (e >= 0)
            mine.x = (sigmoid ? exact_sigmoid(cl) : exact_softmax(cl, soft.shift, total)) + static_cast<double>(cb);
          id = -1;
          for (int j = 0; j < k; ++j) {
            const Best b = warp_best(mine);
            if (b.e < 0) break;
            const int at = __ffs(__ballot_sync(kAll, e == b.e)) - 1;
            if (lane == j) id = b.e, src = at;
            if (lane == at) mine.e = -1;
          }
        }
      }
      w = __shfl_sync(kAll, cs, src);
      if (lane >= k || id < 0) id = -1, w = 0.f;
    } else {
      id = exact_choice<Row>(r, p, a.bias, group_inv, lane);
      if (lane >= k) id = -1;
      if (id >= 0) {
        const float li = to_float(p[id]);
        w = sigmoid ? sigmoid_of(li) : expf(li - soft.shift) * soft.inv;
      }
    }
    if (r.normalise) {
      // in fp32, over the chosen ones
      const float sum = warp_sum(w) + kTiny;
      w = __fdiv_rn(w, sum);
    }
    if (lane < k) ids[lane] = id, weight[lane] = w * r.scale;
  }
}

}  // namespace

cudaError_t launch_route(const RouteLaunch& a, cudaStream_t s) {
  const int size = a.r.num_experts / a.r.groups, inv = ((1 << 20) + size - 1) / size;  // e / size = e * inv >> 20
  // One warp a row; one row a CTA while there are SMs for it, so that a few rows do not share one.
  const int64_t sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidValue;
  int warps = 1;
  while (warps < kWarps && a.n > sms * warps) warps *= 2;
  const int64_t ctas = (a.n + warps - 1) / warps, most = sms * 16;
  const size_t smem = a.r.groups > 1 ? static_cast<size_t>(warps) * a.r.num_experts * sizeof(float) : 0;
  return with_row(a.r, rows_by_four(a.r, a.logits, a.ld), [&](auto row) {
    return launch_maybe_overlapped(route_kernel<decltype(row)>, static_cast<int>(ctas < most ? ctas : most), 32 * warps, smem,
                                   s, true, a, inv);
  });
}

}  // namespace moe
