// The router's choice of experts (moe_route in moe_router.h).
//
// HBM would bound it (32,768 rows of 384 fp32 logits: 7.9 us); what has to be kept below
// that is the number of instructions, of which a plain "largest, k times" over E / 32 values
// a lane would take most.  So a warp takes a row, or two (below), and in one read of it
//  1. each lane's largest value, and the (k + 1)-th largest of those (of the 16 larger ones of
//     pairs of lanes, by a sort): no value of the k + 1 largest is below it.  Scores here
//     are short ones;
//  2. the values from there up (less a margin for the short scores), some k + 3, one to
//     a lane, and their scores again, within 2^-21 of each;
//  3. the rank of each among them, by comparing with all: no step waits for the last.
// For k up to 15, step 2 finds more than 32 only where many values are equal or a few lanes hold
// most of the large ones; for the latter a sort of all lanes bounds them closer, the others
// take the slow way, k maxima over all values in 64 bits.  From there on the (k + 1)-th
// largest lies below most lanes' maxima, and ordinary rows take that way too: of random rows of
// 384 with a bias 0.4 % at k = 16, 40 % at 20, 98 % at 24.  8,192 x 384, sigmoid, us
// with k = 8, 12, 16, 20, 24, 32: 13, 17, 53, 326, 660, 818 with a bias, 10, 13, 53, 225, 648,
// 819 without.
//
// The choice is that of scores and biases in 64 bits.  With a bias (or groups) fp32 scores
// order two experts wrongly where they are closer than the scores' errors: neighbours among
// the k + 1 largest that are closer than `tolerance` and not equal by their inputs send the
// row (three in a thousand of random ones) to the same ranking in 64 bits.
//
// 32,768 x 384, sigmoid, bias, k = 8, on one GB300: 21 us with two rows a warp, 31 with one;
// some 700 instructions two rows, which the SMs issue in 60 % of the cycles, and 3 us of
// launch.  (Rows a pair ahead by cp.async: 26 us, for the accesses of shared memory that it
// takes; by a prefetch to L2, 22.)
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

// How far two fp32 choices' difference may be from the exact one, twice over.  A sigmoid is within 2^-21 of itself; a
// softmax term within 2^-21 too, its difference from the row's largest rounds (2^-24 of up to 104, below which it is 0)
// and the row's sum has (V + 5) 2^-24; the sums with the bias 2^-24 each.
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

// The rank of this lane's key among those of the lanes (0: none, lanes from `count` on have it), equal ones together.
__device__ __forceinline__ int rank_of(uint32_t key, int count) {
  int rank = 0;
#pragma unroll 1
  for (int j0 = 0; j0 < count; j0 += 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) rank += __shfl_sync(kAll, key, j0 + j) > key ? 1 : 0;
  }
  return rank;
}

// The same in 64 bits: the value is the exact score of logit l plus bias b.
template <typename Row>
__device__ __noinline__ int exact_rank(const typename Row::type* p, int E, bool sigmoid, float shift, float l, float b, int e,
                                       int count) {
  const int lane = threadIdx.x & 31;
  double total = 0.0;
  if (!sigmoid) {
#pragma unroll 1
    for (int at = lane; at < E; at += 32) total += exp(static_cast<double>(to_float(p[at])) - static_cast<double>(shift));
    total = warp_sum(total);
  }
  const double x = (sigmoid ? exact_sigmoid(l) : exact_softmax(l, shift, total)) + static_cast<double>(b);
  int rank = 0;
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    const double xj = __shfl_sync(kAll, x, j);
    const int ej = __shfl_sync(kAll, e, j);
    rank += xj > x || (xj == x && ej < e) ? 1 : 0;
  }
  return rank;
}

// The j-th largest (from 1) of the lanes' values.  K. Batcher's bitonic sort (1968): 15 exchanges; up to the 16th, of the
// larger values of pairs of lanes, 10 (a value no larger, with one or two more from it up among all; not with `all`).  dirs: bit i of a
// lane is whether it keeps the larger one in exchange i.  (Nine maxima of the warp one after the other took 130
// instructions.)
__device__ __forceinline__ uint32_t sort_directions(int lane) {
  uint32_t dirs = 0;
  int i = 0;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2, ++i) dirs |= ((lane & o) == 0) == ((lane & size) == 0) ? 1u << i : 0u;
  // (as the last round of 16 the fourth sorts downwards everywhere)
#pragma unroll
  for (int o = 8; o > 0; o /= 2, ++i) dirs |= (lane & o) == 0 ? 1u << i : 0u;
  return dirs;
}
__device__ __forceinline__ float warp_nth(float v, int j, uint32_t dirs, bool all) {
  auto exchange = [&](int o, int i) {
    const float w = __shfl_xor_sync(kAll, v, o);
    v = dirs >> i & 1u ? fmaxf(v, w) : fminf(v, w);
  };
  if (j <= 16 && !all) {
    v = fmaxf(v, __shfl_xor_sync(kAll, v, 16));
    exchange(1, 0);
    exchange(2, 1), exchange(1, 2);
    exchange(4, 3), exchange(2, 4), exchange(1, 5);
    exchange(8, 15), exchange(4, 16), exchange(2, 17), exchange(1, 18);
  } else {
    exchange(1, 0);
    exchange(2, 1), exchange(1, 2);
    exchange(4, 3), exchange(2, 4), exchange(1, 5);
    exchange(8, 6), exchange(4, 7), exchange(2, 8), exchange(1, 9);
    exchange(16, 10), exchange(8, 11), exchange(4, 12), exchange(2, 13), exchange(1, 14);
  }
  return __shfl_sync(kAll, v, j - 1);
}

// The exact value of group g: the sum of its two largest choices.  Of its experts (their choices in fp32 in `row`, -inf: not to
// be chosen) those from `low` (finite) up are looked at, by a lane each.
template <typename T>
__device__ __forceinline__ double exact_group(const float* row, int g, int size, float low, bool sigmoid, float shift, double total,
                                              const float* bias, const T* p) {
  Best one{0.0, -1}, two{0.0, -1};
  for (int e = g * size + (threadIdx.x & 31); e < (g + 1) * size; e += 32) {
    if (!(row[e] >= low)) continue;
    const float l = to_float(p[e]);
    const double x = (sigmoid ? exact_sigmoid(l) : exact_softmax(l, shift, total)) + (bias ? static_cast<double>(bias[e]) : 0.0);
    if (one.e < 0 || x > one.x) two = one, one = Best{x, e};
    else if (two.e < 0 || x > two.x) two = Best{x, e};
  }
  const Best first = warp_best(one);
  const Best second = warp_best(one.e == first.e ? two : one);
  return first.x + (second.e >= 0 ? second.x : 0.0);
}
// Which of the groups in `near` (their bits) are the `slots` best, exactly: of equal ones those of lowest index.  low: on lane
// g * share, from where in fp32 group g's experts can be among its two largest.
template <typename T>
__device__ __noinline__ uint32_t exact_groups(uint32_t near, int slots, const float* row, int size, int share, float low,
                                              bool sigmoid, float shift, int E, const float* bias, const T* p) {
  const int lane = threadIdx.x & 31;
  double total = 0.0;
  if (!sigmoid) {
#pragma unroll 1
    for (int e = lane; e < E; e += 32) total += exp(static_cast<double>(to_float(p[e])) - static_cast<double>(shift));
    total = warp_sum(total);
  }
  Best mine{0.0, -1};  // lane g: group g's
#pragma unroll 1
  for (uint32_t left = near; left != 0; left &= left - 1) {
    const int g = __ffs(left) - 1;
    const double v = exact_group(row, g, size, __shfl_sync(kAll, low, g * share), sigmoid, shift, total, bias, p);
    if (lane == g) mine = Best{v, g};
  }
  uint32_t kept = 0;
#pragma unroll 1
  for (int j = 0; j < slots; ++j) {
    const Best b = warp_best(mine);
    if (b.e < 0) break;
    kept |= 1u << b.e;
    if (b.e == lane) mine.e = -1;
  }
  return kept;
}

// The kept groups' bits.  x: the warp's choices (-inf: not to be chosen), by way of `row` in shared memory.  A group's value is off
// by its two choices' errors, each relative to the choice (the sum may be small beside them), and its own rounding.  Kept groups
// that another one may reach, within the errors of both, and those others are told apart in 64 bits.
template <typename Row>
__device__ __forceinline__ uint32_t kept_groups(const moe_router& r, const float (&x)[Row::width], float* row, float most,
                                                float shift, const float* bias, const typename Row::type* p) {
  const int E = r.num_experts, lane = threadIdx.x & 31;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < Row::width; ++i) {
    const int e = Row::expert(i, lane);
    if (e < E) row[e] = x[i];
  }
  __syncwarp();
  // A group's experts over 32 / groups lanes (rounded down to a power of two).
  const int share = 1 << (31 - __clz(32 / r.groups)), size = E / r.groups, g = lane / share;
  float one = -kInf, two = -kInf;
  if (g < r.groups)
    for (int i = lane % share; i < size; i += share) {
      const float v = row[g * size + i];
      two = fmaxf(two, fminf(one, v));
      one = fmaxf(one, v);
    }
  for (int o = share >> 1; o > 0; o >>= 1) {
    const float q1 = __shfl_xor_sync(kAll, one, o), q2 = __shfl_xor_sync(kAll, two, o);
    two = fmaxf(fmaxf(two, q2), fminf(one, q1));
    one = fmaxf(one, q1);
  }
  // one value a group, on its first lane
  const bool mine = lane % share == 0 && one > -kInf;
  const float less = two > -kInf ? two : 0.f, value = one + less;
  uint32_t key = mine ? key_of(value) : 0u, kept = 0;
  for (int j = 0; j < r.top_groups; ++j) {
    const uint32_t best = __reduce_max_sync(kAll, key);
    if (best == 0) break;
    const int at = __ffs(__ballot_sync(kAll, key == best)) - 1;
    kept |= 1u << (at / share);
    if (lane == at) key = 0;
  }
  // The least and the most that the exact value may be (twice as far as it may be off).  An infinite choice's group has exactly
  // that value; a sum past fp32's range may be anything.
  const float wide = tolerance(sigmoid, 2.f * most, fabsf(one) + fabsf(less));
  const bool in = kept >> (lane / share) & 1u, infinite = one == kInf;
  const uint32_t least = key_of(infinite ? kInf : fmaxf(value - wide, -kInf)),
                 greatest = key_of(infinite ? kInf : fminf(value + wide, kInf));
  const uint32_t last = __reduce_min_sync(kAll, mine && in ? least : kAll),
                 next = __reduce_max_sync(kAll, mine && !in ? greatest : 0u);
  if (last <= next) {
    const bool close = mine && (in ? least <= next : greatest >= last);
    uint32_t near = 0;  // by group
    for (uint32_t left = __ballot_sync(kAll, close); left != 0; left &= left - 1) near |= 1u << ((__ffs(left) - 1) / share);
    const int slots = __popc(near & kept);
    // (every expert that can be chosen where the bound is none: below the range, or inf - inf of infinite choices)
    const float low = fmaxf((two > -kInf ? two : one) - wide, -3.4028234663852886e38f);
    kept = (kept & ~near) | exact_groups(near, slots, row, size, share, low, sigmoid, shift, E, bias, p);
  }
  return kept;
}

// Row t by a warp (GROUPS: more than one).  bias: of this lane's experts, -inf of one that is not to be chosen, whatever its score.
template <typename Row, bool GROUPS>
__device__ __forceinline__ void route_row(const RouteLaunch& a, int group_inv, int64_t t, const float (&bias)[Row::width],
                                          uint32_t dirs, int* list, float* group_row) {
  using T = typename Row::type;
  constexpr int V = Row::width;
  const int lane = threadIdx.x & 31;
  const moe_router& r = a.r;
  const int E = r.num_experts, k = r.top_k;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  const bool by_logit = a.bias == nullptr;  // the choice within the groups is the logits' order
  const bool by_score = !by_logit || GROUPS;
  const int deep = by_logit ? k : k + 1;    // of the logits' order nothing is unsure
  const T* p = static_cast<const T*>(a.logits) + t * a.ld;
  int32_t* ids = a.ids + t * k;
  float* weight = a.weight + t * k;
  float x[V];
  Row::load(p, E, lane, -kInf, x);
  SoftmaxRow soft{0.f, 0.f};
  bool bad = false, slow = false;
  if (!sigmoid) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, x[i]);
    top = warp_max_nan(top);
    bad = !(top < kInf);
    float s[V];
    soft = softmax_row(x, top, s);
    if (by_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = x[i] == -kInf ? -kInf : s[i] + bias[i];
    }
  } else if (by_score) {
    float low = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) low = fminf(low, x[i]);
    const bool masked = __any_sync(kAll, low == -kInf);
    uint32_t off = 0;
    if (masked) {
#pragma unroll
      for (int i = 0; i < V; ++i) off |= x[i] == -kInf ? 1u << i : 0u;
    }
    // Short scores (without groups): the exponent's rounding, 2^-24 of |l|, weighs s (1 - s) |l| < 2^-1; the two
    // functions and the sum 2^-21 of s.
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 l = make_float2(x[i], x[i + 1]);
      float2 s;
      if (GROUPS) {
        s = sigmoid_of(l);
      } else {
        const float2 h = mul2(l, both(-1.44269504f));
        const float2 d = add2(both(1.0f), make_float2(exp2_approx(h.x), exp2_approx(h.y)));
        s = make_float2(reciprocal(d.x), reciprocal(d.y));
      }
      s = add2(s, make_float2(bias[i], bias[i + 1]));
      x[i] = s.x, x[i + 1] = s.y;
    }
    if (masked) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (off >> i & 1u) x[i] = -kInf;
    }
  }
  const float most = sigmoid ? 1.f : soft.inv;  // no score is larger
  float local = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) local = max_nan(local, x[i]);
  bad |= local != local;
  if (__any_sync(kAll, bad)) {
    if (lane < k) ids[lane] = -1, weight[lane] = kNaN;
    return;
  }
  if constexpr (GROUPS) {
    const uint32_t kept = kept_groups<Row>(r, x, group_row, most, soft.shift, a.bias, p);
    if (by_logit) Row::load(p, E, lane, -kInf, x);
    local = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = Row::expert(i, lane);
      if (e >= E || !(kept >> ((e * group_inv >> 20) & 31) & 1u)) x[i] = -kInf;
      local = fmaxf(local, x[i]);
    }
  }
  // the k + 1st largest of the lanes' largest, less the margin of the short scores (twice their error); that of all lanes where
  // the shorter sort's leaves too many from there up
  int found = 0;
#pragma unroll 1
  for (bool all = false;; all = true) {
    float low = deep <= 32 ? warp_nth(local, deep, dirs, all) : -kInf;
    if (!by_logit) low -= fmaf(0x1p-21f, fabsf(low), fmaxf(0x1p-18f, tolerance(sigmoid, most, 0.f)));
    if (!(low > -kInf)) low = -3.4028234663852886e38f;  // all that can be chosen
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mask |= x[i] >= low ? 1u << i : 0u;
    found = 0;
    for (uint32_t who; (who = __ballot_sync(kAll, mask != 0)) != 0;) {
      if (mask != 0) {
        const int at = found + __popc(who & ((1u << lane) - 1u));
        if (at < 32) list[at] = Row::expert(__ffs(mask) - 1, lane);
        mask &= mask - 1;
      }
      found += __popc(who);
    }
    if (found <= 32 || all || deep > 16) break;
    __syncwarp();
  }
  __syncwarp();
  if (found > 32) slow = true;
  int id = -1, rank = lane;
  float w = 0.f;
  if (!slow) {
    // one of them to a lane
    id = lane < found ? list[lane] : -1;
    float l = -kInf, b = 0.f, y = 0.f;
    uint32_t key = 0;
    if (id >= 0) {
      l = to_float(p[id]);
      w = sigmoid ? sigmoid_of(l) : softmax_term(l, soft.shift) * soft.inv;
      if (!by_logit) b = __ldg(a.bias + id);
      y = by_logit ? l : w + b;
      key = key_of(y);
    }
    rank = rank_of(key, found);
    // The lanes by rank: an equal one's place is another's.
    if (id >= 0) list[rank] = lane;
    __syncwarp();
    bool close = false;
    if (__any_sync(kAll, id >= 0 && list[rank & 31] != lane)) {
      // Equal values go by index, if they are of the same inputs; else they are not known to be equal.
      const uint32_t same = __match_any_sync(kAll, key);
      const int first = __ffs(same) - 1;
      const float l0 = __shfl_sync(kAll, l, first), b0 = __shfl_sync(kAll, b, first);
      close = !by_logit && id >= 0 && rank <= k && !(l == l0 && b == b0);
      int before = 0;
      for (int j = 0; j < found; ++j) before += __shfl_sync(kAll, id, j) < id && (same >> j & 1u) ? 1 : 0;
      rank += before;
      if (id >= 0) list[rank] = lane;
      __syncwarp();
    }
    if (!by_logit) {
      // the one in front, where both are not behind the k + 1st (equal ones: as above)
      const float front = __shfl_sync(kAll, y, id >= 0 && rank > 0 ? list[rank - 1] : lane);
      close |= id >= 0 && rank > 0 && rank <= k && front != y &&
               !(front - y > tolerance(sigmoid, most, fabsf(y) + fabsf(front)));
      if (__any_sync(kAll, close)) rank = exact_rank<Row>(p, E, sigmoid, soft.shift, l, b, id, found);
    }
    if (id < 0) rank = lane;  // behind those that were found
    if (rank >= k) w = 0.f;
  } else {
    id = exact_choice<Row>(r, p, a.bias, group_inv, lane);
    if (lane >= k) id = -1;
    if (id >= 0) {
      const float l = to_float(p[id]);
      w = sigmoid ? sigmoid_of(l) : softmax_term(l, soft.shift) * soft.inv;
    }
  }
  __syncwarp();  // the list is read
  if (r.normalise) w = __fdividef(w, warp_sum(w) + kTiny);  // (a sum of 1e-20 to 32)
  if (rank < k) ids[rank] = id, weight[rank] = w * r.scale;
}

template <typename Row>
__device__ __forceinline__ void bias_of(const RouteLaunch& a, int lane, float (&bias)[Row::width]) {
#pragma unroll
  for (int i = 0; i < Row::width; ++i) {
    const int e = Row::expert(i, lane);
    const float b = e < a.r.num_experts && a.bias ? __ldg(a.bias + e) : 0.f;
    bias[i] = e < a.r.num_experts && b == b ? b : -kInf;
  }
}

// CTAs that an SM holds (64 or 128 registers a thread).
template <typename Row>
constexpr int kResident = Row::width <= 16 ? 4 : 2;

template <typename Row, bool GROUPS>
__global__ void __launch_bounds__(32 * kWarps, kResident<Row>)
route_kernel(const RouteLaunch a, const int group_inv) {
  __shared__ int list[kWarps][32];
  extern __shared__ float group_row[];  // with groups: [warps][E]
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float bias[Row::width];
  bias_of<Row>(a, lane, bias);
  const uint32_t dirs = sort_directions(lane);
  const int64_t rows = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp; t < a.n; t += rows)
    route_row<Row, GROUPS>(a, group_inv, t, bias, dirs, list[warp], group_row + warp * a.r.num_experts);
}

// ---------------------------------------------------------------- two rows a warp
// A row over 16 lanes, V values to a lane, four neighbours together.
template <typename T, int V>
struct HalfRow {
  using type = T;
  static constexpr int width = V;
  using Whole = WarpRow<T, (V < 8 ? 4 : V / 2), true>;  // by a whole warp
  static __device__ __forceinline__ int expert(int i, int h) { return 64 * (i >> 2) + 4 * h + (i & 3); }
  template <bool FULL>  // E = 16 V
  static __device__ __forceinline__ void load(const T* p, int E, int h, float fill, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      if (FULL || 64 * j + 4 * h < E) {
        if constexpr (sizeof(T) == 4) {
          const float4 q = *reinterpret_cast<const float4*>(p + 64 * j + 4 * h);
          v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(p + 64 * j + 4 * h);
          v[4 * j] = __uint_as_float(q.x << 16), v[4 * j + 1] = __uint_as_float(q.x & 0xffff0000u);
          v[4 * j + 2] = __uint_as_float(q.y << 16), v[4 * j + 3] = __uint_as_float(q.y & 0xffff0000u);
        }
      } else {
        v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = fill;
      }
    }
  }
};

__device__ __forceinline__ float tanh_approx(float v) {
  float r;
  asm("tanh.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int V>
__device__ __forceinline__ float largest(const float (&x)[V]) {
  float m = max_nan(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < V; i += 2) m = max3_nan(m, x[i], x[i + 1]);
  return m;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// The values of 16 lanes sorted downwards (see warp_nth).
__device__ __forceinline__ float half_sorted(float v, uint32_t dirs) {
  auto exchange = [&](int o, int i) {
    const float w = __shfl_xor_sync(kAll, v, o);
    v = dirs >> i & 1u ? fmaxf(v, w) : fminf(v, w);
  };
  exchange(1, 0);
  exchange(2, 1), exchange(1, 2);
  exchange(4, 3), exchange(2, 4), exchange(1, 5);
  exchange(8, 15), exchange(4, 16), exchange(2, 17), exchange(1, 18);
  return v;
}

// Sums of the lanes up to this one.
__device__ __forceinline__ int half_scan(int v, int h) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const int w = __shfl_up_sync(kAll, v, o, 16);
    if (h >= o) v += w;
  }
  return v;
}

// exact_rank of a sigmoid over a half.  (A function of its own, and small: the first to need it on an SM waits for its
// instructions.)
__device__ __noinline__ int exact_rank_half(float l, float b, int id) {
  const double x = exact_sigmoid(l) + static_cast<double>(b);
  int rank = 0;
#pragma unroll 1
  for (int j = 0; j < 16; ++j) {
    const double xj = __shfl_sync(kAll, x, j, 16);
    const int ij = __shfl_sync(kAll, id, j, 16);
    rank += ij >= 0 && (xj > x || (xj == x && ij < id)) ? 1 : 0;
  }
  return rank;
}

// A row that its half of a warp has not settled.
template <typename Row>
__device__ __noinline__ void route_whole(const RouteLaunch& a, int64_t t, int* list) {
  const int lane = threadIdx.x & 31;
  float bias[Row::width];
  bias_of<Row>(a, lane, bias);
  route_row<Row, false>(a, 0, t, bias, sort_directions(lane), list, nullptr);
}

template <typename Row>
constexpr int kResidentPairs = Row::width <= 24 ? 4 : 3;  // CTAs that an SM holds
constexpr int kHalfDeep = 9;  // see launch_route

// Two rows a warp, without groups, by the same steps: what is done once a row (the threshold, the list, the candidates'
// scores and ranks, two thirds of a warp's instructions) is done for both rows at once.  A half has room for 16
// candidates; a row of more, one with a masked candidate or a NaN and one of softmax scores whose order fp32 does not
// settle are left to the whole warp.
template <typename Row>
__global__ void __launch_bounds__(32 * kWarps, kResidentPairs<Row>)
route_pairs_kernel(const RouteLaunch a) {
  using T = typename Row::type;
  constexpr int V = Row::width;
  __shared__ __align__(16) float bias[16 * V];  // (and a sigmoid's 1/2) -inf: not to be chosen
  __shared__ __align__(16) int list[kWarps][32];
  __shared__ __align__(16) uint32_t keys[kWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = lane & 15, half = lane & 16;
  const moe_router& r = a.r;
  const int E = r.num_experts, k = r.top_k;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID, by_logit = a.bias == nullptr;
  const int deep = by_logit ? k : k + 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (2 * kWarps);
  int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * 2;
  for (int e = threadIdx.x; e < 16 * V; e += 32 * kWarps) {
    const float b = e < E && !by_logit ? __ldg(a.bias + e) : 0.f;
    bias[e] = e < E && b == b ? (sigmoid ? 0.5f + b : b) : -kInf;
  }
  __syncthreads();
  int* const mine = list[warp] + half;
  const uint32_t dirs = sort_directions(lane);
  for (; t0 < a.n; t0 += step) {
    const bool live = t0 + (half >> 4) < a.n;
    const int64_t t = live ? t0 + (half >> 4) : t0;
    const T* const p = static_cast<const T*>(a.logits) + t * a.ld;
    float x[V];
    if (E == 16 * V) Row::template load<true>(p, E, h, -kInf, x);
    else Row::template load<false>(p, E, h, -kInf, x);
    SoftmaxRow soft{0.f, 0.f};
    bool fall = false;  // to the whole warp
    // x = f (lo, hi) + bias
    auto add_bias = [&](int j, float f, float2 lo, float2 hi) {
      const float4 b = *reinterpret_cast<const float4*>(bias + 64 * j + 4 * h);
      lo = fma2(lo, both(f), make_float2(b.x, b.y));
      hi = fma2(hi, both(f), make_float2(b.z, b.w));
      x[4 * j] = lo.x, x[4 * j + 1] = lo.y, x[4 * j + 2] = hi.x, x[4 * j + 3] = hi.y;
    };
    if (!sigmoid) {
      float top = largest(x);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(kAll, top, o));
      fall = !(top < kInf);
      soft.shift = top == -kInf ? 0.f : top;
      float2 sum = both(0.f);
      float s[V];
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 e = softmax_term(make_float2(x[i], x[i + 1]), soft.shift);
        s[i] = e.x, s[i + 1] = e.y;
        sum = add2(sum, e);
      }
      const float total = half_sum(sum.x + sum.y);
      soft.inv = total == 0.f ? 0.f : reciprocal(total);
      if (!by_logit) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
          add_bias(j, soft.inv, make_float2(s[4 * j], s[4 * j + 1]), make_float2(s[4 * j + 2], s[4 * j + 3]));
      }
    } else if (!by_logit) {
      // Shorter scores than a whole warp's: 1/2 + tanh(l / 2) / 2, within 2^-12 (tanh.approx: 2^-11 of the value).
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        const float2 lo = mul2(make_float2(x[4 * j], x[4 * j + 1]), both(0.5f)),
                     hi = mul2(make_float2(x[4 * j + 2], x[4 * j + 3]), both(0.5f));
        add_bias(j, 0.5f, make_float2(tanh_approx(lo.x), tanh_approx(lo.y)), make_float2(tanh_approx(hi.x), tanh_approx(hi.y)));
      }
    }
    // (A masked expert has a choice here too, of its bias alone: it matters only where it is a candidate.)
    const float most = sigmoid ? 1.f : soft.inv;
    // a lane's values in two parts: the larger of their largest, and the other one
    float local = max_nan(x[0], x[1]), other = max_nan(x[V / 2], x[V / 2 + 1]);
#pragma unroll
    for (int i = 2; i < V / 2; i += 2) {
      local = max3_nan(local, x[i], x[i + 1]);
      other = max3_nan(other, x[V / 2 + i], x[V / 2 + i + 1]);
    }
    {
      const float less = fminf(local, other);
      local = max_nan(local, other), other = less;
    }
    fall |= local != local;
    const float sorted = half_sorted(local, dirs);
    float low = __shfl_sync(kAll, sorted, deep - 1, 16);
    // The j lanes' largest and as many others from the j-th up make deep: tried for one and two others, which
    // leaves 10.6 candidates for 12.2 (k = 8 of 384 random values) and more than 16 in one row of 250, not of 20.
#pragma unroll
    for (int d = 1; d <= 2; ++d) {
      const float t = __shfl_sync(kAll, sorted, max(deep - 1 - d, 0), 16);
      if (__popc(__ballot_sync(kAll, other >= t) >> half & 0xffffu) >= d && deep > d) low = t;
    }
    auto margin = [&](float v) {
      return by_logit ? 0.f : fmaf(0x1p-21f, fabsf(v), sigmoid ? 0x1.1p-11f : fmaxf(0x1p-18f, tolerance(false, most, 0.f)));
    };
    low -= margin(low);
    if (!(low > -kInf)) low = -3.4028234663852886e38f;
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mask |= x[i] >= low ? 1u << i : 0u;
    int at = half_scan(__popc(mask), h), found = __shfl_sync(kAll, at, 15, 16);
    // Too many: from a larger one of the lanes' largest up, if the deep-th of those turns out to be above all others.
    float sure = -kInf;
    for (int j = deep - 1; j > 0 && __any_sync(kAll, found > 16); --j) {
      const float t = __shfl_sync(kAll, sorted, j - 1, 16);
      if (found > 16 && t < kInf) {  // (an infinite one is left to the whole warp)
        sure = t - margin(t), low = sure - margin(t);
        mask = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) mask |= x[i] >= low ? 1u << i : 0u;
      }
      at = half_scan(__popc(mask), h);
      found = __shfl_sync(kAll, at, 15, 16);
    }
    at -= __popc(mask);
    fall |= found > 16 || (sure > -kInf && found < deep);
    for (; mask != 0 && at < 16; mask &= mask - 1) mine[at++] = Row::expert(__ffs(mask) - 1, h);
    __syncwarp();
    int id = h < found ? mine[h] : -1, rank = 0;
    float l = -kInf, b = 0.f, w = 0.f, y = 0.f;
    uint32_t key = 0;
    if (id >= 0) {
      if (!by_logit) b = __ldg(a.bias + id);
      l = to_float(p[id]);
      fall |= l == -kInf;
      w = sigmoid ? sigmoid_of(l) : softmax_term(l, soft.shift) * soft.inv;
      y = by_logit ? l : w + b;
      key = key_of(y);
    }
    keys[warp][lane] = key;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 q = reinterpret_cast<const uint4*>(keys[warp] + half)[j];
      rank += (q.x > key ? 1 : 0) + (q.y > key ? 1 : 0) + (q.z > key ? 1 : 0) + (q.w > key ? 1 : 0);
    }
    if (id >= 0) mine[rank] = h;  // (of equal ones the place is another's)
    __syncwarp();
    bool close = false;
    if (__any_sync(kAll, id >= 0 && mine[rank] != h)) {
      int before = 0;
      bool same = true;  // of the same inputs
      for (int j = 0; j < 16; ++j) {
        const bool equal = __shfl_sync(kAll, key, j, 16) == key;
        const float lj = __shfl_sync(kAll, l, j, 16), bj = __shfl_sync(kAll, b, j, 16);
        if (__shfl_sync(kAll, id, j, 16) < id && equal) ++before;
        same &= !equal || (lj == l && bj == b);
      }
      close = !by_logit && id >= 0 && rank <= k && !same;
      __syncwarp();
      rank += before;
      if (id >= 0) mine[rank] = h;
      __syncwarp();
    }
    if (!by_logit) {
      const float front = __shfl_sync(kAll, y, id >= 0 && rank > 0 ? mine[rank - 1] : h, 16);
      close |= id >= 0 && rank > 0 && rank <= k && front != y && !(front - y > tolerance(sigmoid, most, fabsf(y) + fabsf(front)));
      if (!sigmoid) fall |= close;
      else if (__any_sync(kAll, close)) rank = exact_rank_half(l, b, id);
    }
    fall |= id >= 0 && rank == deep - 1 && y < sure;
    if (id < 0) rank = h;  // behind those that were found
    if (rank >= k) w = 0.f;
    if (r.normalise) w = __fdividef(w, half_sum(w) + kTiny);
    const uint32_t falls = __ballot_sync(kAll, fall && live);
    if (live && rank < k && (falls >> half & 0xffffu) == 0) {
      a.ids[t * k + rank] = id;
      a.weight[t * k + rank] = w * r.scale;
    }
    if (falls != 0) {
      if (falls & 0xffffu) route_whole<typename Row::Whole>(a, t0, list[warp]);
      __syncwarp();
      if (falls >> 16) route_whole<typename Row::Whole>(a, t0 + 1, list[warp]);
    }
    __syncwarp();  // the lists are read
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
  const int64_t ctas = (a.n + warps - 1) / warps;
  // Two rows a warp where there are enough for every SM to be busy, and few enough candidates for a half.  Measured, in us on
  // one GB300 (sigmoid, fp32, 384 experts, k = 8, bias; two rows a warp | one): 2,432 rows 14.0 | 13.0, 4,864 15.0 | 15.0,
  // 9,728 17.2 | 19.1, 32,768 21.3 | 31.5, 131,072 70 | 113.  Of k = 10 a half would be too small for every second row.
  if (a.n >= sms * 4 * kWarps && a.r.groups == 1 && a.r.top_k + (a.bias ? 1 : 0) <= kHalfDeep && a.r.num_experts <= 512 &&
      rows_by_four(a.r, a.logits, a.ld)) {
    auto launch = [&](auto row) {
      const int64_t pairs = (a.n + 2 * kWarps - 1) / (2 * kWarps), most = sms * kResidentPairs<decltype(row)>;
      return launch_maybe_overlapped(route_pairs_kernel<decltype(row)>, static_cast<int>(pairs < most ? pairs : most),
                                     32 * kWarps, 0, s, true, a);
    };
    auto by_width = [&](auto type) {
      using T = decltype(type);
      const int E = a.r.num_experts;
      return E <= 64    ? launch(HalfRow<T, 4>{})
             : E <= 128 ? launch(HalfRow<T, 8>{})
             : E <= 256 ? launch(HalfRow<T, 16>{})
             : E <= 384 ? launch(HalfRow<T, 24>{})
                        : launch(HalfRow<T, 32>{});
    };
    return a.r.logits_type == MOE_LOGITS_F32 ? by_width(float{}) : by_width(__nv_bfloat16{});
  }
  const size_t smem = a.r.groups > 1 ? static_cast<size_t>(warps) * a.r.num_experts * sizeof(float) : 0;
  return with_row(a.r, rows_by_four(a.r, a.logits, a.ld), [&](auto row) {
    const int64_t most = sms * kResident<decltype(row)> * kWarps / warps;
    auto kern = a.r.groups > 1 ? route_kernel<decltype(row), true> : route_kernel<decltype(row), false>;
    return launch_maybe_overlapped(kern, static_cast<int>(ctas < most ? ctas : most), 32 * warps, smem, s, true, a, inv);
  });
}

}  // namespace moe
