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
// with c[e] = d_loss coef E / (S k T^2) count_e.
//
// HBM would bound all three; what they spend beyond it is a row's way through its reductions
// (202 instructions a row of 384 in the first, 385 in the gradient, issued in 50 to 60 % of
// the cycles) with the warps that registers leave.  65,536 x 384 fp32, sigmoid, k = 8, 16
// sequences, on one GB300: loss 25.7 us (4.0 TB/s), 19 of them the first kernel; gradient
// 39.5 us (5.2 TB/s).  (Two rows a warp, half the instructions a row and half the warps: 21.5
// for the first kernel's 21.)
#include "router.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRowWarps = 8;
constexpr float kTiny = 1e-20f;

// Shares are quotients of scores, whatever the scores' size: where a row's sigmoids add up to less than this (all logits below
// -44) they are e^l to 2^-64 and their shares the softmax's, which fp32 holds while the sigmoids leave its range.  (Above it a
// score that is flushed to 0 has a share below 2^-62.)
constexpr float kLowTotal = 0x1p-64f;

// The scores of a row and what makes shares of them (0 where every logit is -inf, and for sigmoids below kLowTotal).
template <typename Row>
__device__ __forceinline__ float share_scores(bool sigmoid, const float (&l)[Row::width], float2 (&s)[Row::width / 2],
                                              uint32_t mask) {
  constexpr int V = Row::width;
  float shift = 0.f;
  if (!sigmoid) {
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
    top = lanes_max_nan<Row::lanes>(top, mask);
    shift = top == -kInf ? 0.f : top;
  }
  float2 sum = both(0.f);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 v = make_float2(l[2 * i], l[2 * i + 1]);
    s[i] = sigmoid ? sigmoid_short(v) : softmax_term(v, shift);
    sum = add2(sum, s[i]);
  }
  const float total = lanes_sum<Row::lanes>(sum.x + sum.y, mask);
  return total < kLowTotal ? 0.f : reciprocal(total);  // (a softmax's is 0 or 1 and more)
}

// Row ranges of sequence s, held within [0, n] whatever the offsets say.
__device__ __forceinline__ int64_t within(int64_t o, int64_t n) { return o < 0 ? 0 : o > n ? n : o; }
__device__ __forceinline__ int64_t offset_at(const int32_t* offsets, int64_t n, int s) {
  if (!offsets) return s == 0 ? 0 : n;
  return within(offsets[s], n);
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

// The offsets in shared memory where they fit (one read of all instead of one behind the other).
constexpr int kHeld = 1025;
__device__ __forceinline__ const int32_t* hold_offsets(const int32_t* offsets, int sequences, int32_t* held) {
  if (!offsets || sequences + 1 > kHeld) return offsets;
  for (int i = threadIdx.x; i <= sequences; i += blockDim.x) held[i] = __ldg(offsets + i);
  return held;
}

template <typename Row>
constexpr int kRowsAtOnce = 32 * kRowWarps / Row::lanes;  // of a CTA

// (A kernel for each kind of score: with both in one the low rows of sigmoids, which none of these cases has, cost up to a
// twentieth.  Both | each, us: gradient of 65,536 x 384 40.9 | 39.8, of 200,000 x 8 32.2 | 26.5, loss of 20,000 x 1000 38.0 | 32.2.)
template <typename Row, bool SIGMOID>
__global__ void __launch_bounds__(32 * kRowWarps, Row::width <= 12 ? 4 : 1)
balance_rows_kernel(const BalanceLaunch a, const BalancePlan plan) {
  using T = typename Row::type;
  constexpr int V = Row::width, L = Row::lanes, kRows = kRowsAtOnce<Row>;
  __shared__ int32_t held[kHeld];
  extern __shared__ __align__(16) float joined[];  // [rows at once][E], the counts [E], the rings
  pdl_wait();
  pdl_launch_dependents();
  const int sub = threadIdx.x / L, lane = threadIdx.x % L;
  const uint32_t mask = lanes_mask<L>();
  const int E = a.r.num_experts, k = a.r.top_k;
  constexpr bool sigmoid = SIGMOID;
  const int64_t r0 = blockIdx.x * plan.chunk, r1 = min(r0 + plan.chunk, a.n);
  const T* logits = static_cast<const T*>(a.logits);
  // this warp's (or part of one's) rows: r0 + sub and every kRows-th from there on
  const int64_t first = r0 + sub;
  const RowRing<Row> ring{smem_u32(joined + (kRows + 1) * E) + static_cast<uint32_t>(sub * RowRing<Row>::warp_bytes(E)),
                          RowRing<Row>::row_bytes(E)};
  auto row_at = [&](int64_t t) { return t < r1 ? logits + t * a.ld : nullptr; };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ring.ask(i, row_at(first + kRows * i), E, lane);
  const int32_t* offsets = hold_offsets(a.offsets, a.sequences, held);
  int32_t* hist = reinterpret_cast<int32_t*>(joined + kRows * E);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  int64_t t = first;
  int number = 0;  // t's in the ring
  // the chosen experts of the next two rows, one a lane
  auto id_at = [&](int64_t t) { return lane < k && t < r1 ? a.ids[t * k + lane] : -1; };
  int ids[2] = {id_at(first), id_at(first + kRows)};
  for (int s = sequence_of(offsets, a.sequences, a.n, r0); s < a.sequences; ++s) {
    const int64_t lo = max(r0, offset_at(offsets, a.n, s)), hi = min(r1, offset_at(offsets, a.n, s + 1));
    if (lo >= r1) break;
    if (lo >= hi) continue;
    float2 sum[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) sum[i] = both(0.f);
    bool low = false;
    for (; t < hi; t += kRows, ++number) {
      const bool in = t >= lo;  // (rows in front of the first sequence are not)
      float l[V];
      ring.take(number, logits + t * a.ld, E, lane, -kInf, l);
      ring.ask(number + kAhead, row_at(t + kRows * kAhead), E, lane);
      if (in && ids[0] >= 0 && ids[0] < E) atomicAdd(hist + ids[0], 1);
      ids[0] = ids[1];
      ids[1] = id_at(t + 2 * kRows);
      float2 q[V / 2];
      const float inv = share_scores<Row>(sigmoid, l, q, mask);
      low |= inv == 0.f;
      if (in) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) sum[i] = fma2(q[i], both(inv), sum[i]);
      }
    }
    // Rows of low sigmoids once more, by themselves: in the loop above their branch waits for each row's sum (65,536 x 384
    // 28.6 us, 26.6 this way).
    if (sigmoid && low) {
#pragma unroll 1
      for (int64_t r = first + (lo - first + kRows - 1) / kRows * kRows; r < hi; r += kRows) {
        float l[V];
        float2 q[V / 2];
        Row::load(logits + r * a.ld, E, lane, -kInf, l);
        if (share_scores<Row>(true, l, q, mask) != 0.f) continue;
        const float inv = share_scores<Row>(false, l, q, mask);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) sum[i] = fma2(q[i], both(inv), sum[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (Row::expert(i, lane) < E) joined[sub * E + Row::expert(i, lane)] = i & 1 ? sum[i >> 1].y : sum[i >> 1].x;
    __syncthreads();
    const int64_t piece = static_cast<int64_t>(blockIdx.x) + s;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kRows; ++w) v += joined[w * E + e];
      a.sums[piece * E + e] = v;
      a.hist[piece * E + e] = hist[e];
      hist[e] = 0;
    }
    __syncthreads();
  }
  ring.end();
}

// atomicAdd that releases what this thread has seen written and acquires what the others released.
__device__ __forceinline__ uint32_t take_ticket(uint32_t* p) {
  uint32_t v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Grid (parts, sequences): 32 experts of a sequence, a warp every eighth piece.  What it takes is the way from one access of
// memory to the next (6 us behind the rows' kernel, for 1.4 MB): the offsets are read while that one still runs.
__global__ void __launch_bounds__(256)
balance_loss_kernel(const BalanceLaunch a, const BalancePlan plan) {
  __shared__ float psum[8][32];
  __shared__ int pcount[8][32];
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.r.num_experts, parts = gridDim.x;
  const int e = blockIdx.x * 32 + lane;
  // (The kernel in front waits for those in front of it before it lets this one begin, and writes no offsets; they are read
  // from L2, where those wrote them.)
  auto raw = [&](int s) -> int64_t { return a.offsets ? __ldcg(a.offsets + s) : s == 0 ? 0 : a.n; };
  int s = blockIdx.y;
  int64_t lo = within(raw(s), a.n), hi = within(raw(s + 1), a.n);
  int live = 0;
  bool bad = false;  // offsets that do not ascend within the rows
  auto look = [&](int s) {
    const int64_t o0 = raw(s), o1 = raw(s + 1);
    bad |= o0 < 0 || o1 < o0 || o1 > a.n;
    live += o1 > o0 ? 1 : 0;
  };
  const int seen = min(a.sequences, static_cast<int>(blockDim.x));  // sequences looked at here
  if (static_cast<int>(threadIdx.x) < seen) look(threadIdx.x);
  pdl_wait();
  pdl_launch_dependents();
  while (true) {
    float sum = 0.f;
    int count = 0;
    if (lo < hi && e < E) {
      const uint32_t chunk = static_cast<uint32_t>(plan.chunk);  // (rows and runs are below 2^31)
      const int c0 = static_cast<int>(static_cast<uint32_t>(lo) / chunk), c1 = static_cast<int>((static_cast<uint32_t>(hi) - 1) / chunk);
      // eight pieces' values on their way at once
      for (int c = c0 + warp; c <= c1; c += 64) {
        float v[8];
        int n[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t at = static_cast<int64_t>(c + 8 * j + s) * E + e;
          const bool on = c + 8 * j <= c1;
          v[j] = on ? a.sums[at] : 0.f;
          n[j] = on ? a.hist[at] : 0;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[j], count += n[j];
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
      if (lane == 0) a.parts[s * parts + blockIdx.x] = lo < hi ? part : 0.f;
    }
    s += gridDim.y;
    if (s >= a.sequences) break;
    lo = within(raw(s), a.n), hi = within(raw(s + 1), a.n);
    __syncthreads();
  }
  if (threadIdx.x == 0) last = take_ticket(a.ticket) == gridDim.x * gridDim.y - 1;  // (this thread wrote the parts)
  __syncthreads();
  if (!last) return;
  float sum = 0.f;
  // (the parts of a sequence without rows are 0)
#pragma unroll 4
  for (int i = threadIdx.x; i < a.sequences * parts; i += blockDim.x) sum += __ldcg(a.parts + i);
  for (int s = threadIdx.x + seen; s < a.sequences; s += blockDim.x) look(s);
  bad = __syncthreads_or(bad);
  sum = warp_sum(sum);
  live = __reduce_add_sync(kAll, live);
  if (lane == 0) psum[0][warp] = sum, pcount[0][warp] = live;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.f;
    live = 0;
    for (int w = 0; w < 8; ++w) sum += psum[0][w], live += pcount[0][w];
    const float factor = a.coef * static_cast<float>(E) / (static_cast<float>(a.r.top_k) * static_cast<float>(live));
    *a.loss = bad ? kNaN : live ? sum * factor : 0.f;
  }
}

// CTAs of the gradient that an SM holds.
template <typename Row>
constexpr int kGradResident = Row::width <= 12 ? 3 : Row::width <= 16 ? 2 : 1;

template <typename Row, bool SIGMOID>
__global__ void __launch_bounds__(32 * kRowWarps, kGradResident<Row>)
route_grad_kernel(const RouteGradLaunch a, const int64_t run) {
  using T = typename Row::type;
  constexpr int V = Row::width, L = Row::lanes;
  extern __shared__ __align__(16) float scatter[];  // [rows at once][L V]: ds at the chosen experts, zeros elsewhere; the rings
  __shared__ int lives[kRowWarps];
  __shared__ int32_t held[kHeld];
  pdl_wait();
  pdl_launch_dependents();
  const int subs = blockDim.x / L, sub = threadIdx.x / L, lane = threadIdx.x % L;
  const uint32_t mask = lanes_mask<L>();
  const int E = a.r.num_experts, k = a.r.top_k;
  constexpr bool sigmoid = SIGMOID;
  const int32_t* offsets = a.counts ? hold_offsets(a.offsets, a.sequences, held) : nullptr;
  float* ds = scatter + sub * (L * V);
#pragma unroll
  for (int i = 0; i < V; ++i) ds[L * i + lane] = 0.f;
  float factor = 0.f;  // d_loss coef E / (S k)
  if (a.counts) {
    __syncthreads();
    int live = 0;
    for (int s = threadIdx.x; s < a.sequences; s += blockDim.x)
      live += offset_at(offsets, a.n, s + 1) > offset_at(offsets, a.n, s) ? 1 : 0;
    live = __reduce_add_sync(kAll, live);
    if ((threadIdx.x & 31) == 0) lives[threadIdx.x >> 5] = live;
    __syncthreads();
    live = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) live += lives[w];
    factor = (a.d_loss ? __ldg(a.d_loss) : 1.f) * (a.coef * static_cast<float>(E) / (static_cast<float>(k) * live));
  }
  __syncwarp(mask);
  const uint32_t ds_at = smem_u32(ds + 4 * lane);  // this lane's first four
  // a warp's (or part of one's) rows follow one another, so that a sequence's counts stay in its registers
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * subs + sub) * run, t1 = min(t0 + run, a.n);
  if (t0 >= t1) return;
  const T* logits = static_cast<const T*>(a.logits);
  const RowRing<Row> ring{smem_u32(scatter + subs * (L * V)) + static_cast<uint32_t>(sub * RowRing<Row>::warp_bytes(E)),
                          RowRing<Row>::row_bytes(E)};
  auto row_at = [&](int64_t t) { return t < t1 ? logits + t * a.ld : nullptr; };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ring.ask(i, row_at(t0 + i), E, lane);
  // Chosen experts, one a lane (-1: none), and their weights' gradients, of the next two rows.
  int ids[2] = {-1, -1};
  float gs[2] = {0.f, 0.f};
  auto read = [&](int64_t t, int& id, float& g) {
    id = -1;
    g = 0.f;
    if (a.d_weight && lane < k && t < t1) {
      id = a.ids[t * k + lane];
      g = a.d_weight[t * k + lane];
      if (id < 0 || id >= E) id = -1, g = 0.f;
    }
  };
  read(t0, ids[0], gs[0]);
  read(t0 + 1, ids[1], gs[1]);
  float2 c[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) c[i] = both(0.f);
  int seq = a.counts ? sequence_of(offsets, a.sequences, a.n, t0) : 0;
  int64_t until = t0;  // where c changes next
#pragma unroll 1
  for (int64_t t = t0; t < t1; ++t) {
    const int id = ids[0];
    const float g = gs[0] * a.r.scale;
    ids[0] = ids[1];
    gs[0] = gs[1];
    read(t + 2, ids[1], gs[1]);
    float l[V];
    const int number = static_cast<int>(t - t0);
    ring.take(number, logits + t * a.ld, E, lane, -kInf, l);
    ring.ask(number + kAhead, row_at(t + kAhead), E, lane);
    __syncwarp(mask);  // (the row is in the ring for every lane)
    const float lj = id >= 0 ? ring.one(number, logits + t * a.ld, id) : -kInf;
    if (a.counts && t >= until) {
      // sequences that end at or in front of t are over; between two (and behind the last) there are none
      while (seq < a.sequences && offset_at(offsets, a.n, seq + 1) <= t) ++seq;
      const int64_t lo = seq < a.sequences ? offset_at(offsets, a.n, seq) : a.n,
                    hi = seq < a.sequences ? offset_at(offsets, a.n, seq + 1) : a.n;
      const bool in = lo <= t && t < hi;
      const float rows = static_cast<float>(hi - lo), f = in ? factor / (rows * rows) : 0.f;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const int e0 = Row::expert(2 * i, lane), e1 = Row::expert(2 * i + 1, lane);
        const int32_t* p = a.counts + static_cast<int64_t>(seq) * E;
        c[i].x = in && e0 < E ? f * static_cast<float>(__ldg(p + e0)) : 0.f;
        c[i].y = in && e1 < E ? f * static_cast<float>(__ldg(p + e1)) : 0.f;
      }
      until = in ? hi : lo > t ? lo : a.n;
    }
    // v: what the bracket of the gradient's formula is multiplied by
    float2 v[V / 2], total2 = both(0.f), dot2 = both(0.f);
    float top = -kInf, shift = 0.f;
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float2 t2;
        const float2 s = sigmoid_short(make_float2(l[2 * i], l[2 * i + 1]), t2);
        total2 = add2(total2, s);
        dot2 = fma2(c[i], s, dot2);
        v[i] = mul2(mul2(t2, s), s);  // s (1 - s): e^-l s is 1 - s
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) top = max_nan(top, l[i]);
      top = lanes_max_nan<L>(top, mask);
      shift = top == -kInf ? 0.f : top;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[i] = softmax_term(make_float2(l[2 * i], l[2 * i + 1]), shift);
        total2 = add2(total2, v[i]);
        dot2 = fma2(c[i], v[i], dot2);
      }
    }
    const float total = lanes_sum<L>(total2.x + total2.y, mask), inv = total == 0.f ? 0.f : reciprocal(total);
    float dot = dot2.x + dot2.y, dj = 0.f;  // dj: ds of the lane's chosen expert
    const float sj = sigmoid ? sigmoid_of(lj) : softmax_term(lj, shift) * inv;
    if (a.d_weight) {
      dj = g;
      if (a.r.normalise) {
        const float chosen = id >= 0 ? sj : 0.f;
        const float sum = lanes_sum<L>(chosen, mask) + kTiny, with = lanes_sum<L>(g * chosen, mask);
        dj = __fdividef(g - __fdividef(with, sum), sum);
      }
      const uint32_t same = __match_any_sync(mask, id);
      if (__any_sync(mask, id >= 0 && (same & (same - 1u)) != 0)) {
        // an expert named twice: its entries in order
        for (int j = 0; j < k; ++j) {
          if (lane == j && id >= 0) ds[id] += dj;
          __syncwarp(mask);
        }
      } else if (id >= 0) {
        ds[id] = dj;
      }
      __syncwarp(mask);
    }
    // d = (c scale + rest + ds) v
    float scale = 0.f, rest = 0.f;
    if (sigmoid) {
      if (a.counts) {
        dot = lanes_sum<L>(dot, mask) * inv;
        scale = inv;
        rest = -dot * inv;
      }
    } else {
      // of the shares: v inv
      dot = lanes_sum<L>(fmaf(dot, inv, id >= 0 ? dj * sj : 0.f), mask);
      scale = inv;
      rest = -dot * inv;
    }
    const float ds_scale = sigmoid ? 1.f : inv;
    float d[V], add[V];
    if (a.d_weight) {
      if constexpr (Row::vec) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
          const uint4 q = lds128(ds_at + 16 * L * j);
          add[4 * j] = __uint_as_float(q.x), add[4 * j + 1] = __uint_as_float(q.y), add[4 * j + 2] = __uint_as_float(q.z),
                  add[4 * j + 3] = __uint_as_float(q.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) add[i] = ds[L * i + lane];
      }
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      float2 w = fma2(c[i], both(scale), both(rest));
      if (a.d_weight) {
        w = fma2(make_float2(add[2 * i], add[2 * i + 1]), both(ds_scale), w);
      }
      w = mul2(w, v[i]);
      d[2 * i] = w.x, d[2 * i + 1] = w.y;
    }
    if (sigmoid ? !(total >= kLowTotal) : total != total) {
      if (total != total) {  // a row that holds a NaN
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = kNaN;
      } else {  // low sigmoids: s and s (1 - s) are v e^top (d_logits may be logits: this row is not written yet)
        Row::load(logits + t * a.ld, E, lane, -kInf, l);
        scale = share_scores<Row>(false, l, v, mask);
        top = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
        const float by = softmax_term(lanes_max_nan<L>(top, mask), 0.f);
        dot2 = both(0.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) dot2 = fma2(c[i], v[i], dot2);
        rest = -(lanes_sum<L>(dot2.x + dot2.y, mask) * scale) * scale;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float ci = i & 1 ? c[i >> 1].y : c[i >> 1].x, vi = i & 1 ? v[i >> 1].y : v[i >> 1].x;
          d[i] = fmaf(ds[Row::expert(i, lane)], by, fmaf(ci, scale, rest)) * vi;
        }
      }
    }
    Row::store(static_cast<T*>(a.d_logits) + t * a.d_ld, E, lane, d);
    __syncwarp(mask);
    if (id >= 0) ds[id] = 0.f;
    __syncwarp(mask);
  }
  ring.end();
}

}  // namespace

// (A kernel's own 48 KB need no leave.)
template <typename K>
static cudaError_t allow_smem(K kern, size_t bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

BalancePlan balance_plan(int64_t n) {
  // A row a warp at least; at most what the SMs hold at once of 384 experts (64 registers a thread: four an SM).
  constexpr int64_t kMost = 608, kLeast = 8;
  int64_t chunk = (n + kMost - 1) / kMost;
  if (chunk < kLeast) chunk = kLeast;
  if (chunk > n) chunk = n < 1 ? 1 : n;
  const int64_t chunks = (n + chunk - 1) / chunk;
  return BalancePlan{chunk, static_cast<int32_t>(chunks < 1 ? 1 : chunks)};  // without rows one CTA, for the ticket
}

// More rows than the SMs hold at once, one to a warp: short ones several to a warp, so that what is done once a row is done for
// all of them.  (For fewer rows the way through one counts, which is the same: 5,000 rows take 9 and 6.5 us either way.)  On
// one GB300, us, several | one: loss of 50,000 x 48 12.7 | 15.8, of 200,000 x 8 15.8 | 34.2; gradient of 50,000 x 48 21.4 | 26.5, of
// 200,000 x 8 33 | 80.
template <typename F>
static cudaError_t with_rows_of(const moe_router& r, int64_t n, bool vec, F f) {
  return n > 32 * static_cast<int64_t>(device_sms()) ? with_short_row(r, vec, f) : with_row(r, vec, f);
}

cudaError_t launch_balance(const BalanceLaunch& a, cudaStream_t s) {
  const BalancePlan plan = balance_plan(a.n);
  cudaError_t e = with_rows_of(a.r, a.n, rows_by_four(a.r, a.logits, a.ld), [&](auto row) {
    using Row = decltype(row);
    auto kern = a.r.score == MOE_SCORE_SIGMOID ? balance_rows_kernel<Row, true> : balance_rows_kernel<Row, false>;
    const size_t smem = (kRowsAtOnce<Row> + 1) * sizeof(float) * a.r.num_experts +
                        kRowsAtOnce<Row> * RowRing<Row>::warp_bytes(a.r.num_experts);
    const cudaError_t st = allow_smem(kern, smem);
    if (st != cudaSuccess) return st;
    return launch_maybe_overlapped(kern, plan.chunks, 32 * kRowWarps, smem, s, true, a, plan);
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
  const bool vec = rows_by_four(a.r, a.logits, a.ld) && rows_by_four(a.r, a.d_logits, a.d_ld);
  return with_rows_of(a.r, a.n, vec, [&](auto row) {
    using Row = decltype(row);
    // one round of the CTAs that the SMs hold
    const int64_t subs = warps * 32 / Row::lanes, most = sms * kGradResident<Row> * kRowsAtOnce<Row>;
    const int64_t run = (a.n + most - 1) / most, ctas = (a.n + run * subs - 1) / (run * subs);
    const size_t smem = static_cast<size_t>(subs) * (sizeof(float) * Row::lanes * Row::width +
                                                     RowRing<Row>::warp_bytes(a.r.num_experts));
    auto kern = a.r.score == MOE_SCORE_SIGMOID ? route_grad_kernel<Row, true> : route_grad_kernel<Row, false>;
    const cudaError_t st = allow_smem(kern, smem);
    if (st != cudaSuccess) return st;
    return launch_maybe_overlapped(kern, static_cast<int>(ctas), 32 * warps, smem, s, true, a, run);
  });
}

}  // namespace moe
