// Rows of router logits (moe_router.h): how a warp holds one, their scores, and
// the launchers of route.cu and balance.cu.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "moe_router.h"

namespace moe {

constexpr float kInf = __builtin_huge_valf();
constexpr float kNaN = __builtin_nanf("");

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// A row of E values over LANES lanes of a warp, V to a lane.  VEC: four neighbours to a lane,
// read and written together (E and the row stride multiples of 4, rows aligned to four
// values); else every LANES-th.
template <typename T, int V, bool VEC, int LANES = 32>
struct WarpRow {
  using type = T;
  static constexpr int width = V, lanes = LANES;
  static constexpr bool vec = VEC;
  static __device__ __forceinline__ int expert(int i, int lane) {
    return VEC ? 4 * LANES * (i >> 2) + 4 * lane + (i & 3) : LANES * i + lane;
  }
  // Values past the row are `fill`.
  static __device__ __forceinline__ void load(const T* p, int E, int lane, float fill, float (&v)[V]) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        const int e = 4 * LANES * j + 4 * lane;
        if (e < E) {
          if constexpr (sizeof(T) == 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + e);
            v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
          } else {
            const uint2 q = *reinterpret_cast<const uint2*>(p + e);
            v[4 * j] = __uint_as_float(q.x << 16), v[4 * j + 1] = __uint_as_float(q.x & 0xffff0000u);
            v[4 * j + 2] = __uint_as_float(q.y << 16), v[4 * j + 3] = __uint_as_float(q.y & 0xffff0000u);
          }
        } else {
          v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = fill;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = LANES * i + lane < E ? to_float(p[LANES * i + lane]) : fill;
    }
  }
  static __device__ __forceinline__ void store(T* p, int E, int lane, const float (&v)[V]) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        const int e = 4 * LANES * j + 4 * lane;
        if (e >= E) continue;
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float4*>(p + e) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v[4 * j], v[4 * j + 1]),
                               hi = __floats2bfloat162_rn(v[4 * j + 2], v[4 * j + 3]);
          *reinterpret_cast<uint2*>(p + e) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (LANES * i + lane < E) {
          if constexpr (sizeof(T) == 4) p[LANES * i + lane] = v[i];
          else p[LANES * i + lane] = __float2bfloat16_rn(v[i]);
        }
    }
  }
};

// The next rows of a warp on their way to shared memory, kAhead of them, so that a warp waits for none that it has not
// asked for kAhead rows ago.  (One is enough with 24 to 32 warps an SM; three took the place of a CTA: loss of 65,536 x 384
// 27.6 us for 26.1, gradient 40.7 for 39.3.)  A lane copies and reads its own pieces alone: its own wait is enough.  (Rows that are not
// read four values at a time are read where they are used.)
constexpr int kAhead = 1;
template <typename Row>
struct RowRing {
  using T = typename Row::type;
  static constexpr int kPiece = 4 * sizeof(T);
  uint32_t base;  // of this warp's kAhead + 1 rows
  int bytes;      // of one
  static __host__ __device__ constexpr int row_bytes(int E) {
    return Row::vec ? (static_cast<int>(sizeof(T)) * E + 15) / 16 * 16 : 0;
  }
  static __host__ __device__ constexpr size_t warp_bytes(int E) { return static_cast<size_t>(kAhead + 1) * row_bytes(E); }

  // Row number i of the warp, at p (null: none; each call counts all the same).
  __device__ __forceinline__ void ask(int i, const T* p, int E, int lane) const {
    if constexpr (Row::vec) {
      if (p) {
        const uint32_t to = base + (i & kAhead) * bytes + kPiece * lane;
#pragma unroll
        for (int j = 0; j < Row::width / 4; ++j)
          if (4 * Row::lanes * j + 4 * lane < E)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + Row::lanes * kPiece * j),
                         "l"(p + 4 * Row::lanes * j + 4 * lane), "n"(kPiece)
                         : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // Before the warp ends: nothing is on its way any more.
  __device__ __forceinline__ void end() const {
    if constexpr (Row::vec) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  // Row number i, asked for kAhead calls ago; values past the row are `fill`.
  __device__ __forceinline__ void take(int i, const T* p, int E, int lane, float fill, float (&v)[Row::width]) const {
    if constexpr (Row::vec) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      const uint32_t at = base + (i & kAhead) * bytes + kPiece * lane;
#pragma unroll
      for (int j = 0; j < Row::width / 4; ++j) {
        const bool on = 4 * Row::lanes * j + 4 * lane < E;
        if constexpr (sizeof(T) == 4) {
          uint4 q = make_uint4(0u, 0u, 0u, 0u);
          if (on) q = lds128(at + Row::lanes * kPiece * j);
          v[4 * j] = __uint_as_float(q.x), v[4 * j + 1] = __uint_as_float(q.y), v[4 * j + 2] = __uint_as_float(q.z),
                v[4 * j + 3] = __uint_as_float(q.w);
        } else {
          uint32_t x = 0, y = 0;
          if (on) asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(at + Row::lanes * kPiece * j));
          v[4 * j] = __uint_as_float(x << 16), v[4 * j + 1] = __uint_as_float(x & 0xffff0000u);
          v[4 * j + 2] = __uint_as_float(y << 16), v[4 * j + 3] = __uint_as_float(y & 0xffff0000u);
        }
        if (!on) v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = fill;
      }
    } else {
      Row::load(p, E, lane, fill, v);
    }
  }
  // One value of row number i, which every lane of the warp has taken and not yet asked over.
  __device__ __forceinline__ float one(int i, const T* p, int e) const {
    if constexpr (!Row::vec) return to_float(p[e]);
    const uint32_t at = base + (i & kAhead) * bytes + sizeof(T) * e;
    if constexpr (sizeof(T) == 4) {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
      return v;
    } else {
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
      return __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
  }
};
static_assert((kAhead & (kAhead + 1)) == 0, "rows of the ring are numbered by bits");

// The larger value, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The same over each LANES lanes; mask: the caller's.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max_nan(float v, uint32_t mask) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(mask, v, o));
  return v;
}
// The lanes that share this thread's row.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_mask() {
  return LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
}

// Two values at a time (each rounded as one alone would be): an issue slot for both.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return reinterpret_cast<const float2&>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return reinterpret_cast<const float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return reinterpret_cast<const float2&>(d);
}
__device__ __forceinline__ float exp2_approx(float h) {
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(h));
  return t;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// e^x for -128 <= x <= 88.1 (0 below -87.3): 2^h (1 + r) with h = x log2(e) rounded to a float and r = x - h ln(2), which
// two FMAs get from h in two parts of ln(2).  |r| is below 2^-17, so 1 + r is e^r to 2^-35; ex2.approx is within 2^-22:
// together 2^-22 + 2^-24 of the value.
__device__ __forceinline__ float2 exp_of(float2 x) {
  constexpr float kLog2E = 1.44269504f, kLn2Hi = 0.693147182f, kLn2Lo = -1.90465421e-9f;
  const float2 h = mul2(x, both(kLog2E));
  const float2 r = fma2(h, both(-kLn2Lo), fma2(h, both(-kLn2Hi), x));
  const float2 t = make_float2(exp2_approx(h.x), exp2_approx(h.y));
  return fma2(t, r, t);
}

// 1 / (1 + e^-l), NaN of a NaN.  From -88.1 down e^-l is above 2^127 and its reciprocal is flushed to 0.  The
// reciprocal is within an ulp: together below 2^-21 of the score.
__device__ __forceinline__ float2 sigmoid_of(float2 l) {
  const float2 t = exp_of(make_float2(max_nan(min_nan(-l.x, 88.1f), -128.f), max_nan(min_nan(-l.y, 88.1f), -128.f)));
  const float2 d = add2(both(1.0f), t);
  return make_float2(reciprocal(d.x), reciprocal(d.y));
}
__device__ __forceinline__ float sigmoid_of(float l) { return sigmoid_of(both(l)).x; }

// The same with e^-l by one rounded product, which is within |l| 2^-24 of it (and what the others are): for sums over many
// rows and gradients, whose own roundings are no smaller.
__device__ __forceinline__ float2 sigmoid_short(float2 l, float2& t) {
  const float2 h = mul2(l, both(-1.44269504f));
  t = make_float2(exp2_approx(min_nan(h.x, 127.f)), exp2_approx(min_nan(h.y, 127.f)));
  const float2 d = add2(both(1.0f), t);
  return make_float2(reciprocal(d.x), reciprocal(d.y));
}
// (No value needs a bound here: beyond the range of floats the reciprocal is 0 or 1.)
__device__ __forceinline__ float2 sigmoid_short(float2 l) {
  const float2 h = mul2(l, both(-1.44269504f));
  const float2 d = add2(both(1.0f), make_float2(exp2_approx(h.x), exp2_approx(h.y)));
  return make_float2(reciprocal(d.x), reciprocal(d.y));
}

// What a row's softmax needs of the whole row: score = e^(l - shift) inv.  A row of -inf alone has
// shift 0 and scores 0.
struct SoftmaxRow {
  float shift, inv;
};
__device__ __forceinline__ float2 softmax_term(float2 l, float shift) {
  const float2 x = add2(l, both(-shift));
  return exp_of(make_float2(max_nan(x.x, -128.f), max_nan(x.y, -128.f)));
}
__device__ __forceinline__ float softmax_term(float l, float shift) { return softmax_term(both(l), shift).x; }
template <int V>
__device__ __forceinline__ SoftmaxRow softmax_row(const float (&l)[V], float top, float (&s)[V]) {
  SoftmaxRow r;
  r.shift = top == -kInf ? 0.f : top;
  float2 sum = both(0.f);
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float2 e = softmax_term(make_float2(l[i], l[i + 1]), r.shift);
    s[i] = e.x, s[i + 1] = e.y;
    sum = add2(sum, e);
  }
  const float total = warp_sum(sum.x + sum.y);
  r.inv = total == 0.f ? 0.f : reciprocal(total);
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] *= r.inv;
  return r;
}

struct RouteLaunch {
  moe_router r;
  int64_t n;
  const void* logits;
  int64_t ld;
  const float* bias;
  int32_t* ids;
  float* weight;
};
cudaError_t launch_route(const RouteLaunch& a, cudaStream_t s);

// Rows of a CTA and the number of CTAs of the loss's first kernel.
struct BalancePlan {
  int64_t chunk;
  int32_t chunks;
};
BalancePlan balance_plan(int64_t n);

struct BalanceLaunch {
  moe_router r;
  int64_t n;
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  float coef;
  const int32_t* offsets;  // null: one sequence
  int32_t sequences;
  int32_t* counts;
  float* loss;
  // workspace: a ticket, the sequences' parts of the loss [S][balance_parts(E)], and of each piece (the rows of
  // one CTA in one sequence, piece CTA + sequence) the shares' sums [E] and the counts [E]
  uint32_t* ticket;
  float* parts;
  float* sums;
  int32_t* hist;
};
constexpr int kBalanceCols = 32;  // experts of a CTA of the loss's second kernel
inline int32_t balance_parts(int32_t E) { return (E + kBalanceCols - 1) / kBalanceCols; }
cudaError_t launch_balance(const BalanceLaunch& a, cudaStream_t s);

struct RouteGradLaunch {
  moe_router r;
  int64_t n;
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  const float* d_weight;
  float coef;
  const int32_t* counts;
  const float* d_loss;
  const int32_t* offsets;
  int32_t sequences;
  void* d_logits;
  int64_t d_ld;
};
cudaError_t launch_route_grad(const RouteGradLaunch& a, cudaStream_t s);

// Calls f with a WarpRow for the logits' type, number and alignment.
template <typename F>
cudaError_t with_row(const moe_router& r, bool vec, F f) {
  auto by_width = [&](auto type) -> cudaError_t {
    using T = decltype(type);
    const int E = r.num_experts;
    if (vec) {
      if (E <= 128) return f(WarpRow<T, 4, true>{});
      if (E <= 256) return f(WarpRow<T, 8, true>{});
      if (E <= 384) return f(WarpRow<T, 12, true>{});
      if (E <= 512) return f(WarpRow<T, 16, true>{});
      return f(WarpRow<T, 32, true>{});
    }
    if (E <= 64) return f(WarpRow<T, 2, false>{});
    if (E <= 256) return f(WarpRow<T, 8, false>{});
    if (E <= 512) return f(WarpRow<T, 16, false>{});
    return f(WarpRow<T, 32, false>{});
  };
  return r.logits_type == MOE_LOGITS_F32 ? by_width(float{}) : by_width(__nv_bfloat16{});
}
// The same with two or four short rows to a warp, whose lanes hold the chosen experts too; else as above.
template <typename F>
cudaError_t with_short_row(const moe_router& r, bool vec, F f) {
  auto by_width = [&](auto type) -> cudaError_t {
    using T = decltype(type);
    const int E = r.num_experts, k = r.top_k;
    if (vec && E <= 32 && k <= 8) return f(WarpRow<T, 4, true, 8>{});
    if (vec && E <= 64 && k <= 16) return f(WarpRow<T, 4, true, 16>{});
    if (!vec && E <= 16 && k <= 8) return f(WarpRow<T, 2, false, 8>{});
    if (!vec && E <= 64 && k <= 16) return f(WarpRow<T, 4, false, 16>{});
    return with_row(r, vec, f);
  };
  return r.logits_type == MOE_LOGITS_F32 ? by_width(float{}) : by_width(__nv_bfloat16{});
}
// Rows that can be read four values at a time.
inline bool rows_by_four(const moe_router& r, const void* p, int64_t ld) {
  return r.num_experts % 4 == 0 && ld % 4 == 0 &&
         reinterpret_cast<uintptr_t>(p) % (r.logits_type == MOE_LOGITS_F32 ? 16 : 8) == 0;
}

}  // namespace moe
