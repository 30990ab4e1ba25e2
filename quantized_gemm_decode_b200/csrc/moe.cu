// Routing to experts, the sort of (token, expert) pairs by expert, and the
// weighted sum of a token's expert outputs.
#include <cuda_bf16.h>
#include <float.h>

#include <atomic>

#include "qgd_internal.h"
#include "sm100.cuh"

namespace qgd {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Routing: one warp per token, lane l holding kVPT consecutive experts.
//   x = logit (NaN counts as -inf, +inf as the largest float)
//   s = exp(x - max) / sum exp(x - max), or 1 / (1 + exp(-x))
//   choice value c = s + bias; the k largest c of the kept groups, ties to the
//   lowest index; an expert at -inf is never chosen (id -1, weight 0).
//   w_j = scale * s_j (/ sum of the chosen s)
// The choice is that of 64-bit values: two experts whose scores are equal in 32
// bits would otherwise be ordered by the rounding of an exponential.  Without a
// bias the scores' order is the logits', which needs no rounding at all.  With
// one (and for sums of two scores) a row is first chosen from 32-bit values of
// known error; only where two values that decide something lie closer than
// that error, and are not the same logit with the same bias, the row is chosen
// again in 64 bits (of random rows of 256 experts with a bias, 0.15 % with sigmoid
// scores and 0.4 to 0.7 % with softmax).  Weights are computed from the chosen
// logits in 64 bits; the 64-bit sum that divides them is of the chosen ones' scores,
// or, for a softmax that is not renormalised, of all exponentials, each within 2^-22.
// Bound by its instructions (about 1100 a row of 256 experts in 8 groups, 8
// chosen): 28 us for 16384 such rows, 3.1 us for one; 64-bit values throughout
// took 91 and 9.3 us.
// ---------------------------------------------------------------------------
// Error of a 32-bit score.  The fast exponential is within (2 + 1.2 |d|) 2^-23 of
// exp(-d), relative.  Sigmoid, 1 / (1 + e): at most 0.63 * 2^-23 from e, then the
// sum's and the quotient's roundings, below 2^-21.5 together.  Softmax: the sum of
// up to 1024 positive terms (32 in a lane, 5 exchanges) is off by 37 * 2^-24 and by
// its terms' weighted error, at most 8 * 2^-23: with the quotient below 2^-18.
constexpr float kSigmoidErr = 0x1p-21f, kSoftmaxErr = 0x1p-18f;

template <int kVPT, bool kBf16>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int t, int lane, float (&x)[kVPT]) {
  const size_t row = static_cast<size_t>(t) * a.ldl;
  constexpr int kPer = kBf16 ? 8 : 4;  // logits per 16 bytes
  if constexpr (kVPT >= kPer) {
    if (a.vec) {  // whole vectors: rows 16-byte aligned, E a multiple of kVPT
#pragma unroll
      for (int j = 0; j < kVPT; j += kPer) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const bool in = lane * kVPT < a.E;
        if (in)
          v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.logits) +
                                                   (row + lane * kVPT + j) * (kBf16 ? 2 : 4)));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float f = kBf16 ? __uint_as_float(i & 1 ? w[i / 2 % 4] & 0xffff0000u : w[i / 2 % 4] << 16)
                                : __uint_as_float(w[i % 4]);
          x[j + i] = !in || f != f ? -INFINITY : fminf(f, FLT_MAX);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int e = lane * kVPT + j;
    float v = -INFINITY;
    if (e < a.E) {
      if constexpr (kBf16)
        v = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + row + e)) << 16);
      else
        v = __ldg(static_cast<const float*>(a.logits) + row + e);
    }
    x[j] = v != v ? -INFINITY : fminf(v, FLT_MAX);
  }
}

template <bool kBf16>
__device__ __forceinline__ float logit_at(const RouteArgs& a, int t, int e) {
  const size_t at = static_cast<size_t>(t) * a.ldl + e;
  const float v = kBf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + at)) << 16)
                        : __ldg(static_cast<const float*>(a.logits) + at);
  return fminf(v, FLT_MAX);
}

__device__ __forceinline__ float warp_max_f(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// Order-preserving integers (the key 0, below every number's, marks "not a candidate").
__device__ __forceinline__ unsigned key32(float v) {
  const unsigned u = __float_as_uint(v + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key32_value(unsigned k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }
__device__ __forceinline__ unsigned warp_max_key(unsigned k) { return __reduce_max_sync(kFull, k); }

__device__ __forceinline__ unsigned long long key64(double v) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key64_value(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}
__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long k) {
  const unsigned hi = __reduce_max_sync(kFull, static_cast<unsigned>(k >> 32));
  const unsigned lo = __reduce_max_sync(kFull, static_cast<unsigned>(k >> 32) == hi ? static_cast<unsigned>(k) : 0u);
  return (static_cast<unsigned long long>(hi) << 32) | lo;
}

struct Key32 {
  using K = unsigned;
  using V = float;
  static __device__ __forceinline__ K key(V v) { return key32(v); }
  static __device__ __forceinline__ V value(K k) { return key32_value(k); }
};
struct Key64 {
  using K = unsigned long long;
  using V = double;
  static __device__ __forceinline__ K key(V v) { return key64(v); }
  static __device__ __forceinline__ V value(K k) { return key64_value(k); }
};

// Two largest of two pairs of keys.
template <typename K>
__device__ __forceinline__ void merge2(K& b1, K& b2, K o1, K o2) {
  const K lo = b1 < o1 ? b1 : o1;
  b1 = b1 < o1 ? o1 : b1;
  b2 = b2 < o2 ? o2 : b2;
  b2 = b2 < lo ? lo : b2;
}

// Clears the keys outside the kept groups.  gkey: the keys that a group's value
// is made of.  Returns how far the worst kept group's value is above the best
// other one's (infinity where all or no others are left).
template <typename T, int kVPT>
__device__ __forceinline__ typename T::V keep_groups(const RouteArgs& a, int lane, const typename T::K (&gkey)[kVPT],
                                                     typename T::K (&key)[kVPT]) {
  using K = typename T::K;
  using V = typename T::V;
  const int per = a.per;
  auto group_value = [&](K b1, K b2) -> K { return a.top == 2 && b2 ? T::key(T::value(b1) + T::value(b2)) : b1; };
  K mine = 0;  // lane g: group g's value
  const bool whole_lanes = a.span_log >= 0;  // a group is a power of two of whole lanes
  const int span = 1 << (whole_lanes ? a.span_log : 0);
  if (whole_lanes) {
    K b1 = 0, b2 = 0;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) merge2<K>(b1, b2, gkey[j], K(0));
    for (int o = 1; o < span; o <<= 1) {
      const K o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
      merge2<K>(b1, b2, o1, o2);
    }
    const K v = group_value(b1, b2);
    mine = __shfl_sync(kFull, v, (lane << a.span_log) & 31);
    if (lane >= a.groups) mine = 0;
  } else {
    for (int g = 0; g < a.groups; ++g) {
      K b1 = 0, b2 = 0;
#pragma unroll
      for (int j = 0; j < kVPT; ++j) {
        const int e = lane * kVPT + j;
        merge2<K>(b1, b2, e >= g * per && e < (g + 1) * per ? gkey[j] : K(0), K(0));
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const K o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
        merge2<K>(b1, b2, o1, o2);
      }
      const K v = group_value(b1, b2);
      if (lane == g) mine = v;
    }
  }
  // a group's rank: the groups before it in the order of values, then of indices
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const K v = __shfl_sync(kFull, mine, g);
    rank += v > mine || (v == mine && g < lane) ? 1 : 0;
  }
  const bool in = lane < a.groups && rank < a.keep;
  const unsigned kept = __ballot_sync(kFull, in);
  if (whole_lanes) {
    const bool mine_kept = (kept >> (lane >> a.span_log)) & 1u;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) key[j] = mine_kept ? key[j] : K(0);
  } else {
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
      const int e = lane * kVPT + j;
      if (e < a.E && !((kept >> (e / per)) & 1u)) key[j] = 0;
    }
  }
  const K last = ~warp_max_key(in ? ~mine : K(0)), next = warp_max_key(in ? K(0) : mine);
  return last && next ? T::value(last) - T::value(next) : static_cast<V>(INFINITY);
}

__device__ __forceinline__ double exact_score(bool sigmoid, float x, float mx) {
  if (!(x > -INFINITY)) return 0.0;
  return sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x))) : exp(static_cast<double>(x) - static_cast<double>(mx));
}

// exp(x) within 1e-11: x = n ln 2 + r, |r| <= ln 2 / 2, the series of exp(r) to its
// ninth power, times 2^n.  (The library's function, for its last bits, takes about
// five times the instructions.)
__device__ __forceinline__ double exp_series(double x) {
  if (!(fabs(x) < 700.0)) return exp(x);
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(-n, 0.6931471805599453, x);
  double p = 1.0 / 362880.0;
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return p * __hiloint2double((static_cast<int>(n) + 1023) << 20, 0);
}

// 1 / d to about 2^-42 for d well inside fp32's range: a 32-bit reciprocal and one Newton step.
__device__ __forceinline__ double reciprocal(double d) {
  const double r = static_cast<double>(__fdividef(1.f, static_cast<float>(d)));
  return fma(r, fma(-d, r, 1.0), r);
}

// Weights of the chosen experts (lane i: the i-th, its logit xs) and the row's
// outputs.  total: the softmax's sum, where the weights are not renormalised.
__device__ __forceinline__ void write_row(const RouteArgs& a, int t, int lane, int id, float xs, float mx, double total) {
  double w = 0.0;
  if (id >= 0) {
    if (a.sigmoid) {
      const double e = exp_series(-static_cast<double>(xs));
      w = e < 1e30 ? reciprocal(1.0 + e) : 1.0 / (1.0 + e);
    } else {
      w = exp_series(static_cast<double>(xs) - static_cast<double>(mx));
    }
  }
  double sum = total;
  if (a.renorm) {
    sum = w;
    for (int o = 1; o < a.k; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    sum = __shfl_sync(kFull, sum, 0);
  }
  if (a.renorm || !a.sigmoid) {
    if (sum > 1e-30 && sum < 1e30) w *= reciprocal(sum);
    else if (sum > 0.0) w /= sum;
  }
  if (lane < a.k) {
    a.weights[static_cast<size_t>(t) * a.k + lane] = static_cast<float>(w * static_cast<double>(a.scale));
    a.ids[static_cast<size_t>(t) * a.k + lane] = id;
  }
}

// A row in 64 bits.
template <int kVPT, bool kBf16>
__device__ __noinline__ void route_row_exact(const RouteArgs& a, int t, int lane) {
  using K = Key64::K;
  float x[kVPT];
  load_logits<kVPT, kBf16>(a, t, lane, x);
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < kVPT; ++j) mx = fmaxf(mx, x[j]);
  mx = warp_max_f(mx);
  double s[kVPT], total = 0.0;
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    s[j] = exact_score(a.sigmoid, x[j], mx);
    total += s[j];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  K key[kVPT], gkey[kVPT];
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int e = lane * kVPT + j;
    const double v = a.sigmoid ? s[j] : (total > 0.0 ? s[j] / total : 0.0);
    const double c = a.bias ? v + static_cast<double>(e < a.E ? __ldg(a.bias + e) : 0.f) : static_cast<double>(x[j]);
    const bool can = x[j] > -INFINITY && c > -INFINITY;  // (a bias of -inf or NaN excludes too)
    key[j] = can ? key64(c) : 0;
    gkey[j] = a.top == 2 && !a.bias && can ? key64(v) : key[j];
  }
  if (a.keep < a.groups) keep_groups<Key64, kVPT>(a, lane, gkey, key);
  int my_id = -1;
  float my_x = 0.f;
  for (int i = 0; i < a.k; ++i) {
    K b = 0;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) b = key[j] > b ? key[j] : b;
    const K best = warp_max_key(b);
    if (best == 0) break;
    const int owner = __ffs(__ballot_sync(kFull, b == best)) - 1;
    int at = -1;
    float xv = 0.f;
#pragma unroll
    for (int j = kVPT - 1; j >= 0; --j)
      if (key[j] == best) {
        at = j;
        xv = x[j];
      }
#pragma unroll
    for (int j = 0; j < kVPT; ++j)
      if (lane == owner && j == at) key[j] = 0;
    at = __shfl_sync(kFull, at, owner);
    xv = __shfl_sync(kFull, xv, owner);
    if (lane == i) {
      my_id = owner * kVPT + at;
      my_x = xv;
    }
  }
  write_row(a, t, lane, my_id, my_x, mx, total);
}

constexpr int kRouteWarps = 4;

template <int kVPT, bool kBf16>
__global__ void __launch_bounds__(kRouteWarps * 32, kVPT <= 8 ? 8 : 1) route_kernel(const __grid_constant__ RouteArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const unsigned row = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);  // (the last block's may pass 2^31)
  if (row >= static_cast<unsigned>(a.T)) return;
  const int t = static_cast<int>(row);
  float x[kVPT], bias[kVPT];
  load_logits<kVPT, kBf16>(a, t, lane, x);
#pragma unroll
  for (int j = 0; j < kVPT; ++j) bias[j] = 0.f;
  if (a.bias) {
    if (kVPT >= 4 && a.vec_bias) {
#pragma unroll
      for (int j = 0; j + 3 < kVPT; j += 4)
        if (lane * kVPT < a.E) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(a.bias + lane * kVPT + j));
          bias[j] = f.x;
          bias[j + 1] = f.y;
          bias[j + 2] = f.z;
          bias[j + 3] = f.w;
        }
    } else {
#pragma unroll
      for (int j = 0; j < kVPT; ++j)
        if (lane * kVPT + j < a.E) bias[j] = __ldg(a.bias + lane * kVPT + j);
    }
  }
  float mx = -INFINITY;
  if (!a.sigmoid) {
#pragma unroll
    for (int j = 0; j < kVPT; ++j) mx = fmaxf(mx, x[j]);
    mx = warp_max_f(mx);
  }
  const bool grouped = a.keep < a.groups;
  const bool by_score = a.bias != nullptr || (grouped && a.top == 2);  // scores decide something
  const bool need_total = !a.sigmoid && !a.renorm;
  double total = 0.0;
  if (need_total) {
    // the weights' denominator: exponentials within 2^-22, the rounding of x - max undone to first order
    for (int j = 0; j < kVPT; ++j) {
      if (x[j] > -INFINITY) {
        const double d = static_cast<double>(x[j]) - static_cast<double>(mx);
        const float r = static_cast<float>(d);
        const float ex = expf(r);
        // (d may lie below fp32's range, a masked logit under an infinite one: r and d - r are infinite there)
        if (ex > 0.f) total += static_cast<double>(ex) * (1.0 + (d - static_cast<double>(r)));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  }
  // keys of the choice: the value's upper bits, then the index inside the lane
  // (lowest first among equals), so that a key names its expert
  constexpr unsigned kIdx = kVPT - 1;  // kVPT is a power of two
  constexpr float kCut = kVPT * 0x1p-23f;  // what the index's bits cut off a value, relative
  unsigned key[kVPT];
  bool sure = true;
  const float err = a.sigmoid ? kSigmoidErr : kSoftmaxErr;
  float s[kVPT];
  if (by_score) {
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < kVPT; ++j) s[j] = __fdividef(1.f, 1.f + __expf(fminf(-x[j], 80.f)));
    } else {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kVPT; ++j) {
        s[j] = x[j] > -INFINITY ? __expf(x[j] - mx) : 0.f;
        sum += s[j];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const float inv = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
#pragma unroll
      for (int j = 0; j < kVPT; ++j) s[j] *= inv;
    }
  }
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const float c = a.bias ? s[j] + bias[j] : x[j];
    key[j] = x[j] > -INFINITY && c > -INFINITY ? key32(c) : 0u;
  }
  if (grouped) {
    const bool sums = a.top == 2 && !a.bias;
    unsigned gkey[kVPT];
#pragma unroll
    for (int j = 0; j < kVPT; ++j) gkey[j] = sums && key[j] ? key32(s[j]) : key[j];
    const float gap = keep_groups<Key32, kVPT>(a, lane, gkey, key);
    if (by_score) {
      // (a group's value: up to two choice values, each off by the score's error and a rounding of the sum)
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < kVPT; ++j) most = fmaxf(most, fabsf(bias[j]));
      most = warp_max_f(most);
      sure = gap > 4.f * err + (1.f + most) * 0x1p-20f;
    }
  }
  unsigned b = 0u;
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    key[j] = key[j] ? (key[j] & ~kIdx) | (kIdx - j) : 0u;
    b = key[j] > b ? key[j] : b;
  }
  // The k best and one more; lane i keeps the i-th.
  // (lane i also keeps whose it was; with k = 32 the one behind is kept apart)
  unsigned my_key = 0u, last_key = 0u;
  int my_owner = 0;
  const int rounds = sure ? a.k + 1 : 0;
  for (int i = 0; i < rounds; ++i) {
    const unsigned most = warp_max_key(b);
    if (most == 0u) {
      last_key = 0u;
      break;
    }
    const int owner = __ffs(__ballot_sync(kFull, (b | kIdx) == (most | kIdx))) - 1;  // the lowest lane of equals
    const unsigned best = __shfl_sync(kFull, b, owner);
    last_key = best;
    if (lane == i) {
      my_key = best;
      my_owner = owner;
    }
    const unsigned gone = lane == owner ? best : 0xffffffffu;
    b = 0u;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
      key[j] = key[j] == gone ? 0u : key[j];
      b = key[j] > b ? key[j] : b;
    }
  }
  // Neighbours in the order must be further apart than their errors (without a
  // bias: than the cut) or equal by construction (same logit, same bias); the
  // first one left out must be apart, since its equals behind it were not seen.
  const int my_id = lane < a.k && my_key ? my_owner * kVPT + static_cast<int>(kIdx - (my_key & kIdx)) : -1;
  const float my_x = my_id >= 0 ? logit_at<kBf16>(a, t, my_id) : 0.f;
  const float my_b = a.bias && my_id >= 0 ? __ldg(a.bias + my_id) : 0.f;
  if (a.bias || !kBf16) {  // (the cut takes nothing from a bf16 logit: its keys are exact)
    const unsigned down = __shfl_down_sync(kFull, my_key, 1);
    const float next_x = __shfl_down_sync(kFull, my_x, 1), next_b = __shfl_down_sync(kFull, my_b, 1);
    const unsigned next = lane == a.k - 1 ? last_key : down;
    bool ok = true;
    if (lane < a.k && my_key && next) {
      ok = (my_key ^ next) > kIdx;  // the cut keys differ: so do the logits
      if (a.bias) {
        const float hi = key32_value(my_key & ~kIdx), lo = key32_value(next | kIdx);
        ok = hi - lo > 2.f * err + (fabsf(hi) + fabsf(lo)) * (kCut + 0x1p-22f);
      }
      ok = ok || (lane < a.k - 1 && my_x == next_x && my_b == next_b);
    }
    sure = sure && __all_sync(kFull, ok);
  }
  if (!sure) {
    route_row_exact<kVPT, kBf16>(a, t, lane);
    return;
  }
  write_row(a, t, lane, my_id, my_x, mx, total);
}

// ---------------------------------------------------------------------------
// Sort of the pairs by expert (stable counting sort).  A warp takes kRounds x 32
// consecutive pairs and counts them per expert in shared memory; the counts
// become start positions (experts before, blocks before, warps before), and a
// second pass over the same pairs places them, 32 at a time: a pair's rank among
// the 32 is the number of lower lanes with the same expert.  One block does a
// decode step; more blocks first count their pairs in a kernel of their own.
// Bound by latency: 1.8 us for 256 pairs, 12.4 us for 262144 over 256 experts.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;                          // several blocks: rounds per warp
constexpr int kSortChunk = kSortThreads * kSortRounds;  // and pairs per block

__host__ __device__ inline int count_stride(int E) { return (E + 3) & ~3; }  // a block's row of counts, whole vectors

// Up to 64 K counts each block adds the others' up for itself: no launch in
// between, but loads that grow with the square of the blocks.  Above, a kernel of
// its own replaces the counts by their running sums, in time that grows with the
// pairs.  By themselves / by the kernel, on B200: 262144 pairs over 256 experts (32 K
// counts) 12.7 / 12.9 us, 524288 (64 K) 17.6 / 17.2, 2 M 133 / 56; 2 M over 16
// (16 K) 24 / 43, 8 M (64 K) 163 / 163; 64 M over 1024, 780 ms / 2.6 ms.
__host__ __device__ inline bool sums_apart(int blocks, int stride) { return blocks * stride > (1 << 16); }

// Counts of each block's pairs per expert.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int* __restrict__ ids, int P, int E,
                                                                  int* __restrict__ counts) {
  extern __shared__ int hist[];
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  griddep_wait();
  const long long p0 = static_cast<long long>(blockIdx.x) * kSortChunk;
  int id[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const long long p = p0 + r * kSortThreads + threadIdx.x;
    id[r] = p < P ? __ldg(ids + p) : -1;
  }
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    if (id[r] >= 0 && id[r] < E) atomicAdd(hist + id[r], 1);
  __syncthreads();
  const int stride = count_stride(E);
  for (int e = threadIdx.x; e < stride; e += kSortThreads)
    counts[static_cast<size_t>(blockIdx.x) * stride + e] = e < E ? hist[e] : 0;
}

// Each block's counts become the counts of the blocks before it; the row behind
// the last block's, the totals.  A thread per expert, 16 blocks' loads in flight.
constexpr int kScanThreads = 64;

__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(int* counts, int blocks, int stride) {
  griddep_launch_dependents();
  griddep_wait();
  const int e = blockIdx.x * kScanThreads + threadIdx.x;
  if (e >= stride) return;
  int sum = 0;
  for (int b0 = 0; b0 < blocks; b0 += 16) {
    int c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i] = b0 + i < blocks ? counts[static_cast<size_t>(b0 + i) * stride + e] : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (b0 + i < blocks) counts[static_cast<size_t>(b0 + i) * stride + e] = sum;
      sum += c[i];
    }
  }
  counts[static_cast<size_t>(blocks) * stride + e] = sum;
}

template <int kRounds>
__global__ void __launch_bounds__(kSortThreads)
    sort_place_kernel(const int* __restrict__ ids, int P, int E, int* __restrict__ offsets, int* __restrict__ order,
                      int* __restrict__ pos, const int* __restrict__ counts) {
  extern __shared__ int sh[];
  const int stride = count_stride(E);
  int* cnt = sh;                            // [warps][E]: a warp's count, then its next position
  int* total = sh + kSortWarps * stride;    // [E]: pairs of the expert in all blocks, then its first position
  int* before = total + stride;             // [E]: pairs of the expert in the blocks before
  __shared__ int scan[kSortWarps + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool alone = gridDim.x == 1;
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < (kSortWarps + 2) * stride; i += kSortThreads) sh[i] = 0;
  __syncthreads();
  griddep_wait();
  const long long p0 = static_cast<long long>(blockIdx.x) * (kSortThreads * kRounds) + warp * (32 * kRounds) + lane;
  int id[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const long long p = p0 + r * 32;
    const int e = p < P ? __ldg(ids + p) : -1;
    id[r] = e >= 0 && e < E ? e : -1;
  }
  if (sums_apart(gridDim.x, stride)) {
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
      before[e] = __ldg(counts + static_cast<size_t>(blockIdx.x) * stride + e);
      total[e] = __ldg(counts + static_cast<size_t>(gridDim.x) * stride + e);
    }
  } else if (!alone) {
    // the blocks' counts, four experts a thread, the blocks dealt to as many threads as there are
    const int vecs = stride / 4, teams = kSortThreads / vecs;
    const int team = threadIdx.x / vecs, v = threadIdx.x - team * vecs;
    if (team < teams) {
      int4 all = make_int4(0, 0, 0, 0), prior = all;
#pragma unroll 8
      for (int b = team; b < static_cast<int>(gridDim.x); b += teams) {
        const int4 c = __ldg(reinterpret_cast<const int4*>(counts + static_cast<size_t>(b) * stride) + v);
        const int m = b < static_cast<int>(blockIdx.x) ? -1 : 0;
        all = make_int4(all.x + c.x, all.y + c.y, all.z + c.z, all.w + c.w);
        prior = make_int4(prior.x + (c.x & m), prior.y + (c.y & m), prior.z + (c.z & m), prior.w + (c.w & m));
      }
      const int s4[4] = {all.x, all.y, all.z, all.w}, p4[4] = {prior.x, prior.y, prior.z, prior.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (s4[i]) atomicAdd(total + 4 * v + i, s4[i]);
        if (p4[i]) atomicAdd(before + 4 * v + i, p4[i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (id[r] >= 0) {
      atomicAdd(cnt + warp * stride + id[r], 1);
      if (alone) atomicAdd(total + id[r], 1);
    }
  __syncthreads();
  // exclusive sum over the experts
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    const int own = e < E ? total[e] : 0;
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += up;
    }
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    int lead = carry, all = carry;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = scan[w];
      lead += w < warp ? c : 0;
      all += c;
    }
    if (e < E) {
      const int first = lead + v - own;
      if (blockIdx.x == 0) offsets[e] = first;
      // the warps' start positions of this expert
      int c[kSortWarps], at = first + before[e];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = cnt[w * stride + e];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        cnt[w * stride + e] = at;
        at += c[w];
      }
    }
    carry = all;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = carry;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const long long p = p0 + r * 32;
    const unsigned same = __match_any_sync(kFull, id[r]);
    int at = -1;
    if (id[r] >= 0) at = cnt[warp * stride + id[r]] + __popc(same & ((1u << lane) - 1u));
    if constexpr (kRounds > 1) {
      __syncwarp();
      if (id[r] >= 0 && lane == __ffs(same) - 1) cnt[warp * stride + id[r]] += __popc(same);
      __syncwarp();
    }
    if (p < P) {
      pos[p] = at;
      if (at >= 0) order[at] = static_cast<int>(p);
      if (p >= carry) order[p] = -1;  // behind the last pair
    }
  }
}

// ---------------------------------------------------------------------------
// Weighted sum of a token's expert outputs: 8 columns per thread, the k rows'
// loads in flight together, sums in 32 bits in slot order.  Bound by its reads:
// 8192 tokens of 8 rows of 4096: 100 us, 6.4 TB/s.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const uint16_t* __restrict__ h, int P, const int* __restrict__ pos, const float* __restrict__ weights,
                   const uint16_t* add, int lda, uint16_t* y, int T, int k, int nvec) {  // (y may be add)
  griddep_launch_dependents();
  griddep_wait();
  const long long i = static_cast<long long>(blockIdx.x) * kCombineThreads + threadIdx.x;
  if (i >= static_cast<long long>(T) * nvec) return;
  const int t = static_cast<int>(i / nvec), v = static_cast<int>(i - static_cast<long long>(t) * nvec);
  float acc[8];
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  if (add) {
    const uint4 a4 = *(reinterpret_cast<const uint4*>(add + static_cast<size_t>(t) * lda) + v);
    acc[0] = lo(a4.x); acc[1] = hi(a4.x); acc[2] = lo(a4.y); acc[3] = hi(a4.y);
    acc[4] = lo(a4.z); acc[5] = hi(a4.z); acc[6] = lo(a4.w); acc[7] = hi(a4.w);
  }
  for (int j0 = 0; j0 < k; j0 += 8) {
    uint4 r[8];
    float w[8];
    bool live[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      live[j] = false;
      if (j0 + j < k) {
        const size_t at = static_cast<size_t>(t) * k + j0 + j;
        const int p = __ldg(pos + at);
        live[j] = p >= 0 && p < P;
        if (live[j]) {
          w[j] = __ldg(weights + at);
          r[j] = __ldg(reinterpret_cast<const uint4*>(h) + static_cast<size_t>(p) * nvec + v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (live[j]) {
        acc[0] = fmaf(w[j], lo(r[j].x), acc[0]); acc[1] = fmaf(w[j], hi(r[j].x), acc[1]);
        acc[2] = fmaf(w[j], lo(r[j].y), acc[2]); acc[3] = fmaf(w[j], hi(r[j].y), acc[3]);
        acc[4] = fmaf(w[j], lo(r[j].z), acc[4]); acc[5] = fmaf(w[j], hi(r[j].z), acc[5]);
        acc[6] = fmaf(w[j], lo(r[j].w), acc[6]); acc[7] = fmaf(w[j], hi(r[j].w), acc[7]);
      }
    }
  }
  auto pack = [](float a, float b) {
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(a))) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(b))) << 16);
  };
  reinterpret_cast<uint4*>(y)[static_cast<size_t>(t) * nvec + v] =
      make_uint4(pack(acc[0], acc[1]), pack(acc[2], acc[3]), pack(acc[4], acc[5]), pack(acc[6], acc[7]));
}

template <int kVPT, bool kBf16>
cudaError_t launch_route_v(RouteArgs a, cudaStream_t st) {
  const bool whole = a.E % kVPT == 0;
  a.vec = whole && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && static_cast<size_t>(a.ldl) * (kBf16 ? 2 : 4) % 16 == 0;
  a.per = a.E / a.groups;
  a.span_log = -1;
  if (a.per % kVPT == 0)
    for (int l = 0; l <= 5; ++l)
      if (a.per == kVPT << l) a.span_log = l;
  a.vec_bias = whole && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  return launch_pdl(route_kernel<kVPT, kBf16>, (static_cast<unsigned>(a.T) + kRouteWarps - 1) / kRouteWarps,
                    kRouteWarps * 32, 0, st, a);
}

template <bool kBf16>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t st) {
  const int vpt = (a.E + 31) / 32;
  if (vpt <= 1) return launch_route_v<1, kBf16>(a, st);
  if (vpt <= 2) return launch_route_v<2, kBf16>(a, st);
  if (vpt <= 4) return launch_route_v<4, kBf16>(a, st);
  if (vpt <= 8) return launch_route_v<8, kBf16>(a, st);
  if (vpt <= 16) return launch_route_v<16, kBf16>(a, st);
  return launch_route_v<32, kBf16>(a, st);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_route_t<true>(a, stream) : launch_route_t<false>(a, stream);
}

int sort_blocks(int P) { return static_cast<int>((static_cast<long long>(P) + kSortChunk - 1) / kSortChunk); }

size_t sort_workspace(int P, int E) {
  const int blocks = sort_blocks(P);
  const int stride = count_stride(E);
  return blocks > 1 ? static_cast<size_t>(blocks + (sums_apart(blocks, stride) ? 1 : 0)) * stride * 4 : 0;
}

template <int kRounds>
static cudaError_t launch_place(unsigned blocks, const int* ids, int P, int E, int* offsets, int* order, int* pos,
                                const int* counts, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      allow_smem(sort_place_kernel<kRounds>, static_cast<size_t>(kSortWarps + 2) * kMaxExperts * 4, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(sort_place_kernel<kRounds>, blocks, kSortThreads,
                    static_cast<size_t>(kSortWarps + 2) * count_stride(E) * 4, stream, ids, P, E, offsets, order, pos,
                    counts);
}

cudaError_t launch_sort(const int* ids, int P, int E, int* offsets, int* order, int* pos, int* counts,
                        cudaStream_t stream) {
  if (P <= kSortThreads) return launch_place<1>(1, ids, P, E, offsets, order, pos, counts, stream);
  const unsigned blocks = static_cast<unsigned>(sort_blocks(P));
  if (blocks > 1) {
    cudaError_t e =
        launch_pdl(sort_count_kernel, blocks, kSortThreads, static_cast<size_t>(E) * 4, stream, ids, P, E, counts);
    if (e != cudaSuccess) return e;
    const int stride = count_stride(E);
    if (sums_apart(static_cast<int>(blocks), stride)) {
      e = launch_pdl(sort_scan_kernel, (stride + kScanThreads - 1) / kScanThreads, kScanThreads, 0, stream, counts,
                     static_cast<int>(blocks), stride);
      if (e != cudaSuccess) return e;
    }
  }
  return launch_place<kSortRounds>(blocks, ids, P, E, offsets, order, pos, counts, stream);
}

cudaError_t launch_combine(const uint16_t* h, int P, const int* pos, const float* weights, const uint16_t* add, int lda,
                           uint16_t* y, int T, int k, int H, cudaStream_t stream) {
  const int nvec = H / 8;
  const long long n = static_cast<long long>(T) * nvec;
  const unsigned grid = static_cast<unsigned>((n + kCombineThreads - 1) / kCombineThreads);
  return launch_pdl(combine_kernel, grid, kCombineThreads, 0, stream, h, P, pos, weights, add, lda, y, T, k, nvec);
}

}  // namespace qgd
