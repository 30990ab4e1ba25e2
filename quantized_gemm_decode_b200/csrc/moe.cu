// Routing to experts, the sort of (token, expert) pairs by expert, and the
// weighted sum of a token's expert outputs.
#include <cuda_bf16.h>
#include <float.h>

#include <atomic>
#include <utility>

#include "qgd_internal.h"
#include "sm100.cuh"

namespace qgd {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Routing: one warp per token, lane l holding experts l, l + 32, ...
//   x = logit (NaN counts as -inf, +inf as the largest float)
//   s = exp(x - max) / sum exp(x - max), or 1 / (1 + exp(-x))
//   choice value c = s + bias; the k largest c of the kept groups, ties to the
//   lowest index; an expert at -inf is never chosen (id -1, weight 0).
//   w_j = scale * s_j (/ sum of the chosen s)
// Values and comparisons are in 64 bits: two experts whose scores are equal in
// 32 bits would otherwise be ordered by the rounding of an exponential.
// Without a bias the order of the scores is the order of the logits.
// ---------------------------------------------------------------------------
// Order-preserving integer of a double; 0 (below every number's) marks "not a candidate".
__device__ __forceinline__ unsigned long long sort_key(double v) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double key_value(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long k) {
  const unsigned hi = __reduce_max_sync(kFull, static_cast<unsigned>(k >> 32));
  const unsigned lo = __reduce_max_sync(kFull, static_cast<unsigned>(k >> 32) == hi ? static_cast<unsigned>(k) : 0u);
  return (static_cast<unsigned long long>(hi) << 32) | lo;
}

constexpr int kRouteWarps = 4;

template <int kVPT, bool kBf16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int E = a.E;
  float x[kVPT];
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int e = j * 32 + lane;
    x[j] = -INFINITY;
    if (e < E) {
      const size_t at = static_cast<size_t>(t) * a.ldl + e;
      if constexpr (kBf16)
        x[j] = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + at)) << 16);
      else
        x[j] = __ldg(static_cast<const float*>(a.logits) + at);
      x[j] = x[j] != x[j] ? -INFINITY : fminf(x[j], FLT_MAX);
    }
    mx = fmaxf(mx, x[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  // scores
  double s[kVPT];
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < kVPT; ++j) s[j] = x[j] > -INFINITY ? 1.0 / (1.0 + exp(-static_cast<double>(x[j]))) : 0.0;
  } else {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
      s[j] = x[j] > -INFINITY ? exp(static_cast<double>(x[j]) - static_cast<double>(mx)) : 0.0;
      sum += s[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) s[j] *= inv;
  }
  // choice keys; with groups, gkey holds what a group's value is made of
  unsigned long long key[kVPT];
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int e = j * 32 + lane;
    const double c = a.bias ? s[j] + static_cast<double>(e < E ? __ldg(a.bias + e) : 0.f) : static_cast<double>(x[j]);
    key[j] = x[j] > -INFINITY && c > -INFINITY ? sort_key(c) : 0ull;  // (a bias of -inf or NaN excludes too)
  }
  if (a.keep < a.groups) {
    const int per = E / a.groups;
    unsigned long long mine = 0ull;  // lane g: group g's value
    for (int g = 0; g < a.groups; ++g) {
      // the lane's two best of the group, then the warp's
      unsigned long long b1 = 0ull, b2 = 0ull;
#pragma unroll
      for (int j = 0; j < kVPT; ++j) {
        const int e = j * 32 + lane;
        unsigned long long v = e >= g * per && e < (g + 1) * per ? key[j] : 0ull;
        if (a.top == 2 && !a.bias && v) v = sort_key(s[j]);
        if (v > b1) { b2 = b1; b1 = v; } else if (v > b2) { b2 = v; }
      }
      const unsigned long long m1 = warp_max_key(b1);
      unsigned long long value = m1;
      if (a.top == 2 && m1) {
        const unsigned owner = __ffs(__ballot_sync(kFull, b1 == m1)) - 1;
        const unsigned long long m2 = warp_max_key(lane == static_cast<int>(owner) ? b2 : b1);
        if (m2) value = sort_key(key_value(m1) + key_value(m2));
      }
      if (lane == g) mine = value;
    }
    unsigned kept = 0u;
    for (int i = 0; i < a.keep; ++i) {
      const unsigned long long best = warp_max_key(mine);
      if (best == 0ull) break;
      const int g = __ffs(__ballot_sync(kFull, mine == best)) - 1;
      kept |= 1u << g;
      if (lane == g) mine = 0ull;
    }
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
      const int e = j * 32 + lane;
      if (e < E && !((kept >> (e / per)) & 1u)) key[j] = 0ull;
    }
  }
  // the k best; lane i keeps the i-th
  double my_s = 0.0;
  int my_id = -1;
  for (int i = 0; i < a.k; ++i) {
    unsigned long long b = 0ull;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) b = key[j] > b ? key[j] : b;
    const unsigned long long best = warp_max_key(b);
    if (best == 0ull) break;
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int j = kVPT - 1; j >= 0; --j)
      if (key[j] == best) at = j * 32 + lane;
    at = __reduce_min_sync(kFull, at);
    double sv = 0.0;
#pragma unroll
    for (int j = 0; j < kVPT; ++j)
      if (static_cast<unsigned>(j * 32 + lane) == at) {
        sv = s[j];
        key[j] = 0ull;
      }
    sv = __shfl_sync(kFull, sv, at & 31);
    if (lane == i) {
      my_s = sv;
      my_id = static_cast<int>(at);
    }
  }
  if (a.renorm) {
    double sum = my_s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (sum > 0.0) my_s /= sum;
  }
  if (lane < a.k) {
    a.weights[static_cast<size_t>(t) * a.k + lane] = static_cast<float>(my_s * static_cast<double>(a.scale));
    a.ids[static_cast<size_t>(t) * a.k + lane] = my_id;
  }
}

// ---------------------------------------------------------------------------
// Sort of the pairs by expert (stable counting sort).  A block takes
// kSortRounds x 32 consecutive pairs per warp; each warp counts its own pairs
// per expert in shared memory, the counts become start positions (experts
// before, blocks before, warps before), and a second pass over the same pairs
// places them, 32 at a time: a pair's rank among the 32 is the number of
// lower lanes with the same expert.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 8;
constexpr int kSortChunk = kSortThreads * kSortRounds;  // pairs per block

// Counts of this block's pairs per expert.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int* __restrict__ ids, int P, int E,
                                                                  int* __restrict__ counts) {
  extern __shared__ int hist[];
  griddep_launch_dependents();
  griddep_wait();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const long long p0 = static_cast<long long>(blockIdx.x) * kSortChunk;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const long long p = p0 + r * kSortThreads + threadIdx.x;
    const int e = p < P ? __ldg(ids + p) : -1;
    if (e >= 0 && e < E) atomicAdd(hist + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
}

__global__ void __launch_bounds__(kSortThreads)
    sort_place_kernel(const int* __restrict__ ids, int P, int E, int* __restrict__ offsets, int* __restrict__ order,
                      int* __restrict__ pos, const int* __restrict__ counts) {
  extern __shared__ int sh[];
  int* cnt = sh;                       // [warps][E]: a warp's count, then its next position
  int* total = sh + kSortWarps * E;    // [E]: pairs of the expert in all blocks, then its first position
  int* before = total + E;             // [E]: pairs of the expert in the blocks before
  __shared__ int scan[kSortWarps + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const long long p0 = static_cast<long long>(blockIdx.x) * kSortChunk + warp * (32 * kSortRounds) + lane;
  int id[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const long long p = p0 + r * 32;
    const int e = p < P ? __ldg(ids + p) : -1;
    id[r] = e >= 0 && e < E ? e : -1;
    if (id[r] >= 0) atomicAdd(cnt + warp * E + id[r], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int all = 0, prior = 0;
    if (gridDim.x == 1) {
      for (int w = 0; w < kSortWarps; ++w) all += cnt[w * E + e];
    } else {
#pragma unroll 8
      for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
        const int c = __ldg(counts + static_cast<size_t>(b) * E + e);
        all += c;
        prior += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    total[e] = all;
    before[e] = prior;
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
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) lead += scan[w];
      all += scan[w];
    }
    if (e < E) total[e] = lead + v - own;
    carry = all;
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < E; e += kSortThreads) offsets[e] = total[e];
    if (threadIdx.x == 0) offsets[E] = carry;
  }
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int at = total[e] + before[e];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const long long p = p0 + r * 32;
    const unsigned same = __match_any_sync(kFull, id[r]);
    int at = -1;
    if (id[r] >= 0) at = cnt[warp * E + id[r]] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (id[r] >= 0 && lane == __ffs(same) - 1) cnt[warp * E + id[r]] += __popc(same);
    __syncwarp();
    if (p < P) {
      pos[p] = at;
      if (at >= 0) order[at] = static_cast<int>(p);
      if (p >= carry) order[p] = -1;  // behind the last pair
    }
  }
}

// ---------------------------------------------------------------------------
// Weighted sum of a token's expert outputs: 8 columns per thread, the k rows'
// loads in flight together, sums in 32 bits in slot order.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const uint16_t* __restrict__ h, int P, const int* __restrict__ pos, const float* __restrict__ weights,
                   const uint16_t* __restrict__ add, int lda, uint16_t* __restrict__ y, int T, int k, int nvec) {
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
    const uint4 a4 = __ldg(reinterpret_cast<const uint4*>(add + static_cast<size_t>(t) * lda) + v);
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

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kBf16>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((a.T + kRouteWarps - 1) / kRouteWarps), block = kRouteWarps * 32;
  const int vpt = (a.E + 31) / 32;
  if (vpt <= 1) return launch_pdl(route_kernel<1, kBf16>, grid, block, 0, st, a);
  if (vpt <= 2) return launch_pdl(route_kernel<2, kBf16>, grid, block, 0, st, a);
  if (vpt <= 4) return launch_pdl(route_kernel<4, kBf16>, grid, block, 0, st, a);
  if (vpt <= 8) return launch_pdl(route_kernel<8, kBf16>, grid, block, 0, st, a);
  if (vpt <= 16) return launch_pdl(route_kernel<16, kBf16>, grid, block, 0, st, a);
  return launch_pdl(route_kernel<32, kBf16>, grid, block, 0, st, a);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_route_t<true>(a, stream) : launch_route_t<false>(a, stream);
}

int sort_blocks(int P, int E) {
  (void)E;
  return static_cast<int>((static_cast<long long>(P) + kSortChunk - 1) / kSortChunk);
}

cudaError_t launch_sort(const int* ids, int P, int E, int* offsets, int* order, int* pos, int* counts,
                        cudaStream_t stream) {
  const unsigned blocks = P > 0 ? static_cast<unsigned>(sort_blocks(P, E)) : 1u;
  cudaError_t e;
  if (blocks > 1) {
    e = launch_pdl(sort_count_kernel, blocks, kSortThreads, static_cast<size_t>(E) * 4, stream, ids, P, E, counts);
    if (e != cudaSuccess) return e;
  }
  const size_t smem = static_cast<size_t>(kSortWarps + 2) * E * 4;
  static std::atomic<uint64_t> done{0};
  e = allow_smem(sort_place_kernel, static_cast<size_t>(kSortWarps + 2) * kMaxExperts * 4, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(sort_place_kernel, blocks, kSortThreads, smem, stream, ids, P, E, offsets, order, pos,
                    static_cast<const int*>(counts));
}

cudaError_t launch_combine(const uint16_t* h, int P, const int* pos, const float* weights, const uint16_t* add, int lda,
                           uint16_t* y, int T, int k, int H, cudaStream_t stream) {
  const int nvec = H / 8;
  const long long n = static_cast<long long>(T) * nvec;
  const unsigned grid = static_cast<unsigned>((n + kCombineThreads - 1) / kCombineThreads);
  return launch_pdl(combine_kernel, grid, kCombineThreads, 0, stream, h, P, pos, weights, add, lda, y, T, k, nvec);
}

}  // namespace qgd
