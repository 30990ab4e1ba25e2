// Grouped quantized products of a mixture of experts: rows sorted by expert,
// each expert's rows times its own weights.
//
//   row i of the sorted order, offsets[e] <= i < offsets[e+1], source row
//   r = order[i] / div (or i):
//     sx = max(max |x[r]|, 1e-12) / qmax,  xq = convert(x[r] / sx)
//     v[n] = (sum_k xq[k] wq[e][n][k]) * sx * sw[e][n]
//     y[i][n] = bf16(v[n]), or with the gated activation over 2N weight rows
//               bf16(silu(v[n]) * v[N + n]),  silu(g) = g / (1 + exp(-g))
//
// Two kernels: the quantizer writes the codes in sorted order, then one
// persistent kernel walks the (expert, token tile, weight tile) tiles, whose
// number only the device knows, from the offsets.  Orientation as in the
// dense decode kernel (weights in the MMA's 128-row M slot, tokens in its N),
// because an expert's row count is ragged: N follows the tile's rows in steps
// of 16, where M would round every expert up to 128.
//
// Warp roles (192 threads): warp 0 issues TMA loads, warp 1 owns TMEM and
// issues MMAs, warps 2-5 drain the accumulator.  Every wait is bounded.
#include <cuda_bf16.h>

#include <atomic>
#include <utility>

#include "qgd_internal.h"
#include "quantcore.cuh"
#include "sm100.cuh"

namespace qgd {

// First error code recorded by the kernels of this file on this device.
__device__ unsigned int g_experts_error = 0;

namespace {

__device__ __forceinline__ void record_error(unsigned int code) { atomicCAS(&g_experts_error, 0u, code); }

// ---------------------------------------------------------------------------
// Quantizer: one CTA per sorted row.  Rows behind the last expert's are left
// alone; a source row outside x reads as zeros.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

template <int kVPT, int kQType>
__global__ void __launch_bounds__(kRowThreads)
    experts_quant_kernel(const uint16_t* __restrict__ x, int K, int ldx, int x_rows, const int* __restrict__ order,
                         int div, const int* __restrict__ offsets, int E, int P, uint8_t* __restrict__ q,
                         float* __restrict__ s, unsigned* __restrict__ tickets, int ntickets) {
  __shared__ float red[33];
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < ntickets; i += kRowThreads) tickets[i] = 0u;
  const int row = blockIdx.x;
  if (row >= min(__ldg(offsets + E), P)) return;
  const int pair = order ? __ldg(order + row) : row;
  const int src = order ? pair / div : row;
  const bool have = pair >= 0 && src < x_rows;
  const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(have ? src : 0) * ldx);
  uint2* qr = reinterpret_cast<uint2*>(q + static_cast<size_t>(row) * K);
  const int nvec = K / 8;
  uint4 v[kVPT];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int idx = threadIdx.x + j * kRowThreads;
    v[j] = make_uint4(0, 0, 0, 0);
    if (have && idx < nvec) {
      v[j] = __ldg(xr + idx);
      amax = fmaxf(amax, absmax8(v[j]));
    }
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = red[threadIdx.x & (kRowThreads / 32 - 1)];
#pragma unroll
  for (int o = kRowThreads / 64; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  amax = fmaxf(amax, kAmaxFloor);
  const float sc = __fdiv_rn(amax, kQType == 0 ? kE4M3Max : kInt8Max);
  if (threadIdx.x == 0) s[row] = sc;
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int idx = threadIdx.x + j * kRowThreads;
    if (idx < nvec) qr[idx] = encode8<kQType>(v[j], sc);
  }
}

// ---------------------------------------------------------------------------
// Grouped GEMM
// ---------------------------------------------------------------------------
struct Ctl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int last_flag;
  int epi_ok;
  int scan[8];
};
constexpr uint32_t kCtlBytes = 512;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block too large");
constexpr int kEpiThreads = 128;
constexpr uint32_t kOutBytes = 2 * 16 * 256;  // two staging buffers of 16 tokens x 128 bf16

// Shared-memory map of one CTA (after 1024-byte alignment):
//   ring of `stages` x kps x (128 weight rows + kTok token rows) x 128 bytes,
//   output staging, token scales [2][kTok], control block, expert tile prefix.
template <int kTok, int kKps>
struct Layout {
  static constexpr uint32_t kW = kSwapTileN * kTileK;
  static constexpr uint32_t kX = kTok * kTileK;
  static constexpr uint32_t kStage = kKps * (kW + kX);
  static constexpr uint32_t kTail = kOutBytes + 2 * kTok * 4 + kCtlBytes + (kMaxExperts + 1) * 4;
  static constexpr int kStages0 = static_cast<int>((kSmemBudget - 1024 - kTail) / kStage);
  static constexpr int kStages = kStages0 > kMaxStages ? kMaxStages : kStages0;
  static constexpr size_t kBytes = 1024 + static_cast<size_t>(kStages) * kStage + kTail;
};

// Where a tile lies: its expert, first sorted row, row count and weight tile.
struct Tile {
  int e, row0, n, nt;
};

__device__ __forceinline__ int clamp_off(int v, int P) { return v < 0 ? 0 : (v > P ? P : v); }

// Tile w of the list: weight tiles fastest, then an expert's token tiles, then
// the experts (pre[e]: token tiles of the experts before e).  An expert's rows
// are dealt to its token tiles evenly, in multiples of 16.
__device__ __forceinline__ Tile find_tile(const ExpertArgs& a, const int* pre, int tok, int w) {
  Tile t;
  const int g = w / a.n_tiles;
  t.nt = w - g * a.n_tiles;
  int lo = 0, hi = a.E;  // pre[lo] <= g < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= g) lo = mid;
    else hi = mid;
  }
  t.e = lo;
  const int o0 = clamp_off(__ldg(a.offsets + lo), a.P), o1 = clamp_off(__ldg(a.offsets + lo + 1), a.P);
  const int cnt = o1 - o0, tiles = pre[lo + 1] - pre[lo];
  const int per = ((cnt + tiles - 1) / tiles + 15) & ~15;
  const int j = g - pre[lo];
  t.row0 = o0 + j * per;
  t.n = min(per, cnt - j * per);
  return t;
}

__device__ __forceinline__ int unit_owner(long long u, long long G, long long U) {
  return static_cast<int>(((u + 1) * G - 1) / U);
}

// The CTA's work as a sequence of segments (tile, K units [k0, k1)).  kSplit:
// all (tile, K unit) units dealt out in equal contiguous ranges, one per CTA,
// so that every SM streams the same share of the weights; else whole tiles,
// round-robin.
template <bool kSplit>
struct Walk {
  long long u, ue;  // kSplit: units left; else: next tile and the tile count
  int nku;
  __device__ __forceinline__ Walk(int total, int nku_, int cta, int G) : nku(nku_) {
    if (kSplit) {
      const long long U = static_cast<long long>(total) * nku;
      u = static_cast<long long>(cta) * U / G;
      ue = static_cast<long long>(cta + 1) * U / G;
    } else {
      u = cta;
      ue = total;
    }
  }
  __device__ __forceinline__ bool next(int& w, int& k0, int& k1, int G) {
    if (u >= ue) return false;
    if (kSplit) {
      w = static_cast<int>(u / nku);
      k0 = static_cast<int>(u - static_cast<long long>(w) * nku);
      const long long left = ue - u;
      k1 = left < nku - k0 ? k0 + static_cast<int>(left) : nku;
      u += k1 - k0;
    } else {
      w = static_cast<int>(u);
      k0 = 0;
      k1 = nku;
      u += G;
    }
    return true;
  }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int v, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(v), "l"(policy)
      : "memory");
}

// exp(-g) overflows to infinity for very negative g, where the quotient is the
// -0 that silu tends to; the fast exponential's 2^-21 is far below bf16's step.
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + __expf(fminf(-g, 80.f))); }

template <int kFmt>
__device__ __forceinline__ float acc_value(uint32_t bits) {
  if constexpr (kFmt == kFmtINT8) return static_cast<float>(static_cast<int32_t>(bits));
  else return __uint_as_float(bits);
}

template <int kFmt>
__device__ __forceinline__ uint32_t add_acc(uint32_t x, uint32_t y) {
  if constexpr (kFmt == kFmtINT8) return x + y;
  else return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
}

// Sixteen tokens of this thread's weight row, finished and stored.  r: the
// accumulators of tokens c0 .. c0 + 15 of the tile.  The epilogue warps write
// bf16 rows [token][column] to shared memory and then store whole 16-byte
// vectors, so that y leaves in 128- or 256-byte runs although a thread holds
// one column.  With the activation a warp holds 16 gate rows (lanes 0-15) and
// their 16 up rows (lanes 16-31): each pair of lanes swaps halves, the lower
// lane finishes the even tokens, the upper one the odd ones.
template <int kFmt, bool kAct>
__device__ __forceinline__ void finish16(const ExpertArgs& a, const Tile& t, const uint32_t (&r)[16], int c0, float swv,
                                         const float* sxs, uint8_t* out, uint32_t& flip) {
  const int et = threadIdx.x - 64, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3;
  uint16_t* buf = reinterpret_cast<uint16_t*>(out + (flip & 1u) * (16 * 256));
  flip ^= 1u;
  if constexpr (kAct) {
    const bool up = lane >= 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float even = (acc_value<kFmt>(r[2 * j]) * sxs[c0 + 2 * j]) * swv;
      const float odd = (acc_value<kFmt>(r[2 * j + 1]) * sxs[c0 + 2 * j + 1]) * swv;
      const float other = __shfl_xor_sync(0xffffffffu, up ? even : odd, 16);
      const float gate = up ? other : even, lin = up ? odd : other;
      buf[(2 * j + (up ? 1 : 0)) * 64 + q * 16 + (lane & 15)] =
          __bfloat16_as_ushort(__float2bfloat16_rn(silu(gate) * lin));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      buf[j * 128 + q * 32 + lane] =
          __bfloat16_as_ushort(__float2bfloat16_rn((acc_value<kFmt>(r[j]) * sxs[c0 + j]) * swv));
  }
  named_bar_sync(1, kEpiThreads);
  constexpr int kCols = kAct ? 64 : 128;
  constexpr int kVecs = kCols / 8;  // 16-byte vectors per token
#pragma unroll
  for (int p = 0; p < 16 * kVecs / kEpiThreads; ++p) {
    const int idx = p * kEpiThreads + et;
    const int tok = idx / kVecs, vec = idx - tok * kVecs;
    const int col = t.nt * kCols + vec * 8;
    if (c0 + tok < t.n && col < a.N)
      *reinterpret_cast<uint4*>(a.y + static_cast<size_t>(t.row0 + c0 + tok) * a.N + col) =
          *reinterpret_cast<const uint4*>(buf + tok * kCols + vec * 8);
  }
}

template <int kFmt, int kTok, int kKps, bool kSplit, bool kAct>
__global__ void __launch_bounds__(kGemmThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const ExpertArgs a) {
  using L = Layout<kTok, kKps>;
  constexpr bool kInt = (kFmt == kFmtINT8);
  constexpr int kBoxTok = kTok <= 64 ? 16 : 64;  // token rows per TMA box
  constexpr uint32_t kCols = 2 * kTok;           // TMEM: double-buffered accumulator
  constexpr int stages = L::kStages;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  uint8_t* w_ring = base;
  uint8_t* x_ring = base + stages * kKps * L::kW;
  uint8_t* out = base + stages * L::kStage;
  float* sx_s = reinterpret_cast<float*>(out + kOutBytes);
  Ctl* ctl = reinterpret_cast<Ctl*>(sx_s + 2 * kTok);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(ctl) + kCtlBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkt = (a.K + kTileK - 1) / kTileK;
  const int nku = (nkt + kKps - 1) / kKps;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
    for (int i = 0; i < stages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], 1);
      mbar_init(&ctl->tempty[i], 4);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    ctl->last_flag = 0;
    ctl->epi_ok = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  griddep_launch_dependents();
  griddep_wait();  // offsets, codes and scales come from the kernels before
  // token tiles of the experts before e, as a running sum in blocks of 192 experts
  {
    int carry = 0;
    if (threadIdx.x == 0) pre[0] = 0;
    for (int e0 = 0; e0 < a.E; e0 += kGemmThreads) {
      const int e = e0 + threadIdx.x;
      int v = 0;
      if (e < a.E) {
        const int cnt = clamp_off(__ldg(a.offsets + e + 1), a.P) - clamp_off(__ldg(a.offsets + e), a.P);
        v = cnt > 0 ? (cnt + kTok - 1) / kTok : 0;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      if (lane == 31) ctl->scan[warp] = v;
      __syncthreads();
      int before = carry, all = carry;
      for (int i = 0; i < kGemmThreads / 32; ++i) {
        if (i < warp) before += ctl->scan[i];
        all += ctl->scan[i];
      }
      if (e < a.E) pre[e + 1] = before + v;
      carry = all;
      __syncthreads();
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int total = pre[a.E] * a.n_tiles;
  const long long U = static_cast<long long>(total) * nku;
  // CTAs with work: every one gets at least one unit (or tile)
  const long long most = kSplit ? U : total;
  const int G = most < static_cast<long long>(gridDim.x) ? static_cast<int>(most) : static_cast<int>(gridDim.x);
  const int cta = blockIdx.x;
  const bool busy = cta < G;
  int issued = 0;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0 && busy) {
      const uint64_t pol_w = kSplit ? policy_evict_first() : policy_evict_last();
      const uint64_t pol_x = policy_evict_last();
      Walk<kSplit> walk(total, nku, cta, G);
      int w, k0, k1, i = 0;
      bool stop = false;
      while (!stop && walk.next(w, k0, k1, G)) {
        const Tile t = find_tile(a, pre, kTok, w);
        const int boxes = (t.n + kBoxTok - 1) / kBoxTok;
        for (int k = k0; k < k1; ++k, ++i) {
          const int s = i % stages;
          if (!mbar_wait(&ctl->empty[s], ((i / stages) & 1) ^ 1)) {
            record_error(kErrWaitProducer);
            ctl->abort_flag = 1;
            stop = true;
            break;
          }
          if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) {
            stop = true;
            break;
          }
          const int kt = k * kKps, ns = min(kKps, nkt - kt);
          mbar_arrive_expect_tx(&ctl->full[s], ns * (L::kW + boxes * kBoxTok * kTileK));
          for (int h = 0; h < ns; ++h) {
            uint8_t* wd = w_ring + (s * kKps + h) * L::kW;
            if constexpr (kAct) {
              // four boxes of 16 gate rows and the 16 up rows of the same columns
#pragma unroll
              for (int b = 0; b < 4; ++b)
                tma_load_4d(wd + b * 32 * kTileK, &tw, &ctl->full[s], (kt + h) * kTileK, t.nt * 64 + b * 16, 0, t.e,
                            pol_w);
            } else {
              tma_load_3d(wd, &tw, &ctl->full[s], (kt + h) * kTileK, t.nt * 128, t.e, pol_w);
            }
            uint8_t* xd = x_ring + (s * kKps + h) * L::kX;
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(xd + b * kBoxTok * kTileK, &tx, &ctl->full[s], (kt + h) * kTileK, t.row0 + b * kBoxTok,
                          pol_x);
          }
          issued = i + 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0 && busy) {
      const uint32_t w_base = smem_u32(w_ring), x_base = smem_u32(x_ring);
      Walk<kSplit> walk(total, nku, cta, G);
      int w, k0, k1, i = 0, li = 0;
      bool stop = false;
      while (!stop && walk.next(w, k0, k1, G)) {
        const Tile t = find_tile(a, pre, kTok, w);
        const uint32_t idesc = idesc_mma(kInt ? 2 : 1, kInt ? 1 : 0, kSwapTileN, (t.n + 15) & ~15);
        const int b = li & 1;
        if (!mbar_wait(&ctl->tempty[b], ((li >> 1) & 1) ^ 1)) {
          record_error(kErrWaitMma);
          ctl->abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + b * kTok;
        for (int k = k0; k < k1; ++k, ++i) {
          const int s = i % stages;
          if (!mbar_wait(&ctl->full[s], (i / stages) & 1)) {
            record_error(kErrWaitMma);
            ctl->abort_flag = 1;
            stop = true;
            break;
          }
          if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const int ns = min(kKps, nkt - k * kKps);
          for (int h = 0; h < ns; ++h) {
#pragma unroll
            for (int kk = 0; kk < kTileK / 32; ++kk) {
              const uint64_t ad = sdesc_kmajor_sw128(w_base + (s * kKps + h) * L::kW + kk * 32);
              const uint64_t bd = sdesc_kmajor_sw128(x_base + (s * kKps + h) * L::kX + kk * 32);
              mma_issue<kInt>(d, ad, bd, idesc, (k > k0 || h > 0 || kk > 0) ? 1u : 0u);
            }
          }
          mma_commit(&ctl->empty[s]);
        }
        if (stop) break;
        mma_commit(&ctl->tfull[b]);
        ++li;
      }
    }
    __syncwarp();
  } else if (busy) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, et = threadIdx.x - 64;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int lrow = q * 32 + lane;  // row of the weight tile
    Walk<kSplit> walk(total, nku, cta, G);
    int w, k0, k1, li = 0;
    uint32_t flip = 0;
    while (walk.next(w, k0, k1, G)) {
      const Tile t = find_tile(a, pre, kTok, w);
      const int b = li & 1;
      float* sxs = sx_s + b * kTok;
      for (int i = et; i < ((t.n + 15) & ~15); i += kEpiThreads) sxs[i] = i < t.n ? __ldg(a.sx + t.row0 + i) : 0.f;
      // this thread's weight row and its channel scale (0 past the last row)
      float swv = 0.f;
      if constexpr (kAct) {
        const int col = t.nt * 64 + q * 16 + (lane & 15);
        if (col < a.N) swv = __ldg(a.sw + static_cast<size_t>(t.e) * 2 * a.N + (lane >= 16 ? a.N : 0) + col);
      } else {
        const int col = t.nt * 128 + lrow;
        if (col < a.N) swv = __ldg(a.sw + static_cast<size_t>(t.e) * a.N + col);
      }
      const bool ok = warp_wait(&ctl->tfull[b], (li >> 1) & 1);
      if (!ok && lane == 0) {
        record_error(kErrWaitEpilogue);
        ctl->abort_flag = 1;
      }
      if (ok) tc_fence_after();
      named_bar_sync(1, kEpiThreads);
      if (et == 0) ctl->epi_ok = (*reinterpret_cast<volatile int*>(&ctl->abort_flag) == 0);
      named_bar_sync(1, kEpiThreads);
      if (!ctl->epi_ok) break;
      const bool whole = !kSplit || (k0 == 0 && k1 == nku);
      int first = cta, ncontrib = 1;
      uint32_t* slot = nullptr;
      if (!whole) {
        const long long u0 = static_cast<long long>(w) * nku;
        first = unit_owner(u0, G, U);
        ncontrib = unit_owner(u0 + nku - 1, G, U) - first + 1;
        slot = a.partial + (static_cast<size_t>(cta) * 2 + (cta == first ? 1 : 0)) * (kSwapTileN * kTok) + lrow;
      }
      const int chunks = (t.n + 15) >> 4;
      for (int c = 0; c < chunks; ++c) {
        uint32_t r[16];
        __syncwarp();
        tmem_ld16(taddr + b * kTok + c * 16, r);
        tmem_wait_ld();
        if (c == chunks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->tempty[b]);
        }
        if (whole) {
          finish16<kFmt, kAct>(a, t, r, c * 16, swv, sxs, out, flip);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) __stcg(slot + (c * 16 + j) * kSwapTileN, r[j]);
        }
      }
      if (!whole) {
        // the last of the tile's CTAs to arrive adds the partials in CTA order
        named_bar_sync(1, kEpiThreads);
        if (et == 0) {
          unsigned old;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.tickets + first) : "memory");
          ctl->last_flag = (old == static_cast<unsigned>(ncontrib - 1));
        }
        named_bar_sync(1, kEpiThreads);
        if (ctl->last_flag) {
          for (int c = 0; c < chunks; ++c) {
            uint32_t sum[16];
            for (int j = 0; j < ncontrib; ++j) {
              const uint32_t* src =
                  a.partial + (static_cast<size_t>(first + j) * 2 + (j == 0 ? 1 : 0)) * (kSwapTileN * kTok) + lrow;
              uint32_t v[16];
#pragma unroll
              for (int m = 0; m < 16; ++m) v[m] = __ldcg(src + (c * 16 + m) * kSwapTileN);
#pragma unroll
              for (int m = 0; m < 16; ++m) sum[m] = j == 0 ? v[m] : add_acc<kFmt>(sum[m], v[m]);
            }
            finish16<kFmt, kAct>(a, t, sum, c * 16, swv, sxs, out, flip);
          }
        }
      }
      ++li;
    }
  }

  // ---------------- teardown ----------------
  tc_fence_before();
  __syncthreads();
  if (ctl->abort_flag) {
    if (warp == 0 && lane == 0) {
      // the last copies issued into each stage must land before the CTA exits
      for (int i = issued > stages ? issued - stages : 0; i < issued; ++i) {
        if (!mbar_wait(&ctl->full[i % stages], (i / stages) & 1)) {
          record_error(kErrWaitDrain);
          break;
        }
      }
    }
    if (warp == 1 && lane == 0) {
      mma_commit(&ctl->drain);
      if (!mbar_wait(&ctl->drain, 0)) record_error(kErrWaitDrain);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
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

template <int kQType>
cudaError_t launch_quant_t(const ExpertArgs& a, const uint16_t* x, int ldx, int x_rows, const int* order, int div,
                           uint8_t* q, float* s, cudaStream_t st) {
  const int vpt = (a.K / 8 + kRowThreads - 1) / kRowThreads;
  const dim3 grid(a.P), block(kRowThreads);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, st, x, a.K, ldx, x_rows, order, div, a.offsets, a.E, a.P, q, s,
                      a.tickets, a.ctas);
  };
  if (vpt <= 1) return go(experts_quant_kernel<1, kQType>);
  if (vpt <= 2) return go(experts_quant_kernel<2, kQType>);
  if (vpt <= 4) return go(experts_quant_kernel<4, kQType>);
  if (vpt <= 8) return go(experts_quant_kernel<8, kQType>);
  return cudaErrorInvalidValue;
}

template <int kFmt, int kTok, int kKps, bool kSplit, bool kAct>
cudaError_t launch_t(const CUtensorMap& tw, const CUtensorMap& tx, const ExpertArgs& a, cudaStream_t st) {
  using L = Layout<kTok, kKps>;
  static_assert(L::kStages >= 2 && L::kBytes <= kSmemBudget, "ring does not fit");
  auto kernel = experts_kernel<kFmt, kTok, kKps, kSplit, kAct>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, L::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.ctas), dim3(kGemmThreads), L::kBytes, st, tw, tx, a);
}

template <int kFmt, bool kAct>
cudaError_t launch_f(const CUtensorMap& tw, const CUtensorMap& tx, const ExpertArgs& a, cudaStream_t st) {
  return a.tok <= 64 ? launch_t<kFmt, 64, 2, true, kAct>(tw, tx, a, st)
                     : launch_t<kFmt, 256, 1, false, kAct>(tw, tx, a, st);
}

}  // namespace

cudaError_t launch_experts_quant(int fmt, const ExpertArgs& a, const uint16_t* x, int ldx, int x_rows,
                                 const int* order, int div, uint8_t* q, float* s, cudaStream_t stream) {
  return fmt == kFmtINT8 ? launch_quant_t<1>(a, x, ldx, x_rows, order, div, q, s, stream)
                         : launch_quant_t<0>(a, x, ldx, x_rows, order, div, q, s, stream);
}

cudaError_t launch_experts(int fmt, bool act, const CUtensorMap& tw, const CUtensorMap& tx, const ExpertArgs& a,
                           cudaStream_t stream) {
  if (fmt == kFmtINT8)
    return act ? launch_f<kFmtINT8, true>(tw, tx, a, stream) : launch_f<kFmtINT8, false>(tw, tx, a, stream);
  return act ? launch_f<kFmtFP8, true>(tw, tx, a, stream) : launch_f<kFmtFP8, false>(tw, tx, a, stream);
}

cudaError_t read_experts_error(unsigned int* code) {
  return cudaMemcpyFromSymbol(code, g_experts_error, sizeof(unsigned int));
}

cudaError_t clear_experts_error() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_experts_error, &zero, sizeof(unsigned int));
}

}  // namespace qgd
