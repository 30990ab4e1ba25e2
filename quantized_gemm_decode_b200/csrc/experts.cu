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
// The quantizer writes the codes in sorted order, then one persistent kernel
// walks the (expert, token tile, weight tile) tiles, whose number only the device
// knows, from the offsets.  Orientation as in the dense decode kernel (weights in
// the MMA's 128-row M slot, tokens in its N), because an expert's row count is
// ragged: N follows the tile's rows in steps of 16, where M would round every
// expert up to 128.
//
// Few rows per expert: 64- or 128-token tiles, bound by the one pass over the
// weights; (tile, K unit) units are dealt out over all SMs where whole tiles would
// leave too many idle.  Measured on B200, 32 tokens x 8 of 64 experts, 4096 x 1024
// e4m3 weights: 44 us per call (replayed from a graph), of which the weights stream for 40.5 us (6.5
// TB/s) after 5.5 us of quantizer, hand-over and tile search.  Many: 256-token
// tiles of CTA pairs, bound by the MMA, whose operands and the copies that refill
// them share an SM's shared-memory bandwidth: 8192 tokens x 8 of 64 experts, 2048 x
// 4096 int8 gate / up weights: 2.8 PFLOP/s in the GEMM; 472 to 494 us per call in
// short runs (replayed from a graph, box by box), 554 to 569 where calls one behind
// the other bring the GPU to its power limit.
//
// Warp roles: warp 0 issues TMA loads, warp 1 owns TMEM and issues MMAs, the
// groups of four warps behind them drain the accumulator.  Every wait is bounded.
#include <cuda_bf16.h>

#include <atomic>

#include "qgd_internal.h"
#include "quantcore.cuh"
#include "sm100.cuh"

namespace qgd {

// First error code recorded by the kernels of this file on this device.
__device__ unsigned int g_experts_error = 0;

namespace {

__device__ __forceinline__ void record_error(unsigned int code) { atomicCAS(&g_experts_error, 0u, code); }

// ---------------------------------------------------------------------------
// Quantizer: one CTA per sorted row, so that the GEMM reads every tile's rows
// as one box.  (Gathering in the GEMM was slower: four-row tensor gathers cost
// about 80 cycles each, and 16-byte asynchronous copies by four more warps a
// proxy fence per stage; at 8192 tokens, 8 of 64 experts, K = 4096, 2400 and
// 1050 us against 600 for boxes.)  Rows behind the last expert's are left
// alone; a source row outside x reads as zeros.
// ---------------------------------------------------------------------------
template <int kRowThreads, int kVPT, int kQType>
__global__ void __launch_bounds__(kRowThreads)
    experts_quant_kernel(const uint16_t* __restrict__ x, int K, int ldx, int x_rows, const int* __restrict__ order,
                         int div, const int* __restrict__ offsets, int E, int P, uint8_t* __restrict__ q,
                         float* __restrict__ s, unsigned* __restrict__ tickets, int ntickets) {
  __shared__ float red[kRowThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < ntickets; i += kRowThreads) tickets[i] = 0u;
  const int row = blockIdx.x;
  // the offset is looked at last: its load runs beside those of the order and of x
  const int live = offsets ? __ldg(offsets + E) : P;
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
  if (row >= live) return;
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = red[threadIdx.x & (kRowThreads / 32 - 1)];
#pragma unroll
  for (int o = kRowThreads / 64; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  amax = fmaxf(amax, kAmaxFloor);
  const float sc = __fdiv_rn(amax, kQType == 0 ? kE4M3Max : kInt8Max);
  if (threadIdx.x == 0) s[row] = sc;
  const Reciprocals inv = reciprocals(sc);
#pragma unroll
  for (int j = 0; j < kVPT; ++j) {
    const int idx = threadIdx.x + j * kRowThreads;
    if (idx < nvec) qr[idx] = encode8_by_reciprocal<kQType>(v[j], sc, inv);
  }
}

// Many rows that several experts take: each row of x is coded once and the
// codes are copied into sorted order, a warp per row: coding costs about 10
// issue slots a value, so coding k times is bound by the SMs where the copy is
// bound by its stores.
constexpr int kPermuteThreads = 256;

__global__ void __launch_bounds__(kPermuteThreads)
    permute_codes_kernel(const uint4* __restrict__ q0, const float* __restrict__ s0, int x_rows,
                         const int* __restrict__ order, int div, const int* __restrict__ offsets, int E, int P, int nvec,
                         uint4* __restrict__ q, float* __restrict__ s) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kPermuteThreads / 32) + (threadIdx.x >> 5);
  if (row >= P) return;
  const int pair = __ldg(order + row);
  if (row >= __ldg(offsets + E)) return;
  const int src = pair / div;
  const bool have = pair >= 0 && src < x_rows;
  const uint4* from = q0 + static_cast<size_t>(have ? src : 0) * nvec;
  uint4* to = q + static_cast<size_t>(row) * nvec;
  for (int v0 = lane; v0 < nvec; v0 += 8 * 32) {
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v0 + j * 32 < nvec) v[j] = have ? __ldg(from + v0 + j * 32) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v0 + j * 32 < nvec) __stcs(to + v0 + j * 32, v[j]);
  }
  if (lane == 0) s[row] = have ? __ldg(s0 + src) : 0.f;
}

// ---------------------------------------------------------------------------
// Grouped GEMM
// ---------------------------------------------------------------------------
constexpr int kEpiThreads = 128;  // an epilogue group: four warps, one per quarter of the tensor-memory lanes
constexpr int kMaxWarps = 2 + 4 * 4;

struct Ctl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int last_flag;
  int epi_ok[4];
  int scan[kMaxWarps];
};
constexpr uint32_t kCtlBytes = 512;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block too large");

// Shapes of a variant.  kTok: most tokens per tile; kPair: a CTA pair computes
// 256 weight rows, each CTA holding 128 of them and half of the tokens;
// kGroups: epilogue groups, which take a tile's 16-token chunks in turn; kAct: a
// tile's 128 weight rows are 8 gate rows, their 8 up rows, the next 8 gate rows, ...
// Shared memory of one CTA (after 1024-byte alignment): ring of kStages x kKps
// x (128 weight rows + kXRows token rows) x 128 bytes; per epilogue group an
// output staging buffer of 16 tokens x 128 bf16 (with the activation 16 x 64) and
// the token scales [2][kTok]; control block; running tile counts and first rows of the
// experts.
template <int kTok, int kKps, bool kPair, int kGroups, bool kAct>
struct Layout {
  static constexpr int kThreads = 64 + kGroups * kEpiThreads;
  static constexpr uint32_t kOut = kAct ? 16 * 128 : 16 * 256;
  static constexpr uint32_t kGroupBytes = kOut + 2 * kTok * 4;
  static constexpr int kXRows = kPair ? kTok / 2 : kTok;
  static constexpr int kRound = kPair ? 32 : 16;  // tokens of a tile are rounded up to this
  // token rows per copy: few for short tiles, all for long ones (a copy costs
  // the copy engine about 150 cycles whatever its size, a K slice of a full
  // pair tile about 750 cycles of MMA)
  static constexpr int kBoxShort = kXRows / 4, kBoxLong = kXRows;
  static constexpr uint32_t kW = kSwapTileN * kTileK;
  static constexpr uint32_t kX = kXRows * kTileK;
  static constexpr uint32_t kStage = kKps * (kW + kX);
  static constexpr uint32_t kTail = kGroups * kGroupBytes + kCtlBytes + 2 * (kMaxExperts + 1) * 4;
  static constexpr int kStages0 = static_cast<int>((kSmemBudget - 1024 - kTail) / kStage);
  static constexpr int kStages = kStages0 > kMaxStages ? kMaxStages : kStages0;
  static constexpr size_t kBytes = 1024 + static_cast<size_t>(kStages) * kStage + kTail;
};

// First sorted row of expert e.
__device__ __forceinline__ int offset_of(const ExpertArgs& a, int e) {
  const int v = __ldg(a.offsets + e);
  return v < 0 ? 0 : (v > a.P ? a.P : v);
}

// A worker's (CTA's or CTA pair's) work as a sequence of segments (tile, K
// units [k0, k1)).  split: all (tile, K unit) units dealt out in contiguous
// ranges, one per worker, equal up to a unit, so that every SM streams the same
// share of the weights; else whole tiles, round-robin.  (32-bit arithmetic: a
// 64-bit division or two here cost each call about half a microsecond.)
struct Deal {
  int total, nku, G;
  bool split;
  int q, r;  // split: workers before r take q + 1 units, the others q
  __device__ __forceinline__ Deal(int total_, int nku_, int G_, bool split_)
      : total(total_), nku(nku_), G(G_), split(split_), q(0), r(0) {
    if (split) {
      q = total * nku / G;
      r = total * nku - q * G;
    }
  }
  __device__ __forceinline__ int begin(int worker) const { return worker * q + min(worker, r); }
  __device__ __forceinline__ int owner(int u) const {
    const int wide = r * (q + 1);
    return u < wide ? u / (q + 1) : r + (u - wide) / q;
  }
};

// A segment of a tile: the tile's number, expert, first sorted row, row count and
// weight tile, and the K units [k0, k1).
struct Tile {
  int w, e, row0, n, nt, k0, k1;
};

// A worker's segments in order.  Tiles are numbered weight tiles fastest, then an
// expert's token tiles, then the experts (pre[e]: token tiles of the experts
// before e; off[e]: first sorted row); an expert's rows are dealt to its token
// tiles evenly, in multiples of kRound.  The walk goes on from the expert it is
// at: a search and three divisions per tile took the MMA thread 2000 cycles
// between tiles, as much as four K slices' work.
template <int kRound>
struct Walk {
  const int *pre, *off;
  int n_tiles, nku, step, step_g, step_nt;
  bool split;
  int w, k, left;  // next segment's tile and first unit; split: units left, else tiles to go
  int g, nt;       // the tile's token tile (over all experts) and weight tile
  int e, lo, hi;   // its expert and that one's token tiles [lo, hi)
  int first, cnt, per;
  __device__ __forceinline__ Walk(const Deal& d, const int* pre_, const int* off_, int E, int n_tiles_, int worker)
      : pre(pre_), off(off_), n_tiles(n_tiles_), nku(d.nku), step(d.G), split(d.split) {
    if (split) {
      const int u = d.begin(worker);
      w = u / nku;
      k = u - w * nku;
      left = d.q + (worker < d.r ? 1 : 0);
      step = 1;
    } else {
      w = worker;
      k = 0;
      left = d.total - worker;
    }
    step_g = step / n_tiles;
    step_nt = step - step_g * n_tiles;
    g = w / n_tiles;
    nt = w - g * n_tiles;
    int a = 0, b = E;  // pre[a] <= g < pre[b], where there is such a tile
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (pre[mid] <= g) a = mid;
      else b = mid;
    }
    if (left > 0) enter(a);
  }
  __device__ __forceinline__ void enter(int expert) {
    e = expert;
    lo = pre[e];
    hi = pre[e + 1];
    first = off[e];
    cnt = off[e + 1] - first;
    const int tiles = hi - lo;
    per = tiles > 0 ? ((cnt + tiles - 1) / tiles + kRound - 1) & ~(kRound - 1) : 0;
  }
  __device__ __forceinline__ bool next(Tile& t) {
    if (left <= 0) return false;
    if (g >= hi) {
      int x = e + 1;
      while (pre[x + 1] <= g) ++x;
      enter(x);
    }
    const int at = (g - lo) * per;
    t.w = w;
    t.e = e;
    t.row0 = first + at;
    t.n = min(per, cnt - at);
    t.nt = nt;
    t.k0 = k;
    t.k1 = nku;
    if (split) {
      if (left < nku - k) t.k1 = k + left;
      left -= t.k1 - t.k0;
      k = 0;
    } else {
      left -= step;
    }
    w += step;
    g += step_g;
    nt += step_nt;
    if (nt >= n_tiles) {
      nt -= n_tiles;
      ++g;
    }
    return true;
  }
};

// Barriers with warps converged first: the instructions behind them are
// warp-wide, and a lane that comes out of a role's branch later than the rest
// of its warp would arrive on its own.
__device__ __forceinline__ void epi_sync(int group) {
  __syncwarp();
  named_bar_sync(1 + group, kEpiThreads);
}

template <int kGroups>
__device__ __forceinline__ void all_groups_sync() {
  __syncwarp();
  named_bar_sync(1 + 4, kGroups * kEpiThreads);
}

__device__ __forceinline__ void pair_sync() {
  __syncwarp();
  cluster_sync_all();
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Tensor copies completing on the mbarrier at shared address `bar` (of a pair:
// the leader's).
template <bool kPair>
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

// Gate and up rows, 8 and 8: dimensions K, row of 8, gate / up, block of 8 rows, expert.
template <bool kPair>
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int block, int e,
                                            uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(0), "r"(block), "r"(e), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(0), "r"(block), "r"(e), "l"(policy)
        : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, uint32_t cluster_bar,
                                              int x, int y, uint64_t policy) {
  if constexpr (kPair) tma_load_2d_pair(dst, map, cluster_bar, x, y, policy);
  else tma_load_2d(dst, map, bar, x, y, policy);
}

// g / (1 + exp(-g)).  The fast exponential is within (2 + 1.2 |g|) 2^-23, relative,
// and the quotient within 2^-22: far below bf16's half step.  exp(-g) leaves fp32's
// range at -88.7, and the fast quotient gives 0 for divisors above 2^126; below -80
// the divisor is exp(-g) to the last bit, so the result is g * exp(g), which goes
// down to fp32's last subnormal (an infinite gate gives 0 * inf = NaN, as the formula does).
__device__ __forceinline__ float silu(float g) {
  const bool low = g < -80.f;
  const float e = __expf(low ? g : -g);
  return low ? g * e : __fdividef(g, 1.f + e);
}

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

// A 16-token chunk of the accumulator as 8 x 8 fragments: r[8h + 4g + 2x + i] is
// lane 16h + 8x + l / 4 of the warp's 32, token 8g + 2(l % 4) + i (l: the thread's
// lane).  So a gate row and its up row, 8 lanes on, meet in one thread, and two
// tokens of a channel pack into the register that a transposing matrix store takes.
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8m + j gives the address
// of row j of matrix m.
__device__ __forceinline__ void store_matrices_t(uint32_t addr, const uint32_t (&m)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(m[0]),
               "r"(m[1]), "r"(m[2]), "r"(m[3])
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A chunk's accumulators (see load_chunk) finished and stored: tokens c0 .. c0 + 15
// of the tile.  sw: scales of the thread's rows, sw[2h + x].  The group's warps
// write [token][channel] to shared memory, 8 channels of a token at a time, the
// 16-byte vectors of a token swapped by its low three bits (no bank conflicts), and
// store y from there in runs of 128 or 256 bytes.  The operands' stream through
// shared memory bounds the large tiles, so the epilogue has to use little of it:
// with a row per thread, gate and up swapped through shared memory and 2-byte
// stores it took three times as many accesses.
template <int kFmt, bool kAct>
__device__ __forceinline__ void finish16(const ExpertArgs& a, const Tile& t, const uint32_t (&r)[16], int c0,
                                         const float (&sw)[4], const float* sxs, uint8_t* out, int group) {
  const int et = (threadIdx.x - 64) & (kEpiThreads - 1), lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
  constexpr int kCols = kAct ? 64 : 128;
  constexpr int kVecs = kCols / 8;  // 16-byte vectors per token
  uint32_t m[kAct ? 1 : 2][4];
  float v[16];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float2 sx = *reinterpret_cast<const float2*>(sxs + c0 + 8 * g + 2 * (lane & 3));
#pragma unroll
    for (int hx = 0; hx < 4; ++hx) {
      const int at = 8 * (hx >> 1) + 4 * g + 2 * (hx & 1);
      v[at] = (acc_value<kFmt>(r[at]) * sx.x) * sw[hx];
      v[at + 1] = (acc_value<kFmt>(r[at + 1]) * sx.y) * sw[hx];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 8 * h + 4 * g;
      if constexpr (kAct) {
        m[0][2 * h + g] = pack_bf16(silu(v[at]) * v[at + 2], silu(v[at + 1]) * v[at + 3]);
      } else {
        m[h][g] = pack_bf16(v[at], v[at + 1]);
        m[h][2 + g] = pack_bf16(v[at + 2], v[at + 3]);
      }
    }
  }
  // this lane's row: token 8 (lane / 8 % 2) + lane % 8, vector by q, h or x (lane / 16) and the store
  const int tok = lane & 15;
  const uint32_t row = smem_u32(out) + tok * (kCols * 2);
  epi_sync(group);  // the chunk before has left the buffer
  if constexpr (kAct) {
    store_matrices_t(row + (((q * 2 + (lane >> 4)) ^ (tok & 7)) << 4), m[0]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) store_matrices_t(row + (((q * 4 + h * 2 + (lane >> 4)) ^ (tok & 7)) << 4), m[h]);
  }
  epi_sync(group);
#pragma unroll
  for (int p = 0; p < 16 * kVecs / kEpiThreads; ++p) {
    const int idx = p * kEpiThreads + et;
    const int tk = idx / kVecs, vec = idx - tk * kVecs;
    const int col = t.nt * kCols + vec * 8;
    if (c0 + tk < t.n && col < a.N)
      *reinterpret_cast<uint4*>(a.y + static_cast<size_t>(t.row0 + c0 + tk) * a.N + col) =
          *reinterpret_cast<const uint4*>(out + tk * (kCols * 2) + ((vec ^ (tk & 7)) << 4));
  }
}

template <int kFmt, int kTok, int kKps, bool kSplit, bool kPair, int kGroups, bool kAct>
__global__ void __launch_bounds__(Layout<kTok, kKps, kPair, kGroups, kAct>::kThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                   const __grid_constant__ CUtensorMap tx_short, const ExpertArgs a) {
  using L = Layout<kTok, kKps, kPair, kGroups, kAct>;
  constexpr int kThreads = L::kThreads;
  static_assert(!(kSplit && kPair), "pairs take whole tiles");
  constexpr bool kInt = (kFmt == kFmtINT8);
  constexpr uint32_t kCols = 2 * kTok;  // TMEM: double-buffered accumulator
  constexpr int stages = L::kStages;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  uint8_t* w_ring = base;
  uint8_t* x_ring = base + stages * kKps * L::kW;
  uint8_t* groups = base + stages * L::kStage;
  Ctl* ctl = reinterpret_cast<Ctl*>(groups + kGroups * L::kGroupBytes);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(ctl) + kCtlBytes);  // [E + 1]
  int* off = pre + kMaxExperts + 1;                                               // [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkt = (a.K + kTileK - 1) / kTileK;
  const int nku = (nkt + kKps - 1) / kKps;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;  // of a pair: 0 leads (issues the MMAs)

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tx_short);
    for (int i = 0; i < stages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], 1);
      mbar_init(&ctl->tempty[i], (kPair ? 2 : 1) * kGroups * (kEpiThreads / 32));
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    ctl->last_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(&ctl->tmem_base, kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&ctl->tmem_base, kCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  griddep_launch_dependents();
  griddep_wait();  // offsets, codes and scales come from the kernels before
  // token tiles of the experts before e, as a running sum in blocks of experts
  int descends = 0;
  {
    int carry = 0;
    if (threadIdx.x == 0) pre[0] = 0;
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
      const int e = e0 + threadIdx.x;
      int v = 0, below = 0;
      if (e < a.E) {
        const int first = offset_of(a, e), cnt = offset_of(a, e + 1) - first;
        off[e] = first;
        if (e == a.E - 1) off[a.E] = first + cnt;
        v = cnt > 0 ? (cnt + kTok - 1) / kTok : 0;
        below = cnt < 0;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      if (lane == 31) ctl->scan[warp] = v;
      descends |= __syncthreads_or(below);
      int before = carry, all = carry;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += ctl->scan[i];
        all += ctl->scan[i];
      }
      if (e < a.E) pre[e + 1] = before + v;
      carry = all;
      __syncthreads();
    }
  }
  if constexpr (kPair) pair_sync();  // both CTAs' barriers and tensor memory exist
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int n_tiles = kPair ? (a.n_tiles + 1) / 2 : a.n_tiles;
  // (no tiles where the offsets do not ascend: ranges could hold rows over and over,
  // more than the host's check of the sizes counts on, and rows behind offsets[E],
  // which the quantizer has not coded)
  const int total = descends ? 0 : pre[a.E] * n_tiles;
  const int U = total * nku;
  const int workers = static_cast<int>(gridDim.x) / (kPair ? 2 : 1);
  // Whole tiles leave workers idle at the end, split ones cost a hand-over (about
  // 3 us: partials, arrival, sum); a K unit of 32 KB takes an SM's share of the
  // bandwidth about 0.75 us: split where idling would be more than kSplitPays units.
  constexpr int kSplitPays = 4;
  const int rounds = (total + workers - 1) / workers;
  const bool split = kSplit && (rounds * nku - kSplitPays) * workers > U;
  const int most = split ? U : total;
  const int G = most < workers ? most : workers;  // workers with work
  const Deal deal(total, nku, G > 0 ? G : 1, split);
  const int me = static_cast<int>(blockIdx.x) / (kPair ? 2 : 1);
  const bool busy = me < G;
  int issued = 0;

  // shared::cluster addresses of the leader's barriers (this CTA's own without a pair)
  const uint32_t full0 = kPair ? mapa_shared(smem_u32(&ctl->full[0]), 0) : smem_u32(&ctl->full[0]);
  const uint32_t partner_abort = kPair ? mapa_shared(smem_u32(&ctl->abort_flag), rank ^ 1u) : 0u;
  auto fail = [&](unsigned int code) {
    record_error(code);
    ctl->abort_flag = 1;
    if constexpr (kPair) st_cluster_u32(partner_abort, 1u);
  };
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&ctl->abort_flag) != 0; };

  if (warp == 0) {
    // ---------------- TMA producer (of a pair: both CTAs, their halves) ----------------
    if (lane == 0 && busy) {
      const uint64_t pol_w = kSplit ? policy_evict_first() : policy_evict_last();
      const uint64_t pol_x = policy_evict_last();
      Walk<L::kRound> walk(deal, pre, off, a.E, n_tiles, me);
      Tile t;
      int i = 0;
      bool stop = false;
      while (!stop && walk.next(t)) {
        const int wt = kPair ? t.nt * 2 + static_cast<int>(rank) : t.nt;  // this CTA's 128 weight rows
        const int all = (t.n + L::kRound - 1) & ~(L::kRound - 1);
        const int mine = kPair ? all / 2 : all;  // token rows in this CTA's shared memory
        const int xrow = t.row0 + static_cast<int>(rank) * mine;
        const bool few = mine <= L::kBoxShort;   // rows past the tile's go unused
        const CUtensorMap* xmap = few ? &tx_short : &tx;
        const uint32_t bytes = L::kW + (few ? L::kBoxShort : L::kBoxLong) * kTileK;
        for (int k = t.k0; k < t.k1; ++k, ++i) {
          const int s = i % stages;
          if (!mbar_wait(&ctl->empty[s], ((i / stages) & 1) ^ 1)) {
            fail(kErrWaitProducer);
            stop = true;
            break;
          }
          if (aborted()) {
            stop = true;
            break;
          }
          const int kt = k * kKps, ns = min(kKps, nkt - kt);
          const uint32_t fb = full0 + static_cast<uint32_t>(s) * 8u;
          // the leader's barrier expects both CTAs' bytes (a copy may land first)
          if (rank == 0) mbar_arrive_expect_tx(&ctl->full[s], (kPair ? 2 : 1) * ns * bytes);
          for (int h = 0; h < ns; ++h) {
            const int x = (kt + h) * kTileK;
            uint8_t* wd = w_ring + (s * kKps + h) * L::kW;
            if constexpr (kAct) tma_load_5d<kPair>(wd, &tw, fb, x, wt * 8, t.e, pol_w);
            else tma_load_3d<kPair>(wd, &tw, fb, x, wt * 128, t.e, pol_w);
            tma_load_rows<kPair>(x_ring + (s * kKps + h) * L::kX, xmap, &ctl->full[s], fb, x, xrow, pol_x);
          }
          issued = i + 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer (of a pair: the leader's) ----------------
    if (lane == 0 && rank == 0 && busy) {
      const uint32_t w_base = smem_u32(w_ring), x_base = smem_u32(x_ring);
      Walk<L::kRound> walk(deal, pre, off, a.E, n_tiles, me);
      Tile t;
      int i = 0, li = 0;
      bool stop = false;
      while (!stop && walk.next(t)) {
        const uint32_t idesc = idesc_mma(kInt ? 2 : 1, kInt ? 1 : 0, (kPair ? 2 : 1) * kSwapTileN,
                                         (t.n + L::kRound - 1) & ~(L::kRound - 1));
        const int b = li & 1;
        if (!mbar_wait(&ctl->tempty[b], ((li >> 1) & 1) ^ 1)) {
          fail(kErrWaitMma);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + b * kTok;
        for (int k = t.k0; k < t.k1; ++k, ++i) {
          const int s = i % stages;
          if (!mbar_wait(&ctl->full[s], (i / stages) & 1)) {
            fail(kErrWaitMma);
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
              const uint32_t acc = (k > t.k0 || h > 0 || kk > 0) ? 1u : 0u;
              if constexpr (kPair) mma_issue_pair<kInt>(d, ad, bd, idesc, acc);
              else mma_issue<kInt>(d, ad, bd, idesc, acc);
            }
          }
          if constexpr (kPair) mma_commit_pair(&ctl->empty[s], 0x3);
          else mma_commit(&ctl->empty[s]);
        }
        if (stop) break;
        if constexpr (kPair) mma_commit_pair(&ctl->tfull[b], 0x3);
        else mma_commit(&ctl->tfull[b]);
        ++li;
      }
    }
    __syncwarp();
  } else if (busy) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, group = (warp - 2) >> 2, et = (threadIdx.x - 64) & (kEpiThreads - 1);
    uint8_t* out = groups + group * L::kGroupBytes;
    float* sx_s = reinterpret_cast<float*>(out + L::kOut);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int lrow = q * 32 + lane;
    const uint32_t tempty0 = kPair ? mapa_shared(smem_u32(&ctl->tempty[0]), 0) : 0u;
    // A tile's token scales and the scale of the row at this thread's lane are loaded while the
    // tile before is finished.
    constexpr int kPerThread = (kTok + kEpiThreads - 1) / kEpiThreads;
    float sx_next[kPerThread], sw_next;
    auto prefetch = [&](const Tile& t) {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const int r = i * kEpiThreads + et;
        sx_next[i] = r < t.n ? __ldg(a.sx + t.row0 + r) : 0.f;
      }
      const int col = kAct ? t.nt * 64 + (lrow >> 4) * 8 + (lane & 7) : t.nt * 128 + lrow;
      const size_t from = kAct ? (static_cast<size_t>(t.e) * 2 + (lane >> 3 & 1)) * a.N : static_cast<size_t>(t.e) * a.N;
      sw_next = col < a.N ? __ldg(a.sw + from + col) : 0.f;  // (0 past the last row)
    };
    Walk<L::kRound> walk(deal, pre, off, a.E, n_tiles, me);
    auto next_tile = [&](Tile& t) {
      if (!walk.next(t)) return false;
      if constexpr (kPair) t.nt = t.nt * 2 + static_cast<int>(rank);
      prefetch(t);
      return true;
    };
    Tile t, coming;
    int li = 0;
    for (bool more = next_tile(t); more; t = coming, ++li) {
      const int b = li & 1;
      float* sxs = sx_s + b * kTok;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (i * kEpiThreads + et < kTok) sxs[i * kEpiThreads + et] = sx_next[i];
      float sw[4];
#pragma unroll
      for (int hx = 0; hx < 4; ++hx) sw[hx] = __shfl_sync(0xffffffffu, sw_next, 8 * hx + (lane >> 2));
      more = next_tile(coming);
      const bool ok = warp_wait(&ctl->tfull[b], (li >> 1) & 1);
      if (!ok && lane == 0) fail(kErrWaitEpilogue);
      if (ok) tc_fence_after();
      // go on or leave: one answer for all that meet at a barrier later (a group's
      // warps; with split tiles all groups)
      const int table = kSplit ? 0 : group;
      if constexpr (kSplit) all_groups_sync<kGroups>();
      else epi_sync(group);
      if (kSplit ? threadIdx.x == 64 : et == 0) ctl->epi_ok[table] = !aborted();
      if constexpr (kSplit) all_groups_sync<kGroups>();
      else epi_sync(group);
      if (!ctl->epi_ok[table]) break;
      const bool whole = !kSplit || !split || (t.k0 == 0 && t.k1 == nku);
      int first = me, ncontrib = 1;
      uint32_t* slot = nullptr;
      if (!whole) {
        first = deal.owner(t.w * nku);
        ncontrib = deal.owner(t.w * nku + nku - 1) - first + 1;
        slot = a.partial + (static_cast<size_t>(me) * 2 + (me == first ? 1 : 0)) * (kSwapTileN * kTok) + lrow;
      }
      const int chunks = (t.n + 15) >> 4;
      auto release = [&]() {  // this warp has read all it needs of the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) mbar_arrive_remote(tempty0 + static_cast<uint32_t>(b) * 8u);
          else mbar_arrive(&ctl->tempty[b]);
        }
      };
      if (group >= chunks) release();
      for (int c = group; c < chunks; c += kGroups) {
        uint32_t r[16];
        __syncwarp();
        load_chunk(taddr + b * kTok + c * 16, r);
        if (c + kGroups >= chunks) release();
        if (whole) {
          finish16<kFmt, kAct>(a, t, r, c * 16, sw, sxs, out, group);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) __stcg(slot + (c * 16 + j) * kSwapTileN, r[j]);
        }
      }
      if (!whole) {
        // the last of the tile's CTAs to arrive adds the partials in CTA order
        all_groups_sync<kGroups>();
        if (threadIdx.x == 64) {
          unsigned old;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.tickets + first) : "memory");
          ctl->last_flag = (old == static_cast<unsigned>(ncontrib - 1));
        }
        all_groups_sync<kGroups>();
        if (ctl->last_flag) {
          for (int c = group; c < chunks; c += kGroups) {
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
            finish16<kFmt, kAct>(a, t, sum, c * 16, sw, sxs, out, group);
          }
        }
      }
    }
  }

  // ---------------- teardown ----------------
  __syncwarp();
  tc_fence_before();
  // one answer for every thread (a partner may set the flag at any time)
  if (__syncthreads_or(ctl->abort_flag != 0)) {
    if (warp == 0 && lane == 0) {
      // the last copies issued into each stage (both CTAs') must land before either CTA exits
      if (rank == 0)
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i) {
          if (!mbar_wait(&ctl->full[i % stages], (i / stages) & 1)) {
            record_error(kErrWaitDrain);
            break;
          }
        }
    }
    if (rank == 0 && warp == 1 && lane == 0) {
      if constexpr (kPair) mma_commit_pair(&ctl->drain, 0x1);
      else mma_commit(&ctl->drain);
      if (!mbar_wait(&ctl->drain, 0)) record_error(kErrWaitDrain);
    }
    __syncthreads();
  }
  if constexpr (kPair) pair_sync();  // neither CTA leaves while its partner may still signal its barriers
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem, kCols);
    else tmem_dealloc(tmem, kCols);
  }
}

constexpr int kManyRows = 1184;  // a wave of 8 CTAs on each of 148 SMs

// rows of x in sorted order (offsets), or all of them in place (no offsets)
template <int kQType>
cudaError_t launch_quant_t(const ExpertArgs& a, const uint16_t* x, int ldx, int x_rows, const int* order, int div,
                           const int* offsets, int rows, uint8_t* q, float* s, cudaStream_t st) {
  const int nvec = a.K / 8;
  const dim3 grid(rows);
  auto go = [&](auto kernel, int threads) {
    return launch_pdl(kernel, grid, dim3(threads), 0, st, x, a.K, ldx, x_rows, order, div, offsets, a.E, rows, q, s,
                      a.tickets, a.ctas);
  };
  // few rows: more threads a row, for latency (one row of 4096: 2.3 against 2.8 us);
  // many: fewer, each with more loads in flight (8192 such rows: 22.3 against 24.4 us)
  if (rows <= kManyRows) {
    if (nvec <= 256) return go(experts_quant_kernel<256, 1, kQType>, 256);
    if (nvec <= 512) return go(experts_quant_kernel<256, 2, kQType>, 256);
    if (nvec <= 1024) return go(experts_quant_kernel<256, 4, kQType>, 256);
    return go(experts_quant_kernel<256, 8, kQType>, 256);
  }
  if (nvec <= 128) return go(experts_quant_kernel<128, 1, kQType>, 128);
  if (nvec <= 256) return go(experts_quant_kernel<128, 2, kQType>, 128);
  if (nvec <= 512) return go(experts_quant_kernel<128, 4, kQType>, 128);
  if (nvec <= 1024) return go(experts_quant_kernel<128, 8, kQType>, 128);
  return go(experts_quant_kernel<128, 16, kQType>, 128);
}

template <int kFmt, int kTok, int kKps, bool kSplit, bool kPair, int kGroups, bool kAct>
cudaError_t launch_t(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx_short, const ExpertArgs& a, cudaStream_t st) {
  using L = Layout<kTok, kKps, kPair, kGroups, kAct>;
  static_assert(L::kStages >= 2 && L::kBytes <= kSmemBudget, "ring does not fit");
  // more than half an SM's shared memory, so that no two of these CTAs, which
  // may take all tensor-memory columns, share an SM
  static_assert(L::kBytes > kSmemPerSM / 2, "two CTAs would fit");
  auto kernel = experts_kernel<kFmt, kTok, kKps, kSplit, kPair, kGroups, kAct>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, L::kBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if constexpr (kPair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
    // no more pairs than fit on the GPU at once: the tiles are dealt out over
    // the grid, so a pair that had to wait for a place would end last
    static std::atomic<int> fit[64];
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int pairs = fit[dev & 63].load(std::memory_order_relaxed);
    cfg.gridDim = dim3(a.ctas & ~1);
    if (pairs == 0) {
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs < 1) {
        (void)cudaGetLastError();
        pairs = a.ctas / 2;
      }
      fit[dev & 63].store(pairs, std::memory_order_relaxed);
    }
    if (a.ctas / 2 > pairs) cfg.gridDim = dim3(2 * pairs);
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  e = cudaLaunchKernelEx(&cfg, kernel, tw, tx, tx_short, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int kFmt, bool kAct>
cudaError_t launch_f(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx_short, const ExpertArgs& a,
                     cudaStream_t st) {
  switch (a.tok) {
    case 64: return launch_t<kFmt, 64, 2, true, false, 2, kAct>(tw, tx, tx_short, a, st);
    case 128: return launch_t<kFmt, 128, 2, true, false, 2, kAct>(tw, tx, tx_short, a, st);
    case 256: return launch_t<kFmt, 256, 2, false, true, 3, kAct>(tw, tx, tx_short, a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int experts_box_rows(int tok, bool few) {
  const int long_rows = tok == 256 ? 128 : tok;  // a pair's CTAs hold half of the tokens each
  return few ? long_rows / 4 : long_rows;
}

cudaError_t launch_experts_quant(int fmt, const ExpertArgs& a, const uint16_t* x, int ldx, int x_rows,
                                 const int* order, int div, uint8_t* q, float* s, uint8_t* q0, float* s0,
                                 cudaStream_t stream) {
  auto quant = [&](const int* ord, const int* offsets, int rows, uint8_t* qd, float* sd) {
    return fmt == kFmtINT8 ? launch_quant_t<1>(a, x, ldx, x_rows, ord, div, offsets, rows, qd, sd, stream)
                           : launch_quant_t<0>(a, x, ldx, x_rows, ord, div, offsets, rows, qd, sd, stream);
  };
  if (!q0) return quant(order, a.offsets, a.P, q, s);
  const cudaError_t e = quant(nullptr, nullptr, x_rows, q0, s0);
  if (e != cudaSuccess) return e;
  constexpr int kWarps = kPermuteThreads / 32;
  return launch_pdl(permute_codes_kernel, dim3((a.P + kWarps - 1) / kWarps), dim3(kPermuteThreads), 0, stream,
                    reinterpret_cast<const uint4*>(q0), static_cast<const float*>(s0), x_rows, order, div, a.offsets,
                    a.E, a.P, a.K / 16, reinterpret_cast<uint4*>(q), s);
}

cudaError_t launch_experts(int fmt, bool act, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx_short, const ExpertArgs& a,
                           cudaStream_t stream) {
  if (fmt == kFmtINT8)
    return act ? launch_f<kFmtINT8, true>(tw, tx, tx_short, a, stream) : launch_f<kFmtINT8, false>(tw, tx, tx_short, a, stream);
  return act ? launch_f<kFmtFP8, true>(tw, tx, tx_short, a, stream) : launch_f<kFmtFP8, false>(tw, tx, tx_short, a, stream);
}

cudaError_t read_experts_error(unsigned int* code) {
  return cudaMemcpyFromSymbol(code, g_experts_error, sizeof(unsigned int));
}

cudaError_t clear_experts_error() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_experts_error, &zero, sizeof(unsigned int));
}

}  // namespace qgd
