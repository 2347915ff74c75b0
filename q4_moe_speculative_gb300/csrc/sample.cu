// sample.cu — a token per row of logits with temperature, top-k, top-p and min-p, drawn with a
// given uniform (arithmetic in include/dsmoe.h).
//
// A row belongs to a cluster of CTAs (up to 8), each of which keeps its part of the logits in shared
// memory, so that they are read from memory once; what the CTAs have to agree on goes through
// distributed shared memory. Without top-k and top-p every weight is taken once, for its warp's sum;
// the draw finds the CTA, the warp, the round of 128 tokens and the lane that it falls to.
//
// Masses are integers: weight exp((l - max) / T) in units of 2^-scale, the scale such that a
// vocabulary's sum fits 63 bits. Sums of integers do not depend on their order, so the borders and
// the draw are the same whatever the grid, and no token is drawn beyond its share by rounding. The
// weights come from fp32 pairs, a table and integers (Row::units2), good to 2^-35: fp64 exponentials,
// which this GPU has few units for, took 1050 us for 64 rows of 129,280 with top-p.
//
// Where the order is cut (the k-th largest logit; the logit at which the mass before it reaches
// top_p), the border is found by counts or masses per bin: first 1024 bins of equal width in
// (max - l) / T, which spread a vocabulary's logits (with 2048 only one CTA fits an SM), then the
// border bin's tokens, which one CTA gathers, by their keys (logits as ordered integers) in 1024
// bins, until a bin is one key. Of the tokens with the border's logit the lowest ids are kept. Up to
// 512 tokens that top-k keeps are finished by one CTA without further exchanges.
//
// Bound by the latency of what the CTAs exchange, one step after another, and by instruction issue while
// weights are taken (about 50 per token with its bin), not by memory. Cycles of a CTA, 64 rows of
// 129,280: top-p 0.9 59,000, of which reading 6500, the largest logit 3300, weights and bins 16,300,
// the border 29,200 (its bin over the cluster, gathering its tokens, one CTA's search), the sums 4000, and
// in the CTA that is drawn 12,500 more; temperature alone 25,000, weights 9600. Weights and bins
// are 23% to 44% over all settings and sizes measured.
// Measured, logits normal with twice unit deviation, in us: 64 rows of 129,280 in fp32 (5 at the copy
// rate) with temperature alone 31, top-k 50 32, top-p 0.9 69, and with min-p 0.02 54; 200 rows of
// 32,003 in bf16 25; one row of 129,280 11, 13 with top-k 50, 28 with top-p.
#include <cooperative_groups.h>

#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace dsmoe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr float kReach = 46.f;       // log2: a lighter token has the weight 0
constexpr float kBinsPerLog2 = kBins / kReach;
constexpr float kNegInf = -INFINITY;
constexpr int kRoots = 1024, kRootBits = 10;
constexpr float kMagic = 12582912.f;   // 1.5 x 2^23: added, it leaves an integer in the lowest bits
constexpr int kMagicBits = 0x4B400000;
constexpr int kPad = 4 * kThreads;   // tokens without weight behind a CTA's last one
constexpr int kFew = 512;           // kept tokens that one CTA finishes alone
constexpr int kGathered = 2048;      // tokens of a border's bin that one CTA sorts out

struct SampleArgs {
  SampleProblem p;
  int chunk;        // tokens per CTA, a multiple of 8
  int scale;        // log2 of the weight 1
  unsigned long long coarse[32], fine[32];   // 2^(j / 32) and 2^(j / 1024) in units of 2^-63
};

struct Shared {
  union {
    struct {
      unsigned lo[kBins], hi[kBins];       // sums of the bins, in two words
    };
    struct {                               // rank 0, when few tokens are kept:
      unsigned long long units[kFew];      // weights in falling order
      int ids[kFew];                       // of the tokens in keys
    };
  };
  unsigned long long upto[kBins];          // of this CTA's slice of the bins, over the cluster
  unsigned keys[kGathered];                // rank 0: of the tokens in the border's bin
  int list[kThreads];                      // this CTA's tokens there
  unsigned long long slice[kMaxCluster];   // totals of the slices
  unsigned long long mass[kMaxCluster];    // of the CTAs: mass above the border
  unsigned long long ties[kMaxCluster];    // and tokens at it
  unsigned long long warp_mass[kWarps];
  unsigned long long warp_ties[kWarps];
  unsigned long long root[kRoots];         // 2^(j / kRoots) in units of 2^-63
  unsigned long long above;                // a border found: what is above its bin
  unsigned long long border_ties;
  unsigned border_key;
  float top[kMaxCluster];
  float warp_top[kWarps];
  double less;                             // T log(min_p)
  float least;
  int bin, listed, gathered;
  unsigned long long inside;               // with a border found: what is in its bin and above
  unsigned sorted[kFew];                   // and with units: their keys in falling order
  unsigned low[kWarps], high[kWarps];
};

// Logits as integers in the same order (NaN never gets here).
__device__ __forceinline__ unsigned key_of(float l) {
  const unsigned b = __float_as_uint(l);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(unsigned k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// What a row's weights need.
struct Row {
  float top, per_log2, per_log2_low;     // the largest logit; log2(e) / T, in two parts
  int scale;
  const unsigned long long* root;        // 2^(j / kRoots) in units of 2^-63
  // (max - l) / T in log2: never rises with l; NaN or beyond kReach: no weight
  __device__ __forceinline__ float reach(float l) const {
    return __fmul_rn(__fsub_rn(top, l), per_log2);
  }
  static __device__ __forceinline__ int bin_of(float reach) {
    return min(kBins - 1, __float_as_int(__fmaf_rn(reach, kBinsPerLog2, kMagic)) - kMagicBits);
  }
  // The weights of two logits: 2^s, s = (l - top) log2(e) / T <= 0 as a pair of fp32 values (the
  // difference and the product with their rounding errors), off by 2^-41. With k = 1024 s rounded,
  // s = k / 1024 + r, |r| <= 1 / 2048: a root from the table, shifted, times e^y, y = r log(2), |y| <=
  // 2^-11.5. e^y - 1 = y + y^2 / 2 + y^3 / 6, the next term being 2^-50, is an integer f in units of
  // 2^-37. It is formed in fp32, whose rounding at its size, 2^-36, is the largest error; with the
  // root's upper part (below) and f's own rounding a weight is off by 2^-35 relative.
  // (where[]: the reach of each, negative; beyond kReach the weight is 0)
  __device__ __forceinline__ void units2(float l0, float l1, unsigned long long* u0,
                                         unsigned long long* u1, float2* where) const {
    constexpr float kLn2 = 0.693147182f, kBeyond = -kReach - 1.5f;
    const f2 minus = pair(-1.f, -1.f), magic = pair(kMagic, kMagic), unmagic = pair(-kMagic, -kMagic);
    const f2 l = pair(l0, l1), m_top = pair(-top, -top);
    const f2 n = add2(l, m_top), bb = fma2(l, minus, n);     // n + e = l - top
    const f2 e = add2(fma2(fma2(bb, minus, n), minus, l), fma2(bb, minus, m_top));
    const f2 c = pair(per_log2, per_log2), cl = pair(per_log2_low, per_log2_low);
    const f2 t = mul2(n, c);
    const f2 te = fma2(e, c, fma2(n, cl, fma2(n, c, mul2(n, pair(-per_log2, -per_log2)))));
    const float2 t2 = parts(t);
    // (what is far below, and NaN, to where the shift leaves nothing of any f)
    const f2 near = pair(t2.x > -kReach ? t2.x : kBeyond, t2.y > -kReach ? t2.y : kBeyond);
    const f2 km = fma2(near, pair(1.f * kRoots, 1.f * kRoots), magic);
    const f2 r = fma2(add2(km, unmagic), pair(-1.f / kRoots, -1.f / kRoots), near);
    const f2 y = fma2(te, pair(kLn2, kLn2), mul2(r, pair(kLn2, kLn2)));
    const f2 q = fma2(mul2(y, y), fma2(y, pair(0x1p37f / 6, 0x1p37f / 6), pair(0x1p36f, 0x1p36f)),
                      mul2(te, pair(kLn2 * 0x1p37f, kLn2 * 0x1p37f)));
    const float2 f = parts(fma2(r, pair(kLn2 * 0x1p37f, kLn2 * 0x1p37f), q)), k2 = parts(km);
    *u0 = compose(__float_as_int(k2.x), __float2int_rn(f.x));
    *u1 = compose(__float_as_int(k2.y), __float2int_rn(f.y));
    *where = t2;
  }
  __device__ __forceinline__ unsigned long long units(float l) const {
    unsigned long long u, v;
    float2 where;
    units2(l, l, &u, &v, &where);
    return u;
  }
  // A logit's weight over a total of units, rounded to fp32 (within 2^-10 of half a step): the weight
  // before it is shifted, and the total, as fp32 pairs; the quotient and its remainder's.
  __device__ __forceinline__ float share(float l, unsigned long long total) const {
    const float t = __fmul_rn(__fsub_rn(l, top), per_log2);
    const int k = __float_as_int(__fmaf_rn(t, 1.f * kRoots, kMagic)) - kMagicBits;
    Row wide = *this;
    wide.scale = 45 - (k >> kRootBits);   // (the root is shifted by 18)
    const unsigned long long w = wide.units(l);
    auto high = [](unsigned long long x) { return __ull2float_rn(x); };
    auto low = [](unsigned long long x, float h) {
      return __ll2float_rn((long long)(x - __float2ull_rn(h)));
    };
    const float wh = high(w), wl = low(w, wh), th = high(total), tl = low(total, th);
    const float q = __fdiv_rn(wh, th);
    const float r = __fadd_rn(__fmaf_rn(-q, th, wh), __fmaf_rn(-q, tl, wl));
    return scalbnf(__fadd_rn(q, __fdiv_rn(r, th)), scale - wide.scale);
  }
  // Root k mod 1024 times 1 + f 2^-37, shifted by k / 1024 (k behind the magic number's bits, whose
  // lowest ten are 0). The product takes the root's upper 27 bits: off by 2^-26 of f.
  __device__ __forceinline__ unsigned long long compose(int k_bits, int f) const {
    const unsigned long long z = root[k_bits & (kRoots - 1)];
    unsigned long long w = z + (unsigned long long)((long long)f * (int)(z >> 37));
    const int shift = 62 + (kMagicBits >> kRootBits) - scale - (k_bits >> kRootBits);
    asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(w), "r"(shift));   // (64 and more: 0)
    return (w + 1) >> 1;
  }
};

// Where the order is cut: tokens with a larger key are kept, and `ties` of those with this one.
struct Border {
  unsigned key;
  unsigned long long ties;
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long warp_upto(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// Inclusive sums over the CTA's threads; `sums`: a word per warp.
__device__ __forceinline__ unsigned long long block_upto(unsigned long long v,
                                                         unsigned long long* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_upto(v, lane);
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps - 1; ++w) v += w < warp ? sums[w] : 0ull;
  return v;
}

// The smallest integer not below total * p, 0 < p < 1, total < 2^63.
__device__ __forceinline__ unsigned long long share_of(unsigned long long total, float p) {
  const int bits = __float_as_int(p), exponent = bits >> 23;
  const unsigned long long m = (bits & 0x7FFFFF) | (exponent ? 0x800000 : 0);
  const unsigned long long lo = total * m, hi = __umul64hi(total, m);
  const int s = 150 - max(exponent, 1);   // of m, 24 .. 149
  if (s >= 128) return 1ull;              // (total is not 0, hi below 2^23)
  if (s >= 64) {
    const unsigned long long whole = s == 64 ? hi : hi >> (s - 64);
    return whole + ((s > 64 && (hi & ((1ull << (s - 64)) - 1))) || lo ? 1 : 0);
  }
  return (hi << (64 - s) | lo >> s) + (lo & ((1ull << s) - 1) ? 1 : 0);
}
// The smallest q with q u >= x, for q below 2^25 (the estimate is off by less than 32).
__device__ __forceinline__ unsigned long long ceil_div(unsigned long long x, unsigned long long u) {
  unsigned long long q = (unsigned long long)__fdividef((float)x, (float)u);   // off by a few
  for (int i = 0; i < 32 && q * u < x; ++i) ++q;
  for (int i = 0; i < 32 && q && (q - 1) * u >= x; ++i) --q;
  return q;
}
// Sorts m <= kFew different values in shared memory, the largest first. All threads of the CTA together.
// Up to 128 by counting, a warp for each value in turn, what is larger; above bitonic, with zeros
// behind them (a warp's 32 pairs are among 64 neighbours where they are 32 or less apart). Top-k of
// 50, one row: 14.3 us by counting, 16.8 bitonic; of 200 26.7 and 20.7; of 500 81 and 28.
__device__ __forceinline__ void sort_down(unsigned long long* v, int m, unsigned long long* counted) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  int n = 2;
  while (n < m) n *= 2;
  if (t >= m && t < n) v[t] = 0ull;
  __syncthreads();
  if (m <= 128) {
    unsigned long long mine[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) mine[e] = 32 * e + lane < m ? v[32 * e + lane] : 0ull;
    for (int i = warp; i < m; i += kWarps) {
      const unsigned long long x = v[i];
      int larger = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) larger += __popc(__ballot_sync(0xffffffffu, mine[e] > x));
      if (lane == 0) counted[larger] = x;
    }
    __syncthreads();
    if (t < m) v[t] = counted[t];
    __syncthreads();
    return;
  }
  for (int size = 2; size <= n; size *= 2) {
    for (int apart = size / 2; apart > 0; apart /= 2) {
      if (t < n / 2) {
        const int i = 2 * t - (t & (apart - 1)), j = i + apart;
        const unsigned long long x = v[i], y = v[j];
        if ((x < y) == ((i & size) == 0)) v[i] = y, v[j] = x;
      }
      if (apart > 32 || (apart == 1 && size > 32)) __syncthreads();
      else __syncwarp();
    }
  }
  __syncthreads();
}
// Adds u to a bin's sum in two words.
__device__ __forceinline__ void bin_add(Shared& sh, int at, unsigned long long u) {
  const unsigned add = (unsigned)u, old = atomicAdd(&sh.lo[at], add);
  const unsigned up = (unsigned)(u >> 32) + (old + add < old ? 1u : 0u);
  if (up) atomicAdd(&sh.hi[at], up);
}

// The two halves of a cluster barrier, here to show that every CTA of the cluster has started: before
// that none may access another's shared memory.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

template <bool kBf16, bool kStaged>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) float stage_mem[];
  __shared__ Shared sh;
  using Raw = typename std::conditional<kBf16, uint16_t, float>::type;
  const SampleProblem& p = a.p;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cluster_arrive();   // (waited for behind the logits' loads)
  const int v0 = min(p.V, rank * a.chunk), n = min(p.V, v0 + a.chunk) - v0;
  for (int i = tid; i < kRoots; i += kThreads) {
    const unsigned long long c = a.coarse[i >> 5], f = a.fine[i & 31];
    sh.root[i] = __umul64hi(c, f) << 1 | c * f >> 63;
  }
  pdl_wait();
  // ------------------------------------------------------------------ the row's settings
  float T = p.temperatures ? p.temperatures[b] : p.temperature;
  int k = p.top_ks ? p.top_ks[b] : p.top_k;
  const float top_p = p.top_ps ? p.top_ps[b] : p.top_p;
  const float min_p = p.min_ps ? p.min_ps[b] : p.min_p;
  const double u = p.u[b];
  if (!(T > 0x1p-64f)) T = 1.f, k = 1;
  // log2(e) / T as a pair: quotient and remainder
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;
  const float per_log2 = __fdiv_rn(kLog2e, T);
  const float per_log2_low =
      T < INFINITY ? __fdiv_rn(__fadd_rn(__fmaf_rn(-per_log2, T, kLog2e), kLog2eLow), T) : 0.f;
  if (tid == kThreads - 1)   // (fp64: one thread, beside the loads)
    sh.less = min_p > 0.f && min_p < 1.f ? (double)T * log((double)min_p) : 0.0;
  const Raw* const from = static_cast<const Raw*>(p.logits) + (int64_t)b * p.stride + v0;
  auto widen = [](Raw x) {   // (NaN is never drawn, and -0 is 0)
    float l;
    if constexpr (kBf16) l = bf16_bits_to_f32(x);
    else l = x;
    return l == l ? __fadd_rn(l, 0.f) : kNegInf;
  };
  // ------------------------------------------------------------------ the largest logit
  // (vectors of 16 bytes between a head and a tail of single values; places in shared memory are
  // shifted so that they are vectors there as well)
  constexpr int kVec = 16 / sizeof(Raw);
  const int skew = (int)(reinterpret_cast<uintptr_t>(from) / sizeof(Raw)) & (kVec - 1);
  float* const stage = stage_mem + skew;
  float top = kNegInf;
  if constexpr (kStaged) {
    const int head = min(n, (kVec - skew) & (kVec - 1)), vectors = (n - head) / kVec;
    auto single = [&](int i) {
      const float l = widen(from[i]);
      stage[i] = l;
      top = fmaxf(top, l);
    };
    if (tid < head) single(tid);
    const int tail = head + vectors * kVec;
    if (tid < n - tail) single(tail + tid);
    const uint4* const vec = reinterpret_cast<const uint4*>(from + head);
    float4* const to = reinterpret_cast<float4*>(stage + head);
    constexpr int kAt = 4;
    for (int i0 = tid; i0 < vectors; i0 += kAt * kThreads) {
      uint4 x[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j)
        if (i0 + j * kThreads < vectors) x[j] = __ldcs(vec + i0 + j * kThreads);
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int i = i0 + j * kThreads;
        if (i >= vectors) break;
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        float l[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          if constexpr (kBf16) l[e] = widen((uint16_t)(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu));
          else l[e] = widen(__uint_as_float(w[e]));
          top = fmaxf(top, l[e]);
        }
#pragma unroll
        for (int e = 0; e < kVec; e += 4)
          to[i * (kVec / 4) + e / 4] = make_float4(l[e], l[e + 1], l[e + 2], l[e + 3]);
      }
    }
  } else {
    for (int i = tid; i < n; i += kThreads) top = fmaxf(top, widen(from[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.warp_top[w]);
  cluster_wait();
  if (tid < C) *cluster.map_shared_rank(&sh.top[rank], tid) = top;
  cluster.sync();
  for (int c = 0; c < C; ++c) top = fmaxf(top, sh.top[c]);
  if (top == kNegInf) {   // (the same for the whole cluster)
    if (rank == 0 && tid == 0) {
      p.out[b] = -1;
      if (p.prob) p.prob[b] = 0.f;
    }
    return;
  }
  const bool endless = top == INFINITY;   // only the infinite ones count, all alike
  if (endless) {
    top = 0.f;
    if (kStaged)
      for (int i = tid; i < n; i += kThreads) stage[i] = stage[i] == INFINITY ? 0.f : kNegInf;
  }
  if (kStaged)   // tokens past the CTA's last one have no weight
    for (int i = n + tid; i < n + kPad; i += kThreads) stage[i] = kNegInf;
  auto logit = [&](int i) {   // (i < n + kPad)
    if constexpr (kStaged) return stage[i];
    if (i >= n) return kNegInf;
    const float l = widen(from[i]);
    return endless ? (l == INFINITY ? 0.f : kNegInf) : fminf(l, top);   // (read anew: never above)
  };
  Row row;
  row.top = top;
  row.per_log2 = per_log2;
  row.per_log2_low = per_log2_low;
  row.scale = a.scale;
  row.root = sh.root;
  if (tid == 0) {   // the smallest logit that min-p leaves
    float least = kNegInf;
    if (min_p > 0.f) {
      const double less = sh.less;
      auto enough = [&](float l) { return (double)l - (double)top >= less; };
      // its key: not below `lo`, at most `hi`; mostly the first guess, else in growing steps, since
      // near 0 more logits than there is time for can have one difference in fp64
      const unsigned first = key_of(kNegInf), last = key_of(top);
      unsigned hi = key_of(fminf(top, __double2float_ru((double)top + less))), lo = hi, step = 1;
      if (enough(from_key(hi))) {
        while (hi > first) {
          lo = hi - first > step ? hi - step : first;
          if (!enough(from_key(lo))) break;
          hi = lo;
          step *= 2;
        }
      } else {
        do {
          lo = hi;
          hi = last - hi > step ? hi + step : last;
          step *= 2;
        } while (hi < last && !enough(from_key(hi)));
      }
      while (hi > lo + 1) {   // lo is not enough
        const unsigned middle = lo + (hi - lo) / 2;
        if (enough(from_key(middle))) hi = middle;
        else lo = middle;
      }
      least = from_key(hi);
    }
    sh.least = least;
  }
  __syncthreads();
  const float least = sh.least;
  const unsigned least_key = key_of(least);
  // Calls f(place, logit) for this thread's tokens whose reach passes the test, few of all.
  auto scan = [&](auto&& test, auto&& f) {
    for (int i = tid; i < n; i += 4 * kThreads) {
      float l[4];
      unsigned pass = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[e] = logit(i + e * kThreads);
        pass |= test(row.reach(l[e])) ? 1u << e : 0u;
      }
      if (!pass) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (pass >> e & 1u) f(i + e * kThreads, l[e]);
    }
  };
  // Among the tokens that each(f) gives to f, keys low .. high: the key at which what is above, with
  // `above` beside them, reaches target. all: every CTA of the cluster has some of the tokens, and
  // finds the same; else the CTA that calls has them.
  auto find = [&](bool masses, unsigned long long target, unsigned long long above, unsigned low,
                  unsigned high, const Border& limit, bool all, auto&& each) {
    constexpr int kPer = kBins / kThreads;
    for (;;) {
      int shift = 0;
      while ((high - low) >> shift >= kBins) ++shift;
      for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0u;
      __syncthreads();
      auto place = [&](unsigned key) { return (int)((high - key) >> shift); };
      each([&](unsigned key) {
        if (key > high || key < low) return;
        if (masses) bin_add(sh, place(key), row.units(from_key(key)));
        else atomicAdd(&sh.lo[place(key)], 1u);
      });
      if (rank == 0 && tid == 0 && limit.key && limit.key <= high && limit.key >= low)
        bin_add(sh, place(limit.key), (masses ? row.units(from_key(limit.key)) : 1ull) * limit.ties);
      if (all) {
        cluster.sync();
        for (int i = tid; i < kBins; i += kThreads) {
          unsigned long long v = 0;
          for (int c = 0; c < C; ++c)
            v += ((unsigned long long)cluster.map_shared_rank(sh.hi, c)[i] << 32) +
                 cluster.map_shared_rank(sh.lo, c)[i];
          sh.upto[i] = v;
        }
        cluster.sync();
      } else {
        __syncthreads();
      }
      unsigned long long v[kPer], sum = 0;   // of neighbouring bins
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int i = tid * kPer + e;
        v[e] = all ? sh.upto[i] : ((unsigned long long)sh.hi[i] << 32) + sh.lo[i];
        sum += v[e];
      }
      unsigned long long lower = above + block_upto(sum, sh.warp_mass) - sum;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (lower < target && lower + v[e] >= target) {   // (one of them)
          sh.bin = tid * kPer + e;
          sh.above = lower;
        }
        lower += v[e];
      }
      __syncthreads();
      above = sh.above;
      high -= (unsigned)sh.bin << shift;
      const unsigned span = (1u << shift) - 1;
      low = high - low > span ? high - span : low;
      if (high == low) {
        const unsigned long long u = masses ? row.units(from_key(high)) : 1ull;
        unsigned long long ties = ceil_div(target - above, u);
        if (high == limit.key && ties > limit.ties) ties = limit.ties;
        return Border{high, ties};
      }
      __syncthreads();   // (sh.bin and the bins may be overwritten)
    }
  };
  // Sums over the CTA's threads, for the last one.
  auto sum_up = [&](unsigned long long mass, unsigned long long ties, unsigned long long* own,
                    unsigned long long* own_ties) {
    mass = warp_sum(mass);
    ties = warp_sum(ties);
    __syncthreads();
    if (lane == 0) sh.warp_mass[warp] = mass, sh.warp_ties[warp] = ties;
    __syncthreads();
    if (warp < kWarps - 1) return;
    *own = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0ull);
    *own_ties = warp_sum(lane < kWarps ? sh.warp_ties[lane] : 0ull);
  };
  // The border at which, from above, the count reaches `target`, or the mass top_p of what `limit`
  // keeps; key 0 where there is not as much, or where min-p cuts before. *own: this CTA's mass above
  // the border and its tokens at it, if *weighed. All threads of the cluster together.
  auto cut = [&](bool masses, unsigned long long target, const Border& limit, bool* weighed,
                 unsigned long long* own, unsigned long long* own_ties) {
    *weighed = false;
    for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0u;
    if (tid == 0) sh.listed = sh.gathered = 0;
    __syncthreads();
    if (!masses) {
      for (int i = tid; i < n; i += 4 * kThreads) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = row.reach(logit(i + e * kThreads));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t[e] < kReach) atomicAdd(&sh.lo[Row::bin_of(t[e])], 1u);
      }
    } else {
      const float limit_l = limit.key ? from_key(limit.key) : kNegInf;
      for (int i = tid; i < n; i += 4 * kThreads) {
        float l[4];
        bool in[4], any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[e] = logit(i + e * kThreads);
          // (those at the limit's key: their number is known, and they are counted once below)
          in[e] = l[e] > limit_l;
          any |= in[e];
        }
        if (!any) continue;
        unsigned long long u[4];
        float2 t[2];
        row.units2(l[0], l[1], &u[0], &u[1], &t[0]);
        row.units2(l[2], l[3], &u[2], &u[3], &t[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float reach = e & 1 ? t[e / 2].y : t[e / 2].x;
          if (in[e] && reach > -kReach) bin_add(sh, Row::bin_of(-reach), u[e]);
        }
      }
    }
    if (rank == 0 && tid == 0 && limit.key) {
      const float l = from_key(limit.key);
      bin_add(sh, Row::bin_of(row.reach(l)), (masses ? row.units(l) : 1ull) * limit.ties);
    }
    cluster.sync();
    // this CTA's slice of the bins, over all CTAs (neighbouring bins to a thread)
    const int per = kBins / C, first = rank * per;
    constexpr int kMost = kBins / kThreads;
    const int mine = max(1, per / kThreads), i0 = tid * mine;
    unsigned long long v[kMost], sum = 0;
#pragma unroll
    for (int e = 0; e < kMost; ++e) {
      v[e] = 0;
      if (e < mine && i0 < per) {
        auto from_cta = [&](int c) {
          return ((unsigned long long)cluster.map_shared_rank(sh.hi, c)[first + i0 + e] << 32) +
                 cluster.map_shared_rank(sh.lo, c)[first + i0 + e];
        };
        if (C == kMaxCluster) {   // (all loads on their way together)
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c) v[e] += from_cta(c);
        } else {
          for (int c = 0; c < C; ++c) v[e] += from_cta(c);
        }
      }
      sum += v[e];
    }
    unsigned long long upto_mine = block_upto(sum, sh.warp_mass) - sum;
#pragma unroll
    for (int e = 0; e < kMost; ++e) {
      upto_mine += v[e];
      if (e < mine && i0 < per) sh.upto[i0 + e] = upto_mine;
    }
    if (tid == kThreads - 1)   // (all of it)
      for (int c = 0; c < C; ++c) *cluster.map_shared_rank(&sh.slice[rank], c) = upto_mine;
    cluster.sync();
    unsigned long long slice_to[kMaxCluster], total = 0;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) slice_to[c] = total += c < C ? sh.slice[c] : 0ull;
    if (masses) target = top_p > 0.f ? share_of(total, top_p) : 1ull;
    if (total < target) return Border{0u, ~0ull};
    unsigned long long start = 0;
    int owner = 0;
#pragma unroll
    for (int c = 0; c < kMaxCluster - 1; ++c)
      if (slice_to[c] < target) start = slice_to[c], owner = c + 1;
    const unsigned long long* const upto = cluster.map_shared_rank(sh.upto, owner);
    for (int i = tid; i < per; i += kThreads) {
      const unsigned long long lower = start + (i ? upto[i - 1] : 0);
      if (lower < target && start + upto[i] >= target) {   // (one of them)
        sh.bin = owner * per + i;
        sh.above = lower;
        sh.inside = start + upto[i];
      }
    }
    __syncthreads();
    int bin = sh.bin;
    const unsigned long long above = sh.above;
    // where min-p cuts in an earlier bin, its own tokens decide
    const int least_bin = least > kNegInf ? (row.reach(least) < kReach ? Row::bin_of(row.reach(least)) : kBins)
                                          : kBins;
    const bool min_p_cuts = masses && least_bin < bin;
    if (min_p_cuts) bin = least_bin;
    *weighed = masses && !limit.key;
    unsigned long long part = 0, ties = 0;
    if (*weighed)
      for (int i = tid; i < bin; i += kThreads)
        part += ((unsigned long long)sh.hi[i] << 32) + sh.lo[i];
    // few tokens down to the bin's end: one CTA finishes the row with them
    if (!masses && sh.inside <= kFew) {
      unsigned* const to = cluster.map_shared_rank(sh.keys, 0);
      int* const ids = cluster.map_shared_rank(sh.ids, 0);
      int* const count = cluster.map_shared_rank(&sh.gathered, 0);
      scan([&](float t) { return t < kReach && Row::bin_of(t) <= bin; }, [&](int i, float l) {
        const int at = atomicAdd(count, 1);   // (below kFew: as many as were counted)
        if (at < kFew) to[at] = key_of(l), ids[at] = v0 + i;
      });
      cluster.sync();
      return Border{1u, 0ull};
    }
    // the tokens of the bin
    unsigned* const keys = cluster.map_shared_rank(sh.keys, 0);
    int* const gathered = cluster.map_shared_rank(&sh.gathered, 0);
    scan([&](float t) { return t < kReach && Row::bin_of(t) == bin; }, [&](int i, float l) {
      if (key_of(l) <= limit.key) return;
      if (min_p_cuts) {
        if (key_of(l) >= least_key) part += row.units(l);
        return;
      }
      const int place = atomicAdd(&sh.listed, 1), at = atomicAdd(gathered, 1);
      if (place < kThreads) sh.list[place] = i;
      if (at < kGathered) keys[at] = key_of(l);
    });
    if (min_p_cuts) {
      sum_up(part, 0ull, own, own_ties);
      return Border{0u, ~0ull};
    }
    cluster.sync();
    Border found;
    const int all = *gathered;
    auto each_own = [&](auto&& f) {   // this CTA's tokens in the bin
      if (sh.listed <= kThreads) {
        if (tid < sh.listed) f(key_of(logit(sh.list[tid])));
        return;
      }
      for (int i = tid; i < n; i += kThreads) {
        const float l = logit(i), t = row.reach(l);
        if (t < kReach && Row::bin_of(t) == bin && key_of(l) > limit.key) f(key_of(l));
      }
    };
    if (all > kGathered) {   // (many equal logits, mostly)
      found = find(masses, target, above, 0u, 0xFFFFFFFFu, limit, true, each_own);
    } else {
      if (rank == 0) {
        unsigned low = 0xFFFFFFFFu, high = 0u;
        if (limit.key && Row::bin_of(row.reach(from_key(limit.key))) == bin) low = high = limit.key;
        for (int i = tid; i < all; i += kThreads) {
          low = min(low, sh.keys[i]);
          high = max(high, sh.keys[i]);
        }
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        if (lane == 0) sh.low[warp] = low, sh.high[warp] = high;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) low = min(low, sh.low[w]), high = max(high, sh.high[w]);
        found = find(masses, target, above, low, high, limit, false, [&](auto&& f) {
          for (int i = tid; i < all; i += kThreads) f(sh.keys[i]);
        });
        if (tid < C) {
          *cluster.map_shared_rank(&sh.border_key, tid) = found.key;
          *cluster.map_shared_rank(&sh.border_ties, tid) = found.ties;
        }
      }
      cluster.sync();
      found = Border{sh.border_key, sh.border_ties};
    }
    if (*weighed) {
      each_own([&](unsigned key) {
        if (key < least_key) return;
        if (key > found.key) part += row.units(from_key(key));
        else if (key == found.key) ++ties;
      });
      sum_up(part, ties, own, own_ties);
    }
    return found;
  };

  // floor(u * total), u in units of 2^-64: drawn is the first token beyond it
  auto place_of = [&](unsigned long long total) {
    unsigned long long u64 = 0;
    if (u >= 1.0) u64 = ~0ull << 11;   // the last value below 1: 1 - 2^-53
    else if (u > 0x1p-1000) {
      const unsigned long long bits = (unsigned long long)__double_as_longlong(u);
      const int shift = (int)(bits >> 52) - 1011;   // of the mantissa
      const unsigned long long m = (bits & ((1ull << 52) - 1)) | 1ull << 52;
      u64 = shift >= 0 ? m << shift : (shift > -53 ? m >> -shift : 0ull);
    }
    return __umul64hi(u64, total);
  };
  // Top-k, top-p, min-p and the draw among the few tokens in sh.keys and sh.ids, by this CTA: sorted by
  // their logits, then what is kept by ids.
  auto finish = [&] {
    const int m = min(sh.gathered, kFew);
    unsigned long long* const order = sh.upto;
    // in falling order, of equal logits the lowest ids first
    if (tid < m) order[tid] = (unsigned long long)sh.keys[tid] << 32 | ~(unsigned)sh.ids[tid];
    sort_down(order, m, order + kFew);
    const int first = min(k, m);   // top-k's
    const unsigned my_key = tid < first ? (unsigned)(order[tid] >> 32) : 0u;
    const unsigned not_id = tid < first ? (unsigned)order[tid] : 0u;
    const unsigned long long mine = tid < first ? row.units(from_key(my_key)) : 0ull;
    const unsigned long long to = block_upto(mine, sh.warp_mass);
    if (tid == kThreads - 1) sh.above = to;
    __syncthreads();
    const unsigned long long all = sh.above;
    const unsigned long long limit =
        top_p < 1.f ? (top_p > 0.f ? share_of(all, top_p) : 1ull) : ~0ull;
    const bool kept = tid < first && (to - mine < limit) && my_key >= least_key;
    sh.units[tid] = kept ? mine : 0ull;
    const unsigned long long total_to = block_upto(kept ? mine : 0ull, sh.warp_ties);
    if (tid == kThreads - 1) sh.inside = total_to;
    __syncthreads();
    const unsigned long long total = sh.inside, place = place_of(total);
    // by their ids; what is not kept has no weight
    if (tid < first) order[tid] = (unsigned long long)not_id << 32 | tid;
    sh.sorted[tid] = my_key;
    sort_down(order, first, order + kFew);
    const unsigned long long my = tid < first ? order[tid] : 0ull;
    const int from = (int)(unsigned)my;   // where it was among the sorted
    const unsigned long long weight = tid < first ? sh.units[from] : 0ull;
    const unsigned long long upto = block_upto(weight, sh.warp_mass);
    if (place < upto - weight || place >= upto) return;
    p.out[b] = (int)~(unsigned)(my >> 32);
    if (p.prob) p.prob[b] = row.share(from_key(sh.sorted[from]), total);
  };
  Border border{0u, ~0ull};
  unsigned long long own = 0, own_ties = 0;
  bool weighed = false;
  if (k > 0 && k < p.V) {
    border = cut(false, (unsigned long long)k, border, &weighed, &own, &own_ties);
    if (border.key && border.ties == 0) {
      if (rank == 0) finish();
      return;
    }
  }
  if (top_p < 1.f) border = cut(true, 0ull, border, &weighed, &own, &own_ties);
  // ------------------------------------------------------------------ the draw
  // the mass above the border, and the tokens at it, of each warp's stretch
  // (whole rounds of the loop below; the logits' order is their keys')
  constexpr int kRound = 128;
  static_assert(kRound * kWarps <= kGathered, "a round per warp in sh.keys");
  const int stretch = (n + kRound * kWarps - 1) / (kRound * kWarps) * kRound;
  const float border_l = border.key ? from_key(border.key) : kNegInf;
  auto weigh = [&] {
    unsigned long long mass = 0, ties = 0;
    // where few of a round's tokens are above the border, they wait in shared memory until 64 are there
    float* const room = reinterpret_cast<float*>(sh.keys) + warp * kRound;
    int held = 0, taken = 0;
    const bool all = !border.key && least == kNegInf;
    auto add = [&](float l0, float l1) {
      unsigned long long u0, u1;
      float2 t;
      row.units2(l0, l1, &u0, &u1, &t);
      mass += u0 + u1;
    };
    for (int i = warp * stretch + lane; i < min(n + lane, (warp + 1) * stretch); i += kRound) {
      float l[4];   // (behind the last token: -infinity, which has no weight)
#pragma unroll
      for (int e = 0; e < 4; ++e) l[e] = logit(i + 32 * e);
      if (all) {
        add(l[0], l[1]);
        add(l[2], l[3]);
        continue;
      }
      unsigned over[4];
      int count = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = l[e] >= least;
        ties += in && l[e] == border_l ? 1 : 0;
        over[e] = __ballot_sync(0xffffffffu, in && l[e] > border_l);
        count += __popc(over[e]);
      }
      if (count > kRound / 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e] = over[e] >> lane & 1u ? l[e] : kNegInf;
        add(l[0], l[1]);
        add(l[2], l[3]);
      } else if (count) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (over[e] >> lane & 1u)
            room[(held + __popc(over[e] & ((1u << lane) - 1u))) & (kRound - 1)] = l[e];
          held += __popc(over[e]);
        }
        __syncwarp();
        if (held - taken >= kRound / 2) {
          add(room[(taken + lane) & (kRound - 1)], room[(taken + 32 + lane) & (kRound - 1)]);
          taken += kRound / 2;
          __syncwarp();
        }
      }
    }
    if (held > taken)
      add(taken + lane < held ? room[(taken + lane) & (kRound - 1)] : kNegInf,
          taken + 32 + lane < held ? room[(taken + 32 + lane) & (kRound - 1)] : kNegInf);
    if (!border.key) ties = 0;
    mass = warp_sum(mass);
    ties = warp_sum(ties);
    if (lane == 0) {
      sh.warp_mass[warp] = mass;
      sh.warp_ties[warp] = ties;
    }
    __syncthreads();
  };
  if (!weighed) {
    weigh();
    if (warp == kWarps - 1) {
      own = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0ull);
      own_ties = warp_sum(lane < kWarps ? sh.warp_ties[lane] : 0ull);
    }
  }
  if (tid == kThreads - 1)
    for (int c = 0; c < C; ++c) {
      *cluster.map_shared_rank(&sh.mass[rank], c) = own;
      *cluster.map_shared_rank(&sh.ties[rank], c) = own_ties;
    }
  cluster.sync();
  const unsigned long long each = border.key ? row.units(from_key(border.key)) : 0ull;
  // (a lane per CTA of the cluster)
  const unsigned long long tied_here = lane < C ? sh.ties[lane] : 0ull;
  const unsigned long long ties_upto = warp_upto(tied_here, lane);
  const unsigned long long kept =
      min(ties_upto, border.ties) - min(ties_upto - tied_here, border.ties);
  const unsigned long long mass_here = (lane < C ? sh.mass[lane] : 0ull) + kept * each;
  const unsigned long long mass_upto = warp_upto(mass_here, lane);
  const unsigned long long total = __shfl_sync(0xffffffffu, mass_upto, 31);
  const unsigned long long mine = __shfl_sync(0xffffffffu, mass_here, rank);
  const unsigned long long start = __shfl_sync(0xffffffffu, mass_upto, rank) - mine;
  const unsigned long long ties_start = __shfl_sync(0xffffffffu, ties_upto - tied_here, rank);
  const unsigned long long target = place_of(total);   // drawn: the first beyond it
  if (target < start || target >= start + mine) return;
  // (one CTA of the cluster) the warp's stretch that crosses it, a lane per warp
  if (weighed) weigh();
  const unsigned long long warp_tied = lane < kWarps ? sh.warp_ties[lane] : 0ull;
  const unsigned long long tied_to = ties_start + warp_upto(warp_tied, lane);
  const unsigned long long warp_mass =
      (lane < kWarps ? sh.warp_mass[lane] : 0ull) +
      (min(tied_to, border.ties) - min(tied_to - warp_tied, border.ties)) * each;
  const unsigned long long mass_to = start + warp_upto(warp_mass, lane);
  const unsigned crossing = __ballot_sync(0xffffffffu, target < mass_to);
  const int w = crossing ? __ffs(crossing) - 1 : kWarps - 1;   // (there is one)
  unsigned long long at = __shfl_sync(0xffffffffu, mass_to - warp_mass, w);
  unsigned long long tied = __shfl_sync(0xffffffffu, tied_to - warp_tied, w);
  // four neighbouring tokens of a round: their weights above the border, and which are at it
  auto round_of = [&](int r, unsigned long long (&u)[4], unsigned (&tie)[4]) {
    float l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      l[e] = logit(w * stretch + r * kRound + 4 * lane + e);
      const bool in = l[e] >= least;
      tie[e] = __ballot_sync(0xffffffffu, in && border.key && l[e] == border_l);
      l[e] = in && l[e] > border_l ? l[e] : kNegInf;
    }
    float2 where;
    row.units2(l[0], l[1], &u[0], &u[1], &where);
    row.units2(l[2], l[3], &u[2], &u[3], &where);
  };
  // its rounds (1024 at most: 2^24 tokens in 8 CTAs of 16 warps)
  const int rounds = stretch / kRound;
  for (int r = warp; r < rounds; r += kWarps) {
    unsigned long long u[4];
    unsigned tie[4];
    round_of(r, u, tie);
    const unsigned long long mass = warp_sum(u[0] + u[1] + u[2] + u[3]);
    if (lane == 0) {
      sh.upto[r] = mass;
      sh.lo[r] = __popc(tie[0]) + __popc(tie[1]) + __popc(tie[2]) + __popc(tie[3]);
    }
  }
  __syncthreads();
  if (warp) return;
  int r = 0;
  for (int r0 = 0; r0 < rounds; r0 += 32) {
    const bool there = r0 + lane < rounds;
    const unsigned long long t = there ? sh.lo[r0 + lane] : 0u, t_to = tied + warp_upto(t, lane);
    const unsigned long long m = (there ? sh.upto[r0 + lane] : 0ull) +
                                 (min(t_to, border.ties) - min(t_to - t, border.ties)) * each;
    const unsigned long long m_to = at + warp_upto(m, lane);
    const unsigned found = __ballot_sync(0xffffffffu, target < m_to);
    const int last = found ? __ffs(found) - 1 : 31;
    r = min(r0 + last, rounds - 1);
    at = __shfl_sync(0xffffffffu, found ? m_to - m : m_to, last);
    tied = __shfl_sync(0xffffffffu, found ? t_to - t : t_to, last);
    if (found) break;
  }
  // and its tokens
  unsigned long long of[4], sum = 0;
  unsigned tie[4];
  round_of(r, of, tie);
#pragma unroll
  for (int e = 0; e < 4; ++e) tied += __popc(tie[e] & ((1u << lane) - 1u));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((tie[e] >> lane & 1u) && tied++ < border.ties) of[e] = each;
    sum += of[e];
  }
  unsigned long long from_lane = at + warp_upto(sum, lane) - sum;
  if (target < from_lane || target >= from_lane + sum) return;   // (one lane)
  int e = 0;
  while (e < 3 && target >= from_lane + of[e]) from_lane += of[e++];
  const int i = w * stretch + r * kRound + 4 * lane + e;
  p.out[b] = v0 + i;
  if (p.prob) p.prob[b] = row.share(logit(i), total);
}

}  // namespace

cudaError_t launch_sample(const SampleProblem& p, cudaStream_t s) {
  SampleArgs a{};
  a.p = p;
  int bits = 0;
  while ((1 << bits) < p.V) ++bits;
  a.scale = 62 - bits < 45 ? 62 - bits : 45;
  // CTAs per row: as many as give each 16k tokens, so that two fit an SM (64 rows of 129,280 with
  // top-p: eight 69 us, four 78, two 93; with temperature alone 31, 30, 33), and for few rows more, down
  // to 1024 tokens (one row of 129,280: eight 11 us, two 33; four of 32,003: eight 8, two 11). Where
  // the rows fill the GPU, more only add exchanges: 512 rows of 4000 with one 18.5 us, with two 30;
  // 200 of 32,003 with two 25, four 32.
  int C = 1;
  while (C < kMaxCluster && p.V > 16384 * C) C *= 2;
  while (C < kMaxCluster && p.V > 1024 * C && (int64_t)p.B * C < 2 * device_sm_count()) C *= 2;
  a.chunk = ((p.V + C - 1) / C + 7) / 8 * 8;
  struct Roots {
    unsigned long long coarse[32], fine[32];
    Roots() {
      for (int j = 0; j < 32; ++j) {
        coarse[j] = (unsigned long long)std::exp2(63.0 + j / 32.0);
        fine[j] = (unsigned long long)std::exp2(63.0 + j / 1024.0);
      }
    }
  };
  static const Roots roots;
  std::memcpy(a.coarse, roots.coarse, sizeof a.coarse);
  std::memcpy(a.fine, roots.fine, sizeof a.fine);
  const int room = 160 * 1024, stage = (a.chunk + 8 + kPad) * 4;
  const bool staged = stage <= room;
  const auto kernel = p.bf16 ? (staged ? k_sample<true, true> : k_sample<true, false>)
                             : (staged ? k_sample<false, true> : k_sample<false, false>);
  static OncePerDevice ready;
  const cudaError_t e = ready.run([&] {
    const cudaError_t x = cudaFuncSetAttribute(
        k_sample<true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
    return x != cudaSuccess
               ? x
               : cudaFuncSetAttribute(k_sample<false, true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, room);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = staged ? stage : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace dsmoe
