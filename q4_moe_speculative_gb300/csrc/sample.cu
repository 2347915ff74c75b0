// sample.cu — a token per row of logits with temperature, top-k, top-p and min-p, drawn with a
// given uniform (arithmetic in include/dsmoe.h).
//
// A row belongs to a cluster of CTAs (up to 8), each of which keeps its part of the logits in shared
// memory, so that they are read from memory once; what the CTAs have to agree on goes through
// distributed shared memory.
//
// Masses are integers: weight exp((l - max) / T) in units of 2^-scale, the scale such that a
// vocabulary's sum fits 63 bits. Sums of integers do not depend on their order, so the borders and
// the draw are the same whatever the grid, and no token is drawn beyond its share by rounding.
//
// Where the order is cut (the k-th largest logit; the logit at which the mass before it reaches
// top_p), the border is found by counts or masses per bin: first 2048 bins of equal width in
// (max - l) / T, which spread a vocabulary's logits, then the border bin's range of keys (logits as
// ordered integers) in 2048 bins, until a bin is one key. Of the tokens with the border's logit the
// lowest ids are kept.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace dsmoe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr float kReach = 46.f;       // log2: a lighter token has the weight 0
constexpr float kBinsPerLog2 = kBins / kReach;
constexpr float kNegInf = -INFINITY;

struct SampleArgs {
  SampleProblem p;
  int chunk;        // tokens per CTA, a multiple of 8
  int scale;        // log2 of the weight 1
  bool staged;      // the chunk is kept in shared memory
};

struct Shared {
  unsigned lo[kBins], hi[kBins];
  unsigned long long upto[kBins];          // of this CTA's slice of the bins, merged
  unsigned long long slice[kMaxCluster];   // totals of the slices
  unsigned long long mass[kMaxCluster];    // of the CTAs: mass above the border
  unsigned long long ties[kMaxCluster];    // and tokens at it
  unsigned long long warp_mass[kWarps];
  unsigned long long warp_ties[kWarps];
  unsigned long long above;                // a border found: what is above its bin
  float top[kMaxCluster];
  float warp_top[kWarps];
  int bin;
  unsigned range[2];
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
  float top, per_log2;     // the largest logit; log2(e) / T
  double inv_t;
  int scale;
  // (max - l) / T in log2: never falls as l does; NaN or beyond kReach: no weight
  __device__ __forceinline__ float reach(float l) const {
    return l == top ? 0.f : __fmul_rn(__fsub_rn(top, l), per_log2);
  }
  __device__ __forceinline__ bool alive(float l) const { return reach(l) < kReach; }
  __device__ __forceinline__ double weight(float l) const {
    return l == top ? 1.0 : exp(((double)l - (double)top) * inv_t);
  }
  __device__ __forceinline__ unsigned long long units(float l) const {
    return __double2ull_rn(weight(l) * (double)(1ull << scale));
  }
  __device__ __forceinline__ int bin(float l) const {
    return min(kBins - 1, (int)__fmul_rn(reach(l), kBinsPerLog2));
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
  unsigned long long before = 0;
  for (int w = 0; w < warp; ++w) before += sums[w];
  return v + before;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleArgs a) {
  extern __shared__ float stage[];
  __shared__ Shared sh;
  const SampleProblem& p = a.p;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = min(p.V, rank * a.chunk), n = min(p.V, v0 + a.chunk) - v0;
  pdl_wait();
  const int64_t row_at = (int64_t)b * p.stride + v0;
  auto raw = [&](int i) {   // NaN is never drawn
    float l;
    if constexpr (kBf16)
      l = bf16_bits_to_f32(static_cast<const uint16_t*>(p.logits)[row_at + i]);
    else
      l = static_cast<const float*>(p.logits)[row_at + i];
    return l == l ? __fadd_rn(l, 0.f) : kNegInf;   // (and -0 is 0)
  };
  // ------------------------------------------------------------------ the largest logit
  float top = kNegInf;
  for (int i = tid; i < n; i += kThreads) {
    const float l = raw(i);
    if (a.staged) stage[i] = l;
    top = fmaxf(top, l);
  }
  auto logit = [&](int i) { return a.staged ? stage[i] : raw(i); };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.warp_top[w]);
  if (tid < C) *cluster.map_shared_rank(&sh.top[rank], tid) = top;
  cluster.sync();
  for (int c = 0; c < C; ++c) top = fmaxf(top, sh.top[c]);
  if (top == kNegInf) {   // (the same for the whole cluster)
    if (rank == 0 && tid == 0) {
      p.out[b] = -1;
      if (p.prob) p.prob[b] = 0.f;
    }
    cluster.sync();
    return;
  }
  // ------------------------------------------------------------------ the row's settings
  float T = p.temperatures ? p.temperatures[b] : p.temperature;
  int k = p.top_ks ? p.top_ks[b] : p.top_k;
  const float top_p = p.top_ps ? p.top_ps[b] : p.top_p;
  float min_p = p.min_ps ? p.min_ps[b] : p.min_p;
  const bool greedy = !(T > 0x1p-64f);
  if (greedy) T = 1.f, k = 1;
  Row row;
  row.top = top;
  row.inv_t = 1.0 / (double)T;
  row.per_log2 = (float)(row.inv_t * 1.4426950408889634);
  row.scale = a.scale;

  // The border at which counts (masses) from above reach `target` (>= 1) units; tokens all kept: key
  // 0 with no limit of ties. All threads of the cluster together.
  auto cut = [&](bool masses, unsigned long long target, const Border& limit) {
    unsigned high = 0xFFFFFFFFu, low = 0u;   // the range of keys of the bin (level 0: none yet)
    int shift = 0;
    unsigned long long above = 0;
    for (int level = 0;; ++level) {
      for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0u;
      __syncthreads();
      for (int i = tid; i < n; i += kThreads) {
        const float l = logit(i);
        if (!row.alive(l)) continue;
        const unsigned key = key_of(l);
        // (tokens at the limit's key: their number is known, and counted once below)
        if (key <= limit.key) continue;
        int at;
        if (level == 0) {
          at = row.bin(l);
        } else {
          if (key > high || key < low) continue;
          at = (int)((high - key) >> shift);
        }
        const unsigned long long u = masses ? row.units(l) : 1ull;
        const unsigned add = (unsigned)u, old = atomicAdd(&sh.lo[at], add);
        const unsigned up = (unsigned)(u >> 32) + (old + add < old ? 1u : 0u);
        if (up) atomicAdd(&sh.hi[at], up);
      }
      if (rank == 0 && tid == 0 && limit.key) {
        const float l = from_key(limit.key);
        const int at = level == 0 ? row.bin(l)
                                  : (limit.key <= high && limit.key >= low
                                         ? (int)((high - limit.key) >> shift) : -1);
        if (at >= 0) {
          const unsigned long long u = (masses ? row.units(l) : 1ull) * limit.ties;
          const unsigned add = (unsigned)u, old = atomicAdd(&sh.lo[at], add);
          const unsigned up = (unsigned)(u >> 32) + (old + add < old ? 1u : 0u);
          if (up) atomicAdd(&sh.hi[at], up);
        }
      }
      cluster.sync();
      // this CTA's slice of the bins, over all CTAs
      const int per = kBins / C, first = rank * per;
      unsigned long long before = 0;
      for (int i0 = 0; i0 < per; i0 += kThreads) {
        const int i = i0 + tid;
        unsigned long long v = 0;
        if (i < per)
          for (int c = 0; c < C; ++c)
            v += ((unsigned long long)cluster.map_shared_rank(sh.hi, c)[first + i] << 32) +
                 cluster.map_shared_rank(sh.lo, c)[first + i];
        const unsigned long long upto = before + block_upto(v, sh.warp_mass);
        if (i < per) sh.upto[i] = upto;
        __syncthreads();
        before = sh.upto[min(per, i0 + kThreads) - 1];
      }
      if (tid < C) *cluster.map_shared_rank(&sh.slice[rank], tid) = before;
      cluster.sync();
      unsigned long long start = above;
      int owner = 0;
      while (owner < C && start + sh.slice[owner] < target) start += sh.slice[owner++];
      if (owner == C) return Border{0u, ~0ull};   // (level 0 only: there is not as much)
      if (owner == rank) {
        for (int i = tid; i < per; i += kThreads) {
          const unsigned long long lower = start + (i ? sh.upto[i - 1] : 0);
          if (lower < target && start + sh.upto[i] >= target)
            for (int c = 0; c < C; ++c) {
              *cluster.map_shared_rank(&sh.bin, c) = first + i;
              *cluster.map_shared_rank(&sh.above, c) = lower;
            }
        }
      }
      cluster.sync();
      const int bin = sh.bin;
      above = sh.above;
      if (level == 0) {
        // the keys of the bin: those of the largest and the smallest logit that fall into it
        if (tid < 2) {
          unsigned in = 0u, ex = 0xFFFFFFFFu;   // tid 0: the largest key whose bin is >= bin
          const unsigned top_key = key_of(row.top);
          // (bins fall as keys rise; no key above the top's counts)
          ex = top_key + 1;
          in = key_of(-INFINITY);
          while (ex - in > 1) {
            const unsigned mid = in + (ex - in) / 2;
            const float l = from_key(mid);
            const bool beyond = !row.alive(l) || row.bin(l) > bin;
            const bool inside = !beyond && row.bin(l) == bin;
            if (tid == 0 ? (beyond || inside) : beyond) in = mid;
            else ex = mid;
          }
          sh.range[tid] = tid == 0 ? in : ex;   // (tid 1: the smallest key that is not beyond)
        }
        __syncthreads();
        high = sh.range[0];
        low = sh.range[1];
      } else {
        const unsigned span = shift ? (1u << shift) - 1 : 0u;
        high = high - ((unsigned)bin << shift);
        low = high - low > span ? high - span : low;
      }
      if (high == low) {
        const unsigned long long each = masses ? row.units(from_key(high)) : 1ull;
        unsigned long long ties = (target - above + each - 1) / each;
        if (high == limit.key && ties > limit.ties) ties = limit.ties;
        return Border{high, ties};
      }
      shift = 0;
      while ((high - low) >> shift >= kBins) ++shift;
    }
  };
  // Mass above the border and tokens at it: of each warp's stretch and each CTA. The total.
  const int stretch = (n + kWarps - 1) / kWarps;
  auto weigh = [&](const Border& cutoff, float least) {
    unsigned long long mass = 0, ties = 0;
    const int end = min(n, (warp + 1) * stretch);
    for (int i = warp * stretch + lane; i < end; i += 32) {
      const float l = logit(i);
      if (!row.alive(l) || l < least) continue;
      const unsigned key = key_of(l);
      if (key > cutoff.key) mass += row.units(l);
      else if (key == cutoff.key) ++ties;
    }
    mass = warp_sum(mass);
    ties = warp_sum(ties);
    __syncthreads();
    if (lane == 0) {
      sh.warp_mass[warp] = mass;
      sh.warp_ties[warp] = ties;
    }
    __syncthreads();
    if (tid < C) {
      mass = ties = 0;
      for (int w = 0; w < kWarps; ++w) {
        mass += sh.warp_mass[w];
        ties += sh.warp_ties[w];
      }
      *cluster.map_shared_rank(&sh.mass[rank], tid) = mass;
      *cluster.map_shared_rank(&sh.ties[rank], tid) = ties;
    }
    cluster.sync();
  };

  Border border{0u, ~0ull};
  if (k > 0 && k < p.V) border = cut(false, (unsigned long long)k, border);
  const bool nucleus = top_p < 1.f;
  if (nucleus) {
    // the mass of what top-k kept
    weigh(border, kNegInf);
    unsigned long long total = 0, ties = 0;
    for (int c = 0; c < C; ++c) {
      total += sh.mass[c];
      ties += sh.ties[c];
    }
    if (border.key) total += min(ties, border.ties) * row.units(from_key(border.key));
    double share = ceil((double)total * (double)top_p);
    unsigned long long target = share >= 1.0 ? __double2ull_rz(share) : 1ull;
    if (target > total) target = total;
    border = cut(true, target, border);
  }
  float least = kNegInf;   // the smallest logit that min-p leaves
  if (min_p > 0.f) {
    const double less = min_p < 1.f ? (double)T * log((double)min_p) : 0.0;
    least = fminf(top, __double2float_ru((double)top + less));
    auto enough = [&](float l) { return (double)l - (double)top >= less; };
    while (least < top && !enough(least)) least = from_key(key_of(least) + 1);
    while (least > kNegInf && enough(from_key(key_of(least) - 1)))
      least = from_key(key_of(least) - 1);
  }
  // ------------------------------------------------------------------ the draw
  weigh(border, least);
  const unsigned long long each = border.key ? row.units(from_key(border.key)) : 0ull;
  unsigned long long total = 0, mine = 0, start = 0, ties_start = 0, ties_upto = 0;
  for (int c = 0; c < C; ++c) {
    const unsigned long long first = min(ties_upto, border.ties);
    ties_upto += sh.ties[c];
    const unsigned long long kept = min(ties_upto, border.ties) - first;
    if (c == rank) {
      start = total;
      ties_start = ties_upto - sh.ties[c];
      mine = sh.mass[c] + kept * each;
    }
    total += sh.mass[c] + kept * each;
  }
  const double u = p.u[b];
  // floor(u * total), u in units of 2^-64
  const unsigned long long u64 = u > 0.0 ? (u < 1.0 ? __double2ull_rz(u * 0x1p64) : ~0ull) : 0ull;
  const unsigned long long target = __umul64hi(u64, total);   // drawn: the first beyond it
  if (target >= start && target < start + mine) {   // (one CTA of the cluster)
    // the warp's stretch that crosses it, and the same again inside that stretch
    unsigned long long at = start, tied = ties_start;
    int w = 0;
    for (; w < kWarps - 1; ++w) {
      const unsigned long long next = tied + sh.warp_ties[w];
      const unsigned long long m =
          sh.warp_mass[w] + (min(next, border.ties) - min(tied, border.ties)) * each;
      if (target < at + m) break;
      at += m;
      tied = next;
    }
    const int begin = w * stretch, end = min(n, begin + stretch);
    __syncthreads();
    const int per = (stretch + kThreads - 1) / kThreads;
    const int i0 = begin + tid * per, i1 = min(end, i0 + per);
    unsigned long long mass = 0, ties = 0;
    for (int i = i0; i < i1; ++i) {
      const float l = logit(i);
      if (!row.alive(l) || l < least) continue;
      if (key_of(l) > border.key) mass += row.units(l);
      else if (key_of(l) == border.key) ++ties;
    }
    const unsigned long long ties_to = tied + block_upto(ties, sh.warp_ties);
    const unsigned long long ties_from = ties_to - ties;
    mass += (min(ties_to, border.ties) - min(ties_from, border.ties)) * each;
    const unsigned long long to = at + block_upto(mass, sh.warp_mass), from = to - mass;
    if (target >= from && target < to) {
      unsigned long long sum = from, place = ties_from;
      for (int i = i0; i < i1; ++i) {
        const float l = logit(i);
        if (!row.alive(l) || l < least) continue;
        const unsigned key = key_of(l);
        if (key > border.key || (key == border.key && place++ < border.ties)) sum += row.units(l);
        if (sum > target) {
          p.out[b] = v0 + i;
          if (p.prob)
            p.prob[b] = (float)(row.weight(l) / ((double)total / (double)(1ull << row.scale)));
          break;
        }
      }
    }
  }
  cluster.sync();   // (no CTA leaves while others may reach into its shared memory)
}

}  // namespace

cudaError_t launch_sample(const SampleProblem& p, cudaStream_t s) {
  SampleArgs a{};
  a.p = p;
  int bits = 0;
  while ((1 << bits) < p.V) ++bits;
  a.scale = 62 - bits < 45 ? 62 - bits : 45;
  int C = 1;
  while (C < kMaxCluster && p.V > 2048 * C) C *= 2;
  a.chunk = ((p.V + C - 1) / C + 7) / 8 * 8;
  const int room = 160 * 1024;
  a.staged = a.chunk * 4 <= room;
  const auto kernel = p.bf16 ? k_sample<true> : k_sample<false>;
  static OncePerDevice ready;
  cudaError_t e = ready.run([&] {
    const cudaError_t x = cudaFuncSetAttribute(
        k_sample<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
    return x != cudaSuccess ? x
                            : cudaFuncSetAttribute(
                                  k_sample<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.staged ? a.chunk * 4 : 0;
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
