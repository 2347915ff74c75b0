// cache.cu — rows of head_dim values on their way to and from the paged key-value cache:
// norms of queries and keys per head with the position rotation, 8-bit quantisation as the
// cache is written, and reading it back (arithmetic and layouts in include/dsmoe.h).
//
// k_rows: a row (one head of one token) belongs to D / 8 lanes of 8 values each, one 16-byte
// load and one store per lane, so a warp takes 2 (D = 128) or 4 (D = 64) tokens at a time and
// no shared memory is needed: the norm's sum and the quantiser's maximum are butterfly
// shuffles inside the row's lanes, and the rotation's partner values (n / 2 values away) come
// as bf16 from one fixed lane, because n / 2 is a multiple of a lane's 8 values. A warp's rows
// are of the same head, so what is done to queries, keys and values branches for whole warps.
// The angle of a pair is position * freq modulo one turn, with freq in units of 2^-64 turn:
// a 64-bit integer product that wraps, exact at any position, of which the upper 32 bits go
// to sincospif. Each lane computes the angles of its own 8 values once per token, times the
// weights, and keeps them in registers over the heads of its chunk. Memory-bound by bytes,
// by instruction issue in practice (55 to 70% of the slots): fp32 arithmetic is done two values
// at a time (f32x2). 16,384 tokens x 20 heads of 128, rotated: 31.8 us, 5.3 TB/s; 32,768 tokens x
// 8 heads into a Q8 cache: 40 us, 5.1 TB/s.
#include "common.cuh"
#include "kernels.h"

namespace dsmoe {
namespace {

constexpr int kThreads = 256;

struct RowsArgs {
  RowsProblem p;
  CacheView c;
  int groups;              // warps per chunk of heads: 32 * 8 / D tokens each
  int chunks, per_chunk;   // the heads of a token in chunks of per_chunk
};

__device__ __forceinline__ void pairs_of(const uint4& w, f2 (&x)[4]) {
  x[0] = pair(bf16_lo(w.x), bf16_hi(w.x));
  x[1] = pair(bf16_lo(w.y), bf16_hi(w.y));
  x[2] = pair(bf16_lo(w.z), bf16_hi(w.z));
  x[3] = pair(bf16_lo(w.w), bf16_hi(w.w));
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// Where a row of the cache starts, in values; slot is inside the cache.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int slot, int head, int D) {
  const int page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
  return page * c.stride + (((int64_t)head << c.page_shift) + off) * D;
}
__device__ __forceinline__ int64_t scale_at(const CacheView& c, int slot, int head) {
  const int page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
  return page * c.scale_stride + ((int64_t)head << c.page_shift) + off;
}
__device__ __forceinline__ bool slot_ok(const CacheView& c, int slot) {
  return slot >= 0 && (slot >> c.page_shift) < c.pages;
}

// The larger of two bf16 pairs of magnitudes, NaN above all.
__device__ __forceinline__ uint32_t max_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 1 / x to an ulp, x normal and not near the largest.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Writes the codes and the scale of a row of the cache: code = 127 x / a rounded to nearest,
// ties to even, a the row's largest magnitude (its bits in `top`, already the maximum over the
// row's lanes). The quotient is the product with 1 / a (to an ulp) and one correction by its
// remainder (Markstein, IBM J. Res. Dev. 34, 1990), which makes a half-integer exactly that: for
// bf16 values 127 x / a is a ratio of small integers, so no other value comes near one. Rounding
// is the addition of 1.5 * 2^23, whose low byte is the code. a / 127 by the same theorem, with
// 1 / 127 rounded correctly, is the correctly rounded quotient where it is normal.
template <int D>
__device__ __forceinline__ void put_codes(const f2 (&x)[4], uint32_t top, uint8_t* dst,
                                          float* scale, int j, bool store) {
  const bool bad = top >= 0x7F800000u, none = top == 0u || bad;
  const float amax = __uint_as_float(top);
  // 127 x and 1 / a stay finite: both sides by 2^-8 or 2^64 where they would not (exact)
  const float pre = amax > 3.3230699e35f ? 0.00390625f : (amax < 7.8886091e-31f ? 1.8446744e19f : 1.f);
  const float den = __fmul_rn(amax, pre), inv = none ? 0.f : rcp(den);
  const float mult = __fmul_rn(127.f, pre);
  const f2 mult2 = pair(mult, mult), inv2 = pair(inv, inv), den2 = pair(-den, -den);
  const f2 magic = pair(12582912.f, 12582912.f);
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 t = mul2(x[i], mult2), u = mul2(t, inv2);
    const float2 m = parts(add2(fma2(fma2(u, den2, t), inv2, u), magic));
    q[2 * i] = __float_as_uint(m.x);
    q[2 * i + 1] = __float_as_uint(m.y);
  }
  if (!store) return;
  const uint32_t lo =
      __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  const uint32_t hi =
      __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  reinterpret_cast<uint2*>(dst)[j] = make_uint2(none ? 0u : lo, none ? 0u : hi);
  if (j == 0) {
    constexpr float k127 = 1.f / 127.f;
    const float t = __fmul_rn(amax, k127);
    float q127 = __fmaf_rn(__fmaf_rn(-127.f, t, amax), k127, t);
    if (amax < 7.8886091e-31f) q127 = __fdiv_rn(amax, 127.f);
    *scale = bad ? __uint_as_float(0x7FC00000u) : q127;
  }
}
// Bits of the largest magnitude of a row: of bf16 values, and of fp32 ones (as integers they
// order as the values do, NaN above all).
template <int LPH>
__device__ __forceinline__ uint32_t top_of(const uint4& x) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = max_bf2(max_bf2(x.x & kAbs, x.y & kAbs), max_bf2(x.z & kAbs, x.w & kAbs));
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) m = max_bf2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max_bf2(m, m << 16) & 0xFFFF0000u;
}
template <int LPH>
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// kCache: 0 keys to k_out, 1 keys and values to a bf16 cache, 2 to a Q8 cache.
// kTurn: 0 rows are stored as they are; norms and rotation of halves (1) or neighbours (2).
// kPerSm: CTAs per SM the registers are limited for.
template <int D, int kCache, int kTurn, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm)
    k_rows(const __grid_constant__ RowsArgs a) {
  constexpr int LPH = D / 8, kTokens = 32 / LPH;   // lanes per row, tokens per warp
  // rows whose loads are in flight together (the write above: 2 50 us, 4 43, 8 40, but of one
  // head, 16,384 tokens with the reading back, 4 8.2 and 8 8.6; the rotation: 4 31.9 us, 5 36.4.
  // With four CTAs per SM the rotating forms spill with 4 as well, 40 to 80 bytes a thread)
  constexpr int kBatch = kTurn ? 4 : 8;
  pdl_trigger();
  pdl_wait();
  const RowsProblem& p = a.p;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int chunk = (int)(w / a.groups);
  if (chunk >= a.chunks) return;                   // (a whole warp)
  const int lane = threadIdx.x & 31, j = lane % LPH;
  const int t_mine = (int)(w % a.groups) * kTokens + lane / LPH;
  const bool live = t_mine < p.T;
  const int t = live ? t_mine : p.T - 1;           // (every lane takes part in the shuffles)

  int slot = -1;
  if (kCache) slot = p.slots[t];
  const bool keep = live && (kCache == 0 || slot_ok(a.c, slot));

  // this lane's 8 angles: value e becomes x[e] * co[e] + partner[e] * si[e]
  const int half = p.rot / 16;                     // lanes per half of the rotated values
  const bool turned = kTurn && j < 2 * half;
  const int partner = kTurn != 1 || !turned ? j : (j < half ? j + half : j - half);
  float co[8], si[8];
  if constexpr (kTurn != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) co[e] = 1.f, si[e] = 0.f;
    if (turned) {
      const uint64_t pos = (uint64_t)(int64_t)p.positions[t];
      const int64_t* f = p.freqs + (kTurn == 2 ? 4 * j : 8 * (j < half ? j : j - half));
#pragma unroll
      for (int e = 0; e < (kTurn == 2 ? 4 : 8); ++e) {
        const uint64_t turn = pos * (uint64_t)f[e];
        float sn, cs;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31
        if constexpr (kTurn == 2) {
          co[2 * e] = co[2 * e + 1] = cs;
          si[2 * e] = -sn, si[2 * e + 1] = sn;
        } else {
          co[e] = cs;
          si[e] = j < half ? -sn : sn;
        }
      }
    }
  }
  const uint32_t other = turned ? 0xFFFFFFFFu : 0u;   // (0 x infinity is not 0)

  // heads [from, to) of one kind, rows `stride` values apart per token
  auto rows = [&](const uint16_t* src, int64_t stride, int from, int to, const uint16_t* weight,
                  bool turn, auto&& emit) {
    f2 c2[4], s2[4];
    if (kTurn && turn) {
      float c[8], s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = co[e], s[e] = si[e];
      if (weight) {
        float wo[8], wp[8];
        unpack8(reinterpret_cast<const uint4*>(weight)[j], wo);
        unpack8(reinterpret_cast<const uint4*>(weight)[partner], wp);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          c[e] = __fmul_rn(c[e], wo[e]);
          s[e] = __fmul_rn(s[e], wp[kTurn == 2 ? e ^ 1 : e]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c2[i] = pair(c[2 * i], c[2 * i + 1]), s2[i] = pair(s[2 * i], s[2 * i + 1]);
    }
    const uint4* row = reinterpret_cast<const uint4*>(src + t * stride) + j;
    for (int h0 = from; h0 < to; h0 += kBatch) {
      uint4 in[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        in[b] = h0 + b < to ? row[(h0 + b) * LPH] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (h0 + b >= to) break;
        float x[8];
        f2 x2[4];
        if (kTurn && turn) {
          f2 y2[4];
          pairs_of(in[b], x2);
          if constexpr (kTurn == 1) {
            uint4 y;
            y.x = __shfl_sync(0xffffffffu, in[b].x, partner, LPH) & other;
            y.y = __shfl_sync(0xffffffffu, in[b].y, partner, LPH) & other;
            y.z = __shfl_sync(0xffffffffu, in[b].z, partner, LPH) & other;
            y.w = __shfl_sync(0xffffffffu, in[b].w, partner, LPH) & other;
            pairs_of(y, y2);
          } else {
            const uint4 y = make_uint4(__byte_perm(in[b].x, 0u, 0x1032) & other,
                                       __byte_perm(in[b].y, 0u, 0x1032) & other,
                                       __byte_perm(in[b].z, 0u, 0x1032) & other,
                                       __byte_perm(in[b].w, 0u, 0x1032) & other);
            pairs_of(y, y2);
          }
          if (weight) {
            f2 sum = mul2(x2[0], x2[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) sum = fma2(x2[i], x2[i], sum);
            const float2 two = parts(sum);
            float ss = __fadd_rn(two.x, two.y);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1)
              ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
            const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.f / D), p.eps));
            const f2 r2 = pair(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) x2[i] = mul2(x2[i], r2), y2[i] = mul2(y2[i], r2);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x2[i] = fma2(y2[i], s2[i], mul2(x2[i], c2[i]));
            const float2 o = parts(x2[i]);
            x[2 * i] = o.x;
            x[2 * i + 1] = o.y;
          }
        } else {
          pairs_of(in[b], x2);
        }
        emit(h0 + b, x, x2, in[b]);
      }
    }
  };
  // the row of head 0 in the cache; heads are head_rows rows apart
  const int64_t row0 = keep && kCache ? cache_row(a.c, slot, 0, D) : 0;
  const int64_t scale0 = keep && kCache == 2 ? scale_at(a.c, slot, 0) : 0;
  const int begin = chunk * a.per_chunk, end = begin + a.per_chunk;
  if constexpr (kTurn != 0)
    rows(p.q, p.q_stride, begin, min(end, p.Hq), p.q_weight, true,
         [&](int h, const float(&x)[8], const f2(&)[4], const uint4&) {
           if (live) reinterpret_cast<uint4*>(p.q_out + ((int64_t)t * p.Hq + h) * D)[j] = pack8(x);
         });
  rows(p.k, p.k_stride, max(begin - p.Hq, 0), min(end - p.Hq, p.Hkv), p.k_weight, true,
       [&](int h, const float(&x)[8], const f2(&x2)[4], const uint4& in) {
         const int64_t at = row0 + ((int64_t)h << a.c.page_shift) * D;
         if constexpr (kCache == 0) {
           if (live) reinterpret_cast<uint4*>(p.k_out + ((int64_t)t * p.Hkv + h) * D)[j] = pack8(x);
         } else if constexpr (kCache == 1) {
           if (keep)
             reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.c.k) + at)[j] =
                 kTurn ? pack8(x) : in;
         } else {
           uint32_t top;
           if constexpr (kTurn != 0) top = top_of<LPH>(x);
           else top = top_of<LPH>(in);
           put_codes<D>(x2, top, a.c.k + at, a.c.k_scale + scale0 + ((int64_t)h << a.c.page_shift), j,
                        keep);
         }
       });
  if constexpr (kCache != 0)
    rows(p.v, p.v_stride, max(begin - p.Hq - p.Hkv, 0), min(end - p.Hq - p.Hkv, p.Hkv), nullptr,
         false, [&](int h, const float(&)[8], const f2(&x2)[4], const uint4& in) {
           const int64_t at = row0 + ((int64_t)h << a.c.page_shift) * D;
           if constexpr (kCache == 1) {
             if (keep) reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.c.v) + at)[j] = in;
           } else {
             put_codes<D>(x2, top_of<LPH>(in), a.c.v + at,
                          a.c.v_scale + scale0 + ((int64_t)h << a.c.page_shift), j, keep);
           }
         });
}

// k_cache_read: one thread per 8 values of a (token, head), keys and values. Bound by memory's
// latency over scattered rows: 32,768 tokens x 8 heads from a Q8 cache 33 us, 6.1 TB/s.
template <int D, bool kQ8>
__global__ void __launch_bounds__(kThreads) k_cache_read(const CacheView c, const int32_t* slots,
                                                         int n, uint16_t* k_out,
                                                         uint16_t* v_out) {
  constexpr int LPH = D / 8;
  pdl_trigger();
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)n * c.heads * LPH) return;
  const int j = (int)(i % LPH);
  const int64_t row = i / LPH;
  const int head = (int)(row % c.heads);
  const int slot = slots[row / c.heads];
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (slot_ok(c, slot)) {
    const int64_t at = cache_row(c, slot, head, D);
    if constexpr (kQ8) {
      const uint2 kc = reinterpret_cast<const uint2*>(c.k + at)[j];
      const uint2 vc = reinterpret_cast<const uint2*>(c.v + at)[j];
      const int64_t sa = scale_at(c, slot, head);
      const float ks = c.k_scale[sa], vs = c.v_scale[sa];
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int sh = 8 * (e & 3);
        x[e] = __fmul_rn((float)(int8_t)((e < 4 ? kc.x : kc.y) >> sh), ks);
        y[e] = __fmul_rn((float)(int8_t)((e < 4 ? vc.x : vc.y) >> sh), vs);
      }
      k = pack8(x);
      v = pack8(y);
    } else {
      k = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(c.k) + at)[j];
      v = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(c.v) + at)[j];
    }
  }
  reinterpret_cast<uint4*>(k_out)[i] = k;
  reinterpret_cast<uint4*>(v_out)[i] = v;
}

template <int D, int kCache, int kTurn, int kPerSm>
cudaError_t start_rows(const RowsProblem& p, const CacheView* c, cudaStream_t s) {
  constexpr int kTokens = 256 / D;
  RowsArgs a{};
  a.p = p;
  if (c) a.c = *c;
  const int heads = p.Hq + (c ? 2 : 1) * p.Hkv;
  a.groups = (p.T + kTokens - 1) / kTokens;
  // A token's heads go to one warp after another in chunks. Long chunks share what a warp does
  // once (the angles: about as long as 6 heads; else addresses, 3), short ones keep every SM's
  // warps busy: the fewest steps over the waves of resident warps. (384 tokens x 40 heads, as
  // many warps as two waves have: 8.8 us, this 5.0; 2048 tokens 14.7 and 10.8.)
  const int64_t resident = (int64_t)device_sm_count() * kPerSm * (kThreads / 32);
  constexpr int kAngles = kTurn ? 6 : 3;
  int64_t best = INT64_MAX;
  for (int chunks = 1; chunks <= heads; chunks += (chunks + 3) / 4) {
    const int per = (heads + chunks - 1) / chunks;
    const int64_t warps = (int64_t)a.groups * ((heads + per - 1) / per);
    const int64_t cost = (warps + resident - 1) / resident * (per + kAngles);
    if (cost < best) best = cost, a.per_chunk = per;
  }
  a.chunks = (heads + a.per_chunk - 1) / a.per_chunk;
  const int64_t grid = ((int64_t)a.groups * a.chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(k_rows<D, kCache, kTurn, kPerSm>, dim3((unsigned)grid), kThreads, 0, s, a);
}

template <int D, int kCache, int kPerSm>
cudaError_t pick_turn(const RowsProblem& p, const CacheView* c, cudaStream_t s) {
  return p.interleaved ? start_rows<D, kCache, 2, kPerSm>(p, c, s)
                       : start_rows<D, kCache, 1, kPerSm>(p, c, s);
}

template <int D>
cudaError_t pick_rows(const RowsProblem& p, const CacheView* c, cudaStream_t s) {
  if (p.Hq == 0) return c->q8 ? start_rows<D, 2, 0, 4>(p, c, s) : start_rows<D, 1, 0, 4>(p, c, s);
  // CTAs per SM: four have 64 registers a thread. Into a Q8 cache that is too few (16,384
  // tokens x 32 + 8 heads, halves 85.2 us, with four 86.3, with two 98.1; neighbours 78.3, 82.7, 93.0),
  // into a bf16 one it is as good (halves 76.0, with three 77.1; neighbours 73.5, 72.3); without a cache three are faster while all
  // tokens fit the SMs at once (384 tokens x 40 heads 5.0 against 6.4 us, 2048 10.8 against 13.0),
  // four beyond (16,384 tokens x 20 heads 31.8 against 34.8).
  if (c) return c->q8 ? pick_turn<D, 2, 3>(p, c, s) : pick_turn<D, 1, 4>(p, c, s);
  const bool many = (int64_t)p.T * D / 256 > (int64_t)device_sm_count() * 4 * (kThreads / 32);
  return many ? pick_turn<D, 0, 4>(p, c, s) : pick_turn<D, 0, 3>(p, c, s);
}

template <int D>
cudaError_t start_read(const CacheView& c, const int32_t* slots, int n, uint16_t* k_out,
                       uint16_t* v_out, cudaStream_t s) {
  const int64_t grid = ((int64_t)n * c.heads * (D / 8) + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return c.q8 ? launch_pdl(k_cache_read<D, true>, dim3((unsigned)grid), kThreads, 0, s, c, slots,
                           n, k_out, v_out)
              : launch_pdl(k_cache_read<D, false>, dim3((unsigned)grid), kThreads, 0, s, c, slots,
                           n, k_out, v_out);
}

}  // namespace

cudaError_t launch_rows(const RowsProblem& p, const CacheView* cache, cudaStream_t s) {
  return p.D == 128 ? pick_rows<128>(p, cache, s) : pick_rows<64>(p, cache, s);
}

cudaError_t launch_cache_read(const CacheView& c, int D, const int32_t* slots, int n,
                              uint16_t* k_out, uint16_t* v_out, cudaStream_t s) {
  return D == 128 ? start_read<128>(c, slots, n, k_out, v_out, s)
                  : start_read<64>(c, slots, n, k_out, v_out, s);
}

}  // namespace dsmoe
