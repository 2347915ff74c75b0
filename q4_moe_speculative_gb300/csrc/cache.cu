// cache.cu — rows of head_dim values on their way to and from the paged key-value cache:
// norms of queries and keys per head with the position rotation, 8-bit quantisation as the
// cache is written, and reading it back (arithmetic and layouts in include/dsmoe.h).
//
// k_rows: a row (one head of one token) belongs to D / 8 lanes of 8 values each, one 16-byte
// load and one store per lane, so a warp takes 2 (D = 128) or 4 (D = 64) rows at a time and
// no shared memory is needed: the norm's sum and the quantiser's maximum are butterfly
// shuffles inside the row's lanes, and the rotation's partner values (n / 2 values away) one
// shuffle from a fixed lane, because n / 2 is a multiple of a lane's 8 values.
// The angle of a pair is position * freq modulo one turn, with freq in units of 2^-64 turn:
// a 64-bit integer product that wraps, exact at any position, of which the upper 32 bits go
// to sincospif. Each lane computes the angles of its own 8 values once per token and keeps
// them in registers over the heads of its chunk. Memory-bound: every value is read once and
// written once.
#include "common.cuh"
#include "kernels.h"

namespace dsmoe {
namespace {

constexpr int kThreads = 256;

struct RowsArgs {
  RowsProblem p;
  CacheView c;
  int chunks, per_chunk;   // the heads of a token in chunks of per_chunk
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
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

// kCache: 0 keys to k_out, 1 keys and values to a bf16 cache, 2 to a Q8 cache.
// kTurn: norms and rotation (false: rows are stored as they are).
template <int D, int kCache, bool kTurn>
__global__ void __launch_bounds__(kThreads) k_rows(const __grid_constant__ RowsArgs a) {
  constexpr int LPH = D / 8;         // lanes per row
  constexpr int kBatch = 4;          // rows whose loads are in flight together
  pdl_trigger();
  pdl_wait();
  const RowsProblem& p = a.p;
  const int64_t sub = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LPH;
  const int j = threadIdx.x % LPH;
  const bool live = sub < (int64_t)p.T * a.chunks;
  const int t = live ? (int)(sub / a.chunks) : 0;
  const int h_begin = live ? (int)(sub % a.chunks) * a.per_chunk : 0;
  const int heads = p.Hq + (kCache ? 2 : 1) * p.Hkv;
  const int h_end = !live ? 0 : min(heads, h_begin + a.per_chunk);

  int slot = -1;
  if (kCache) slot = p.slots[t];
  const bool keep = kCache == 0 || slot_ok(a.c, slot);

  // this lane's 8 angles: value e is x[e] * co[e] + partner[e] * si[e]
  const bool turned = kTurn && j < p.rot / 8;
  float co[8], si[8];
  if constexpr (kTurn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) co[e] = 1.f, si[e] = 0.f;
    if (turned) {
      const uint64_t pos = (uint64_t)(int64_t)p.positions[t];
      const int half = p.rot / 16;   // lanes per half
      const int first = p.interleaved ? 4 * j : 8 * (j < half ? j : j - half);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (p.interleaved && (e & 1)) continue;
        const uint64_t turn = pos * (uint64_t)p.freqs[first + (p.interleaved ? e / 2 : e)];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
        co[e] = c;
        si[e] = (p.interleaved || j < half) ? -s : s;
        if (p.interleaved) co[e + 1] = c, si[e + 1] = s;
      }
    }
  }
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if constexpr (kTurn) {
    if (p.q_weight) wq = reinterpret_cast<const uint4*>(p.q_weight)[j];
    if (p.k_weight) wk = reinterpret_cast<const uint4*>(p.k_weight)[j];
  }
  const int partner = j < p.rot / 16 ? j + p.rot / 16 : (j < p.rot / 8 ? j - p.rot / 16 : j);

  for (int i0 = 0; i0 < a.per_chunk; i0 += kBatch) {
    uint4 in[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h_begin + i0 + b;
      in[b] = make_uint4(0, 0, 0, 0);
      if (i0 + b >= a.per_chunk || h >= h_end) continue;
      const uint16_t* src;
      if (h < p.Hq) src = p.q + t * p.q_stride + (int64_t)h * D;
      else if (h < p.Hq + p.Hkv) src = p.k + t * p.k_stride + (int64_t)(h - p.Hq) * D;
      else src = p.v + t * p.v_stride + (int64_t)(h - p.Hq - p.Hkv) * D;
      in[b] = reinterpret_cast<const uint4*>(src)[j];
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i0 + b >= a.per_chunk) break;   // the same for the whole grid
      const int h = h_begin + i0 + b;
      const bool store = h < h_end;
      const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
      float x[8];
      unpack8(in[b], x);
      if constexpr (kTurn) {
        // (every lane shuffles, whatever its row: rows of one warp may be of different kinds)
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __fmaf_rn(x[e], x[e], ss);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1)
          ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
        const bool normed = is_q ? p.q_weight != nullptr : (is_k && p.k_weight != nullptr);
        const uint4 w4 = is_q ? wq : wk;
        float w[8], y[8];
        unpack8(w4, w);
        const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.f / D), p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = normed ? __fmul_rn(__fmul_rn(x[e], r), w[e]) : x[e];
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner, LPH);
        }
        if (turned && (is_q || is_k)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fmaf_rn(y[e], si[e], __fmul_rn(x[e], co[e]));
        }
      }
      if constexpr (kCache == 2) {
        // the largest magnitude, by its bits: they order as the values do, NaN above all
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (store && !is_q && keep) {
          const int head = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
          const bool bad = top >= 0x7F800000u;
          const float amax = __uint_as_float(top);
          // 127 x stays finite: both sides down by 2^-8 where it could not
          const float pre = amax > 3.3230699e35f ? 0.00390625f : 1.f;   // 2^118
          const float den = __fmul_rn(amax, pre);
          uint32_t q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            q[e] = top == 0u || bad
                       ? 0u
                       : (uint32_t)__float2int_rn(
                             __fdiv_rn(__fmul_rn(127.f, __fmul_rn(x[e], pre)), den)) & 0xFFu;
          const uint2 code = make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24,
                                        q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
          uint8_t* dst = (is_k ? a.c.k : a.c.v) + cache_row(a.c, slot, head, D);
          reinterpret_cast<uint2*>(dst)[j] = code;
          if (j == 0)
            (is_k ? a.c.k_scale : a.c.v_scale)[scale_at(a.c, slot, head)] =
                bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 127.f);
        }
      }
      if (store && is_q)
        reinterpret_cast<uint4*>(p.q_out + ((int64_t)t * p.Hq + h) * D)[j] = pack8(x);
      if (kCache == 0 && store && is_k)
        reinterpret_cast<uint4*>(p.k_out + ((int64_t)t * p.Hkv + h - p.Hq) * D)[j] = pack8(x);
      if (kCache == 1 && store && !is_q && keep) {
        const int head = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
        uint16_t* dst = reinterpret_cast<uint16_t*>(is_k ? a.c.k : a.c.v) +
                        cache_row(a.c, slot, head, D);
        reinterpret_cast<uint4*>(dst)[j] = pack8(x);
      }
    }
  }
}

// k_cache_read: one thread per 8 values of a (token, head), keys and values.
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

template <int D, int kCache, bool kTurn>
cudaError_t start_rows(const RowsProblem& p, const CacheView* c, cudaStream_t s) {
  RowsArgs a{};
  a.p = p;
  if (c) a.c = *c;
  const int heads = p.Hq + (c ? 2 : 1) * p.Hkv;
  // Few tokens: a row per group of lanes, so that the call is one short wave. Many: a token's
  // heads share its angles, as long as every SM keeps its lanes busy.
  const int64_t groups = (int64_t)device_sm_count() * 2048 / (D / 8);
  int64_t chunks = (groups + p.T - 1) / p.T;
  chunks = chunks > heads ? heads : chunks;
  a.per_chunk = (int)((heads + chunks - 1) / chunks);
  a.chunks = (heads + a.per_chunk - 1) / a.per_chunk;
  const int64_t threads = (int64_t)p.T * a.chunks * (D / 8);
  const int64_t grid = (threads + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(k_rows<D, kCache, kTurn>, dim3((unsigned)grid), kThreads, 0, s, a);
}

template <int D>
cudaError_t pick_rows(const RowsProblem& p, const CacheView* c, cudaStream_t s) {
  if (p.Hq == 0) return c->q8 ? start_rows<D, 2, false>(p, c, s) : start_rows<D, 1, false>(p, c, s);
  if (!c) return start_rows<D, 0, true>(p, c, s);
  return c->q8 ? start_rows<D, 2, true>(p, c, s) : start_rows<D, 1, true>(p, c, s);
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
