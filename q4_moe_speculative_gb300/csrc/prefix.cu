// prefix.cu — attention of sequences that share prefixes (arithmetic in include/dsmoe.h): every
// prefix is read once for all its sequences.
//
// Three kernels. The sequences' own tokens go through the kernels of the paged attention, which leave
// their maxima, normalisers and sums in the workspace (paged_attn.cu). k_prefix_tc (prefix_tc.cu) does
// the same for the rows of all of a prefix's sequences together over its tokens. k_prefix_join
// merges both per row, in a fixed order. The second starts as the first's CTAs leave, the third as the
// second's do. Measured: 64 sequences x 6 rows, 32 heads on 8, with up to 512 tokens of their own after
// 16k 136 us, of which the second 109; with 6 after 16k 123, after 128 30 (14, 8 and 8); 16 x 1
// rows, 16 heads on one, after 100k 35 us.
#include "prefix.cuh"

namespace dsmoe {
namespace {

using namespace prefix;

// k_prefix_join: kWarps warps per row of the result (one head of one new token); with 1, a row for
// each of 8 warps. 32 pieces at a time: a lane looks one up, and the warp adds up those there are,
// four at a time, each lane D / 32 of the values. Its time is latency (8 us for 12,288 rows of 4
// pieces, which are in L2): where rows are few and pieces many, 8 warps, with registers for what they
// have on their way (56; with 32 the 100k tokens below took 38 instead of 34 us).
template <int D, int kWarps>
__global__ void __launch_bounds__(256, kWarps == 1 ? 6 : 4) k_prefix_join(const __grid_constant__ PrefixArgs a) {
  constexpr int V = D / 32;
  __shared__ float acc_s[kWarps][D];
  __shared__ float2 l_s[kWarps];
  const PagedArgs& o = a.own;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row64 = kWarps > 1 ? blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
  if (row64 >= (int64_t)o.B * o.R * o.Hq) return;
  const unsigned row = (unsigned)row64;   // (4096 sequences x 128 rows x 256 heads: below 2^32)
  const unsigned hq = row % o.Hq, br = row / o.Hq, h = hq / o.G;
  const unsigned b = br / o.R, m = br % o.R * o.G + hq % o.G;
  uint16_t* const dst = o.out + row64 * D + V * lane;
  // the pieces of the prefix: of the CTAs that share the row's unit, one or two (its streams) of each
  const unsigned p = b / a.per, mp = (b % a.per) * o.M + m, u = mp / (2 * kRows);
  const int w = unit_tiles(a, u), subs = w == 2 ? 1 : 2;
  const int sub0 = w == 2 ? mp / kRows % 2 : 0;
  const int unit = (p * o.c.heads + h) * a.units + u;
  pdl_wait();
  if (row64 == 0 && lane == 0) *o.ready = 0ull;   // (no prefix kernel of this call looks any more)
  const int own_len = o.lengths[b], prefix_tokens = prefix_len(a, p);
  const int2 first = __ldcg(reinterpret_cast<const int2*>(a.span) + unit);
  // and those of its own tokens
  const unsigned bh = b * o.c.heads + h;
  const int2 span = __ldcg(reinterpret_cast<const int2*>(o.span) + bh);
  const bool absent = own_len < 0;
  // (spans that were not noted: the kernel gave up, and the status says so)
  const bool has_prefix = !absent && prefix_tokens > 0 && first.x >= 0 && first.y >= first.x &&
                          first.y < a.grid;
  const bool has_own = own_len > 0 && span.x >= 0 && span.y >= span.x && span.y < o.grid;
  const int n_prefix = has_prefix ? (first.y - first.x + 1) * subs : 0;
  const int n_all = n_prefix + (has_own ? span.y - span.x + 1 : 0);

  float top = kNegInf, norm = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int i0 = kWarps > 1 ? warp : 0; i0 < n_all; i0 += 32 * kWarps) {
    const int i = i0 + kWarps * lane;
    float2 ml = make_float2(kNegInf, 0.f);
    const float* from = a.part_o;
    if (i < n_prefix) {
      const int c = first.x + (subs == 2 ? i >> 1 : i), sub = subs == 2 ? i & 1 : sub0;
      const int64_t at = ((int64_t)(unit + c) * 2 + sub) * a.rows + mp % kRows;
      ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at);
      from = a.part_o + at * D;
    } else if (i < n_all) {
      const int c = span.x + i - n_prefix;
      const int64_t piece = span.x == span.y ? 2 * (int64_t)o.grid + bh
                                             : 2 * (int64_t)c + (c == span.x ? 1 : 0);
      const int64_t at = piece * o.M + m;
      ml = __ldcg(reinterpret_cast<const float2*>(o.part_ml) + at);
      from = o.part_o + at * D;
    }
    float now = ml.x;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, x));
    now = fmaxf(now, top);
    const float f = top == kNegInf ? 0.f : exp2_fast(__fsub_rn(top, now));
    const bool has = ml.x != kNegInf;
    const float g = has ? exp2_fast(__fsub_rn(ml.x, now)) : 0.f;
    top = now;
    float part = has ? __fmul_rn(g, ml.y) : 0.f;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) part = __fadd_rn(part, __shfl_xor_sync(0xffffffffu, part, x));
    norm = __fmaf_rn(norm, f, part);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __fmul_rn(acc[e], f);
    unsigned left = __ballot_sync(0xffffffffu, has);
    while (left) {
      float x[4][V], gx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int l = left ? __ffs(left) - 1 : -1;
        left &= left - 1;
        gx[j] = __shfl_sync(0xffffffffu, g, l < 0 ? 0 : l);
        const float* const at = reinterpret_cast<const float*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(from), l < 0 ? 0 : l));
#pragma unroll
        for (int e = 0; e < V; ++e) x[j][e] = 0.f;
        if (l < 0) continue;
        if constexpr (V == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(at) + lane);
          x[j][0] = v.x, x[j][1] = v.y, x[j][2] = v.z, x[j][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(at) + lane);
          x[j][0] = v.x, x[j][1] = v.y;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(x[j][e], gx[j], acc[e]);
    }
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc_s[warp][V * lane + e] = acc[e];
    if (lane == 0) l_s[warp] = make_float2(top, norm);
    __syncthreads();
    if (warp) return;
    for (int x = 1; x < kWarps; ++x) top = fmaxf(top, l_s[x].x);
    norm = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    for (int x = 0; x < kWarps; ++x) {
      const float2 l = l_s[x];
      if (l.x == kNegInf) continue;
      const float g = exp2_fast(__fsub_rn(l.x, top));
      norm = __fmaf_rn(l.y, g, norm);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(acc_s[x][V * lane + e], g, acc[e]);
    }
  }
  float y[V];
#pragma unroll
  for (int e = 0; e < V; ++e)
    y[e] = absent || norm == 0.f ? 0.f : __fdiv_rn(acc[e], norm);
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2(y[0], y[1]);
}

struct Plan {
  int grid;
  int64_t pieces;
  size_t span, ml, po, total;
};

Plan make_plan(const PrefixAttnProblem& p, PrefixArgs* a) {
  a->P = p.P;
  a->per = p.own.B / p.P;
  const int M = p.own.R * (p.own.Hq / p.own.cache.heads);
  a->MP = a->per * M;
  a->tiles = (a->MP + kRows - 1) / kRows;
  a->units = (a->tiles + 1) / 2;
  a->rows = a->MP < kRows ? a->MP : kRows;
  a->m_inverse = (uint32_t)((((uint64_t)1 << 32) + M - 1) / M);
  a->max_pages = p.max_pages;
  const int64_t cap = ((int64_t)p.max_pages << p.own.cache.page_shift), T = (cap + kTok - 1) / kTok;
  const int64_t heads = (int64_t)p.P * p.own.cache.heads;
  const int64_t most = heads * (a->tiles * T + (int64_t)a->units * kBegin);
  const int64_t sms = device_sm_count();
  Plan pl{};
  pl.grid = (int)(most < sms ? most : sms);
  pl.pieces = heads * a->units + pl.grid;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl.span = up(pieces_workspace(p.own));
  pl.ml = pl.span + up((size_t)heads * a->units * 2 * sizeof(int));
  pl.po = pl.ml + up((size_t)pl.pieces * 2 * a->rows * 2 * sizeof(float));
  pl.total = pl.po + up((size_t)pl.pieces * 2 * a->rows * p.own.D * sizeof(float));
  return pl;
}

template <int D>
cudaError_t join(const PrefixArgs& a, int64_t units, cudaStream_t s) {
  const int64_t rows = (int64_t)a.own.B * a.own.R * a.own.Hq;
  // Eight warps where rows are few and their pieces many: at least 12 CTAs that share a unit, and at
  // most 12 rows per SM. With 152 CTAs (100k tokens for 16 rows of a head) 34 us against 76 with one
  // warp, with 19 and 512 rows of the result 21.5 against 32, with 1536 rows 29.8 against 30.8; with
  // 19 and 1920 rows 32.0 against 31.6, with 12.7 and 3072 39.6 against 33.4, with 9.5 38.9
  // against 35.0.
  if (a.grid >= 12 * units && rows <= 12 * a.grid)
    return launch_pdl(k_prefix_join<D, 8>, dim3((unsigned)rows), 256, 0, s, a);
  return launch_pdl(k_prefix_join<D, 1>, dim3((unsigned)((rows + 7) / 8)), 256, 0, s, a);
}

}  // namespace

size_t prefix_attn_workspace(const PrefixAttnProblem& p) {
  PrefixArgs a{};
  return make_plan(p, &a).total;
}

cudaError_t launch_prefix_attn(const PrefixAttnProblem& p, uint8_t* ws, cudaStream_t s) {
  PrefixArgs a{};
  const Plan pl = make_plan(p, &a);
  a.table = p.table;
  a.lengths = p.lengths;
  a.grid = pl.grid;
  a.span = reinterpret_cast<int*>(ws + pl.span);
  a.part_ml = reinterpret_cast<float*>(ws + pl.ml);
  a.part_o = reinterpret_cast<float*>(ws + pl.po);
  cudaError_t e = launch_pieces(p.own, ws, s, &a.own);   // (it clears the status word)
  if (e != cudaSuccess) return e;
  e = launch_prefix_tc(a, p.own.D, s);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.P * a.own.c.heads * a.units;
  return p.own.D == 128 ? join<128>(a, units, s) : join<64>(a, units, s);
}

}  // namespace dsmoe
