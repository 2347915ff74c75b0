// paged_few.cu — attention over the paged cache for up to 32 query rows per key head (plain
// decode steps, and verify steps of models with few heads per key head).
//
// The list of tiles, its division among the CTAs and the partial results are those of
// paged_attn.cu. Here each of the four warps works alone on its 16 tokens of every tile: it
// fetches them into a ring of its own, scores them, and adds them to its own maximum,
// normaliser and sums over all D values of the head, so nothing is exchanged and no warp waits
// for another until the (sequence, key head) ends and the four are added up.
//
// The products are turned over: S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16), with tokens
// and values along the 16 and query rows along the 8, so that 1 to 8 rows cost one tile, 17 to
// 24 three. P^T comes out of the first product with a token per group of four lanes and goes
// into the second with a query row per group: movmatrix turns each 8 x 8 tile over in registers.
// Codes of a Q8 cache are widened exactly to bf16; the key's scale multiplies the score, the
// value's scale P, and P enters as a high and a low bf16 part (relative error 2^-17). The
// reference of a row moves only when a score exceeds it by 2^8.
//
// Measured on 32 sequences x 8 heads of 8k tokens, D = 128: bf16 (1.05 GB) 160 us for 1 to 8
// rows, 6.6 TB/s, bound by memory, and 176 us for 32 rows; Q8 (0.54 GB) 102, 127, 160 and 198 us
// for 8, 16, 24 and 32 rows, bound by the latency of dependent instructions (700 per 16 tokens and
// warp at 16 rows, of which 224 widen codes and 48 are products; at 24 rows, with two warps per
// scheduler, 47% of the issue slots are used). A single head of 500 tokens: 6.4 us, of which
// launching the two kernels is most.
#include <type_traits>

#include "paged.cuh"

namespace dsmoe {
namespace paged {
namespace {

constexpr int kTile = 64, kWarps = 4, kTok = kTile / kWarps;

// Turns an 8 x 8 tile of 16-bit values over: lane 4 i + j has values 2 j, 2 j + 1 of row i.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Shapes of one instantiation: NT tiles of 8 query rows.
template <int D, bool kQ8, int NT>
struct Few {
  static constexpr int kRows = 8 * NT;
  static constexpr int RB = D * (kQ8 ? 1 : 2);   // bytes of a cached row
  static constexpr int kMat = kTok * RB;
  static constexpr int kStage = 2 * kMat + (kQ8 ? 2 * kTok * 4 : 0);
  static constexpr int kPart = kQ8 || NT <= 2 ? D : 64;   // values that are added up at a time
  // The next queries wait in registers while results are added up, where the loop has the
  // registers for it: Q8, 24 rows 158 against 163 us, but 32 rows 222 against 196.
  static constexpr bool kHold = NT % 2 == 1;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSum = kRows * kPart * 4;
  static constexpr int kStat = kWarps * kRows * 4;
  static constexpr int kFixed = kQ + kSum + 2 * kStat;
  // CTAs per SM. Three leave 168 registers a thread and room for fewer stages. On the case at
  // the top of this file, three against two: Q8, D = 128, 8 rows 104 against 115 us, 16 rows 127
  // against 140, 24 rows 177 against 167, 32 rows (spilled) 445 against 197; bf16, 8 rows 195
  // (two stages) against 161; D = 64 Q8, 8 rows 71 against 100, 32 rows 132 against 133, bf16 32
  // rows 113 against 124.
  static constexpr int kPerSm = D == 64 || (kQ8 && NT <= 2) ? 3 : 2;
  static constexpr int kFit = (228 * 1024 / kPerSm - 1024 - kFixed) / (kWarps * kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kFixed + kWarps * kStages * kStage;
  static_assert(kStages >= 2, "a ring of at least two stages");
};

template <int D, bool kQ8, int NT>
__global__ void __launch_bounds__(32 * kWarps, (Few<D, kQ8, NT>::kPerSm))
    k_paged_few(const __grid_constant__ PagedArgs a) {
  using C = Few<D, kQ8, NT>;
  constexpr int RB = C::RB, S = C::kStages, DT = D / 16;
  extern __shared__ __align__(128) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  uint8_t* const ring = sm + warp * S * C::kStage;
  uint8_t* const sQ = sm + kWarps * S * C::kStage;
  float* const sum = reinterpret_cast<float*>(sQ + C::kQ);          // [row][kPart]
  float* const top_s = reinterpret_cast<float*>(sQ + C::kQ + C::kSum);   // [warp][row]
  float* const norm_s = top_s + kWarps * C::kRows;
  pdl_wait();

  if (blockIdx.x == 0 && tid == 0) *a.status = 0u;
  if (a.pieces && tid == 0) began(a);
  Cursor cur{};
  const int n = cta_run(a, blockIdx.x, lane, &cur);   // tiles of this CTA
  if (n == 0) return;

  // ---------------------------------------------------------------- this warp's loads ------
  // Its tokens of a tile lie in one page; where they start is looked up a tile ahead (in
  // values; -1: nowhere, there are none or the table's entry is bad).
  Cursor ahead = cur;
  const int page_mask = (1 << a.c.page_shift) - 1;
  int64_t run_at, run_scale = 0;
  auto look_up = [&] {
    const int t = ahead.tile * kTile + kTok * warp, page = page_of(a, ahead.b, t, ahead.len);
    const int64_t in_page = ((int64_t)ahead.h << a.c.page_shift) + (t & page_mask);
    run_at = page < 0 ? -1 : page * a.c.stride + in_page * D;
    if (kQ8) run_scale = page * a.c.scale_stride + in_page;
  };
  constexpr int kChunks = RB / 16, kStep = 32 / kChunks;   // rows per copy instruction
  const int my_row = lane / kChunks, my_chunk = lane % kChunks;
  const uint32_t my_dst = swz<RB>(my_row, my_chunk);
  static_assert(C::kStage % 128 == 0 && (RB != 64 || kStep % 8 == 0), "see the swizzle below");
  int fetched = 0, stage_in = 0;
  uint32_t have = 0;   // stages that hold tokens
  auto fetch = [&] {
    if (fetched < n) {
      have &= ~(1u << stage_in);
      if (run_at >= 0) {
        have |= 1u << stage_in;
        const int left = ahead.len - ahead.tile * kTile - kTok * warp;
        const int64_t off = (run_at + my_row * D) * (kQ8 ? 1 : 2) + my_chunk * 16;
        const uint8_t* const kp = a.c.k + off;
        const uint8_t* const vp = a.c.v + off;
        const int mine = left - my_row;
        const uint32_t dst = smem_at(ring + stage_in * C::kStage);
        // row it * kStep + my_row: the swizzle of it * kStep and that of my_row share no bits
#pragma unroll
        for (int it = 0; it < kTok / kStep; ++it) {
          constexpr int kTurn = RB == 64 ? 0 : 7;
          const uint32_t to = ((dst + my_dst) ^ ((it * kStep & kTurn) << 4)) + it * kStep * RB;
          const bool there = it * kStep < mine;
          cp_async16(to, kp + it * kStep * RB, there);
          cp_async16(to + C::kMat, vp + it * kStep * RB, there);
        }
        if (kQ8 && lane < 8) {   // 4 scales per copy: 16 of the keys, 16 of the values
          const int r = 4 * (lane & 3);
          cp_async16(dst + 2 * C::kMat + 16 * lane,
                     (lane < 4 ? a.c.k_scale : a.c.v_scale) + run_scale + r, r < left);
        }
      }
      if (++fetched < n) {
        ahead.next(a);
        look_up();
      }
    }
    cp_async_commit();
    stage_in = stage_in + 1 == S ? 0 : stage_in + 1;
  };
  look_up();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch();

  // The queries of a (sequence, key head): to registers, then to shared memory. Rows behind M
  // are zero. For a Q8 cache the 16 values of a step are stored even ones first, the order in
  // which codes are widened.
  constexpr int kPairs = D / 16, kLoads = (C::kRows * kPairs + 32 * kWarps - 1) / (32 * kWarps);
  uint4 next_q[kLoads][2];
  auto load_queries = [&](const Cursor& at) {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int idx = x * 32 * kWarps + tid, r = idx / kPairs, pr = idx % kPairs;
      next_q[x][0] = next_q[x][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < a.M) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (((int64_t)at.b * a.R + r / a.G) * a.Hq + at.h * a.G + r % a.G) * D) + 2 * pr;
        next_q[x][0] = src[0];
        next_q[x][1] = src[1];
      }
    }
  };
  auto store_queries = [&] {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int idx = x * 32 * kWarps + tid, r = idx / kPairs, pr = idx % kPairs;
      if (r >= C::kRows) continue;
      uint4 x0 = next_q[x][0], x1 = next_q[x][1];
      if constexpr (kQ8) {
        const uint4 e0 = make_uint4(
            __byte_perm(x0.x, x0.y, 0x5410), __byte_perm(x0.z, x0.w, 0x5410),
            __byte_perm(x1.x, x1.y, 0x5410), __byte_perm(x1.z, x1.w, 0x5410));
        x1 = make_uint4(__byte_perm(x0.x, x0.y, 0x7632), __byte_perm(x0.z, x0.w, 0x7632),
                        __byte_perm(x1.x, x1.y, 0x7632), __byte_perm(x1.z, x1.w, 0x7632));
        x0 = e0;
      }
      *reinterpret_cast<uint4*>(sQ + swz<2 * D>(r, 2 * pr)) = x0;
      *reinterpret_cast<uint4*>(sQ + swz<2 * D>(r, 2 * pr + 1)) = x1;
    }
  };
  load_queries(cur);
  store_queries();
  __syncthreads();

  int rr[NT][2];   // verify row of this lane's query rows 8 nt + 2 q + e
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) rr[nt][e] = (8 * nt + 2 * q + e) / a.G;

  // per query row: the reference (log2), what a score may be before it has to move (-infinity:
  // nothing seen yet), the lanes' shares of the normaliser, and the sums
  float m[NT][2], lim[NT][2], l[NT][2], o[DT][NT][4];
  bool starts = true;
  int stage = 0;
  for (int i = 0; i < n; ++i) {
    if (starts) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = 0.f;
        lim[nt][0] = lim[nt][1] = kNegInf;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
          o[dt][nt][0] = o[dt][nt][1] = o[dt][nt][2] = o[dt][nt][3] = 0.f;
      }
    }
    cp_async_wait<S - 2>();
    __syncwarp();   // the tokens are there; every lane is done with the stage before
    const bool some = have >> stage & 1;
    fetch();
    if (some) {
      const uint32_t kb = smem_at(ring + stage * C::kStage), vb = kb + C::kMat;
      const uint32_t qb = smem_at(sQ);
      const int t0 = cur.tile * kTile + kTok * warp;
      const int seen0 = cur.len - (a.R - 1);   // row r sees t < seen0 + r
      // -------------------------------------------------------- S^T = K Q^T ------------
      // (few rows: even and odd steps in accumulators of their own, for shorter chains)
      constexpr int kSets = NT <= 2 || D == 64 ? 2 : 1;
      float s[NT][4], s_odd[kSets == 2 ? NT : 1][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = 0.f;
          if constexpr (kSets == 2) s_odd[nt][e] = 0.f;
        }
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        uint32_t kf[2][4];   // two steps of 16 values
        const int row = lane & 15, half = lane >> 4;
        if constexpr (kQ8) {
          uint32_t w[4];
          ldsm_x4(kb + swz<RB>(row, 2 * kk + half), w);
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            kf[st][0] = code_pair(w[2 * st]);
            kf[st][1] = code_pair(w[2 * st + 1]);
            kf[st][2] = code_pair(w[2 * st] >> 8);
            kf[st][3] = code_pair(w[2 * st + 1] >> 8);
          }
        } else {
#pragma unroll
          for (int st = 0; st < 2; ++st) ldsm_x4(kb + swz<RB>(row, 4 * kk + 2 * st + half), kf[st]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t qf[4];
          ldsm_x4(qb + swz<2 * D>(8 * nt + (lane & 7), 4 * kk + (lane >> 3)), qf);
          mma16816(s[nt], kf[0], qf[0], qf[1]);
          if constexpr (kSets == 2)
            mma16816(s_odd[nt], kf[1], qf[2], qf[3]);
          else
            mma16816(s[nt], kf[1], qf[2], qf[3]);
        }
      }
      if constexpr (kSets == 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = __fadd_rn(s[nt][e], s_odd[nt][e]);
      }
      // ---------------------------------------------- scale, mask, P = 2^(S - m) --------
      // this lane: tokens g (s[.][0, 1]) and g + 8 (2, 3), query rows 8 nt + 2 q and the next
      float f[2] = {a.scale_log2, a.scale_log2}, vs[2] = {1.f, 1.f};
      if constexpr (kQ8) {
        const float* sc = reinterpret_cast<const float*>(ring + stage * C::kStage + 2 * C::kMat);
        f[0] = __fmul_rn(f[0], sc[g]);
        f[1] = __fmul_rn(f[1], sc[g + 8]);
        vs[0] = sc[kTok + g];
        vs[1] = sc[kTok + g + 8];
      }
      bool over = false;
      const bool edge = t0 + kTok > seen0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = __fmul_rn(s[nt][e], f[e >> 1]);
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (t0 + g + 8 * (e >> 1) >= seen0 + rr[nt][e & 1]) s[nt][e] = kNegInf;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          over |= fmaxf(s[nt][e], s[nt][2 + e]) > lim[nt][e];
      }
      if (__any_sync(0xffffffffu, over)) {   // some row's reference moves
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[nt][e], s[nt][2 + e]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            // up to the row's largest score so far, or down to the first ones
            const bool first = lim[nt][e] == kNegInf;
            const float now = first ? (x == kNegInf ? 0.f : x) : fmaxf(x, m[nt][e]);
            const float c = first ? 0.f : exp2_fast(__fsub_rn(m[nt][e], now));
            m[nt][e] = now;
            if (x > kNegInf) lim[nt][e] = __fadd_rn(now, kSlack);
            l[nt][e] = __fmul_rn(l[nt][e], c);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
              o[dt][nt][e] = __fmul_rn(o[dt][nt][e], c);
              o[dt][nt][2 + e] = __fmul_rn(o[dt][nt][2 + e], c);
            }
          }
      }
      uint32_t hi[NT][2], lo[NT][2];   // [tokens g, g + 8]: P of the two rows, then turned over
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float p0 = exp2_fast(__fsub_rn(s[nt][2 * h], m[nt][0]));
          float p1 = exp2_fast(__fsub_rn(s[nt][2 * h + 1], m[nt][1]));
          l[nt][0] = __fadd_rn(l[nt][0], p0);
          l[nt][1] = __fadd_rn(l[nt][1], p1);
          if constexpr (kQ8) {
            p0 = __fmul_rn(p0, vs[h]);
            p1 = __fmul_rn(p1, vs[h]);
            if (edge) {   // a masked token's scale may be anything
              p0 = s[nt][2 * h] == kNegInf ? 0.f : p0;
              p1 = s[nt][2 * h + 1] == kNegInf ? 0.f : p1;
            }
          }
          hi[nt][h] = pack2(p0, p1);
          lo[nt][h] = pack2(__fsub_rn(p0, bf16_lo(hi[nt][h])), __fsub_rn(p1, bf16_hi(hi[nt][h])));
        }
      }
      // -------------------------------------------------------- O^T += V^T P^T ----------
      // A bf16 value that only some rows see may hold anything, and 0 x infinity is not 0: where
      // the (at most 7) tokens from seen0 on have such values, they are left out of the product
      // and added row by row.
      bool apart = false;
      if (!kQ8 && a.R > 1 && edge) {
        const uint8_t* const values = ring + stage * C::kStage + C::kMat;
        const int first = seen0 > t0 ? seen0 - t0 : 0;
        const int last = cur.len - t0 < kTok ? cur.len - t0 : kTok;
        for (int x = first * (RB / 16) + lane; x < last * (RB / 16); x += 32) {
          const uint4 v = *reinterpret_cast<const uint4*>(values + 16 * x);   // (swizzled in a row)
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int y = 0; y < 4; ++y)
            apart |= (w[y] & 0x7F80u) == 0x7F80u || (w[y] & 0x7F800000u) == 0x7F800000u;
        }
        apart = __any_sync(0xffffffffu, apart);
        for (int t = apart ? first : last; t < last; ++t) {
          const int from = 4 * (t & 7) + q;
          float v[DT][2];
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              v[dt][h] = bf16_bits_to_f32(
                  *reinterpret_cast<const uint16_t*>(values + swz<RB>(t, 2 * dt + h) + 2 * g));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t ph = __shfl_sync(0xffffffffu, t < 8 ? hi[nt][0] : hi[nt][1], from);
            const uint32_t pl = __shfl_sync(0xffffffffu, t < 8 ? lo[nt][0] : lo[nt][1], from);
            const float p[2] = {__fadd_rn(bf16_lo(ph), bf16_lo(pl)),
                                __fadd_rn(bf16_hi(ph), bf16_hi(pl))};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (t0 + t >= seen0 + rr[nt][e]) continue;
#pragma unroll
              for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  o[dt][nt][2 * h + e] = __fmaf_rn(p[e], v[dt][h], o[dt][nt][2 * h + e]);
            }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          hi[nt][h] = turned(hi[nt][h]);
          lo[nt][h] = turned(lo[nt][h]);
        }
      // (two tiles of 16 values at a time, so that no product waits for the one before)
      const int row = kQ8 ? lane & 15 : (lane & 7) + 8 * (lane >> 4);
      const int half = kQ8 ? lane >> 4 : lane >> 3 & 1;
      const int t = t0 + 2 * q;
      const uint32_t k0 = (t < seen0 ? 0xFFFFu : 0u) | (t + 1 < seen0 ? 0xFFFF0000u : 0u);
      const uint32_t k1 = (t + 8 < seen0 ? 0xFFFFu : 0u) | (t + 9 < seen0 ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int dp = 0; dp < DT / 2; ++dp) {
        uint32_t vf[2][4];
        if constexpr (kQ8) {   // 16 codes per chunk: the even ones are the tile's first 8
          uint32_t w[4];
          ldsm_x4_t(vb + swz<RB>(row, 2 * dp + half), w);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            vf[x][0] = code_pair(w[2 * x]);
            vf[x][1] = code_pair(w[2 * x] >> 8);
            vf[x][2] = code_pair(w[2 * x + 1]);
            vf[x][3] = code_pair(w[2 * x + 1] >> 8);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ldsm_x4_t(vb + swz<RB>(row, 4 * dp + 2 * x + half), vf[x]);
            if (apart) vf[x][0] &= k0, vf[x][1] &= k0, vf[x][2] &= k1, vf[x][3] &= k1;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[2 * dp + x][nt], vf[x], hi[nt][0], hi[nt][1]);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[2 * dp + x][nt], vf[x], lo[nt][0], lo[nt][1]);
      }
    }
    stage = stage + 1 == S ? 0 : stage + 1;
    // --------------------------------------- the end of this run of the (sequence, head)
    const bool whole_end = cur.tile + 1 == cur.tiles;
    starts = whole_end || i + 1 == n;
    if (starts) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = l[nt][e];
          v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 16));
          if (g == 0) {
            top_s[warp * C::kRows + 8 * nt + 2 * q + e] = lim[nt][e] == kNegInf ? kNegInf : m[nt][e];
            norm_s[warp * C::kRows + 8 * nt + 2 * q + e] = v;
          }
        }
      __syncthreads();   // (and no warp needs this run's queries any more)
      const Cursor here = cur;
      if (i + 1 < n) {
        cur.next(a);
        load_queries(cur);
        if (!C::kHold) store_queries();
      }
      auto top_of = [&](int row) {
        return fmaxf(fmaxf(top_s[row], top_s[C::kRows + row]),
                     fmaxf(top_s[2 * C::kRows + row], top_s[3 * C::kRows + row]));
      };
      const int run = i < here.tile ? i : here.tile;   // tiles before this one in it
      const bool all = whole_end && here.tile == run, whole = all && !a.pieces;
      const int64_t slot = piece_at(a, here.b, here.h, here.tile == run, all);
      if (tid == 0) note_span(a, here, here.tile == run, whole_end);
      if (tid < a.M) {
        const float top = top_of(tid);
        float norm = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float t = top_s[w * C::kRows + tid];
          norm = __fmaf_rn(norm_s[w * C::kRows + tid],
                           t == kNegInf ? 0.f : exp2_fast(__fsub_rn(t, top)), norm);
        }
        norm_s[tid] = norm;   // (in place of what only this thread reads)
        norm_s[C::kRows + tid] = __frcp_rn(norm);
        if (!whole)
          *reinterpret_cast<float2*>(a.part_ml + 2 * (slot * a.M + tid)) = make_float2(top, norm);
      }
      float c[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          c[nt][e] = lim[nt][e] == kNegInf
                         ? 0.f
                         : exp2_fast(__fsub_rn(m[nt][e], top_of(8 * nt + 2 * q + e)));
#pragma unroll
      for (int part = 0; part < D / C::kPart; ++part) {
        // four rounds: in each, every warp adds a quarter of its sums to the common ones, always
        // in the same order (places of a row are turned so that no two lanes meet in a bank)
        constexpr int kTiles = C::kPart / 64;   // tiles of 16 values in a quarter
#pragma unroll 1
        for (int round = 0; round < kWarps; ++round) {
          const int x = (warp + round) & 3;
#pragma unroll
          for (int y = 0; y < kTiles; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int d0 = 4 * kTiles * part + y;
                const float lower = x & 1 ? o[d0 + kTiles][nt][e] : o[d0][nt][e];
                const float upper = x & 1 ? o[d0 + 3 * kTiles][nt][e] : o[d0 + 2 * kTiles][nt][e];
                const float v = __fmul_rn(x & 2 ? upper : lower, c[nt][e & 1]);
                float* to = sum + (8 * nt + 2 * q + (e & 1)) * C::kPart +
                            ((16 * (kTiles * x + y) + g + 8 * (e >> 1)) ^ (8 * q));
                *to = round == 0 ? v : __fadd_rn(*to, v);
              }
          __syncthreads();
        }
        if (C::kHold && part == 0) store_queries();
        for (int idx = tid; idx < a.M * (C::kPart / 2); idx += 32 * kWarps) {
          const int row = idx / (C::kPart / 2), d = 2 * (idx % (C::kPart / 2));
          const int p0 = kQ8 ? (d & ~15) + (d & 15) / 2 : d, p1 = kQ8 ? p0 + 8 : d + 1;
          const float* from = sum + row * C::kPart;
          const int turn = 8 * ((row >> 1) & 3);
          const float y0 = from[p0 ^ turn], y1 = from[p1 ^ turn];
          const int at = C::kPart * part + d;
          if (whole) {
            const float norm = norm_s[row], inv = norm_s[C::kRows + row];
            *reinterpret_cast<uint32_t*>(
                a.out +
                (((int64_t)here.b * a.R + row / a.G) * a.Hq + here.h * a.G + row % a.G) * D + at) =
                norm == 0.f ? 0u : pack2(__fmul_rn(y0, inv), __fmul_rn(y1, inv));   // 0: sees nothing
          } else {
            *reinterpret_cast<float2*>(a.part_o + (slot * a.M + row) * D + at) = make_float2(y0, y1);
          }
        }
        __syncthreads();   // sums and statistics may be overwritten; the next queries are there
      }
    } else {
      cur.next(a);
    }
  }
  cp_async_wait<0>();
}

// Calls f with the number of 8-row tiles.
template <typename F>
auto with_tiles(int M, F&& f) {
  if (M <= 8) return f(std::integral_constant<int, 1>{});
  if (M <= 16) return f(std::integral_constant<int, 2>{});
  if (M <= 24) return f(std::integral_constant<int, 3>{});
  return f(std::integral_constant<int, 4>{});
}

template <int D, bool kQ8>
cudaError_t launch(const PagedArgs& a, cudaStream_t s) {
  return with_tiles(a.M, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    using C = Few<D, kQ8, NT>;
    static OncePerDevice ready;
    const cudaError_t e = ready.run([&] {
      return cudaFuncSetAttribute(k_paged_few<D, kQ8, NT>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(k_paged_few<D, kQ8, NT>, dim3(a.grid), 32 * kWarps, C::kSmem, s, a);
  });
}

}  // namespace

int few_ctas_per_sm(int M, int D, bool q8) {
  return with_tiles(M, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if (D == 128) return q8 ? Few<128, true, NT>::kPerSm : Few<128, false, NT>::kPerSm;
    return q8 ? Few<64, true, NT>::kPerSm : Few<64, false, NT>::kPerSm;
  });
}

cudaError_t launch_few(const PagedArgs& p, int D, cudaStream_t s) {
  if (D == 128) return p.c.q8 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return p.c.q8 ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace paged
}  // namespace dsmoe
