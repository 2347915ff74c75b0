// paged_attn.cu — attention of each sequence's last R tokens over its paged key-value cache
// (arithmetic in include/dsmoe.h): a plain decode step for R = 1, a verify step for R <= 8.
//
// All query rows of one key head, M = R x heads per key head (row m = r * G + j), read the
// same keys and values, so they are the M dimension of one problem whose cost is the bytes
// of the cache. Tokens come in tiles. The tiles of all sequences and key heads form one list
// that is cut into equal runs, one per CTA: a long sequence is split over many CTAs, a batch
// of ragged ones is balanced, and no CTA waits for another. A (sequence, head) that lies
// inside one run is finished there; one that crosses a boundary leaves its running maximum,
// normaliser and sums per CTA in the workspace, and k_paged_join merges those in CTA order, so
// results do not depend on timing.
//
// Three kernels do the runs: paged_few.cu up to 32 rows, k_paged here for more, paged_tc.cu
// for 25 rows and more of long contexts (rules and figures at which()). None of them lets the next
// kernel start early: waiting CTAs of the join took room from this kernel's and of the next
// kernel from the join's (16 rows, 8 sequences x 8 heads at 4k, Q8: 32 against 27 us).
//
// k_paged (8 warps, one CTA per SM): tiles of 64 tokens are copied by cp.async into a ring of
// stages (rows swizzled in 16-byte chunks, so that ldmatrix is free of bank conflicts). Per
// tile, warp w of each group of four scores tokens 16 w .. 16 w + 15 for its group's rows
// (S = Q K^T, mma.sync m16n8k16), P = 2^(S - m) goes to shared memory as bf16, and then the
// warp accumulates its quarter of the head's values for all 64 tokens (O += P V): a key or
// value byte is read from shared memory (and an int8 one widened) once per group, and the
// accumulators are a quarter of M x D per warp. Codes of a Q8 cache are widened exactly to
// bf16; the key's scale multiplies the score, the value's scale P. The reference m of a row
// moves only when a score exceeds it by 2^8 (P stays in range and bf16's relative precision
// does not depend on it), so the usual tile needs no exchange of maxima and no rescaling: the
// CTA votes on it at the barrier that publishes P anyway. P (with a Q8 cache the value's scale is
// in it) goes in as a high and a low bf16 part, off by 2^-16 relative; rounded once it would be
// off by 2^-8, and a result by 1.4 times its own rounding, for 52 instead of 60 us below. Its
// bound is the issue of instructions: 4 sequences x 8 heads of 8k tokens, 64 rows, 60 us for 132
// MB of bf16 as for 68 MB of Q8.
#include <type_traits>

#include "paged.cuh"

namespace dsmoe {
namespace {

using namespace paged;

constexpr int kTile = 64;

// Shapes of one instantiation: MT m16 tiles of rows per warp, two groups of four warps.
template <int D, bool kQ8, int MT>
struct Shape {
  static constexpr int kThreads = 256;
  static constexpr int kRows = 32 * MT;
  static constexpr int RB = D * (kQ8 ? 1 : 2);          // bytes of a cached row
  static constexpr int kMat = kTile * RB;
  static constexpr int kStage = 2 * kMat + (kQ8 ? 2 * kTile * 4 : 0);
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kP = kRows * kTile * 2;          // one of the two parts of P
  static constexpr int kRed = 4 * kRows * 4;
  static constexpr int kFixed = kQ + 2 * kP + kRed + 64;
  static constexpr int kFit = (227 * 1024 - kFixed) / kStage;
  static constexpr int kStages = kFit > 5 ? 5 : kFit;
  static constexpr int kSmem = kFixed + kStages * kStage;
  static_assert(kStages >= 2 && kStages <= 8, "a ring of two to eight stages");
};

template <int D, bool kQ8, int MT>
__global__ void __launch_bounds__(256, 1) k_paged(const __grid_constant__ PagedArgs a) {
  using C = Shape<D, kQ8, MT>;
  constexpr int RB = C::RB, S = C::kStages, NT = D / 32;
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* sQ = sm + S * C::kStage;
  uint8_t* sP = sQ + C::kQ;
  float* red = reinterpret_cast<float*>(sP + 2 * C::kP);   // [4][kRows]
  bool* there = reinterpret_cast<bool*>(red + 4 * C::kRows);   // [stage][4] 16-token groups
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w4 = warp & 3, row0 = (warp >> 2) * MT * 16;
  const int g = lane >> 2, q = lane & 3;
  pdl_wait();

  if (blockIdx.x == 0 && tid == 0) *a.status = 0u;
  Cursor cur{};
  const int n = cta_run(a, blockIdx.x, lane, &cur);   // tiles of this CTA
  if (n == 0) return;
  Cursor ahead = cur;

  const int page_mask = (1 << a.c.page_shift) - 1;
  // Each run of 16 tokens lies in one page. Lane x of every warp holds where run x & 3 of the
  // tile to be fetched next starts (in values, -1: nowhere), looked up a tile ahead.
  int64_t run_at, run_scale;
  auto look_up = [&](const Cursor& at) {
    const int t = at.tile * kTile + 16 * (lane & 3), page = page_of(a, at.b, t, at.len);
    const int64_t in_page = ((int64_t)at.h << a.c.page_shift) + (t & page_mask);
    run_at = page < 0 ? -1 : page * a.c.stride + in_page * D;
    if (kQ8) run_scale = page < 0 ? -1 : page * a.c.scale_stride + in_page;
  };
  constexpr int kChunks = RB / 16, kStep = C::kThreads / kChunks;   // rows per iteration
  const int my_row = tid / kChunks, my_chunk = tid % kChunks;
  const uint32_t my_dst = swz<RB>(my_row, my_chunk);   // (kStep is a multiple of 8 rows)
  auto load_tile = [&](const Cursor& at, int stage) {
    const uint32_t k0 = smem_at(sm + stage * C::kStage) + my_dst, v0 = k0 + C::kMat;
    const int left = at.len - at.tile * kTile;   // tokens from the tile's first on
    int64_t run = 0;
#pragma unroll
    for (int it = 0; it < kTile / kStep; ++it) {
      const int r = it * kStep + my_row;
      if (it * kStep % 16 == 0 || kStep > 16) run = __shfl_sync(0xffffffffu, run_at, (r >> 4) & 3);
      const bool ok = run >= 0 && r < left;
      const int64_t off = ok ? (run + (r & 15) * D) * (kQ8 ? 1 : 2) + my_chunk * 16 : 0;
      cp_async16(k0 + it * kStep * RB, a.c.k + off, ok);
      cp_async16(v0 + it * kStep * RB, a.c.v + off, ok);
    }
    if (warp == 0) {
      if constexpr (kQ8) {   // 4 scales per copy: 16 of the keys, 16 of the values
        const int r = 4 * (lane & 15);
        const int64_t at_s = __shfl_sync(0xffffffffu, run_scale, r >> 4);
        const bool ok = at_s >= 0 && r < left;
        cp_async16(smem_at(sm + stage * C::kStage) + 2 * C::kMat + 16 * lane,
                   (lane < 16 ? a.c.k_scale : a.c.v_scale) + (ok ? at_s + (r & 15) : 0), ok);
      }
      if (lane < 4) there[4 * stage + lane] = run_at >= 0;
    }
  };

  int fetched = 0;
  auto fetch = [&](int stage) {
    if (fetched < n) {
      load_tile(ahead, stage);
      if (++fetched < n) {
        ahead.next(a);
        look_up(ahead);
      }
    }
    cp_async_commit();
  };
  look_up(ahead);
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);

  int rr[MT][2];   // verify row of this lane's query rows
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) rr[mt][e] = (row0 + 16 * mt + g + 8 * e) / a.G;

  float m[MT][2], l[MT][2], o[MT][NT][4];
  bool starts = true;
  int stage = S - 1;
  for (int i = 0; i < n; ++i) {
    const int refill = stage;   // the stage of the tile before
    stage = stage + 1 == S ? 0 : stage + 1;
    const uint8_t* sK = sm + stage * C::kStage;
    const uint8_t* sV = sK + C::kMat;
    if (starts) {
      // queries of this (sequence, key head); rows behind M are zero. For a Q8 cache the 16
      // values of a step are stored even ones first, the order in which codes are widened.
      constexpr int kChunks = D / 8;
      for (int idx = tid; idx < C::kRows * kChunks / 2; idx += C::kThreads) {
        const int r = idx / (kChunks / 2), pr = idx % (kChunks / 2);
        uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
        if (r < a.M) {
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (((int64_t)cur.b * a.R + r / a.G) * a.Hq + cur.h * a.G + r % a.G) * D) + 2 * pr;
          x0 = src[0];
          x1 = src[1];
        }
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
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        m[mt][0] = m[mt][1] = kNegInf;
        l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
      }
    }
    cp_async_wait<S - 2>();
    __syncthreads();   // the tile and the queries are there; the tile before is done with
    fetch(refill);

    const int t0 = cur.tile * kTile, seen0 = cur.len - (a.R - 1);   // row r sees t < seen0 + r
    // ------------------------------------------------------------ S = Q K^T ---------
    // (few rows: even and odd steps in accumulators of their own, for shorter chains)
    constexpr int kSets = MT <= 2 ? 2 : 1;
    float s[MT][2][4], s_odd[kSets == 2 ? MT : 1][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mt][nt][e] = 0.f;
          if constexpr (kSets == 2) s_odd[mt][nt][e] = 0.f;
        }
    {
      const uint32_t kb = smem_at(sK), qb = smem_at(sQ);
      constexpr int kSteps = D / 16, kPer = kQ8 ? 4 : 2;   // 16-value steps per ldmatrix.x4
#pragma unroll
      for (int kk = 0; kk < kSteps / kPer; ++kk) {
        uint32_t kf[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          ldsm_x4(kb + swz<RB>(16 * w4 + 8 * nt + (lane & 7), 4 * kk + (lane >> 3)), kf[nt]);
#pragma unroll
        for (int st = 0; st < kPer; ++st) {
          const int ks = kPer * kk + st;
          uint32_t b[2][2];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            if constexpr (kQ8) {
              b[nt][0] = code_pair(kf[nt][st]);
              b[nt][1] = code_pair(kf[nt][st] >> 8);
            } else {
              b[nt][0] = kf[nt][2 * st];
              b[nt][1] = kf[nt][2 * st + 1];
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t qf[4];
            ldsm_x4(qb + swz<2 * D>(row0 + 16 * mt + (lane & 15), 2 * ks + (lane >> 4)), qf);
            if (kSets == 2 && (ks & 1)) {
              mma16816(s_odd[kSets == 2 ? mt : 0][0], qf, b[0][0], b[0][1]);
              mma16816(s_odd[kSets == 2 ? mt : 0][1], qf, b[1][0], b[1][1]);
            } else {
              mma16816(s[mt][0], qf, b[0][0], b[0][1]);
              mma16816(s[mt][1], qf, b[1][0], b[1][1]);
            }
          }
        }
      }
      if constexpr (kSets == 2) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = __fadd_rn(s[mt][nt][e], s_odd[mt][nt][e]);
      }
    }
    // -------------------------------------------------- scale, mask, P = 2^(S - m) ---
    // this lane: rows g (s[.][.][0, 1]) and g + 8 (2, 3), tokens 8 nt + 2q, 2q + 1 of the warp's
    float vs[2][2], ref[MT][2], top[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      ref[mt][0] = m[mt][0] == kNegInf ? 0.f : m[mt][0];
      ref[mt][1] = m[mt][1] == kNegInf ? 0.f : m[mt][1];
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float f0 = a.scale_log2, f1 = f0;
      if constexpr (kQ8) {
        const float2* sc = reinterpret_cast<const float2*>(sV + C::kMat);
        const float2 kq = sc[8 * w4 + 4 * nt + q], vq = sc[kTile / 2 + 8 * w4 + 4 * nt + q];
        f0 = __fmul_rn(f0, kq.x);
        f1 = __fmul_rn(f1, kq.y);
        vs[nt][0] = vq.x;
        vs[nt][1] = vq.y;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {   // s: scores in log2, before any mask
        s[mt][nt][0] = __fmul_rn(s[mt][nt][0], f0);
        s[mt][nt][1] = __fmul_rn(s[mt][nt][1], f1);
        s[mt][nt][2] = __fmul_rn(s[mt][nt][2], f0);
        s[mt][nt][3] = __fmul_rn(s[mt][nt][3], f1);
      }
    }
    const int wt0 = t0 + 16 * w4;   // the warp's first token
    const bool gone = !there[4 * stage + w4];
    const bool edge = gone || wt0 + 16 > seen0;
    if (edge) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = wt0 + 8 * nt + 2 * q + (e & 1);
            if (gone || t >= seen0 + rr[mt][e >> 1]) s[mt][nt][e] = kNegInf;
          }
    }
    float lt[MT][2];
    auto make_p = [&] {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = row0 + 16 * mt + g + 8 * e;
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const float s0 = s[mt][nt][2 * e], s1 = s[mt][nt][2 * e + 1];
            float p0 = exp2_fast(__fsub_rn(s0, ref[mt][e]));
            float p1 = exp2_fast(__fsub_rn(s1, ref[mt][e]));
            uint8_t* dst = sP + swz<2 * kTile>(row, 2 * w4 + nt) + 4 * q;
            sum = __fadd_rn(sum, __fadd_rn(p0, p1));
            if constexpr (kQ8) {
              p0 = __fmul_rn(p0, vs[nt][0]);
              p1 = __fmul_rn(p1, vs[nt][1]);
              if (edge) {   // a masked token's scale may be anything
                p0 = s0 == kNegInf ? 0.f : p0;
                p1 = s1 == kNegInf ? 0.f : p1;
              }
            }
            const uint32_t w = pack2(p0, p1);
            *reinterpret_cast<uint32_t*>(dst) = w;
            *reinterpret_cast<uint32_t*>(dst + C::kP) =
                pack2(__fsub_rn(p0, bf16_lo(w)), __fsub_rn(p1, bf16_hi(w)));
          }
          lt[mt][e] = sum;
        }
      }
    };
    bool over = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[mt][e] = fmaxf(fmaxf(s[mt][0][2 * e], s[mt][0][2 * e + 1]),
                           fmaxf(s[mt][1][2 * e], s[mt][1][2 * e + 1]));
        over |= top[mt][e] > __fadd_rn(m[mt][e], kSlack);   // (-infinity: nothing seen yet)
      }
    make_p();
    if (__syncthreads_or(over)) {
      // some row's reference moves: exchange the tile's maxima, rescale, and make P again
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = top[mt][e];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          if (q == 0) red[w4 * C::kRows + row0 + 16 * mt + g + 8 * e] = x;
        }
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* rp = red + row0 + 16 * mt + g + 8 * e;
          const float mn = fmaxf(m[mt][e], fmaxf(fmaxf(rp[0], rp[C::kRows]),
                                                 fmaxf(rp[2 * C::kRows], rp[3 * C::kRows])));
          const float f = m[mt][e] == kNegInf ? 0.f : exp2_fast(__fsub_rn(m[mt][e], mn));
          m[mt][e] = mn;
          ref[mt][e] = mn == kNegInf ? 0.f : mn;
          l[mt][e] = __fmul_rn(l[mt][e], f);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[mt][nt][2 * e] = __fmul_rn(o[mt][nt][2 * e], f);
            o[mt][nt][2 * e + 1] = __fmul_rn(o[mt][nt][2 * e + 1], f);
          }
        }
      make_p();
      __syncthreads();
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt][0] = __fadd_rn(l[mt][0], lt[mt][0]);
      l[mt][1] = __fadd_rn(l[mt][1], lt[mt][1]);
    }
    // ---------------------------------------------------------------- O += P V -------
    // A bf16 value that only some rows see may hold anything, and 0 x infinity is not 0: the
    // (at most 7) tokens from seen0 on are left out of the product and added row by row.
    const bool part_seen = !kQ8 && a.R > 1 && t0 + kTile > seen0;
    {
      const uint32_t vb = smem_at(sV), pb = smem_at(sP);
      const int vrow = (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t b[NT][2];
        if constexpr (!kQ8) {
#pragma unroll
          for (int dp = 0; dp < NT / 2; ++dp) {
            uint32_t r[4];
            ldsm_x4_t(vb + swz<RB>(16 * ks + vrow, NT * w4 + 2 * dp + (lane >> 4)), r);
            b[2 * dp][0] = r[0], b[2 * dp][1] = r[1];
            b[2 * dp + 1][0] = r[2], b[2 * dp + 1][1] = r[3];
          }
          if (part_seen) {
            const int t = t0 + 16 * ks + 2 * q;
            const uint32_t k0 = (t < seen0 ? 0xFFFFu : 0u) | (t + 1 < seen0 ? 0xFFFF0000u : 0u);
            const uint32_t k1 = (t + 8 < seen0 ? 0xFFFFu : 0u) | (t + 9 < seen0 ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) b[nt][0] &= k0, b[nt][1] &= k1;
          }
        } else if constexpr (D == 128) {
          uint32_t r[4];
          ldsm_x4_t(vb + swz<RB>(16 * ks + vrow, 2 * w4 + (lane >> 4)), r);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            b[nt][0] = code_pair(r[nt & 2] >> (8 * (nt & 1)));
            b[nt][1] = code_pair(r[(nt & 2) + 1] >> (8 * (nt & 1)));
          }
        } else {
          uint32_t r0, r1;
          ldsm_x2_t(vb + swz<RB>(16 * ks + (lane & 15), w4), r0, r1);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            b[nt][0] = code_pair(r0 >> (8 * nt));
            b[nt][1] = code_pair(r1 >> (8 * nt));
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t pf[4];
          ldsm_x4(pb + swz<2 * kTile>(row0 + 16 * mt + (lane & 15), 2 * ks + (lane >> 4)), pf);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[mt][nt], pf, b[nt][0], b[nt][1]);
          ldsm_x4(pb + C::kP + swz<2 * kTile>(row0 + 16 * mt + (lane & 15), 2 * ks + (lane >> 4)),
                  pf);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[mt][nt], pf, b[nt][0], b[nt][1]);
        }
      }
    }
    if constexpr (!kQ8) {
      if (part_seen) {
        const int first = seen0 > t0 ? seen0 - t0 : 0;
        const int last = cur.len - t0 < kTile ? cur.len - t0 : kTile;
        for (int t = first; t < last; ++t) {
          uint32_t v[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            v[nt] = *reinterpret_cast<const uint32_t*>(sV + swz<RB>(t, NT * w4 + nt) + 4 * q);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (t0 + t >= seen0 + rr[mt][e]) continue;
              const int row = row0 + 16 * mt + g + 8 * e;
              const uint8_t* ps = sP + swz<2 * kTile>(row, t >> 3) + 2 * (t & 7);
              const float p =
                  __fadd_rn(bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(ps)),
                            bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(ps + C::kP)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                o[mt][nt][2 * e] = __fmaf_rn(p, bf16_lo(v[nt]), o[mt][nt][2 * e]);
                o[mt][nt][2 * e + 1] = __fmaf_rn(p, bf16_hi(v[nt]), o[mt][nt][2 * e + 1]);
              }
            }
        }
      }
    }
    // --------------------------------------- the end of this run of the (sequence, head)
    const bool whole_end = cur.tile + 1 == cur.tiles;
    starts = whole_end || i + 1 == n;
    if (starts) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = l[mt][e];
          v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 2));
          if (q == 0) red[w4 * C::kRows + row0 + 16 * mt + g + 8 * e] = v;
        }
      __syncthreads();
      const int run = i < cur.tile ? i : cur.tile;   // tiles before this one in it
      const bool whole = whole_end && cur.tile == run;
      // slot 0: the run began before this CTA; slot 1: it begins here and goes on in the next
      const int64_t slot = 2 * (int64_t)blockIdx.x + (cur.tile == run ? 1 : 0);
      if (tid == 0) note_span(a, cur, cur.tile == run, whole_end);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = row0 + 16 * mt + g + 8 * e;
          if (row >= a.M) continue;
          const float* rp = red + row;
          const float norm = __fadd_rn(__fadd_rn(rp[0], rp[C::kRows]),
                                       __fadd_rn(rp[2 * C::kRows], rp[3 * C::kRows]));
          if (whole) {
            uint16_t* dst = a.out + (((int64_t)cur.b * a.R + rr[mt][e]) * a.Hq + cur.h * a.G +
                                     row % a.G) * D + w4 * (D / 4);
            auto val = [&](int nt, int x) {
              return norm == 0.f ? 0.f : __fdiv_rn(o[mt][nt][2 * e + x], norm);
            };
            if constexpr (!kQ8) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<uint32_t*>(dst + 8 * nt + 2 * q) = pack2(val(nt, 0), val(nt, 1));
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; nt += 2)
                *reinterpret_cast<uint2*>(dst + 8 * nt + 4 * q) =
                    make_uint2(pack2(val(nt, 0), val(nt + 1, 0)), pack2(val(nt, 1), val(nt + 1, 1)));
            }
          } else {
            float* dst = a.part_o + (slot * a.M + row) * D + w4 * (D / 4);
            if constexpr (!kQ8) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<float2*>(dst + 8 * nt + 2 * q) =
                    make_float2(o[mt][nt][2 * e], o[mt][nt][2 * e + 1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; nt += 2)
                *reinterpret_cast<float4*>(dst + 8 * nt + 4 * q) =
                    make_float4(o[mt][nt][2 * e], o[mt][nt + 1][2 * e], o[mt][nt][2 * e + 1],
                                o[mt][nt + 1][2 * e + 1]);
            }
            if (w4 == 0 && q == 0)
              *reinterpret_cast<float2*>(a.part_ml + 2 * (slot * a.M + row)) =
                  make_float2(m[mt][e], norm);
          }
        }
    }
    cur.next(a);
  }
  cp_async_wait<0>();
}

// k_paged_join: block x = (sequence, key head). Those that crossed a CTA boundary are merged
// in CTA order; empty sequences get zeros; the others are already written. kWarps: the warps
// that share a row (a head is cut into many pieces); with 1, a row for each of 8 warps. Its
// time is latency, so pieces are read several at a time (one after the other: 41 against 32 us
// for the whole call of 16 rows, 8 sequences x 8 heads at 4k). One head of 64 pieces or fewer
// takes 8 warps: 24 rows, 8 heads of 38 pieces, 16 us for the call against 19 with 32.
// (top, norm, acc) += the N (m, l, x), in order: sums relative to 2^reference.
template <int V, int N>
__device__ __forceinline__ void merge(float& top, float& norm, float (&acc)[V],
                                      const float2 (&ml)[N], const float (&x)[N][V]) {
  float now = top;
#pragma unroll
  for (int j = 0; j < N; ++j) now = fmaxf(now, ml[j].x);
  const float f = top == kNegInf ? 0.f : exp2_fast(__fsub_rn(top, now));
  top = now;
  norm = __fmul_rn(norm, f);
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = __fmul_rn(acc[e], f);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float g = ml[j].x == kNegInf ? 0.f : exp2_fast(__fsub_rn(ml[j].x, now));
    norm = __fmaf_rn(ml[j].y, g, norm);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(x[j][e], g, acc[e]);
  }
}
template <int D, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 256 : 32 * kWarps)
    k_paged_join(const __grid_constant__ PagedArgs a) {
  constexpr int V = D / 32;   // values per lane
  constexpr bool kShared = kWarps > 1;
  __shared__ float acc_s[kWarps][D];
  __shared__ float2 l_s[kWarps];   // reference, normaliser
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.c.heads, h = blockIdx.x % a.c.heads;
  pdl_trigger();
  pdl_wait();
  const int row = kShared ? blockIdx.y : blockIdx.y * 8 + warp;
  const int2 span = __ldcg(reinterpret_cast<const int2*>(a.span) + blockIdx.x);
  const bool empty = seq_len(a, b) == 0;
  const int c0 = empty ? 0 : span.x, c1 = empty ? -1 : span.y;
  // (in one CTA: already written; not noted: the kernel gave up, and the status says so)
  if (!empty && (c0 < 0 || c1 <= c0 || c1 >= a.grid)) return;
  if (row >= a.M) return;   // (all warps of the block, when they share the row)
  // a warp's pieces, as many at a time as keep memory's latency down, the reference moving up
  constexpr int kAt = kWarps == 32 ? 5 : 8;
  float top = kNegInf, acc[V], norm = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int first = c0 + (kShared ? warp : 0); first <= c1; first += kAt * kWarps) {
    float2 ml[kAt];
    float x[kAt][V];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int c = first + j * kWarps;
      ml[j] = make_float2(kNegInf, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) x[j][e] = 0.f;
      if (c > c1) continue;
      const int64_t at = (2 * (int64_t)c + (c == c0 ? 1 : 0)) * a.M + row;
      ml[j] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at);
      if constexpr (V == 4) {
        const float4 f4 = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + lane);
        x[j][0] = f4.x, x[j][1] = f4.y, x[j][2] = f4.z, x[j][3] = f4.w;
      } else {
        const float2 f2 = __ldcg(reinterpret_cast<const float2*>(a.part_o + at * D) + lane);
        x[j][0] = f2.x, x[j][1] = f2.y;
      }
    }
    merge<V, kAt>(top, norm, acc, ml, x);
  }
  if constexpr (kShared) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc_s[warp][V * lane + e] = acc[e];
    if (lane == 0) l_s[warp] = make_float2(top, norm);
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < kWarps; w += kAt) {
      float2 ml[kAt];
      float x[kAt][V];
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        ml[j] = w + j < kWarps ? l_s[w + j] : make_float2(kNegInf, 0.f);
#pragma unroll
        for (int e = 0; e < V; ++e) x[j][e] = w + j < kWarps ? acc_s[w + j][V * lane + e] : 0.f;
      }
      merge<V, kAt>(top, norm, acc, ml, x);
    }
  }
  uint16_t* dst = a.out + (((int64_t)b * a.R + row / a.G) * a.Hq + h * a.G + row % a.G) * D + V * lane;
  float y[V];
#pragma unroll
  for (int e = 0; e < V; ++e) y[e] = norm == 0.f ? 0.f : __fdiv_rn(acc[e], norm);
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2(y[0], y[1]);
}

// ------------------------------------------------------------------------------- host ----
enum class Kernel { kFew, kRows, kTensor };

struct Plan {
  Kernel kernel;
  int grid;
  size_t span, ml, po, total;
};

// Calls f with the m16 tiles per warp for these rows.
template <typename F>
auto with_rows(int M, F&& f) {
  if (M <= 64) return f(std::integral_constant<int, 2>{});
  if (M <= 96) return f(std::integral_constant<int, 3>{});
  return f(std::integral_constant<int, 4>{});
}

// Up to 32 rows: paged_few.cu, which costs no more for 1 row than it has to (24 rows, 32
// sequences x 8 heads at 8k, bf16 167 us, Q8 160; k_paged's design with 16-row tiles: 207, 186).
// More rows: the tcgen05 kernel (paged_tc.cu) has the higher rate and the longer beginning and
// end, and is ahead from several tiles per SM on. k_paged | paged_tc, us, 4 sequences x 8 heads:
//   tokens per sequence        500      1k       2k       4k        8k       64k
//   bf16, D = 128, 40 rows   13 | 16  15 | 16  23 | 20  35 | 24   60 | 34  397 | 160
//                  96 rows   17 | 20  19 | 21  30 | 25  45 | 30   76 | 43  504 | 195
//                 128 rows   21 | 25  24 | 26  37 | 32  55 | 40   92 | 57  610 | 291
//   Q8,   D = 128, 64 rows   13 | 20  15 | 19  23 | 26  35 | 29   60 | 42  405 | 207
//                  96 rows   16 | 24  19 | 25  29 | 32  45 | 41   77 | 61  524 | 314
//                 128 rows   20 | 33  24 | 38  36 | 38  56 | 48   95 | 68  649 | 356
//   bf16, D = 64,  64 rows   11 | 16  13 | 16  18 | 18  27 | 22   44 | 30  290 | 136
//                 128 rows   17 | 24  18 | 24  26 | 28  39 | 35   66 | 50  433 | 251
//   Q8,   D = 64,  64 rows   11 | 18  12 | 19  18 | 22  26 | 26   45 | 38  301 | 187
//                  96 rows   13 | 25  16 | 29  22 | 32  33 | 33   57 | 47  382 | 224
// One head of 32k, D = 128, 96 rows: bf16 19 | 18, Q8 20 | 20. From 25 rows on it is ahead of
// paged_few.cu as well at D = 128: 32 rows, 32 sequences x 8 heads at 8k, bf16 176 against 162,
// Q8 198 against 164; 8 x 8 heads at 2k, 24.6 against 21.5 and 24.8 against 24.5; at 1k, 17.5
// against 17.1 and 16.3 against 20.2; but 24 rows at 8k 167 against 161 and 160 against 162, and 32
// rows at D = 64 112 against 109 and 127 against 148. `places`: tokens x key heads there can be
// (lengths are not known here: short ones in a table with room for long ones pay paged_tc.cu's
// beginning).
Kernel which(int M, int D, bool q8, int64_t places) {
  const bool lengthy = places >= (int64_t)(q8 ? 4 : 2) * (128 / D) * 128 * device_sm_count();
  static_assert(kPagedMaxRows <= kTcMaxRows, "it takes any rows");
  if (lengthy && M > (D == 128 ? 24 : kFewMaxRows)) return Kernel::kTensor;
  return M <= kFewMaxRows ? Kernel::kFew : Kernel::kRows;
}

// What a (sequence, key head) costs beside its tiles, in tiles. 32 sequences of up to 8k tokens,
// 8 heads: paged_few.cu, 24 rows, Q8: 99 us with 2, 95 with 3, 97 with 6; paged_tc.cu, 48 rows,
// bf16: 121 with 2, 101.6 with 5, 103 with 8; Q8: 140 with 2, 134 with 4, 139 with 8.
int begin_of(Kernel k, bool q8) {
  return k == Kernel::kFew ? 3 : (k == Kernel::kTensor ? (q8 ? 4 : 5) : 2);
}

Plan make_plan(const PagedAttnProblem& p) {
  const int M = p.R * (p.Hq / p.cache.heads);
  Plan pl{};
  const int64_t cap = (int64_t)p.max_pages << p.cache.page_shift;
  const int64_t runs = (int64_t)p.B * p.cache.heads;
  pl.kernel = which(M, p.D, p.cache.q8, runs * cap);
  const int per_sm = pl.kernel == Kernel::kFew ? few_ctas_per_sm(M, p.D, p.cache.q8) : 1;
  // no more CTAs than positions in the list of tiles there can be
  const int tile = pl.kernel == Kernel::kTensor ? 128 : kTile;
  const int64_t most = runs * ((cap + tile - 1) / tile + begin_of(pl.kernel, p.cache.q8));
  const int64_t all = (int64_t)per_sm * device_sm_count();
  pl.grid = (int)(most < all ? most : all);
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl.span = 256;   // behind the status word
  pl.ml = pl.span + up((size_t)runs * 2 * sizeof(int));
  pl.po = pl.ml + up((size_t)2 * pl.grid * M * 2 * sizeof(float));
  pl.total = pl.po + up((size_t)2 * pl.grid * M * p.D * sizeof(float));
  return pl;
}

template <int D, bool kQ8>
cudaError_t run(const PagedAttnProblem& p, uint8_t* ws, cudaStream_t s) {
  const Plan pl = make_plan(p);
  PagedArgs a{};
  a.B = p.B;
  a.R = p.R;
  a.Hq = p.Hq;
  a.G = p.Hq / p.cache.heads;
  a.M = p.R * a.G;
  a.max_pages = p.max_pages;
  a.tile_log = pl.kernel == Kernel::kTensor ? 7 : 6;
  a.begin = begin_of(pl.kernel, p.cache.q8);
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  a.q = p.q;
  a.c = p.cache;
  a.table = p.table;
  a.lengths = p.lengths;
  a.out = p.out;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.span = reinterpret_cast<int*>(ws + pl.span);
  a.part_ml = reinterpret_cast<float*>(ws + pl.ml);
  a.part_o = reinterpret_cast<float*>(ws + pl.po);
  a.grid = pl.grid;
  cudaError_t err;
  if (pl.kernel == Kernel::kFew) {
    err = launch_few(a, D, s);
  } else if (pl.kernel == Kernel::kTensor) {
    err = launch_tc(a, D, s);
  } else {
    err = with_rows(a.M, [&](auto mt) {
      using C = Shape<D, kQ8, decltype(mt)::value>;
      const auto kernel = k_paged<D, kQ8, decltype(mt)::value>;
      static OncePerDevice ready;
      const cudaError_t e = ready.run([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      });
      if (e != cudaSuccess) return e;
      return launch_pdl(kernel, dim3(pl.grid), C::kThreads, C::kSmem, s, a);
    });
  }
  if (err != cudaSuccess) return err;
  const int heads = p.B * p.cache.heads;
  if (pl.grid > 64 * heads)   // pieces per head
    return launch_pdl(k_paged_join<D, 32>, dim3(heads, a.M), 1024, 0, s, a);
  if (pl.grid > 8 * heads) return launch_pdl(k_paged_join<D, 8>, dim3(heads, a.M), 256, 0, s, a);
  return launch_pdl(k_paged_join<D, 1>, dim3(heads, (a.M + 7) / 8), 256, 0, s, a);
}

}  // namespace

size_t paged_attn_workspace(const PagedAttnProblem& p) { return make_plan(p).total; }

cudaError_t launch_paged_attn(const PagedAttnProblem& p, uint8_t* ws, cudaStream_t s) {
  if (p.D == 128) return p.cache.q8 ? run<128, true>(p, ws, s) : run<128, false>(p, ws, s);
  return p.cache.q8 ? run<64, true>(p, ws, s) : run<64, false>(p, ws, s);
}

}  // namespace dsmoe
