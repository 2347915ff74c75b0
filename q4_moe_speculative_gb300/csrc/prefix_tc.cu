// prefix_tc.cu — attention of many query rows over a shared prefix in the paged cache, on the
// 5th-generation tensor cores (list of tiles in prefix.cuh, arithmetic in include/dsmoe.h).
//
// Query rows are the M = 128 rows of both products, so a thread of the softmax owns a row:
//   S = Q K^T     A = the queries, B = the key tile, both K-major in shared memory; TMEM lane = row,
//                 column = token;
//   O += P V      A = P in tensor memory, in place of S, as a high and a low bf16 part (off by
//                 2^-16 relative, against 2^-8 for one), B = the value tile, MN-major.
// Two streams of scores (two row tiles, or two token tiles of one: prefix.cuh), each with its S / P
// and O (512 columns together for D = 128): while one stream's softmax runs, the tensor cores work
// for the other. Their order is S(j), then O of j - 1; an MMA reads P before a later one
// overwrites it, since a CTA's MMAs run in the order of their issue.
// Roles: two groups of four warps turn scores into P and write the sums; one warp each copies key and
// value tiles page by page, by TMA into the swizzled operand layout (bf16), or four warps each widen
// int8 codes to bf16 (Q8; the key's scale multiplies the score, the value's scale P); one thread of
// the last warp issues the MMAs. Bound by the tensor cores with two row tiles: three products of
// 128 x 128 x 128 per 128 tokens and row tile. Every wait is bounded; a give-up sets the status word.
#include "prefix.cuh"

namespace dsmoe {
namespace prefix {

constexpr int kInfo = 8;                  // tiles whose pages and scales are at hand
constexpr uint32_t kWaitPolls = 1u << 20;
constexpr int kScore = 256;               // softmax threads
// Reference of a row that has seen no token yet: the least finite value, so that any score that
// counts is above it by more than kSlack, or is equal to it and has the weight 1.
constexpr float kNothing = -3.402823466e38f;

template <int D, bool kQ8>
struct Tc {
  static constexpr int kHalves = D / 64;
  static constexpr int kMat = kTok * D * 2;             // bytes of an operand tile
  static constexpr int kRing = D == 128 ? 2 : 4;        // stages of keys, and of values
  static constexpr int kWiden = kQ8 ? 128 : 32;         // threads per matrix that bring tiles
  static constexpr int kThreads = kScore + 2 * kWiden + 32;
  static constexpr int kMmaWarp = kThreads / 32 - 1;
  static constexpr int kSmall = 1024 + (kQ8 ? kInfo * 2 * kTok * 4 : 0);
  static constexpr int kSmem = 1024 + kSmall + 2 * kMat + 2 * kRing * kMat;
  static_assert(kSmem <= 227 * 1024 && kSmem > 114 * 1024, "one CTA has an SM's tensor memory");
};

struct Small {
  uint64_t kfull[4], vfull[4], kfree[4], vfree[4];
  uint64_t sfull[2], pfull[2], qfull[2], odone[2];
  uint64_t info[kInfo], vedge, end;
  uint32_t tmem;
  int abort;
  unsigned runs[kInfo];       // which pages of a tile are there
};
static_assert(sizeof(Small) <= 1024, "in front of the tiles");

__device__ __forceinline__ void ld32(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// To 32 columns; tmem_wait_st() waits for it.
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc], issued by one thread.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Page of the prefix's token t, or -1: no such token, or a bad table entry.
__device__ __forceinline__ int prefix_page(const PrefixArgs& a, int p, int t, int len) {
  if (t >= len) return -1;
  const int page = a.table[(int64_t)p * a.max_pages + (t >> a.own.c.page_shift)];
  return page >= 0 && page < a.own.c.pages ? page : -1;
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(Tc<D, kQ8>::kThreads, 1)
    k_prefix_tc(const __grid_constant__ PrefixArgs a, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map) {
  using T = Tc<D, kQ8>;
  constexpr int kRing = T::kRing;
  extern __shared__ uint8_t smem_raw[];
  const PagedArgs& o = a.own;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t pad = (1024u - (smem_at(smem_raw) & 1023u)) & 1023u;
  uint8_t* const base = smem_raw + pad;
  Small& sh = *reinterpret_cast<Small*>(base);
  float* const sScale = reinterpret_cast<float*>(base + 1024);   // Q8: [kInfo][2][tokens]
  uint8_t* const sQ = base + T::kSmall;                          // [2][halves][rows][128 B]
  uint8_t* const sK = sQ + 2 * T::kMat;                          // [ring][halves][tokens][128 B]
  uint8_t* const sV = sK + kRing * T::kMat;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      sm100::mbar_init(&sh.kfull[i], kQ8 ? T::kWiden / 32 : 1);
      sm100::mbar_init(&sh.vfull[i], kQ8 ? T::kWiden / 32 : 1);
      sm100::mbar_init(&sh.kfree[i], 1);
      sm100::mbar_init(&sh.vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&sh.sfull[i], 1);
      sm100::mbar_init(&sh.pfull[i], 4);
      sm100::mbar_init(&sh.qfull[i], 4);
      sm100::mbar_init(&sh.odone[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) sm100::mbar_init(&sh.info[i], 1);
    sm100::mbar_init(&sh.vedge, 1);
    sm100::mbar_init(&sh.end, 1);
    sh.abort = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 0) {
    sm100::tmem_alloc(&sh.tmem, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = sh.tmem;   // S / P of either stream: 128 columns each; then O of either: D
  if (!kQ8 && tid < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid ? &v_map : &k_map) : "memory");
  pdl_wait();

  volatile int* const abort_flag = &sh.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
      if (sm100::mbar_try_wait(bar, parity)) return true;
      if ((i & 63u) == 63u && *abort_flag) return false;
    }
    *abort_flag = 1;
    flag_status(o.status, kStatusTimeout);
    return false;
  };
  const int page_shift = o.c.page_shift, pt = 1 << page_shift;
  Walk walk;
  walk.open(a, blockIdx.x, lane);
  Run run;
  if (blockIdx.x == 0 && warp == 0) {   // for the join
    int64_t total = 0;
    for (int p0 = 0; p0 < a.P; p0 += 32) {
      int64_t n = p0 + lane < a.P ? head_places(a, token_tiles(prefix_len(a, p0 + lane))) : 0;
      n *= o.c.heads;
      int64_t upto = n;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += v;
      }
      if (p0 + lane < a.P) a.starts[p0 + lane] = total + upto - n;
      total += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) a.starts[a.P] = total;
  }
  auto page_full = [&](const Run& r, int t0, unsigned there) {   // every token of the tile is there
    return t0 + kTok <= r.len && there == 0xFFFFFFFFu >> (32 - (kTok >> page_shift));
  };

  if (warp < kScore / 32) {
    // ------------------------------------------------------------ softmax, results ------
    const int w = warp >> 2, quad = warp & 3, mine = 32 * quad + lane;   // stream; row of its tile
    const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_at + w * kTok, tO = tmem + lane_at + 2 * kTok + w * D;
    // (a negative factor becomes its queries' sign, so that the largest product has the largest
    // score)
    const float fk = fabsf(o.scale_log2);
    const uint32_t flip = o.scale_log2 < 0.f ? 0x80008000u : 0u;
    const f2 fk2 = pair(fk, fk);
    uint32_t jobs = 0, runs = 0, tile0 = 0;   // before this run; tiles of the CTA
    bool alive = true;
    while (alive && walk.next(a, &run)) {
      const int n = run.t1 - run.t0, count = run.w == 2 ? n : (n + 1 - w) / 2;   // tiles of the stream
      const int tile_row = run.u * 2 + (run.w == 2 ? w : 0);
      const int row0 = tile_row * kRows;
      if (count > 0) {
        // ---- queries: eight threads of a warp take 64 values of a row
        constexpr int kChunks = D / 8, kStep = 128 / kChunks;
        const int lt = tid & 127, ch = lt % kChunks;
#pragma unroll 4
        for (int r = lt / kChunks; r < kRows; r += kStep) {
          const int gr = row0 + r;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (gr < a.MP) {
            const int s = run.p * a.per + gr / o.M, mm = gr % o.M;
            x = reinterpret_cast<const uint4*>(
                o.q + (((int64_t)s * o.R + mm / o.G) * o.Hq + run.h * o.G + mm % o.G) * D)[ch];
          }
          if constexpr (kQ8) {   // each four values as (0, 2, 1, 3), the order of widened codes
            const uint4 y = x;
            x.x = __byte_perm(y.x, y.y, 0x5410);
            x.y = __byte_perm(y.x, y.y, 0x7632);
            x.z = __byte_perm(y.z, y.w, 0x5410);
            x.w = __byte_perm(y.z, y.w, 0x7632);
          }
          x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
          *reinterpret_cast<uint4*>(sQ + w * T::kMat + (ch >> 3) * (kRows * 128) + r * 128 +
                                    (((ch & 7) ^ (r & 7)) << 4)) = x;
        }
        fence_async();
        warp_arrive(&sh.qfull[w], lane);
      }
      float ref = kNothing, norm = 0.f;
      for (int i = 0; i < count && alive; ++i, ++jobs) {
        const int nt = run.w == 2 ? i : 2 * i + w;   // of the run
        const uint32_t tile = tile0 + nt;            // of the CTA
        const int slot = tile % kInfo, t0 = (run.t0 + nt) * kTok;
        alive = wait(&sh.info[slot], (tile / kInfo) & 1) && wait(&sh.sfull[w], jobs & 1);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
        sm100::tc_fence_after();
        volatile unsigned* const known = sh.runs;
        const unsigned there = known[slot];
        const bool edge = !page_full(run, t0, there);
        const float* const scales = sScale + 2 * slot * kTok;
        // the tokens among 32 that count
        auto seen = [&](int c) {
          unsigned s = 0u;
          for (int x = 0; x < 32; x += 16)
            if (there >> ((c + x) >> page_shift) & 1u) s |= 0xFFFFu << x;
          const int rest = run.len - t0 - c;
          return rest >= 32 ? s : (rest <= 0 ? 0u : s & ((1u << rest) - 1u));
        };
        // 32 scores, in units of log2
        auto scores = [&](int c, float (&t)[32]) {
          __syncwarp();
          ld32(tS + c, t);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            f2 f = fk2;
            if constexpr (kQ8) {
              const float2 k2 = *reinterpret_cast<const float2*>(scales + c + j);
              f = mul2(f, pair(k2.x, k2.y));
            }
            const float2 s = parts(mul2(pair(t[j], t[j + 1]), f));
            t[j] = s.x;
            t[j + 1] = s.y;
          }
          if (edge) {
            const unsigned s = seen(c);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(s >> j & 1u)) t[j] = kNegInf;
          }
        };
        float top = kNegInf;
#pragma unroll 1
        for (int c = 0; c < kTok; c += 32) {
          float t[32];
          scores(c, t);
          float m4[4] = {t[0], t[1], t[2], t[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], t[j]);
          top = fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
        }
        // the reference moves only when a score exceeds it by 2^kSlack, and O with it (at rest: the
        // scores were issued after the product of this stream's tile before)
        const bool up = i == 0 || __fsub_rn(top, ref) > kSlack;
        if (__any_sync(0xffffffffu, up)) {
          const float now = fmaxf(ref, top), f = exp2_fast(__fsub_rn(ref, now));
          ref = now;
          norm = __fmul_rn(norm, f);
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float t[32];
              uint32_t r[32];
              __syncwarp();
              ld32(tO + c, t);
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__fmul_rn(t[j], f));
              st32(tO + c, r);
            }
            tmem_wait_st();
          }
        }
        const f2 less = pair(-1.f, -1.f), back = pair(-ref, -ref);
        f2 sum0 = pair(0.f, 0.f), sum1 = pair(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < kTok; c += 32) {
          float t[32];
          uint32_t r[32];
          scores(c, t);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 d = parts(add2(pair(t[j], t[j + 1]), back));
            f2 p = pair(exp2_fast(d.x), exp2_fast(d.y));
            if (j & 2) sum1 = add2(sum1, p);
            else sum0 = add2(sum0, p);
            if constexpr (kQ8) {
              const float2 v2 = *reinterpret_cast<const float2*>(scales + kTok + c + j);
              p = mul2(p, pair(v2.x, v2.y));
            }
            float2 x = parts(p);
            if (kQ8 && edge) {   // a masked token's scale may be anything
              x.x = t[j] == kNegInf ? 0.f : x.x;
              x.y = t[j + 1] == kNegInf ? 0.f : x.y;
              p = pair(x.x, x.y);
            }
            const uint32_t hi = pack2(x.x, x.y);
            const float2 rest = parts(fma2(pair(bf16_lo(hi), bf16_hi(hi)), less, p));
            r[j / 2] = hi;
            r[16 + j / 2] = pack2(rest.x, rest.y);
          }
          __syncwarp();
          st32(tS + c, r);
        }
        const float2 s2 = parts(add2(sum0, sum1));
        norm = __fadd_rn(norm, __fadd_rn(s2.x, s2.y));
        tmem_wait_st();
        sm100::tc_fence_before();
        warp_arrive(&sh.pfull[w], lane);
      }
      // ---------------------------------------------------------------- results -----------
      if (alive) {
        const int64_t at = (unit_piece(a, run.p, run.h, run.u, blockIdx.x) * 2 + w) * kRows + mine;
        *reinterpret_cast<float2*>(a.part_ml + 2 * at) =
            make_float2(norm == 0.f ? kNegInf : ref, norm);
        if (count > 0) {
          alive = __all_sync(0xffffffffu, wait(&sh.odone[w], runs & 1));
          ++runs;
          if (alive) {
            sm100::tc_fence_after();
            float4* const to = reinterpret_cast<float4*>(a.part_o + at * D);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float t[32];
              __syncwarp();
              ld32(tO + c, t);
              if (row0 + mine < a.MP) {
#pragma unroll
                for (int j = 0; j < 8; ++j)   // (columns of widened codes: (0, 2, 1, 3))
                  to[c / 4 + j] = kQ8 ? make_float4(t[4 * j], t[4 * j + 2], t[4 * j + 1], t[4 * j + 3])
                                      : make_float4(t[4 * j], t[4 * j + 1], t[4 * j + 2], t[4 * j + 3]);
              }
            }
            sm100::tc_fence_before();
          }
        }
      }
      tile0 += n;
    }
  } else if (warp < T::kMmaWarp) {
    // ------------------------------------------------------------- tiles from the pages ---
    const bool values = warp >= (kScore + T::kWiden) / 32;
    uint64_t* const full = values ? sh.vfull : sh.kfull;
    uint64_t* const free_bar = values ? sh.vfree : sh.kfree;
    uint8_t* const tiles = values ? sV : sK;
    const int pages = kTok >> page_shift;
    const bool teller = !values && (warp == kScore / 32);   // fills in the tile information
    int done = 0, edges = 0, st = 0;
    uint32_t par = 1;
    bool alive = true;
    while (alive && walk.next(a, &run)) {
      int page = lane < pages ? prefix_page(a, run.p, run.t0 * kTok + lane * pt, run.len) : -1;
      for (int t = run.t0; t < run.t1; ++t) {
        const int t0 = t * kTok;
        const bool ok = page >= 0;
        const unsigned there = __ballot_sync(0xffffffffu, ok);
        uint4 codes[kQ8 ? 8 : 1];
        int rows_of = 0;
        if constexpr (kQ8) {   // this tile's codes, on their way while the stage gets free
          constexpr int kChunks = D / 16, kStep = 128 / kChunks, kIters = kTok / kStep;
          static_assert(kIters <= 8, "codes");
          const int lt = (tid - kScore) & 127;
          const int my_row = D == 128 ? (lt >> 4) * 2 + ((lt >> 2) & 1) : lt / kChunks;
          const int my_chunk = D == 128 ? (lt & 3) + ((lt >> 1) & 4) : lt % kChunks;
          const uint8_t* const from = values ? o.c.v : o.c.k;
#pragma unroll
          for (int it = 0; it < kIters; ++it) {
            const int r = my_row + it * kStep;
            const int pg = __shfl_sync(0xffffffffu, page, r >> page_shift);
            codes[it] = make_uint4(0u, 0u, 0u, 0u);
            if (pg >= 0 && t0 + r < run.len)
              codes[it] = __ldg(reinterpret_cast<const uint4*>(
                  from + pg * o.c.stride +
                  (((int64_t)run.h << page_shift) + (r & (pt - 1))) * D + my_chunk * 16));
          }
          rows_of = my_row * 128 + (my_chunk >> 2) * (kTok * 128);
        }
        if (done >= kRing) alive = wait(&free_bar[st], par);
        if (!(alive = __all_sync(0xffffffffu, alive))) break;
        if (teller) {   // (its slot is free: the scores of the tile kRing before are done)
          const int slot = done % kInfo;
          if (lane == 0) {
            sh.runs[slot] = there;
            sm100::mbar_arrive_expect_tx(&sh.info[slot], kQ8 ? __popc(there) * pt * 8 : 0);
          }
          __syncwarp();
          if (kQ8 && ok) {
            const int64_t at = page * o.c.scale_stride + ((int64_t)run.h << page_shift);
            float* const dst = sScale + 2 * slot * kTok + lane * pt;
            bulk_copy(dst, o.c.k_scale + at, pt * 4, &sh.info[slot]);
            bulk_copy(dst + kTok, o.c.v_scale + at, pt * 4, &sh.info[slot]);
          }
        }
        if constexpr (kQ8) {
          constexpr int kChunks = D / 16, kStep = 128 / kChunks, kIters = kTok / kStep;
          const int lt = (tid - kScore) & 127;
          const int my_row = D == 128 ? (lt >> 4) * 2 + ((lt >> 2) & 1) : lt / kChunks;
          const int my_chunk = D == 128 ? (lt & 3) + ((lt >> 1) & 4) : lt % kChunks;
          const int c0 = ((2 * my_chunk & 7) ^ (my_row & 7)) << 4;   // (kStep: a multiple of 8 rows)
          uint8_t* const dst = tiles + st * T::kMat + rows_of;
#pragma unroll
          for (int it = 0; it < kIters; ++it) {
            const uint4 v = codes[it];
            *reinterpret_cast<uint4*>(dst + it * (kStep * 128) + c0) = make_uint4(
                code_pair(v.x), code_pair(v.x >> 8), code_pair(v.y), code_pair(v.y >> 8));
            *reinterpret_cast<uint4*>(dst + it * (kStep * 128) + (c0 ^ 16)) = make_uint4(
                code_pair(v.z), code_pair(v.z >> 8), code_pair(v.w), code_pair(v.w >> 8));
          }
          fence_async();
          warp_arrive(&full[st], lane);
        } else {
          const bool edge = values && !page_full(run, t0, there);
          uint64_t* const bar = edge ? &sh.vedge : &full[st];
          if (lane == 0) sm100::mbar_arrive_expect_tx(bar, __popc(there) * pt * 2 * D);
          __syncwarp();
          if (ok) {
#pragma unroll
            for (int hf = 0; hf < T::kHalves; ++hf)
              sm100::tma_load_3d(tiles + st * T::kMat + hf * (kTok * 128) + lane * pt * 128,
                                 values ? &v_map : &k_map, 64 * hf, run.h << page_shift, page, bar);
          }
          if (edge) {   // clear what is no value: 0 x infinity is not 0
            const uint32_t edge_par = edges++ & 1;
            alive = wait(&sh.vedge, edge_par);
            if (!(alive = __all_sync(0xffffffffu, alive))) {   // (no full[] counts these copies)
              sm100::mbar_wait(&sh.vedge, edge_par, kWaitPolls);
              break;
            }
            for (int r = lane; r < kTok; r += 32) {
              if (t0 + r < run.len && (there >> (r >> page_shift) & 1u)) continue;
              for (int x = 0; x < 8 * T::kHalves; ++x)
                *reinterpret_cast<uint4*>(tiles + st * T::kMat + (x >> 3) * (kTok * 128) + r * 128 +
                                          (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) arrive(&full[st]);
          }
        }
        ++done;
        if (++st == kRing) st = 0, par ^= 1;
        page = -1;
        if (t + 1 < run.t1 && lane < pages)
          page = prefix_page(a, run.p, (t + 1) * kTok + lane * pt, run.len);
      }
    }
    if (*abort_flag) {   // copies in flight end (bounded) before the CTA does
      if (!kQ8)
        for (int j = done - kRing < 0 ? 0 : done - kRing; j < done; ++j)
          sm100::mbar_wait(&full[j % kRing], (j / kRing) & 1, kWaitPolls);
      if (teller)
        for (int j = done - kInfo < 0 ? 0 : done - kInfo; j < done; ++j)
          sm100::mbar_wait(&sh.info[j % kInfo], (j / kInfo) & 1, kWaitPolls);
    }
  } else {
    // --------------------------------------------------------------------------- MMAs ----
    // (the whole warp walks the loop; one lane issues)
    const bool leader = elect_one();
    const uint32_t s_idesc = sm100::idesc_bf16_f32(kRows, kTok);
    const uint32_t o_idesc = sm100::idesc_bf16_f32(kRows, D) | (kMajorMN & (1u << 16));
    const uint64_t q_desc = sm100::desc_k_sw128(smem_at(sQ));
    const uint64_t k_desc = sm100::desc_k_sw128(smem_at(sK));
    const uint64_t v_desc = desc_mn_sw128(smem_at(sV), kTok * 128);
    uint32_t ktiles = 0, vtiles = 0;    // tiles taken up
    uint32_t summed[2] = {0, 0}, queries[2] = {0, 0};
    bool alive = true;
    while (alive && walk.next(a, &run)) {
      const int n = run.t1 - run.t0, jobs = n * run.w;
      auto score = [&](int j) {
        const int w = j & 1;
        const bool opens = run.w == 1 || w == 0, closes = run.w == 1 || w == 1;
        const uint32_t tile = opens ? ktiles : ktiles - 1;
        const int st = tile % kRing;
        bool ok = true;
        if (j < 2) ok = wait(&sh.qfull[w], queries[w]++ & 1);
        if (opens) {
          ok = ok && wait(&sh.kfull[st], (tile / kRing) & 1);
          ++ktiles;
        }
        if (!__all_sync(0xffffffffu, ok)) return false;
        sm100::tc_fence_after();
        fence_async();
        if (leader) {
          const uint64_t kd = k_desc + (uint32_t)st * (T::kMat >> 4);
          const uint64_t qd = q_desc + (uint32_t)w * (T::kMat >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {   // 16 values: 32 bytes, or the next 64 values
            const uint32_t off = (ks >> 2) * (kTok * 8) + (ks & 3) * 2;
            sm100::mma_bf16(tmem + w * kTok, qd + off, kd + off, s_idesc, ks > 0);
          }
          sm100::mma_commit(&sh.sfull[w]);
          if (closes) sm100::mma_commit(&sh.kfree[st]);
        }
        __syncwarp();
        return true;
      };
      auto sum = [&](int j) {
        const int w = j & 1;
        const bool opens = run.w == 1 || w == 0, closes = run.w == 1 || w == 1;
        const uint32_t tile = opens ? vtiles : vtiles - 1;
        const int st = tile % kRing;
        bool ok = wait(&sh.pfull[w], summed[w]++ & 1);
        if (opens) {
          ok = ok && wait(&sh.vfull[st], (tile / kRing) & 1);
          ++vtiles;
        }
        if (!__all_sync(0xffffffffu, ok)) return false;
        sm100::tc_fence_after();
        fence_async();
        if (leader) {
          const uint64_t vd = v_desc + (uint32_t)st * (T::kMat >> 4);
          const uint32_t p = tmem + w * kTok, to = tmem + 2 * kTok + w * D;
#pragma unroll
          for (int ks = 0; ks < kTok / 16; ++ks) {   // 16 tokens: 2 KB of values, 8 columns of P
            const uint32_t at = p + 32 * (ks >> 1) + 8 * (ks & 1);
            mma_tmem_a(to, at, vd + ks * 128, o_idesc, j >= 2 || ks > 0);
            mma_tmem_a(to, at + 16, vd + ks * 128, o_idesc, 1u);
          }
          if (closes) sm100::mma_commit(&sh.vfree[st]);
          if (j + 2 >= jobs) sm100::mma_commit(&sh.odone[w]);
        }
        __syncwarp();
        return true;
      };
      for (int j = 0; j <= jobs && alive; ++j) {
        if (j < jobs) alive = score(j);
        if (alive && j > 0) alive = sum(j - 1);
      }
    }
    // MMAs issued but maybe not observed complete: wait (bounded) before TMEM is freed
    if (leader) sm100::mma_commit(&sh.end);
    __syncwarp();
    sm100::mbar_wait(&sh.end, 0, kWaitPolls);
  }
  __syncwarp();
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 0) sm100::tmem_dealloc(tmem, 512);
}

template <int D, bool kQ8>
cudaError_t start(const PrefixArgs& a, cudaStream_t s) {
  using T = Tc<D, kQ8>;
  const auto kernel = k_prefix_tc<D, kQ8>;
  static OncePerDevice ready;
  const cudaError_t e = ready.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap k_map = {}, v_map = {};
  if (!kQ8) {
    const CacheView& c = a.own.c;
    const int pt = 1 << c.page_shift;
    cudaError_t m = page_tile_map(&k_map, c.k, D, c.heads * pt, c.pages, c.stride, pt);
    if (m == cudaSuccess) m = page_tile_map(&v_map, c.v, D, c.heads * pt, c.pages, c.stride, pt);
    if (m != cudaSuccess) return m;
  }
  return launch_pdl(kernel, dim3(a.grid), T::kThreads, T::kSmem, s, a, k_map, v_map);
}

cudaError_t launch_prefix_tc(const PrefixArgs& a, int D, cudaStream_t s) {
  if (D == 128) return a.own.c.q8 ? start<128, true>(a, s) : start<128, false>(a, s);
  return a.own.c.q8 ? start<64, true>(a, s) : start<64, false>(a, s);
}

}  // namespace prefix
}  // namespace dsmoe
