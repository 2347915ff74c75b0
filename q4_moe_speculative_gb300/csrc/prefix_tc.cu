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
// for the other. Their order: O of tile j, and behind it without a pause the scores of the stream's
// next tile; an MMA reads P before a later one overwrites it, since a CTA's MMAs run in the order of
// their issue. P comes in two halves, so that O's products begin at the first.
// Roles: one lane of warp 0 issues the MMAs; one warp each copies key and value tiles page by page, by
// TMA into the swizzled operand layout (bf16), or seven warps widen int8 codes to bf16 (Q8; the
// key's scale multiplies the score, the value's scale P); 16 warps turn scores into P, two threads
// to a row, and write the sums. A row's reference moves, and O with it, only when a score exceeds it
// by 2^8. Every wait is bounded; a give-up sets the status word.
//
// Bound by the tensor cores in bf16: three products of 128 x 128 x 128 per 128 tokens and row tile.
// Measured, 1536 rows of 8 heads, D = 128: 6.0 us per 1024 tokens, 82% of the measured rate; over 16k
// tokens 109 us with its beginning (5 us to the first scores) and end. Q8: 9.0 us per 1024 tokens,
// bound by instruction issue (59 M warp instructions against 33 M in bf16 for 8k tokens: widening and
// the scales) and the order widen, score, weigh, add; three widening warps took 1.6 times as long.
// D = 64: 16k tokens with the other kernels 103 us, in Q8 140; half the products per score, so the
// softmax's instructions weigh twice as much against them (not profiled).
#include <type_traits>

#include "prefix.cuh"

namespace dsmoe {
namespace prefix {

constexpr int kInfo = 8;                  // tiles whose pages and scales are at hand
// Polls of a wait: of one role for another (a test's build has fewer, so that they run out), and of the
// last ones, for copies and products in flight.
#ifndef DS_PREFIX_WAIT_POLLS
#define DS_PREFIX_WAIT_POLLS (1u << 20)
#endif
constexpr uint32_t kWaitPolls = DS_PREFIX_WAIT_POLLS, kEndPolls = 1u << 20;
constexpr int kStream = 256;              // softmax threads of a stream: two per row
constexpr int kScore = 2 * kStream;
// Reference of a row that has seen no token yet: the least finite value, so that any score that
// counts is above it by more than kSlack, or is equal to it and has the weight 1.
constexpr float kNothing = -3.402823466e38f;

template <int D, bool kQ8>
struct Tc {
  static constexpr int kHalves = D / 64;
  static constexpr int kC = kQ8 ? 16 : 32;              // columns of scores at a time (Q8: 80 registers)
  static constexpr int kMat = kTok * D * 2;             // bytes of an operand tile
  static constexpr int kRing = D == 128 ? 2 : 4;        // stages of keys, and of values
  static constexpr int kBringers = kQ8 ? 7 : 2;         // warps that bring tiles
  // warp 0 issues the MMAs, the next bring tiles, then softmax from a multiple of four on
  static constexpr int kFirst = (1 + kBringers + 3) / 4 * 128;
  static constexpr int kThreads = kFirst + kScore;
  static constexpr int kSmall = 6144 + (kQ8 ? kInfo * 2 * kTok * 4 : 0);
  static constexpr int kQ = kRows * 64 * 4;             // of a stream: its queries, then its sums
  static constexpr int kSmem = 1024 + kSmall + 2 * kQ + 2 * kRing * kMat;
  static_assert(kSmem <= 227 * 1024 && kSmem > 114 * 1024, "one CTA has an SM's tensor memory");
};

struct Small {
  uint64_t kfull[4], vfull[4], kfree[4], vfree[4];
  uint64_t sfull[2], pfull[2][2], qfull[2], odone[2];   // P in two parts
  uint64_t qfree[2], info[kInfo], vedge, end;
  uint32_t tmem;
  int abort;
  bool given;                 // what the caller gives is visible
  unsigned runs[kInfo];       // which pages of a tile are there
  int row_at[kPagedMaxRows];  // where a row's values start in a sequence's queries
  Run run[2][4];              // [stream][32 rows]: what their two warps work on
  float top[2][2][2][kRows];  // [tile parity][stream][half of the columns]: largest scores
};
static_assert(sizeof(Small) <= 6144, "in front of the tiles");

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
__device__ __forceinline__ void load_columns(uint32_t at, float (&v)[32]) { ld32(at, v); }
__device__ __forceinline__ void load_columns(uint32_t at, float (&v)[16]) { sm100::tmem_ld16(at, v); }
// To 16 columns; tmem_wait_st() waits for it.
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
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
// Whether three phases are complete (bit 0), and a fourth (bit 1): one round trip.
__device__ __forceinline__ uint32_t ready3_1(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                             uint64_t* c, uint32_t pc, uint64_t* d, uint32_t pd) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q, s, t;\n\t.reg .u32 x;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 s, [%5], %6;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 t, [%7], %8;\n\t"
      "and.pred p, p, q;\n\tand.pred p, p, s;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "selp.u32 x, 2, 0, t;\n\tor.b32 %0, %0, x;\n\t}"
      : "=&r"(r)
      : "r"(smem_at(a)), "r"(pa), "r"(smem_at(b)), "r"(pb), "r"(smem_at(c)), "r"(pc),
        "r"(smem_at(d)), "r"(pd)
      : "memory");
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
  float* const sScale = reinterpret_cast<float*>(base + 6144);   // Q8: [kInfo][2][tokens]
  uint8_t* const sQ = base + T::kSmall;                          // [2][halves][rows][128 B]
  uint8_t* const sK = sQ + 2 * T::kQ;                            // [ring][halves][tokens][128 B]
  uint8_t* const sV = sK + kRing * T::kMat;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      sm100::mbar_init(&sh.kfull[i], kQ8 ? T::kBringers : 1);
      sm100::mbar_init(&sh.vfull[i], kQ8 ? T::kBringers : 1);
      sm100::mbar_init(&sh.kfree[i], 1);
      sm100::mbar_init(&sh.vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&sh.sfull[i], 1);
      sm100::mbar_init(&sh.pfull[i][0], kStream / 32);
      sm100::mbar_init(&sh.pfull[i][1], kStream / 32);
      sm100::mbar_init(&sh.qfull[i], kStream / 32);
      sm100::mbar_init(&sh.qfree[i], kStream / 32);
      sm100::mbar_init(&sh.odone[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) sm100::mbar_init(&sh.info[i], 1);
    sm100::mbar_init(&sh.vedge, 1);
    sm100::mbar_init(&sh.end, 1);
    sh.abort = 0;
    sm100::fence_mbar_init();
  }
  if (tid < o.M) sh.row_at[tid] = (tid / o.G * o.Hq + tid % o.G) * D;
  if (warp == 0) {
    sm100::tmem_alloc(&sh.tmem, 512);
    sm100::tmem_relinquish();
  }
  if (tid == 32) sh.given = given_is_there(o);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  // tensor memory, all of it, so from column 0 on: S / P of either stream, 128 columns each; then O of
  // either, D columns
  constexpr uint32_t tmem = 0;
  if (!kQ8 && tid < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid ? &v_map : &k_map) : "memory");
  pdl_trigger();
  // (Of the kernel of the own tokens before this one nothing is used but that it had waited for those
  // before it. The join needs both: waited for at the end.)
  if (!sh.given) pdl_wait();
  fence_async_global();
  const int lane_len = lane < a.P ? prefix_len(a, lane) : 0;

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
  walk.open(a, blockIdx.x, lane, lane_len);
  Run run;
  auto page_full = [&](const Run& r, int t0, unsigned there) {   // every token of the tile is there
    return t0 + kTok <= r.len && there == 0xFFFFFFFFu >> (32 - (kTok >> page_shift));
  };

  if (tid >= T::kFirst) {
    // ------------------------------------------------------------ softmax, results ------
    // two threads per row, each with half of the columns; the two warps of the same 32 rows agree on
    // the row's reference
    const int st = tid - T::kFirst;
    const int w = st / kStream, quad = warp & 3, half = (st >> 7) & 1;   // w: the stream
    const int mine = 32 * quad + lane;                                      // row of its tile
    constexpr int kCols = kTok / 2;
    const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_at + w * kTok + half * kCols;
    const uint32_t tO = tmem + lane_at + 2 * kTok + w * D + half * (D / 2);
    // (a negative factor becomes its queries' sign, so that the largest product has the largest
    // score)
    const float fk = fabsf(o.scale_log2);
    const uint32_t flip = o.scale_log2 < 0.f ? 0x80008000u : 0u;
    // A barrier of the two warps: whether both are alive. It has no limit, so neither may leave the other
    // there: what they do next is the same for both, since the runs come from one of them (their own
    // walks could differ if the lengths changed under the kernel), and a warp that has given up says
    // so here, at the next meeting, and not by staying away. (Meeting at an mbarrier with a limit
    // instead: 126.9 us against 124.2 for 1536 rows of 8 heads after 16k tokens.)
    auto together = [&](bool alive) {
      int gone;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\t"
          "barrier.cta.red.or.pred q, %1, 64, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
          : "=r"(gone)
          : "r"(1 + 4 * w + quad), "r"((int)!alive)
          : "memory");
      return !gone;
    };
    uint32_t jobs = 0, runs = 0, tile0 = 0;   // before this run; tiles of the CTA
    bool alive = true;   // the same for both warps, but between a wait and the next meeting
    for (;;) {
      if (half == 0) {
        if (!alive || !walk.next(a, &run)) run.t1 = 0;   // no more
        if (lane == 0) sh.run[w][quad] = run;
      }
      together(true);
      run = sh.run[w][quad];
      if (run.t1 == 0) break;
      const int n = run.t1 - run.t0, count = run.w == 2 ? n : (n + 1 - w) / 2;   // tiles of the stream
      const int row0 = (run.u * 2 + (run.w == 2 ? w : 0)) * kRows;
      if (count > 0) {
        // ---- queries: 16 bytes of every kStep-th row (all loads before the first store)
        constexpr int kChunks = D / 8, kStep = kStream / kChunks, kIters = kRows / kStep;
        const int lt = st % kStream, ch = lt % kChunks, r0 = lt / kChunks;
        const int each = over_m(a, kStep), rest = kStep - each * o.M, before = over_m(a, row0 + r0);
        int seq = run.p * a.per + before, m = row0 + r0 - before * o.M;
        uint4 in[kIters];
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          in[it] = make_uint4(0u, 0u, 0u, 0u);
          if (row0 + r0 + it * kStep < a.MP)
            in[it] = reinterpret_cast<const uint4*>(
                o.q + ((int64_t)seq * o.R * o.Hq + run.h * o.G) * D + sh.row_at[m])[ch];
          seq += each;
          m += rest;
          if (m >= o.M) m -= o.M, ++seq;
        }
        // (the sums of the run before have left the room)
        if (runs) alive = __all_sync(0xffffffffu, wait(&sh.qfree[w], (runs - 1) & 1));
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          uint4 x = in[it];
          if constexpr (kQ8) {   // each four values as (0, 2, 1, 3), the order of widened codes
            const uint4 y = x;
            x.x = __byte_perm(y.x, y.y, 0x5410);
            x.y = __byte_perm(y.x, y.y, 0x7632);
            x.z = __byte_perm(y.z, y.w, 0x5410);
            x.w = __byte_perm(y.z, y.w, 0x7632);
          }
          x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
          const int r = r0 + it * kStep;
          *reinterpret_cast<uint4*>(sQ + w * T::kQ + (ch >> 3) * (kRows * 128) + r * 128 +
                                    (((ch & 7) ^ (r & 7)) << 4)) = x;
        }
        fence_async();
        warp_arrive(&sh.qfull[w], lane);
      }
      // ref: a score from which 2^(factor (score - ref)) is taken; norm: this thread's part of the sum
      float ref = kNothing, norm = 0.f;
      for (int i = 0; i < count; ++i, ++jobs) {
        const int nt = run.w == 2 ? i : 2 * i + w;   // of the run
        const uint32_t tile = tile0 + nt;            // of the CTA
        const int slot = tile % kInfo, t0 = (run.t0 + nt) * kTok + half * kCols;
        alive = alive && wait(&sh.info[slot], (tile / kInfo) & 1) && wait(&sh.sfull[w], jobs & 1);
        alive = __all_sync(0xffffffffu, alive);
        sm100::tc_fence_after();
        volatile unsigned* const known = sh.runs;
        const unsigned there = known[slot];
        const bool is_edge = !page_full(run, t0 - half * kCols, there);
        const float* const scales = sScale + 2 * slot * kTok + half * kCols;
        // the tokens among 32 that count
        auto seen = [&](int c) {
          unsigned s = 0u;
          for (int x = 0; x < 32; x += 16)
            if (there >> ((half * kCols + c + x) >> page_shift) & 1u) s |= 0xFFFFu << x;
          const int rest = run.len - t0 - c;
          return rest >= 32 ? s : (rest <= 0 ? 0u : s & ((1u << rest) - 1u));
        };
        // T::kC scores before the factor (edge: masked)
        auto scores = [&](auto edge, int c, float (&x)[T::kC]) {
          __syncwarp();
          load_columns(tS + c, x);
          if constexpr (kQ8) {
#pragma unroll
            for (int j = 0; j < T::kC; j += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(scales + c + j);
              const float2 s0 = parts(mul2(pair(x[j], x[j + 1]), pair(k4.x, k4.y)));
              const float2 s1 = parts(mul2(pair(x[j + 2], x[j + 3]), pair(k4.z, k4.w)));
              x[j] = s0.x, x[j + 1] = s0.y, x[j + 2] = s1.x, x[j + 3] = s1.y;
            }
          }
          if constexpr (edge.value) {
            const unsigned s = seen(c);
#pragma unroll
            for (int j = 0; j < T::kC; ++j)
              if (!(s >> j & 1u)) x[j] = kNegInf;
          }
        };
        using Inner = std::false_type;
        using Edge = std::true_type;
        auto largest = [&](auto edge) {
          float top = kNegInf;
#pragma unroll 1
          for (int c = 0; c < kCols; c += T::kC) {
            float x[T::kC];
            scores(edge, c, x);
            float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < T::kC - 4; j += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], x[j + e], x[j + 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], x[T::kC - 4 + e]);
            top = max3(top, max3(m4[0], m4[1], m4[2]), m4[3]);
          }
          return top;
        };
        float top = is_edge ? largest(Edge{}) : largest(Inner{});
        sh.top[jobs & 1][w][half][mine] = top;
        if (!(alive = together(alive))) break;
        top = fmaxf(top, sh.top[jobs & 1][w][half ^ 1][mine]);
        // the reference moves only when a score exceeds it by 2^kSlack, and O with it (at rest: the
        // scores were issued after the product of this stream's tile before)
        const bool up = i == 0 || __fmul_rn(__fsub_rn(top, ref), fk) > kSlack;
        if (__any_sync(0xffffffffu, up)) {
          const float now = fmaxf(ref, top);
          const float f = i == 0 ? 0.f : exp2_fast(__fmul_rn(__fsub_rn(ref, now), fk));
          ref = now;
          norm = __fmul_rn(norm, f);
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              float x[16];
              uint32_t r[16];
              __syncwarp();
              load_columns(tO + c, x);
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__fmul_rn(x[j], f));
              st16(tO + c, r);
            }
          }
        }
        const f2 less = pair(-1.f, -1.f), back = pair(-ref, -ref), fk2 = pair(fk, fk);
        f2 sum0 = pair(0.f, 0.f), sum1 = pair(0.f, 0.f);
        auto weigh = [&](auto edge) {
#pragma unroll 1
          for (int c = 0; c < kCols; c += T::kC) {
            float x[T::kC];
            scores(edge, c, x);
#pragma unroll
            for (int c16 = 0; c16 < T::kC; c16 += 16) {   // 8 columns of high parts, 8 of low ones
              uint32_t r[16];
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                [[maybe_unused]] float4 v4;
                if constexpr (kQ8)
                  v4 = *reinterpret_cast<const float4*>(scales + kTok + c + c16 + j);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  const float x0 = x[c16 + j + e], x1 = x[c16 + j + e + 1];
                  float2 d = parts(mul2(add2(pair(x0, x1), back), fk2));
                  if constexpr (edge.value) {   // (a factor of 0 makes NaN of -infinity)
                    d.x = x0 == kNegInf ? kNegInf : d.x;
                    d.y = x1 == kNegInf ? kNegInf : d.y;
                  }
                  f2 p = pair(exp2_fast(d.x), exp2_fast(d.y));
                  if (e) sum1 = add2(sum1, p);
                  else sum0 = add2(sum0, p);
                  if constexpr (kQ8) {
                    p = mul2(p, e ? pair(v4.z, v4.w) : pair(v4.x, v4.y));
                    if constexpr (edge.value) {   // a masked token's scale may be anything
                      float2 y = parts(p);
                      y.x = d.x == kNegInf ? 0.f : y.x;
                      y.y = d.y == kNegInf ? 0.f : y.y;
                      p = pair(y.x, y.y);
                    }
                  }
                  const float2 y = parts(p);
                  const uint32_t hi = pack2(y.x, y.y);
                  const float2 rest = parts(fma2(pair(bf16_lo(hi), bf16_hi(hi)), less, p));
                  r[(j + e) / 2] = hi;
                  r[8 + (j + e) / 2] = pack2(rest.x, rest.y);
                }
              }
              __syncwarp();
              st16(tS + c + c16, r);
            }
            if (c + T::kC == kCols / 2) {   // half of this thread's columns: products with these may begin
              tmem_wait_st();
              sm100::tc_fence_before();
              warp_arrive(&sh.pfull[w][0], lane);
            }
          }
        };
        if (is_edge) weigh(Edge{});
        else weigh(Inner{});
        const float2 s2 = parts(add2(sum0, sum1));
        norm = __fadd_rn(norm, __fadd_rn(s2.x, s2.y));
        tmem_wait_st();
        sm100::tc_fence_before();
        warp_arrive(&sh.pfull[w][1], lane);
      }
      // ---------------------------------------------------------------- results -----------
      if (alive) {
        sh.top[jobs & 1][w][half][mine] = norm;
        together(true);
        const float other = sh.top[jobs & 1][w][half ^ 1][mine];
        norm = half ? __fadd_rn(other, norm) : __fadd_rn(norm, other);
        const int64_t at = (unit_piece(a, run.p, run.h, run.u, blockIdx.x) * 2 + w) * a.rows + mine;
        // (never -infinity where there is a sum, of NaN scores for instance: the join leaves those out)
        if (half == 0 && row0 + mine < a.MP)
          *reinterpret_cast<float2*>(a.part_ml + 2 * at) =
              make_float2(norm == 0.f ? kNegInf : fmaxf(__fmul_rn(ref, fk), kNothing), norm);
        if (count > 0) {
          alive = __all_sync(0xffffffffu, wait(&sh.odone[w], runs & 1));
          ++runs;
          if (alive) {
            sm100::tc_fence_after();
            // (32 rows x 32 columns at a time pass through the warp's part of the queries' room, so
            // that whole lines are written)
            float4* const room =
                reinterpret_cast<float4*>(sQ + w * T::kQ + (4 * half + quad) * (T::kQ / 8));
            float* const to = a.part_o + (at - lane) * D + half * (D / 2);
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 32) {
              float x[32];
              __syncwarp();
              ld32(tO + c, x);
#pragma unroll
              for (int j = 0; j < 8; ++j)   // (columns of widened codes: (0, 2, 1, 3))
                room[8 * lane + (j ^ (lane & 7))] =
                    kQ8 ? make_float4(x[4 * j], x[4 * j + 2], x[4 * j + 1], x[4 * j + 3])
                        : make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int r = 4 * j + lane / 8, col = lane % 8;
                if (row0 + 32 * quad + r < a.MP)
                  reinterpret_cast<float4*>(to + r * D + c)[col] = room[8 * r + (col ^ (r & 7))];
              }
            }
            warp_arrive(&sh.qfree[w], lane);
            sm100::tc_fence_before();
          }
        }
        alive = together(alive);   // (and sh.top is free)
        if (alive && half == 0 && w == 0 && quad == 0 && lane == 0) {
          int* const span = a.span + 2 * (((int64_t)run.p * o.c.heads + run.h) * a.units + run.u);
          if (run.t0 == 0) span[0] = blockIdx.x;
          if (run.t1 == (run.len + kTok - 1) / kTok) span[1] = blockIdx.x;
        }
      }
      tile0 += n;
    }
  } else if (warp > 0 && warp <= T::kBringers) {
    // ------------------------------------------------------------- tiles from the pages ---
    // bf16: a warp copies key tiles and one value tiles, page by page. Q8: all widen both, in turn.
    const int pages = kTok >> page_shift;
    const bool values = warp == 2;   // (bf16)
    const bool teller = warp == 1;   // fills in the tile information
    int done = 0, st = 0, told = 0;
    uint32_t par = 1;
    bool alive = true;
    auto tell = [&](int page, unsigned there) {
      // (its slot is free: the scores of the tile kRing before are done)
      const int slot = told++ % kInfo;
      if (lane == 0) {
        sh.runs[slot] = there;
        sm100::mbar_arrive_expect_tx(&sh.info[slot], kQ8 ? __popc(there) * pt * 8 : 0);
      }
      __syncwarp();
      if (kQ8 && page >= 0) {
        const int64_t at = page * o.c.scale_stride + ((int64_t)run.h << page_shift);
        float* const dst = sScale + 2 * slot * kTok + lane * pt;
        bulk_copy(dst, o.c.k_scale + at, pt * 4, &sh.info[slot]);
        bulk_copy(dst + kTok, o.c.v_scale + at, pt * 4, &sh.info[slot]);
      }
    };
    if constexpr (kQ8) {
      // a lane takes 16 codes of a token; a warp 512, of kTokens tokens, every kBringers-th time. One
      // matrix's codes are on their way while the other's are widened.
      constexpr int kTokens = 512 / D, kTurns = kTok / kTokens;
      constexpr int kMost = (kTurns + T::kBringers - 1) / T::kBringers;
      // (eight lanes take 4 chunks of 2 rows, so that a quarter warp's stores meet all banks)
      const int my_row = D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) : lane >> 2;
      const int my_chunk = D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane & 3;
      const int turn0 = warp - 1;
      auto fetch = [&](uint4 (&codes)[kMost], const uint8_t* from, int page, int t0) {
#pragma unroll
        for (int it = 0; it < kMost; ++it) {
          const int turn = turn0 + it * T::kBringers, r = (turn * kTokens + my_row) & (kTok - 1);
          const int pg = __shfl_sync(0xffffffffu, page, r >> page_shift);
          codes[it] = make_uint4(0u, 0u, 0u, 0u);
          if (turn < kTurns && pg >= 0 && t0 + r < run.len)
            codes[it] = __ldg(reinterpret_cast<const uint4*>(
                from + pg * o.c.stride + (((int64_t)run.h << page_shift) + (r & (pt - 1))) * D +
                my_chunk * 16));
        }
      };
      auto widen = [&](const uint4 (&codes)[kMost], uint8_t* tile) {
        tile += (my_chunk >> 2) * (kTok * 128);
#pragma unroll
        for (int it = 0; it < kMost; ++it) {
          const int turn = turn0 + it * T::kBringers, r = turn * kTokens + my_row;
          if (turn >= kTurns) break;
          const uint4 v = codes[it];
          const int c0 = ((2 * my_chunk & 7) ^ (r & 7)) << 4;
          *reinterpret_cast<uint4*>(tile + r * 128 + c0) = make_uint4(
              code_pair(v.x), code_pair(v.x >> 8), code_pair(v.y), code_pair(v.y >> 8));
          *reinterpret_cast<uint4*>(tile + r * 128 + (c0 ^ 16)) = make_uint4(
              code_pair(v.z), code_pair(v.z >> 8), code_pair(v.w), code_pair(v.w >> 8));
        }
      };
      while (alive && walk.next(a, &run)) {
        auto page_of_tile = [&](int t) {
          return lane < pages && t < run.t1 ? prefix_page(a, run.p, t * kTok + lane * pt, run.len) : -1;
        };
        int page = page_of_tile(run.t0);
        uint4 kc[kMost], vc[kMost];
        fetch(kc, o.c.k, page, run.t0 * kTok);
        for (int t = run.t0; t < run.t1; ++t) {
          const int next = page_of_tile(t + 1);
          const unsigned there = __ballot_sync(0xffffffffu, page >= 0);
          fetch(vc, o.c.v, page, t * kTok);
          if (done >= kRing) alive = wait(&sh.kfree[st], par);
          if (!(alive = __all_sync(0xffffffffu, alive))) break;
          if (teller) tell(page, there);
          widen(kc, sK + st * T::kMat);
          fence_async();
          warp_arrive(&sh.kfull[st], lane);
          if (t + 1 < run.t1) fetch(kc, o.c.k, next, (t + 1) * kTok);
          if (done >= kRing) alive = wait(&sh.vfree[st], par);
          if (!(alive = __all_sync(0xffffffffu, alive))) break;
          widen(vc, sV + st * T::kMat);
          fence_async();
          warp_arrive(&sh.vfull[st], lane);
          ++done;
          if (++st == kRing) st = 0, par ^= 1;
          page = next;
        }
      }
      if (teller)   // copies in flight end (bounded) before the CTA does, whoever gives up and when
        for (int j = told - kInfo < 0 ? 0 : told - kInfo; j < told; ++j)
          sm100::mbar_wait(&sh.info[j % kInfo], (j / kInfo) & 1, kEndPolls);
    } else {
      uint64_t* const full = values ? sh.vfull : sh.kfull;
      uint64_t* const free_bar = values ? sh.vfree : sh.kfree;
      uint8_t* const tiles = values ? sV : sK;
      int edges = 0;
      while (alive && walk.next(a, &run)) {
        int page = lane < pages ? prefix_page(a, run.p, run.t0 * kTok + lane * pt, run.len) : -1;
        for (int t = run.t0; t < run.t1; ++t) {
          const int t0 = t * kTok;
          const bool ok = page >= 0;
          const unsigned there = __ballot_sync(0xffffffffu, ok);
          if (done >= kRing) alive = wait(&free_bar[st], par);
          if (!(alive = __all_sync(0xffffffffu, alive))) break;
          if (teller) tell(page, there);
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
              sm100::mbar_wait(&sh.vedge, edge_par, kEndPolls);
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
          ++done;
          if (++st == kRing) st = 0, par ^= 1;
          page = -1;
          if (t + 1 < run.t1 && lane < pages)
            page = prefix_page(a, run.p, (t + 1) * kTok + lane * pt, run.len);
        }
      }
      // copies in flight end (bounded) before the CTA does, whoever gives up and when
      for (int j = done - kRing < 0 ? 0 : done - kRing; j < done; ++j)
        sm100::mbar_wait(&full[j % kRing], (j / kRing) & 1, kEndPolls);
    }
  } else if (warp == 0) {
    // --------------------------------------------------------------------------- MMAs ----
    // One lane issues, but the whole warp walks the loop, and what the MMAs are given is kept the same
    // for all lanes in a way that the compiler sees (constants, tensor memory from column 0 on,
    // reductions of loop bounds): operands then stay in uniform registers, and are not moved there for
    // every MMA (128 against 132 us for 1536 rows of 8 heads over 16k tokens).
    const bool leader = elect_one();
    constexpr uint32_t s_idesc = sm100::idesc_bf16_f32(kRows, kTok);
    constexpr uint32_t o_idesc = sm100::idesc_bf16_f32(kRows, D) | (kMajorMN & (1u << 16));
    const uint64_t q_desc = sm100::desc_k_sw128(smem_at(sQ));
    const uint64_t k_desc = sm100::desc_k_sw128(smem_at(sK));
    const uint64_t v_desc = desc_mn_sw128(smem_at(sV), kTok * 128);
    uint32_t ktiles = 0, vtiles = 0;    // tiles taken up
    uint32_t q_par = 0, p_par = 0;      // bit w: parity of stream w
    bool alive = true;
    while (alive && walk.next(a, &run)) {
      const bool two = __reduce_max_sync(0xffffffffu, run.w) == 2;   // row tiles
      const int jobs = __reduce_max_sync(0xffffffffu, (run.t1 - run.t0) * run.w);
      auto score = [&](auto stream) {
        constexpr int w = decltype(stream)::value;
        const uint32_t st = (ktiles - 1) % kRing;
        const uint64_t kd = k_desc + st * (uint32_t)(T::kMat >> 4);
        const uint64_t qd = q_desc + (uint32_t)w * (T::kQ >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {   // 16 values: 32 bytes, or the next 64 values
          const uint32_t off = (ks >> 2) * (kTok * 8) + (ks & 3) * 2;
          sm100::mma_bf16(w * kTok, qd + off, kd + off, s_idesc, ks > 0);
        }
        sm100::mma_commit(&sh.sfull[w]);
        if (!two || w == 1) sm100::mma_commit(&sh.kfree[st]);
      };
      // half of the sums: the steps whose P comes first (32 of 64 columns), or the others
      auto sum = [&](auto stream, auto part, bool fresh) {
        constexpr int w = decltype(stream)::value, x = decltype(part)::value;
        const uint64_t vd = v_desc + (vtiles - 1) % kRing * (uint32_t)(T::kMat >> 4);
        constexpr uint32_t p = w * kTok, to = 2 * kTok + w * D;
#pragma unroll
        for (int n = 0; n < kTok / 32; ++n) {   // 16 tokens: 2 KB of values, 16 columns of P
          const int ks = (n >> 1) * 4 + 2 * x + (n & 1);
          mma_tmem_a(to, p + 16 * ks, vd + ks * 128, o_idesc, !(fresh && n == 0));
          mma_tmem_a(to, p + 16 * ks + 8, vd + ks * 128, o_idesc, 1u);
        }
      };
      using C0 = std::integral_constant<int, 0>;
      using C1 = std::integral_constant<int, 1>;
      // Tile j's sums, and behind them, without a pause, the scores of its stream's next tile. What they
      // need is looked up together, so that it costs one round trip when all of it is there.
      auto unit = [&](auto stream, int j) {
        constexpr int w = decltype(stream)::value;
        const bool more = j + 2 < jobs, opens = !two || w == 0, keys = opens && more;
        if (opens) ++vtiles;
        if (keys) ++ktiles;
        const uint32_t vt = vtiles - 1, kt = ktiles - 1, p = p_par >> w & 1u;
        uint64_t* const p0 = &sh.pfull[w][0];
        uint64_t* const v = opens ? &sh.vfull[vt % kRing] : p0;
        uint64_t* const k = keys ? &sh.kfull[kt % kRing] : p0;
        const uint32_t vp = opens ? (vt / kRing) & 1 : p, kp = keys ? (kt / kRing) & 1 : p;
        uint64_t* const p1 = &sh.pfull[w][1];
        // (Q8: the sums do not wait for keys that are still being widened)
        const uint32_t found = kQ8 ? ready3_1(v, vp, v, vp, p0, p, p1, p)
                                   : ready3_1(v, vp, k, kp, p0, p, p1, p);
        bool ok = __all_sync(0xffffffffu, found & 1u);
        if (!ok) {
          ok = wait(v, vp) && (kQ8 || wait(k, kp)) && wait(p0, p);
          if (!__all_sync(0xffffffffu, ok)) return false;
        }
        p_par ^= 1u << w;
        auto rest = [&] {
          sum(stream, C1{}, false);
          if (!two || w == 1) sm100::mma_commit(&sh.vfree[vt % kRing]);
          if (!more) sm100::mma_commit(&sh.odone[w]);
          if (!kQ8 && more) score(stream);
        };
        sm100::tc_fence_after();
        if (__all_sync(0xffffffffu, found == 3u)) {   // all of P is there: this warp is late
          if (leader) {
            sum(stream, C0{}, j < 2);
            rest();
          }
        } else {
          if (leader) sum(stream, C0{}, j < 2);
          __syncwarp();
          ok = wait(p1, p);
          if (!__all_sync(0xffffffffu, ok)) return false;
          sm100::tc_fence_after();
          if (leader) rest();
        }
        __syncwarp();
        if (kQ8 && more) {
          if (!__all_sync(0xffffffffu, wait(k, kp))) return false;
          sm100::tc_fence_after();
          if (leader) score(stream);
          __syncwarp();
        }
        return true;
      };
      // a stream's first scores of the run
      auto first = [&](auto stream) {
        constexpr int w = decltype(stream)::value;
        bool ok = wait(&sh.qfull[w], q_par >> w & 1u);
        q_par ^= 1u << w;
        if (!two || w == 0) {
          ++ktiles;
          ok = ok && wait(&sh.kfull[(ktiles - 1) % kRing], ((ktiles - 1) / kRing) & 1);
        }
        if (!__all_sync(0xffffffffu, ok)) return false;
        sm100::tc_fence_after();
        if (leader) score(stream);
        __syncwarp();
        return true;
      };
      alive = first(C0{}) && (jobs < 2 || first(C1{}));
      for (int j = 0; j < jobs && alive; j += 2)
        alive = unit(C0{}, j) && (j + 1 >= jobs || unit(C1{}, j + 1));
    }
    // MMAs issued but maybe not observed complete: wait (bounded) before TMEM is freed
    if (leader) sm100::mma_commit(&sh.end);
    __syncwarp();
    sm100::mbar_wait(&sh.end, 0, kEndPolls);
  }
  __syncwarp();
  pdl_wait();
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 0) sm100::tmem_dealloc(sh.tmem, 512);
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
