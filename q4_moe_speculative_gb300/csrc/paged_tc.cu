// paged_tc.cu — the attention over the paged cache on the 5th-generation tensor cores, for the
// calls whose work pays for it (choice and figures in paged_attn.cu). The list of tiles, the
// split over CTAs and the join are those of paged_attn.cu, with tiles of 128 tokens.
//
// Tokens are the M = 128 rows of both products, so every thread of the softmax owns one token
// and its scales are scalars:
//   S^T = K Q^T      A = the key tile [128 tokens][D], B = the queries [N rows][D], both
//                    K-major; TMEM lane = token, column = query row (N = M up to a multiple
//                    of 32);
//   O^T += V^T P^T   A = the value tile, read MN-major (its rows are tokens, the MMA's K),
//                    B = P [128 tokens][N rows], also MN-major, as a high and a low bf16
//                    part; TMEM lane = value dimension, column = query row (of either part:
//                    see Parts).
// Roles: warps 0-7 turn scores into P (a row's reference maximum moves only when a score
// exceeds it by 2^8, agreed by one barrier vote per tile), keep the normaliser of their
// token in TMEM, and write the results; two warps copy tiles page by page, by TMA straight
// into the swizzled operand layout (bf16) or as raw codes that eight more warps widen to bf16
// (Q8); one thread each of the last two warps issues the MMAs of S and of O. Up to 96 rows S is
// double-buffered: the next tile's scores are computed while this tile's are exponentiated.
// Measured: 96 rows of one head of 300k tokens, D = 128, bf16 (154 MB) 43.5 us with the join,
// which takes 6 to 8 of them; 4 sequences x 8 heads of 64k, bf16 (1.05 GB), 40 and 64 rows 160 us
// (6.6 TB/s, bound by memory), 96 rows 195, 128 rows 291; Q8 (0.54 GB), 64 rows 206, 96 rows 314,
// 128 rows 356, and D = 64, bf16, 64 rows 135 (0.52 GB), bound by the chain of a tile through
// widening, scores and P: beyond 64 rows shared memory has no room for two tiles of all of them.
// (With one part of P beyond 64 rows: 96 rows 165 us, Q8 234; 128 rows 247, Q8 284; results off
// by 1.4 times their own rounding. Bringing the tiles behind the ring into L2 ahead of time
// costs 8% two tiles ahead, 37% with four.)
// A token of a bf16 cache that only some rows see may hold infinities, and 0 x infinity is
// not 0: where one of its values is not finite they are cleared before the product, and the
// (at most 7) such tokens are added row by row when the run ends. Every wait is bounded; a
// give-up sets the status word.
#include "paged.cuh"
#include "sm100.cuh"

namespace dsmoe {
namespace paged_tc {

using namespace paged;

constexpr int kTok = 128;
constexpr int kScore = 256;               // softmax threads: two per token, half of the rows each
constexpr int kMaxN = kTcMaxRows;                 // query rows, as a multiple of 32
constexpr int kMaxRing = 4;
constexpr int kInfo = 8;                  // tiles whose pages and scales are at hand
// Reference of a row that has seen no token yet: the least finite value, so that any score that
// counts is above it by more than kSlack, or is equal to it and has the weight 1.
constexpr float kNothing = -3.402823466e38f;
constexpr uint32_t kWaitPolls = 1u << 20;

struct TcArgs {
  PagedArgs p;
  int N;            // query rows, padded to a multiple of 32
  int k_ring, v_ring;   // stages of the key and of the value operand tiles
  int raw;          // stages of raw codes (Q8)
  int p_bufs;       // 2: P of one tile is multiplied while the next is formed
  int s_bufs;       // 2: the next tile's scores are computed while this tile's are read
  uint32_t tmem_cols;
};

// Where the two parts of P are among its columns, in chunks of 64 (128 bytes of a token), and what
// they are added to in O. Up to 64 rows: side by side, and O has columns of either, so that
// one MMA does both. 128 rows: two chunks each, two MMAs into the same columns (tensor memory
// has 512). 96 rows: high 0..63; high and low 64..95; low 0..63; an MMA for each, the third into
// the columns of the first. MMAs into the same columns follow one another in order because
// their shapes are the same as well.
template <bool kBeside>   // up to 64 rows
struct Parts {
  int N;
  __host__ __device__ int p_chunks() const { return (2 * N + 63) / 64; }
  __host__ __device__ int o_columns() const { return kBeside ? 2 * N : 128; }
  // of the low part of rows c .. c + 15, in P
  __device__ int low_in_p(int c) const {
    return kBeside ? N + c : (N == 96 && c >= 64 ? c + 32 : 128 + c);
  }
  // and in O, where it has columns there
  __device__ bool low_apart(int c) const { return kBeside || (N == 96 && c >= 64); }
  __device__ int low_in_o(int c) const { return kBeside ? N + c : c + 32; }
  // the MMAs of one step, their columns of P, and where the x-th one's sums are in O
  __device__ int mmas() const { return kBeside ? 1 : (N == 96 ? 3 : 2); }
  __device__ int mma_columns() const { return kBeside ? 2 * N : (N == 96 ? 64 : 128); }
  __device__ int mma_at(int x) const { return N == 96 && x == 1 ? 64 : 0; }
  __device__ bool mma_adds(int x) const { return x == mmas() - 1 && x > 0; }   // never the first
};

template <int D, bool kQ8>
struct Tc {
  static constexpr int kHalves = D / 64;
  static constexpr int kMat = kTok * D * 2;             // bytes of an operand tile
  static constexpr int kRawMat = kQ8 ? kTok * D : 0;
  static constexpr int kWiden = kQ8 ? 128 : 0;          // threads per matrix that widen codes
  static constexpr int kThreads = kScore + 2 * kWiden + 128;
  static constexpr int kFetchWarp = kThreads / 32 - 4;  // keys; the next one: values
  static constexpr int kMmaWarp = kThreads / 32 - 2;    // scores; the next one: values
};

struct alignas(16) TcSmem {   // small arrays in front of the tiles
  uint64_t kfull[kMaxRing], vfull[kMaxRing], kfree[kMaxRing], vfree[kMaxRing];
  uint64_t sfull[2], pfull[2], odone[2], qfull;
  uint64_t raw_full[2][kMaxRing], raw_free[2][kMaxRing];   // Q8: codes of keys, of values
  uint64_t info[kInfo], vedge;
  uint32_t tmem;
  int abort;
  alignas(16) float ref[kMaxN];   // (read four at a time)
  float fac[kMaxN], red[4 * kMaxN], norm[kMaxN];
  int row_r[kMaxN];           // verify row of a query row
  int row_at[kMaxN];          // and where its values start in a sequence's queries or results
  alignas(16) float pe[7][kMaxN];   // P of the tokens that only some rows see
  unsigned runs[kInfo];       // which pages of a tile are there
  unsigned apart[kInfo];      // tokens behind seen0 whose values are not finite, and cleared
};
constexpr int kSmallBytes = (sizeof(TcSmem) + 1023) / 1024 * 1024;
static_assert(kSmallBytes <= 10240, "the largest call fills the SM's shared memory");

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Copies bytes (a multiple of 16, both addresses 16-byte aligned), counted by `bar`.
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(smem_at(dst)), "l"(src), "r"(bytes), "r"(smem_at(bar))
      : "memory");
}
// Whether one of two bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(bar)) : "memory");
}
// One arrival for the whole warp, after what its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) arrive(bar);
}
// Whether three phases are complete: one round trip when they are.
__device__ __forceinline__ bool ready3(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                       uint64_t* c, uint32_t pc) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q, s;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 s, [%5], %6;\n\t"
      "and.pred p, p, q;\n\tand.pred p, p, s;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(smem_at(a)), "r"(pa), "r"(smem_at(b)), "r"(pb), "r"(smem_at(c)), "r"(pc)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void score_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool score_any(bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)x)
      : "memory");
  return r != 0;
}
// An operand stored with its K (tokens) as rows of 128 bytes of 64 M or N values, 128-byte
// swizzle: groups of 8 tokens are 1024 bytes apart, the next 64 values `next` bytes further.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(next >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kMajorMN = (1u << 15) | (1u << 16);   // instruction descriptor: A and B

// To 16 columns; tmem_wait_st() waits for it.
__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Twice 16 columns, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t at0, float (&v)[16], uint32_t at1,
                                            float (&w)[16]) {
  uint32_t r[16], x[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]),
        "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]),
        "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
      : "r"(at0), "r"(at1)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]), w[i] = __uint_as_float(x[i]);
}

// Combines 16 columns over the warp's lanes: lanes j and j + 16 end up with column j.
template <typename Op>
__device__ __forceinline__ float over_lanes(float (&v)[16], int lane, Op op) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

template <int D, bool kQ8, bool kBeside>
__global__ void __launch_bounds__(Tc<D, kQ8>::kThreads, 1)
    k_paged_tc(const __grid_constant__ TcArgs ta, const __grid_constant__ CUtensorMap k_map,
               const __grid_constant__ CUtensorMap v_map) {
  using T = Tc<D, kQ8>;
  extern __shared__ uint8_t smem_raw[];
  const PagedArgs& a = ta.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t pad = (1024u - (smem_at(smem_raw) & 1023u)) & 1023u;
  uint8_t* const base = smem_raw + pad;
  TcSmem& sh = *reinterpret_cast<TcSmem*>(base);
  const int N = ta.N;                                           // columns of S
  const Parts<kBeside> cols{N};
  uint8_t* const sQ = base + kSmallBytes;                       // [halves][N][128 B]
  const uint32_t p_size = (uint32_t)cols.p_chunks() * kTok * 128;
  uint8_t* const sP = sQ + T::kHalves * N * 128;                // [buffers][chunks][tokens][128 B]
  uint8_t* const sK = sP + ta.p_bufs * p_size;                  // [ring][halves][tokens][128 B]
  uint8_t* const sV = sK + ta.k_ring * T::kMat;
  uint8_t* const sRaw = sV + ta.v_ring * T::kMat;               // Q8: [2][raw][tokens][D]
  float* const sScale = reinterpret_cast<float*>(sRaw + 2 * ta.raw * T::kRawMat);  // [kInfo][2][tokens]

  if (tid == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      sm100::mbar_init(&sh.kfull[i], kQ8 ? T::kWiden / 32 : 1);
      sm100::mbar_init(&sh.vfull[i], kQ8 ? T::kWiden / 32 : 1);
      sm100::mbar_init(&sh.kfree[i], 1);
      sm100::mbar_init(&sh.vfree[i], 1);
      for (int x = 0; kQ8 && x < 2; ++x) {
        sm100::mbar_init(&sh.raw_full[x][i], 1);
        sm100::mbar_init(&sh.raw_free[x][i], T::kWiden / 32);
      }
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&sh.sfull[i], 1);
      sm100::mbar_init(&sh.pfull[i], kScore / 32);
      sm100::mbar_init(&sh.odone[i], 1);
    }
    sm100::mbar_init(&sh.qfull, kScore / 32);
    for (int i = 0; i < kInfo; ++i) sm100::mbar_init(&sh.info[i], 1);
    sm100::mbar_init(&sh.vedge, 1);
    sh.abort = 0;
    sm100::fence_mbar_init();
  }
  if (tid < kMaxN) {
    sh.row_r[tid] = tid / a.G;
    sh.row_at[tid] = (tid / a.G * a.Hq + tid % a.G) * D;
  }
  if (warp == 0) {
    sm100::tmem_alloc(&sh.tmem, ta.tmem_cols);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (!kQ8 && tid < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid ? &v_map : &k_map) : "memory");
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0) *a.status = 0u;

  Cursor cur{};
  const int n = cta_run(a, blockIdx.x, lane, &cur);   // tiles of this CTA

  volatile int* const abort_flag = &sh.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
      if (sm100::mbar_try_wait(bar, parity)) return true;
      if ((i & 63u) == 63u && *abort_flag) return false;
    }
    *abort_flag = 1;
    flag_status(a.status, kStatusTimeout);
    return false;
  };
  const int page_mask = (1 << a.c.page_shift) - 1;

  if (n == 0) {
    // nothing to do
  } else if (warp < kScore / 32) {
    // ------------------------------------------------------------ softmax, results ------
    // thread = token tk (TMEM lane) x the query rows col0 .. col0 + N / 2 - 1, 16 at a time
    const int quad = warp & 3, tk = 32 * quad + lane, half = N / 2, col0 = (warp >> 2) * half;
    const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + lane_at + ta.s_bufs * N;
    const uint16_t* const q0 = a.q;
    auto seq_at = [&](const Cursor& c) {   // of its queries and results for the key head
      return ((int64_t)c.b * a.R * a.Hq + c.h * a.G) * D;
    };
    auto stage_q = [&](const Cursor& c) {
      constexpr int kChunks = D / 8;
      const int64_t at = seq_at(c);
      // (all loads of a batch before its first store; the Q8 kernel has 96 registers: 32 rows, 32
      // sequences x 8 heads at 8k, 169 us with batches of 2, 179 with 4, 183 with 8)
      constexpr int kMost = (kMaxN * kChunks + kScore - 1) / kScore, kBatch = kQ8 ? 2 : kMost;
#pragma unroll 1
      for (int u0 = 0; u0 < kMost && (tid + u0 * kScore) / kChunks < N; u0 += kBatch) {
        uint4 in[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int idx = tid + (u0 + u) * kScore, r = idx / kChunks;
          in[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < a.M)
            in[u] = reinterpret_cast<const uint4*>(q0 + at + sh.row_at[r])[idx % kChunks];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int idx = tid + (u0 + u) * kScore, r = idx / kChunks, ch = idx % kChunks;
          if (r >= N) break;
          uint4 x = in[u];
          if constexpr (kQ8) {   // each four values as (0, 2, 1, 3), the order of widened codes
            x.x = __byte_perm(in[u].x, in[u].y, 0x5410);
            x.y = __byte_perm(in[u].x, in[u].y, 0x7632);
            x.z = __byte_perm(in[u].z, in[u].w, 0x5410);
            x.w = __byte_perm(in[u].z, in[u].w, 0x7632);
          }
          *reinterpret_cast<uint4*>(sQ + (ch >> 3) * N * 128 + r * 128 +
                                    (((ch & 7) ^ (r & 7)) << 4)) = x;
        }
      }
      fence_async();
      warp_arrive(&sh.qfull, lane);
    };
    Cursor n1 = cur;                   // the next tile
    stage_q(cur);
    bool alive = true;
    for (int i = 0; i < n && alive; ++i) {
      if (i + 1 < n) n1.next(a);
      const bool first = i == 0 || cur.tile == 0;
      const bool ends = cur.tile + 1 == cur.tiles;      // of the (sequence, head)
      const bool last = ends || i + 1 == n;             // of this run
      const int t0 = cur.tile * kTok, tok = t0 + tk;
      const int seen0 = cur.len - (a.R - 1);            // row r sees t < seen0 + r
      const uint32_t tS = tmem + lane_at + (i & (ta.s_bufs - 1)) * N;
      const uint32_t tL = tO + cols.o_columns() + (i & 1) * N;
      const uint32_t tLnew = tO + cols.o_columns() + (~i & 1) * N;
      uint8_t* const p_at = sP + (i & (ta.p_bufs - 1)) * p_size + tk * 128;
      const int slot = i % kInfo;
      // what is known of the tile, its scores, and P's buffer (free after the tile p_bufs before)
      const int before = i - ta.p_bufs;
      uint64_t* const p_free = before >= 0 ? &sh.odone[before & 1] : &sh.sfull[i & 1];
      const uint32_t p_par = before >= 0 ? (before >> 1) & 1 : (i >> 1) & 1;
      if (!ready3(&sh.info[slot], (i / kInfo) & 1, &sh.sfull[i & 1], (i >> 1) & 1, p_free, p_par))
        alive = wait(&sh.info[slot], (i / kInfo) & 1) && wait(&sh.sfull[i & 1], (i >> 1) & 1) &&
                wait(p_free, p_par);
      sm100::tc_fence_after();
      if (last && i + 1 < n) {   // the scores with these queries are done
        alive = !score_any(!alive);
        if (!alive) break;
        stage_q(n1);
      }
      const bool ok = tok < cur.len && (sh.runs[slot] >> (tk >> a.c.page_shift) & 1u);
      const bool edge = __any_sync(0xffffffffu, !ok || tok >= seen0);
      const bool partly = !kQ8 && tok >= seen0 && tok < cur.len;   // some rows may not see it
      const float fk = kQ8 ? __fmul_rn(a.scale_log2, sScale[2 * slot * kTok + tk]) : a.scale_log2;
      const float vs0 = kQ8 ? sScale[(2 * slot + 1) * kTok + tk] : 1.f;
      auto mask = [&](int c, float (&t)[16]) {
        if (!edge) return;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!ok || tok - seen0 >= sh.row_r[c + j]) t[j] = kNegInf;
      };
      // Moves the references up to what this tile needs, and the sums with them. False: a wait
      // gave up (the same for all threads).
      auto move = [&] {
        if (alive && !first) alive = wait(&sh.odone[(i - 1) & 1], ((i - 1) >> 1) & 1);   // O rests
        if (score_any(!alive)) return false;
        sm100::tc_fence_after();
        float t[16];
#pragma unroll 1
        for (int c = col0; c < col0 + half; c += 16) {
          __syncwarp();
          sm100::tmem_ld16(tS + c, t);
#pragma unroll
          for (int j = 0; j < 16; ++j) t[j] = __fmul_rn(t[j], fk);
          mask(c, t);
          const float top = over_lanes(t, lane, [](float x, float y) { return fmaxf(x, y); });
          if (lane < 16) sh.red[kMaxN * quad + c + lane] = top;
        }
        score_sync();
        if (tid < N) {
          const float was = first ? kNothing : sh.ref[tid];
          const float now = fmaxf(was, fmaxf(fmaxf(sh.red[tid], sh.red[kMaxN + tid]),
                                             fmaxf(sh.red[2 * kMaxN + tid], sh.red[3 * kMaxN + tid])));
          sh.ref[tid] = now;
          sh.fac[tid] = exp2_fast(__fsub_rn(was, now));
        }
        score_sync();
        if (first) return true;
#pragma unroll 1
        for (int c = col0; c < col0 + half; c += 16) {
#pragma unroll 1
          for (int x = 0; x < 3; ++x) {    // O, its low part, the sums
            if (x == 1 && !cols.low_apart(c)) continue;
            const uint32_t at = x == 2 ? tL + c : tO + (x ? cols.low_in_o(c) : c);
            __syncwarp();
            sm100::tmem_ld16(at, t);
#pragma unroll
            for (int j = 0; j < 16; ++j) t[j] = __fmul_rn(t[j], sh.fac[c + j]);
            tmem_st(at, t);
          }
        }
        if (!kQ8)
          for (int x = tid; x < 7 * N; x += kScore)
            if (seen0 + x / N < t0) {
              float& pe = sh.pe[x / N][x % N];
              pe = __fmul_rn(pe, sh.fac[x % N]);
            }
        tmem_wait_st();
        return true;
      };
      // (the score is rounded as it was for the reference, so that the largest one is off by
      // nothing from it whatever its size)
      const f2 fk2 = pair(fk, fk), less = pair(-1.f, -1.f);
      auto minus = [&](float& x, float& y, float rx, float ry) {
        const float2 d = parts(fma2(pair(rx, ry), less, mul2(pair(x, y), fk2)));
        x = d.x;
        y = d.y;
      };
      float l[16];
      for (bool settled = first;; settled = true) {   // P of the tile, at most twice
        if (settled) alive = move();
        if (settled && !alive) break;
        bool over = !alive;
#pragma unroll 1
        for (int c = col0; c < col0 + half; c += 16) {
          float t[16];
          float4 r4[4];
#pragma unroll
          for (int j4 = 0; j4 < 4; ++j4)
            r4[j4] = *reinterpret_cast<const float4*>(sh.ref + c + 4 * j4);
          __syncwarp();
          tmem_ld16x2(tS + c, t, tL + c, l);
          if (first) {
#pragma unroll
            for (int j = 0; j < 16; ++j) l[j] = 0.f;
          }
#pragma unroll
          for (int j4 = 0; j4 < 4; ++j4) {
            const float4 r = r4[j4];
            minus(t[4 * j4], t[4 * j4 + 1], r.x, r.y);
            minus(t[4 * j4 + 2], t[4 * j4 + 3], r.z, r.w);
          }
          mask(c, t);
          float top[4] = {t[0], t[1], t[2], t[3]};
#pragma unroll
          for (int j = 4; j < 16; ++j) top[j & 3] = fmaxf(top[j & 3], t[j]);
          over |= fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > kSlack;
          // P, and its sum per row over this thread's tokens
#pragma unroll
          for (int c8 = 0; c8 < 2; ++c8) {
            uint32_t hi4[4], lo4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * c8 + 2 * e;
              float p0 = exp2_fast(t[j]), p1 = exp2_fast(t[j + 1]);
              const float2 sum = parts(add2(pair(l[j], l[j + 1]), pair(p0, p1)));
              l[j] = sum.x;
              l[j + 1] = sum.y;
              if constexpr (kQ8) {
                p0 = __fmul_rn(p0, vs0);
                p1 = __fmul_rn(p1, vs0);
                if (edge) {   // a masked token's scale may be anything
                  p0 = t[j] == kNegInf ? 0.f : p0;
                  p1 = t[j + 1] == kNegInf ? 0.f : p1;
                }
              } else if (partly) {
                sh.pe[tok - seen0][c + j] = p0;
                sh.pe[tok - seen0][c + j + 1] = p1;
              }
              hi4[e] = pack2(p0, p1);
              const float2 rest =
                  parts(fma2(pair(bf16_lo(hi4[e]), bf16_hi(hi4[e])), less, pair(p0, p1)));
              lo4[e] = pack2(rest.x, rest.y);
            }
            auto put = [&](int ch, const uint32_t(&x)[4]) {
              *reinterpret_cast<uint4*>(p_at + (ch >> 3) * kTok * 128 +
                                        (((ch & 7) ^ (tk & 7)) << 4)) =
                  make_uint4(x[0], x[1], x[2], x[3]);
            };
            put(c / 8 + c8, hi4);
            put(cols.low_in_p(c) / 8 + c8, lo4);
          }
          __syncwarp();
          tmem_st(tLnew + c, l);
        }
        if (settled || !score_any(over)) break;
      }
      if (!alive) break;
      tmem_wait_st();
      sm100::tc_fence_before();
      fence_async();
      warp_arrive(&sh.pfull[i & 1], lane);
      if (last) {
        // ------------------------------------------------------------ results -------------
        const int run = i < cur.tile ? i : cur.tile;    // tiles before this one in the run
        const bool whole = ends && cur.tile == run;
        // this thread's dimension of the values (codes are widened as (0, 2, 1, 3))
        const int dim = kQ8 ? (tk & ~3) | ((tk & 1) << 1) | ((tk >> 1) & 1) : tk;
        float v[7];
#pragma unroll 1
        for (int c = col0; c < col0 + half; c += 16) {
          __syncwarp();
          sm100::tmem_ld16(tLnew + c, l);
          const float sum =
              over_lanes(l, lane, [](float x, float y) { return __fadd_rn(x, y); });
          if (lane < 16) sh.red[kMaxN * quad + c + lane] = sum;
        }
        score_sync();
        const int64_t piece = 2 * (int64_t)blockIdx.x + (cur.tile == run ? 1 : 0);
        if (tid == 0) note_span(a, cur, cur.tile == run, ends);
        if (tid < N) {
          const float norm = __fadd_rn(__fadd_rn(sh.red[tid], sh.red[kMaxN + tid]),
                                       __fadd_rn(sh.red[2 * kMaxN + tid], sh.red[3 * kMaxN + tid]));
          sh.norm[tid] = norm == 0.f ? 0.f : __frcp_rn(norm);
          if (!whole && tid < a.M)
            *reinterpret_cast<float2*>(a.part_ml + 2 * (piece * a.M + tid)) =
                make_float2(norm == 0.f ? kNegInf : sh.ref[tid], norm);
        }
        alive = wait(&sh.odone[i & 1], (i >> 1) & 1);
        alive = !score_any(!alive);
        if (!alive) break;
        sm100::tc_fence_after();
        // the partly seen tokens of this run that were left out of the products (they are among
        // its last 7, so in its last two tiles)
        unsigned apart = 0;
        if (!kQ8) {
          volatile unsigned* const left_out = sh.apart;
          apart = left_out[i % kInfo];
          if (run > 0) apart |= left_out[(i + kInfo - 1) % kInfo];
#pragma unroll
          for (int e = 0; e < 7; ++e) {   // (their loads overlap)
            v[e] = 0.f;
            if (!(apart >> e & 1u) || tk >= D) continue;
            const int t = seen0 + e, page = page_of(a, cur.b, t, cur.len);
            if (page >= 0)
              v[e] = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(
                  a.c.v)[page * a.c.stride +
                         (((int64_t)cur.h << a.c.page_shift) + (t & page_mask)) * D + dim]);
          }
        }
        uint16_t* const out = a.out + seq_at(cur) + dim;
        float* const po = a.part_o + piece * a.M * D + dim;
        // (16 rows at a time go through this thread's own words of P's buffers, which nothing else
        // uses now, so that they can be walked in a loop: this code runs once per run)
        float* const words = reinterpret_cast<float*>(sP) + tk;
        float* const mine = words + (col0 ? 16 : 0) * kTok;
        float* const mine_v = words + (col0 ? 39 : 32) * kTok;
        if (apart) {
#pragma unroll
          for (int e = 0; e < 7; ++e) mine_v[e * kTok] = v[e];
        }
#pragma unroll 1
        for (int c = col0; c < col0 + half; c += 16) {
          float o[16];
          __syncwarp();
          sm100::tmem_ld16(tO + c, o);
          if (cols.low_apart(c)) {
            sm100::tmem_ld16(tO + cols.low_in_o(c), l);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __fadd_rn(o[j], l[j]);
          }
          if (!kQ8) {
#pragma unroll 1
            for (unsigned rest = apart; rest; rest &= rest - 1) {
              const int e = __ffs(rest) - 1;
              const float ve = mine_v[e * kTok];
              const bool plain = fabsf(ve) < INFINITY;   // P of a row that does not see it is 0
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (plain || e < sh.row_r[c + j]) o[j] = __fmaf_rn(sh.pe[e][c + j], ve, o[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) mine[j * kTok] = o[j];
          const int rows = tk < D ? min(a.M, c + 16) : 0;   // (D = 64: the upper lanes repeat)
#pragma unroll 4
          for (int row = c; row < rows; ++row) {
            const float o = mine[(row - c) * kTok];
            // (a normaliser of 0 is a row that sees nothing; its sums may hold a token's NaN)
            if (whole)
              out[sh.row_at[row]] =
                  f32_to_bf16_rne(sh.norm[row] == 0.f ? 0.f : __fmul_rn(o, sh.norm[row]));
            else
              po[row * D] = o;
          }
        }
        score_sync();   // (sh is free for the next run)
      }
      cur = n1;
    }
  } else if (warp < T::kFetchWarp) {
    // ----------------------------------------------------- Q8: codes widened to operands ---
    if constexpr (kQ8) {
      const bool values = warp >= (kScore + T::kWiden) / 32;
      const int lt = tid - kScore - (values ? T::kWiden : 0);
      uint64_t* const full = values ? sh.vfull : sh.kfull;
      uint64_t* const free_bar = values ? sh.vfree : sh.kfree;
      const int ring = values ? ta.v_ring : ta.k_ring;
      constexpr int kChunks = D / 16, kStep = T::kWiden / kChunks, kIters = kTok / kStep;
      // (eight lanes take 4 chunks of 2 rows, so that a quarter warp's stores meet all banks)
      const int my_row = D == 128 ? (lt >> 4) * 2 + ((lt >> 2) & 1) : lt / kChunks;
      const int my_chunk = D == 128 ? (lt & 3) + ((lt >> 1) & 4) : lt % kChunks;
      const uint8_t* const raw0 =
          sRaw + (values ? ta.raw * T::kRawMat : 0) + my_row * D + my_chunk * 16;
      uint8_t* const dst0 = (values ? sV : sK) + (my_chunk >> 2) * (kTok * 128) + my_row * 128;
      const int c0 = ((2 * my_chunk & 7) ^ (my_row & 7)) << 4;   // (kStep: a multiple of 8 rows)
      int st = 0, rst = 0;            // stages of the operand tile, of the codes
      uint32_t par = 1, rpar = 0;     // and parities: of the phase before, of this one
      for (int i = 0; i < n; ++i) {
        bool alive = wait(&sh.raw_full[values][rst], rpar);
        if (i >= ring) alive = alive && wait(&free_bar[st], par);
        if (!__all_sync(0xffffffffu, alive)) break;
        uint4 w[kIters];   // (all loads before the first store)
#pragma unroll
        for (int it = 0; it < kIters; ++it)
          w[it] = *reinterpret_cast<const uint4*>(raw0 + rst * T::kRawMat + it * (kStep * D));
        warp_arrive(&sh.raw_free[values][rst], lane);
        uint8_t* const dst = dst0 + st * T::kMat;
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          const uint4 v = w[it];
          *reinterpret_cast<uint4*>(dst + it * (kStep * 128) + c0) = make_uint4(
              code_pair(v.x), code_pair(v.x >> 8), code_pair(v.y), code_pair(v.y >> 8));
          *reinterpret_cast<uint4*>(dst + it * (kStep * 128) + (c0 ^ 16)) = make_uint4(
              code_pair(v.z), code_pair(v.z >> 8), code_pair(v.w), code_pair(v.w >> 8));
        }
        fence_async();
        warp_arrive(&full[st], lane);
        if (++st == ring) st = 0, par ^= 1;
        if (++rst == ta.raw) rst = 0, rpar ^= 1;
      }
    }
  } else if (warp < T::kMmaWarp) {
    // ------------------------------------------------------------- copies from the pages ---
    // A page's tokens of one head are one stretch of memory: lane x copies the x-th page of a
    // tile, by TMA into the swizzled operand tile (bf16) or as raw codes (Q8). What no copy
    // brings is left as it is: its scores are masked, and its values either count as codes
    // (finite) times 0 or are cleared below.
    const bool values = warp == T::kFetchWarp + 1;
    const int pt = 1 << a.c.page_shift, pages = kTok >> a.c.page_shift;
    const int ring = kQ8 ? ta.raw : (values ? ta.v_ring : ta.k_ring);
    uint64_t* const full = kQ8 ? sh.raw_full[values] : (values ? sh.vfull : sh.kfull);
    uint64_t* const free_bar = kQ8 ? sh.raw_free[values] : (values ? sh.vfree : sh.kfree);
    uint8_t* const tiles = kQ8 ? sRaw + (values ? ta.raw * T::kRawMat : 0) : (values ? sV : sK);
    int page = lane < pages ? page_of(a, cur.b, cur.tile * kTok + lane * pt, cur.len) : -1;
    int st = 0, done = 0, edges = 0;
    uint32_t par = 1;
    bool alive = true;
    for (int i = 0; i < n; ++i) {
      if (i >= ring) alive = wait(&free_bar[st], par);
      if (!__all_sync(0xffffffffu, alive)) break;
      const bool ok = page >= 0 && page < a.c.pages;
      const unsigned there = __ballot_sync(0xffffffffu, ok);
      const int count = __popc(there), t0 = cur.tile * kTok, seen0 = cur.len - (a.R - 1);
      if (!values) {   // what the softmax needs to know (its slot is free: see kInfo's use)
        const int slot = i % kInfo;
        if (lane == 0) {
          sh.runs[slot] = there;
          sm100::mbar_arrive_expect_tx(&sh.info[slot], kQ8 ? count * pt * 8 : 0);
        }
        __syncwarp();
        if (kQ8 && ok) {
          const int64_t at = page * a.c.scale_stride + ((int64_t)cur.h << a.c.page_shift);
          float* const dst = sScale + 2 * slot * kTok + lane * pt;
          bulk_copy(dst, a.c.k_scale + at, pt * 4, &sh.info[slot]);
          bulk_copy(dst + kTok, a.c.v_scale + at, pt * 4, &sh.info[slot]);
        }
      }
      const bool edge = !kQ8 && values && (t0 + kTok > seen0 || count < pages);
      // (read when the results of tile i or i + 1 are written: at most the ring ahead of here)
      if (!kQ8 && values && !edge && lane == 0) sh.apart[i % kInfo] = 0u;
      uint64_t* const bar = edge ? &sh.vedge : &full[st];
      if (lane == 0) sm100::mbar_arrive_expect_tx(bar, count * pt * (kQ8 ? D : 2 * D));
      __syncwarp();
      if (ok) {
        if constexpr (kQ8) {
          bulk_copy(tiles + st * T::kRawMat + lane * pt * D,
                    (values ? a.c.v : a.c.k) + page * a.c.stride +
                        (((int64_t)cur.h << a.c.page_shift)) * D,
                    pt * D, bar);
        } else {
#pragma unroll
          for (int hf = 0; hf < T::kHalves; ++hf)
            sm100::tma_load_3d(tiles + st * T::kMat + hf * (kTok * 128) + lane * pt * 128,
                               values ? &v_map : &k_map, 64 * hf, cur.h << a.c.page_shift, page, bar);
        }
      }
      if (edge) {   // clear what is no value, and the partly seen values that are not finite
        const uint32_t edge_par = edges++ & 1;
        alive = wait(&sh.vedge, edge_par);
        if (!__all_sync(0xffffffffu, alive)) {   // (no full[] counts these copies)
          sm100::mbar_wait(&sh.vedge, edge_par, kWaitPolls);
          break;
        }
        unsigned apart = 0;
        for (int r = lane; r < kTok; r += 32) {
          bool none = t0 + r >= cur.len || !(there >> (r >> a.c.page_shift) & 1u);
          auto at = [&](int x) {
            return reinterpret_cast<uint4*>(tiles + st * T::kMat + (x >> 3) * (kTok * 128) +
                                            r * 128 + (x & 7) * 16);
          };
          if (!none && t0 + r >= seen0) {
            for (int x = 0; x < 8 * T::kHalves; ++x) {
              const uint4 v = *at(x);
              none |= not_finite(v.x) || not_finite(v.y) || not_finite(v.z) || not_finite(v.w);
            }
            if (none) apart |= 1u << (t0 + r - seen0);
          }
          if (none)
            for (int x = 0; x < 8 * T::kHalves; ++x) *at(x) = make_uint4(0u, 0u, 0u, 0u);
        }
        apart = __reduce_or_sync(0xffffffffu, apart);
        if (lane == 0) sh.apart[i % kInfo] = apart;
        fence_async();
        __syncwarp();
        if (lane == 0) arrive(&full[st]);
      }
      done = i + 1;
      if (++st == ring) st = 0, par ^= 1;
      if (done < n) {
        cur.next(a);
        const int t = cur.tile * kTok + lane * pt;
        page = -1;
        if (lane < pages && t < cur.len)
          page = a.table[(int64_t)cur.b * a.max_pages + (t >> a.c.page_shift)];
      }
    }
    if (*abort_flag) {   // copies in flight end (bounded) before the CTA does
      for (int j = done - ring < 0 ? 0 : done - ring; j < done; ++j)
        sm100::mbar_wait(&full[j % ring], (j / ring) & 1, kWaitPolls);
      if (!values)
        for (int j = done - kInfo < 0 ? 0 : done - kInfo; j < done; ++j)
          sm100::mbar_wait(&sh.info[j % kInfo], (j / kInfo) & 1, kWaitPolls);
    }
  } else if (warp == T::kMmaWarp) {
    // ---------------------------------------------------------------- MMAs of the scores ---
    // (the whole warp walks the loop, so that descriptors stay in uniform registers; one lane
    // issues)
    const bool leader = elect_one();
    const uint32_t idesc = sm100::idesc_bf16_f32(kTok, N);
    const uint64_t q_desc = sm100::desc_k_sw128(smem_at(sQ));
    const uint64_t k_desc = sm100::desc_k_sw128(smem_at(sK));
    int segs = 0, done = 0, st = 0;
    uint32_t par = 0;
    for (int j = 0; j < n; ++j) {
      const bool new_q = j == 0 || cur.tile == 0;
      // the buffer of S is free once P of the tile s_bufs before is there
      const int before = j - ta.s_bufs;
      bool ok = before < 0 || wait(&sh.pfull[before & 1], (before >> 1) & 1);
      if (new_q) ok = ok && wait(&sh.qfull, segs++ & 1);
      ok = ok && wait(&sh.kfull[st], par);
      if (!__all_sync(0xffffffffu, ok)) break;
      sm100::tc_fence_after();
      fence_async();
      const uint64_t kd = k_desc + (uint32_t)st * (T::kMat >> 4);
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)   // 16 values: 32 bytes, or the next 64 values
          sm100::mma_bf16(tmem + (j & (ta.s_bufs - 1)) * N, kd + (ks >> 2) * (kTok * 8) + (ks & 3) * 2,
                          q_desc + (uint32_t)((ks >> 2) * N * 8 + (ks & 3) * 2), idesc, ks > 0);
        sm100::mma_commit(&sh.sfull[j & 1]);
        sm100::mma_commit(&sh.kfree[st]);
      }
      __syncwarp();
      if (++st == ta.k_ring) st = 0, par ^= 1;
      done = j + 1;
      if (done < n) cur.next(a);
    }
    // MMAs issued but maybe not observed complete: wait (bounded) before TMEM is freed
    if (done) sm100::mbar_wait(&sh.sfull[(done - 1) & 1], ((done - 1) >> 1) & 1, kWaitPolls);
  } else {
    // ---------------------------------------------------------------- MMAs of the values ---
    const bool leader = elect_one();
    const uint32_t idesc = sm100::idesc_bf16_f32(kTok, cols.mma_columns()) | kMajorMN;
    // (D = 64: the upper half of the M rows repeats the lower one)
    const uint64_t v_desc = desc_mn_sw128(smem_at(sV), D == 128 ? kTok * 128 : 0);
    const uint64_t p_desc = desc_mn_sw128(smem_at(sP), kTok * 128);
    int done = 0, st = 0;
    uint32_t par = 0;
    for (int i = 0; i < n; ++i) {
      bool ok = wait(&sh.vfull[st], par);
      ok = ok && wait(&sh.pfull[i & 1], (i >> 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      sm100::tc_fence_after();
      fence_async();
      const uint64_t vd = v_desc + (uint32_t)st * (T::kMat >> 4);
      const uint64_t pd = p_desc + (uint32_t)(i & (ta.p_bufs - 1)) * (p_size >> 4);
      const bool fresh = i == 0 || cur.tile == 0;
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < kTok / 16; ++ks) {   // 16 tokens: 2 KB
          const uint32_t tO = tmem + ta.s_bufs * N, more = !(fresh && ks == 0);
          if constexpr (kBeside) {
            sm100::mma_bf16(tO, vd + ks * 128, pd + ks * 128, idesc, more);
          } else {
            for (int x = 0; x < cols.mmas(); ++x)   // (mma_columns: a chunk or two)
              sm100::mma_bf16(tO + cols.mma_at(x), vd + ks * 128,
                              pd + (uint32_t)(x * cols.mma_columns() * (kTok / 8)) + ks * 128, idesc,
                              cols.mma_adds(x) || more);
          }
        }
        sm100::mma_commit(&sh.odone[i & 1]);
        sm100::mma_commit(&sh.vfree[st]);
      }
      __syncwarp();
      if (++st == ta.v_ring) st = 0, par ^= 1;
      done = i + 1;
      if (done < n) cur.next(a);
    }
    if (done) sm100::mbar_wait(&sh.odone[(done - 1) & 1], ((done - 1) >> 1) & 1, kWaitPolls);
  }
  __syncwarp();
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 0) sm100::tmem_dealloc(tmem, ta.tmem_cols);
}

// Shared memory of a call.
template <int D, bool kQ8, bool kBeside>
int smem_bytes(const TcArgs& a) {
  using T = Tc<D, kQ8>;
  return 1024 + kSmallBytes + T::kHalves * a.N * 128 +
         a.p_bufs * Parts<kBeside>{a.N}.p_chunks() * kTok * 128 + (a.k_ring + a.v_ring) * T::kMat +
         2 * a.raw * T::kRawMat + (kQ8 ? kInfo * 2 * kTok * 4 : 0);
}

template <int D, bool kQ8, bool kBeside>
cudaError_t start_as(const TcArgs& a, int room, int smem, cudaStream_t s) {
  const auto kernel = k_paged_tc<D, kQ8, kBeside>;
  static OncePerDevice ready;
  const cudaError_t e = ready.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap k_map = {}, v_map = {};
  if (!kQ8) {
    const CacheView& c = a.p.c;
    const int pt = 1 << c.page_shift;
    cudaError_t m = page_tile_map(&k_map, c.k, D, c.heads * pt, c.pages, c.stride, pt);
    if (m == cudaSuccess) m = page_tile_map(&v_map, c.v, D, c.heads * pt, c.pages, c.stride, pt);
    if (m != cudaSuccess) return m;
  }
  return launch_pdl(kernel, dim3(a.p.grid), Tc<D, kQ8>::kThreads, smem, s, a, k_map, v_map);
}

template <int D, bool kQ8, bool kBeside>
cudaError_t start_with(const PagedArgs& p, cudaStream_t s) {
  TcArgs a{};
  a.p = p;
  a.N = p.M <= 32 ? 32 : (p.M <= 64 ? 64 : (p.M <= 96 ? 96 : 128));
  a.s_bufs = a.N <= 96 ? 2 : 1;   // (tensor memory has 512 columns)
  const int room = 227 * 1024;
  // The least first, then what fits: two stages of codes, a second buffer of P (Q8, 64 rows, D =
  // 128: 207 us with two, 234 with one and a second value tile; bf16, 96 rows: 195 with two and a
  // second value tile, 263 with two and a second key tile, 262 with one and both), a second
  // value tile, deeper rings. (Q8, 96 rows: 314 us with any that fits.)
  a.p_bufs = 1;
  a.k_ring = a.v_ring = 1;
  a.raw = kQ8 ? 1 : 0;
  auto grow = [&](int TcArgs::*what, int most) {
    while (a.*what < most) {
      ++(a.*what);
      if (smem_bytes<D, kQ8, kBeside>(a) <= room) continue;
      --(a.*what);
      break;
    }
  };
  if (kQ8) grow(&TcArgs::raw, 2);
  grow(&TcArgs::p_bufs, 2);
  grow(&TcArgs::v_ring, 2);
  if (kQ8) {
    grow(&TcArgs::k_ring, 2);
    grow(&TcArgs::raw, kMaxRing);
  } else {
    grow(&TcArgs::k_ring, kMaxRing);
    grow(&TcArgs::v_ring, kMaxRing);
  }
  // Page flags and scales of a tile are overwritten kInfo tiles later. The keys of that tile
  // are fetched once the codes of the tile `raw` before it are widened, so k_ring further
  // back the scores are done, and two further back P (the two buffers of S).
  static_assert(kMaxRing + 2 + 2 <= kInfo, "slots of the tile information");
  a.tmem_cols = 128;
  while ((int)a.tmem_cols < (a.s_bufs + 2) * a.N + Parts<kBeside>{a.N}.o_columns()) a.tmem_cols *= 2;
  // (the results of a run pass through P's buffers)
  if (a.p_bufs * Parts<kBeside>{a.N}.p_chunks() * 128 < (32 + (kQ8 ? 0 : 14)) * 4)
    return cudaErrorInvalidValue;
  // (at least half of the SM's shared memory, so that one CTA has the SM's tensor memory)
  int smem = smem_bytes<D, kQ8, kBeside>(a);
  smem = smem < 120 * 1024 ? 120 * 1024 : smem;
  return start_as<D, kQ8, kBeside>(a, room, smem, s);
}

template <int D, bool kQ8>
cudaError_t start(const PagedArgs& p, cudaStream_t s) {
  return p.M <= 64 ? start_with<D, kQ8, true>(p, s) : start_with<D, kQ8, false>(p, s);
}

}  // namespace paged_tc

namespace paged {

using paged_tc::start;

cudaError_t launch_tc(const PagedArgs& p, int D, cudaStream_t s) {
  if (D == 128) return p.c.q8 ? start<128, true>(p, s) : start<128, false>(p, s);
  return p.c.q8 ? start<64, true>(p, s) : start<64, false>(p, s);
}

}  // namespace paged
}  // namespace dsmoe
