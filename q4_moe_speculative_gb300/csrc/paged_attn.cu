// paged_attn.cu — attention of each sequence's last R tokens over its paged key-value cache
// (arithmetic in include/dsmoe.h): a plain decode step for R = 1, a verify step for R <= 8.
//
// All query rows of one key head, M = R x heads per key head (row m = r * G + j), read the
// same keys and values, so they are the M dimension of one problem whose cost is the bytes
// of the cache. Tokens come in tiles of 64. The tiles of all sequences and key heads form one
// list that is cut into equal runs, one per CTA: a long sequence is split over many CTAs, a
// batch of ragged ones is balanced, and no CTA waits for another. A (sequence, head) that
// lies inside one run is finished there; one that crosses a boundary leaves its running
// maximum, normaliser and sums per CTA in the workspace, and k_paged_join merges those in
// CTA order, so results do not depend on timing.
//
// k_paged (4 or 8 warps): tiles are copied by cp.async into a ring of stages (rows swizzled
// in 16-byte chunks, so that ldmatrix is free of bank conflicts). Per tile, warp w scores
// tokens 16 w .. 16 w + 15 for its rows (S = Q K^T, mma.sync m16n8k16), P = 2^(S - m) goes
// to shared memory as bf16, and then warp w accumulates its quarter of the head's values for
// all 64 tokens (O += P V): a key or value byte is read from shared memory (and an int8 one
// widened) once per CTA, and the accumulators are a quarter of M x D per warp. Codes of a Q8
// cache are widened exactly to bf16; the key's scale multiplies the score, the value's scale
// P. The reference m of a row moves only when a score exceeds it by 2^8 (P stays in range and
// bf16's relative precision does not depend on it), so the usual tile needs no exchange of
// maxima and no rescaling: the CTA votes on it at the barrier that publishes P anyway.
// P is rounded once to bf16, half a step of 2^-8 relative per term; for a bf16 cache the
// normaliser sums the rounded values, so that the weights add up to one.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace dsmoe {
namespace {

constexpr int kTile = 64;
constexpr float kNegInf = -INFINITY;
constexpr float kSlack = 8.f;   // log2 by which a score may exceed the row's reference

struct PagedArgs {
  int B, R, Hq, G, M, max_pages;
  float scale_log2;
  const uint16_t* q;
  CacheView c;
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  float* part_o;    // [2 grid][M][D]
  float* part_ml;   // [2 grid][M][2]
  int grid;         // CTAs of k_paged
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x2_t(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The int8 values at bytes 0 and 2 of w as a bf16 pair, exactly: (128 + low 7 bits) minus
// 128 or, with the sign bit, 256.
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t m, c, d;
  asm("lop3.b32 %0, %1, 0x007F007F, 0x43004300, 0xEA;" : "=r"(m) : "r"(w));
  asm("lop3.b32 %0, %1, 0x00800080, 0x43004300, 0xEA;" : "=r"(c) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of RB bytes: the eight rows of
// an ldmatrix meet eight different bank groups.
template <int RB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (RB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return r * RB + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ int seq_len(const PagedArgs& a, int b) {
  const int n = a.lengths[b], cap = a.max_pages << a.c.page_shift;
  return n < 0 ? 0 : (n > cap ? cap : n);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Tiles of all sequences, per key head (every lane of the warp gets the sum).
__device__ __forceinline__ int64_t all_tiles(const PagedArgs& a, int lane) {
  int64_t sum = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32)
    sum += b0 + lane < a.B ? tiles_of(seq_len(a, b0 + lane)) : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The place of a tile in the list: sequences, then key heads, then tiles along the length.
struct Cursor {
  int b, h, tile, tiles, len;
  __device__ __forceinline__ void open(const PagedArgs& a) {   // first non-empty from b on
    for (; b < a.B; ++b) {
      len = seq_len(a, b);
      tiles = tiles_of(len);
      if (tiles) break;
    }
  }
  __device__ __forceinline__ void next(const PagedArgs& a) {
    if (++tile < tiles) return;
    tile = 0;
    if (++h < a.c.heads) return;
    h = 0;
    ++b;
    open(a);
  }
};

// The cursor of tile `at` (warp-wide search; at is inside the list).
__device__ __forceinline__ Cursor find_tile(const PagedArgs& a, int64_t at, int lane) {
  Cursor cur{};
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int n = b0 + lane < a.B ? tiles_of(seq_len(a, b0 + lane)) : 0;
    int64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, (before + upto) * a.c.heads > at);
    if (past) {
      const int l = __ffs(past) - 1;
      const int64_t first =
          (before + __shfl_sync(0xffffffffu, upto - n, l)) * a.c.heads;   // of sequence b0 + l
      cur.b = b0 + l;
      cur.len = seq_len(a, cur.b);
      cur.tiles = tiles_of(cur.len);
      cur.h = (int)((at - first) / cur.tiles);
      cur.tile = (int)((at - first) % cur.tiles);
      return cur;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  cur.b = a.B;
  return cur;
}

// Shapes of one instantiation: MT m16 tiles of rows per warp, MH groups of four warps.
template <int D, bool kQ8, int MT, int MH>
struct Shape {
  static constexpr int kThreads = 128 * MH;
  static constexpr int kRows = 16 * MT * MH;
  static constexpr int RB = D * (kQ8 ? 1 : 2);          // bytes of a cached row
  static constexpr int kMat = kTile * RB;
  static constexpr int kStage = 2 * kMat + (kQ8 ? 2 * kTile * 4 : 0);
  static constexpr bool kSplit = kQ8 || kRows <= 32;    // P as a high and a low part
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kP = kRows * kTile * 2;
  static constexpr int kRed = 4 * kRows * 4;
  static constexpr int kFixed = kQ + kP * (kSplit ? 2 : 1) + kRed + 64;
  // CTAs per SM: as many as the registers allow (65,536 over the threads at 128, 168 or 255
  // each) with at least two stages each
  static constexpr int kWant = MH == 2 ? 1 : (MT == 1 ? 4 : MT == 2 ? 3 : 2);
  static constexpr int room(int n) { return 228 * 1024 / n - 1024; }
  static constexpr int fit(int n) {
    return n > 1 && kFixed + 2 * kStage > room(n) ? fit(n - 1) : n;
  }
  static constexpr int kPerSm = fit(kWant);
  static constexpr int kFit = (room(kPerSm) - kFixed) / kStage;
  static constexpr int kStages = kFit > 5 ? 5 : kFit;
  static constexpr int kSmem = kFixed + kStages * kStage;
  static_assert(kStages >= 2 && kStages <= 8, "a ring of two to eight stages");
};

template <int D, bool kQ8, int MT, int MH>
__global__ void __launch_bounds__(128 * MH, (Shape<D, kQ8, MT, MH>::kPerSm))
    k_paged(const __grid_constant__ PagedArgs a) {
  using C = Shape<D, kQ8, MT, MH>;
  constexpr int RB = C::RB, S = C::kStages, NT = D / 32;
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* sQ = sm + S * C::kStage;
  uint8_t* sP = sQ + C::kQ;
  float* red = reinterpret_cast<float*>(sP + C::kP * (C::kSplit ? 2 : 1));   // [4][kRows]
  bool* there = reinterpret_cast<bool*>(red + 4 * C::kRows);   // [stage][4] 16-token groups
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w4 = warp & 3, row0 = (warp >> 2) * MT * 16;
  const int g = lane >> 2, q = lane & 3;
  pdl_trigger();
  pdl_wait();

  const int64_t total = all_tiles(a, lane) * a.c.heads;
  const int64_t ctas = total < a.grid ? total : a.grid;   // every one has a tile
  if (blockIdx.x >= ctas) return;
  const int64_t lo = blockIdx.x * total / ctas, hi = (blockIdx.x + 1) * total / ctas;
  Cursor cur = find_tile(a, lo, lane), ahead = cur;

  const int page_mask = (1 << a.c.page_shift) - 1;
  // page of token t of sequence b, or -1: no such token, or a bad page table entry
  auto page_of = [&](int b, int t, int len) {
    if (t >= len) return -1;
    const int p = a.table[(int64_t)b * a.max_pages + (t >> a.c.page_shift)];
    return p >= 0 && p < a.c.pages ? p : -1;
  };
  // Each run of 16 tokens lies in one page. Lane x of every warp holds where run x & 3 of the
  // tile to be fetched next starts (in values, -1: nowhere), looked up a tile ahead.
  int64_t run_at, run_scale;
  auto look_up = [&](const Cursor& at) {
    const int t = at.tile * kTile + 16 * (lane & 3), page = page_of(at.b, t, at.len);
    const int64_t in_page = ((int64_t)at.h << a.c.page_shift) + (t & page_mask);
    run_at = page < 0 ? -1 : page * a.c.stride + in_page * D;
    if (kQ8) run_scale = page < 0 ? -1 : page * a.c.scale_stride + in_page;
  };
  constexpr int kChunks = RB / 16, kStep = C::kThreads / kChunks;   // rows per iteration
  const int my_row = tid / kChunks, my_chunk = tid % kChunks;
  const uint32_t my_dst = swz<RB>(my_row, my_chunk);   // (kStep is a multiple of 8 rows)
  auto load_tile = [&](const Cursor& at, int stage) {
    const uint32_t k0 = smem_u32(sm + stage * C::kStage) + my_dst, v0 = k0 + C::kMat;
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
        cp_async16(smem_u32(sm + stage * C::kStage) + 2 * C::kMat + 16 * lane,
                   (lane < 16 ? a.c.k_scale : a.c.v_scale) + (ok ? at_s + (r & 15) : 0), ok);
      }
      if (lane < 4) there[4 * stage + lane] = run_at >= 0;
    }
  };

  const int n = (int)(hi - lo);   // tiles of this CTA
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
      const uint32_t kb = smem_u32(sK), qb = smem_u32(sQ);
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
      for (int mt = 0; mt < MT; ++mt) {   // s: log2 of p, before any mask
        s[mt][nt][0] = __fmaf_rn(s[mt][nt][0], f0, -ref[mt][0]);
        s[mt][nt][1] = __fmaf_rn(s[mt][nt][1], f1, -ref[mt][0]);
        s[mt][nt][2] = __fmaf_rn(s[mt][nt][2], f0, -ref[mt][1]);
        s[mt][nt][3] = __fmaf_rn(s[mt][nt][3], f1, -ref[mt][1]);
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
            float p0 = exp2_fast(s0), p1 = exp2_fast(s1);
            uint8_t* dst = sP + swz<2 * kTile>(row, 2 * w4 + nt) + 4 * q;
            if constexpr (C::kSplit) sum = __fadd_rn(sum, __fadd_rn(p0, p1));
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
            if constexpr (C::kSplit)
              *reinterpret_cast<uint32_t*>(dst + C::kP) =
                  pack2(__fsub_rn(p0, bf16_lo(w)), __fsub_rn(p1, bf16_hi(w)));
            else
              sum = __fadd_rn(sum, __fadd_rn(bf16_lo(w), bf16_hi(w)));
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
        over |= top[mt][e] > (m[mt][e] == kNegInf ? kNegInf : kSlack);
      }
    make_p();
    if (__syncthreads_or(over)) {
      // some row's reference moves: exchange the tile's maxima, rescale, and make P again
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = __fadd_rn(top[mt][e], ref[mt][e]);
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
          const float move = __fsub_rn(ref[mt][e], mn == kNegInf ? 0.f : mn);
          m[mt][e] = mn;
          l[mt][e] = __fmul_rn(l[mt][e], f);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[mt][nt][2 * e] = __fmul_rn(o[mt][nt][2 * e], f);
            o[mt][nt][2 * e + 1] = __fmul_rn(o[mt][nt][2 * e + 1], f);
          }
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            s[mt][nt][2 * e] = __fadd_rn(s[mt][nt][2 * e], move);
            s[mt][nt][2 * e + 1] = __fadd_rn(s[mt][nt][2 * e + 1], move);
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
      const uint32_t vb = smem_u32(sV), pb = smem_u32(sP);
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
          if constexpr (C::kSplit) {
            ldsm_x4(pb + C::kP + swz<2 * kTile>(row0 + 16 * mt + (lane & 15), 2 * ks + (lane >> 4)),
                    pf);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[mt][nt], pf, b[nt][0], b[nt][1]);
          }
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
              float p = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(ps));
              if constexpr (C::kSplit)
                p = __fadd_rn(p, bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(ps + C::kP)));
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
// in CTA order; empty sequences get zeros; the others are already written. 8 warps: a row
// each, or (many CTAs per head) all on one row.
template <int D>
__global__ void __launch_bounds__(256) k_paged_join(const __grid_constant__ PagedArgs a,
                                                    int rows_per_block) {
  constexpr int V = D / 32;   // values per lane
  __shared__ float acc_s[8][D], l_s[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.c.heads, h = blockIdx.x % a.c.heads;
  pdl_trigger();
  pdl_wait();
  const bool shared_row = rows_per_block == 1;
  const int row = blockIdx.y * rows_per_block + (shared_row ? 0 : warp);
  int64_t before = 0, total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int n = b0 + lane < a.B ? tiles_of(seq_len(a, b0 + lane)) : 0;
    total += n;
    before += b0 + lane < b ? n : 0;
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, x);
    before += __shfl_xor_sync(0xffffffffu, before, x);
  }
  total *= a.c.heads;
  const int n = tiles_of(seq_len(a, b));
  const int64_t first = before * a.c.heads + (int64_t)h * n;
  int c0 = 0, c1 = -1;   // CTAs that hold a piece
  if (n) {
    const int64_t ctas = total < a.grid ? total : a.grid;   // as in k_paged
    c0 = (int)(((first + 1) * ctas - 1) / total);
    c1 = (int)(((first + n) * ctas - 1) / total);
    if (c0 == c1) return;
  }
  if (row >= a.M) return;   // (all warps of the block, when they share the row)
  auto piece = [&](int c) { return (2 * (int64_t)c + (c == c0 ? 1 : 0)) * a.M + row; };
  float top = kNegInf;
  for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, __ldcg(a.part_ml + 2 * piece(c)));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  float acc[V], norm = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  const int step = shared_row ? 8 : 1;
#pragma unroll 4
  for (int c = c0 + (shared_row ? warp : 0); c <= c1; c += step) {
    const int64_t at = piece(c);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at);
    float x[V];
    if constexpr (V == 4) {
      const float4 f4 = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + lane);
      x[0] = f4.x, x[1] = f4.y, x[2] = f4.z, x[3] = f4.w;
    } else {
      const float2 f2 = __ldcg(reinterpret_cast<const float2*>(a.part_o + at * D) + lane);
      x[0] = f2.x, x[1] = f2.y;
    }
    const float f = ml.x == kNegInf ? 0.f : exp2_fast(__fsub_rn(ml.x, top));
    norm = __fmaf_rn(ml.y, f, norm);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(x[e], f, acc[e]);
  }
  if (shared_row) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc_s[warp][V * lane + e] = acc[e];
    if (lane == 0) l_s[warp] = norm;
    __syncthreads();
    if (warp) return;
    norm = l_s[0];
    for (int w = 1; w < 8; ++w) {
      norm = __fadd_rn(norm, l_s[w]);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = __fadd_rn(acc[e], acc_s[w][V * lane + e]);
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
struct Plan {
  int grid, per_sm;
  size_t ml, po, total;
};

// Calls f with the instantiation for these rows: m16 tiles per warp x warp groups.
template <int D, bool kQ8, typename F>
auto with_rows(int M, F&& f) {
  if (M <= 16) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  if (M <= 32) return f(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
  if (M <= 64) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  if (M <= 96) return f(std::integral_constant<int, 3>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
}

template <int D, bool kQ8>
Plan make_plan(const PagedAttnProblem& p) {
  const int M = p.R * (p.Hq / p.cache.heads);
  Plan pl{};
  pl.per_sm = with_rows<D, kQ8>(M, [](auto mt, auto mh) {
    return Shape<D, kQ8, decltype(mt)::value, decltype(mh)::value>::kPerSm;
  });
  // no more CTAs than tiles there can be
  const int64_t cap = (int64_t)p.max_pages << p.cache.page_shift;
  const int64_t most = (int64_t)p.B * p.cache.heads * ((cap + kTile - 1) / kTile);
  const int64_t all = (int64_t)pl.per_sm * device_sm_count();
  pl.grid = (int)(most < all ? most : all);
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl.ml = 0;
  pl.po = up((size_t)2 * pl.grid * M * 2 * sizeof(float));
  pl.total = pl.po + up((size_t)2 * pl.grid * M * D * sizeof(float));
  return pl;
}

template <int D, bool kQ8>
cudaError_t run(const PagedAttnProblem& p, uint8_t* ws, cudaStream_t s) {
  const Plan pl = make_plan<D, kQ8>(p);
  PagedArgs a{};
  a.B = p.B;
  a.R = p.R;
  a.Hq = p.Hq;
  a.G = p.Hq / p.cache.heads;
  a.M = p.R * a.G;
  a.max_pages = p.max_pages;
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  a.q = p.q;
  a.c = p.cache;
  a.table = p.table;
  a.lengths = p.lengths;
  a.out = p.out;
  a.part_ml = reinterpret_cast<float*>(ws + pl.ml);
  a.part_o = reinterpret_cast<float*>(ws + pl.po);
  a.grid = pl.grid;
  cudaError_t err = with_rows<D, kQ8>(a.M, [&](auto mt, auto mh) {
    using C = Shape<D, kQ8, decltype(mt)::value, decltype(mh)::value>;
    const auto kernel = k_paged<D, kQ8, decltype(mt)::value, decltype(mh)::value>;
    // (the attribute belongs to the kernel on a device and lasts: set once on each)
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e != cudaSuccess) return e;
      ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_pdl(kernel, dim3(pl.grid), C::kThreads, C::kSmem, s, a);
  });
  if (err != cudaSuccess) return err;
  // rows of a head over its pieces: all warps on one row when a head is cut into many
  const int heads = p.B * p.cache.heads;
  const int rows = pl.grid > 8 * heads ? 1 : 8;
  return launch_pdl(k_paged_join<D>, dim3(heads, (a.M + rows - 1) / rows), 256, 0, s, a, rows);
}

}  // namespace

size_t paged_attn_workspace(const PagedAttnProblem& p) {
  if (p.D == 128) return (p.cache.q8 ? make_plan<128, true>(p) : make_plan<128, false>(p)).total;
  return (p.cache.q8 ? make_plan<64, true>(p) : make_plan<64, false>(p)).total;
}

cudaError_t launch_paged_attn(const PagedAttnProblem& p, uint8_t* ws, cudaStream_t s) {
  if (p.D == 128) return p.cache.q8 ? run<128, true>(p, ws, s) : run<128, false>(p, ws, s);
  return p.cache.q8 ? run<64, true>(p, ws, s) : run<64, false>(p, ws, s);
}

}  // namespace dsmoe
