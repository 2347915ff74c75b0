// q4.cu — Q4 projections: R rows (R <= 8) through one tile-major Q4 matrix (groups of 1),
// every weight byte loaded once and applied to all rows.
//
// A tile is 16 rows x 64 values in 576 bytes (include/dsmoe.h): lane L = 4g + w holds at
// 16 L the 8-value words w of rows g, g + 8 of both blocks, which are the A fragments of
// mma.sync m16n8k16 (weights 16 rows, the R rows as the 8 columns). A nibble pair becomes a
// bf16 pair exactly by (w & 0x000F000F) | 0x43004300 minus 136; a block's two MMAs are scaled
// once by its fp16 scale. Weights go from global memory to registers in 16-byte loads, a
// batch of tiles ahead of the arithmetic, without shared memory: no other warp needs them.
//
// k_q4_proj: 16 warps; 2^wk_log of them split a unit's (16 rows') K tiles, tile kt to warp
// kt mod 2^wk_log, and the others run units side by side (short K). A warp's tiles of a unit
// come in batches of kTiles. When one batch is all of them the activation fragments stay in
// registers for the whole call (kKeepX); else they are read again through L1. The warps'
// partials meet in shared memory, kGroup units at a time (the barrier is paid once per group),
// in warp order, rounded once. Nothing depends on R. Bound: rows x K x 9/16 bytes; in practice
// the issue of about 80 instructions per tile, of which 44 widen nibbles. 129,280 x 4096, R = 6:
// 57.8 us, 5.2 TB/s; 4096 x 4096, R = 1: 3.8 us. 300 MB of weights (45 us at the copy rate), R = 6:
// K = 4096 58 us, 2048 62, 8192 73, 12,288 73 (beyond 4096 the activations are read again); a K
// that is no multiple of 1024 also pays for the tiles that fill its warps' batches up: 1088 107,
// 2560 84, 4160 131, 5120 109, 7168 82.
#include "common.cuh"
#include "kernels.h"
#include "mma.cuh"

namespace dsmoe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 2;   // rounds per barrier (129,280 x 4096: 1 63.7 us, 2 57.8, 4 60.8)

struct Q4Args {
  const uint8_t* tiles;
  int units, Tk, R;        // 16-row units, 64-value tiles along K, activation rows
  int wk_log;              // log2 of the warps along K
  int batches;             // batches of kTiles tiles per unit and warp
  const uint16_t* x;
  uint16_t* y;
};

__device__ __forceinline__ uint4 ldg_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_once8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// bf16 pair of the nibbles at bits 0-3 and 16-19 of w, minus 8, exactly.
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w) {
  uint32_t p, d;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(p) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(p), "r"(0x43084308u));
  return d;
}

// acc += scales x (block of 16 rows x 32 values) x X: the K order of the two MMAs is
// (8w + {0, 4} | 8w + {1, 5}) and (8w + {2, 6} | 8w + {3, 7}) for lane w of a row. acc: row g
// columns 2w and 2w + 1, then row g + 8.
__device__ __forceinline__ void block_mma(uint32_t lo, uint32_t hi, uint32_t scales,
                                          const uint4& X, float (&acc)[4]) {
  const float z[4] = {0.f, 0.f, 0.f, 0.f};
  float d[4];
  mma16816(d, nibble_pair(lo), nibble_pair(hi), nibble_pair(lo >> 4), nibble_pair(hi >> 4), X.x,
           X.y, z);
  mma16816(d, nibble_pair(lo >> 8), nibble_pair(hi >> 8), nibble_pair(lo >> 12),
           nibble_pair(hi >> 12), X.z, X.w, d);
  const __half2 s2 = *reinterpret_cast<const __half2*>(&scales);
  const float s0 = __low2float(s2), s1 = __high2float(s2);
  acc[0] = __fmaf_rn(s0, d[0], acc[0]);
  acc[1] = __fmaf_rn(s0, d[1], acc[1]);
  acc[2] = __fmaf_rn(s1, d[2], acc[2]);
  acc[3] = __fmaf_rn(s1, d[3], acc[3]);
}

// 8 consecutive activations (one 16-byte load) as the pairs (v0,v4) (v1,v5) (v2,v6) (v3,v7).
__device__ __forceinline__ uint4 x_pairs(const uint4& r) {
  return make_uint4(__byte_perm(r.x, r.z, 0x5410), __byte_perm(r.x, r.z, 0x7632),
                    __byte_perm(r.y, r.w, 0x5410), __byte_perm(r.y, r.w, 0x7632));
}

// kFull: all 16 warps along K (K >= 1024), so that tiles lie at fixed distances.
template <int kTiles, bool kKeepX, bool kFull>
__global__ void __launch_bounds__(kThreads, 1) k_q4_proj(const __grid_constant__ Q4Args a) {
  extern __shared__ float4 part[];   // [2][kGroup][warps][32 lanes]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  const int wk_log = kFull ? 4 : a.wk_log;
  const int wk = 1 << wk_log, wu = kWarps >> wk_log;   // warps along K, units side by side
  const int my_k = warp & (wk - 1), my_u = warp >> wk_log;
  const int rounds = (a.units + wu - 1) / wu;
  const int r0 = (int)((int64_t)blockIdx.x * rounds / gridDim.x);
  const int r1 = (int)((int64_t)(blockIdx.x + 1) * rounds / gridDim.x);
  pdl_trigger();
  pdl_wait();

  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const int64_t round_bytes = (int64_t)wu * a.Tk * kQ4TileBytes;
  const int tile_step = wk * kQ4TileBytes;
  const uint8_t* const lane0 =
      a.tiles + ((int64_t)my_u * a.Tk + my_k) * kQ4TileBytes + r0 * round_bytes + 16 * lane;
  const int scales_at = 512 + 8 * g - 16 * lane;
  const int mine = (a.Tk - my_k + wk - 1) >> wk_log;   // K tiles of a unit that are this warp's
  // The batch to be loaded next, and where its first tile is. Tiles behind the row's end have
  // scale 0.
  int rl = r0, bl = 0;
  const uint8_t* next = lane0;
  auto load = [&](int i, uint4& w, uint2& s) {
    w = none;
    s = make_uint2(0u, 0u);
    if (bl * kTiles + i < mine && rl < r1 && (kFull || rl * wu + my_u < a.units)) {
      w = ldg_once(next + i * tile_step);
      s = ldg_once8(next + i * tile_step + scales_at);
    }
  };
  auto advance = [&] {
    next += kTiles * tile_step;
    if (kKeepX || ++bl == a.batches) {
      bl = 0;
      ++rl;
      next += round_bytes - (int64_t)(kKeepX ? 1 : a.batches) * kTiles * tile_step;
    }
  };
  auto load_x = [&](int b, int i, uint4& x0, uint4& x1) {
    const int kt = ((b * kTiles + i) << wk_log) + my_k;
    x0 = x1 = none;
    if (g < a.R && kt < a.Tk) {
      const uint4* src =
          reinterpret_cast<const uint4*>(a.x + (int64_t)g * a.Tk * 64 + kt * 64 + 8 * q);
      x0 = x_pairs(__ldg(src));
      x1 = x_pairs(__ldg(src + 4));
    }
  };
  uint4 X[kKeepX ? kTiles : 1][2];
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  int r = r0, b = 0, filled = 0, buf = 0;   // rounds whose partials are in this buffer
  // Multiplies a batch; each of its registers is loaded again, two batches ahead, as soon as
  // it is used. False after the last.
  auto step = [&](uint4(&w)[kTiles], uint2(&s)[kTiles]) {
    const bool unit_ends = kKeepX || b + 1 == a.batches;
    const int rn = unit_ends ? r + 1 : r, bn = unit_ends ? 0 : b + 1;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      uint4 x0, x1;
      if constexpr (kKeepX) x0 = X[i][0], x1 = X[i][1];
      else load_x(b, i, x0, x1);
      block_mma(w[i].x, w[i].y, s[i].x, x0, acc);
      block_mma(w[i].z, w[i].w, s[i].y, x1, acc);
      load(i, w[i], s[i]);
    }
    advance();
    if (unit_ends) {
      float4* const group = part + buf * kGroup * kWarps * 32;
      group[(filled * kWarps + warp) * 32 + lane] =
          make_float4(acc[0], acc[1], acc[2], acc[3]);   // rows g and g + 8, columns 2q, 2q + 1
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      if (++filled == kGroup || rn == r1) {
        __syncthreads();   // (the other buffer was read before the last one)
        for (int o = tid; o < filled * wu * 128; o += kThreads) {
          const int at = o & 127, u = (o >> 7) & (wu - 1), f = o >> 7 >> (4 - wk_log);
          const int row = (at >> 4) + 8 * ((at >> 1) & 1), col = 2 * ((at >> 2) & 3) + (at & 1);
          const int unit = (rn - filled + f) * wu + u;
          if (col >= a.R || unit >= a.units) continue;
          const float* p = reinterpret_cast<const float*>(group + (f * kWarps + u * wk) * 32) + at;
          float sum = 0.f;
          for (int k = 0; k < wk; ++k) sum = __fadd_rn(sum, p[k * 128]);
          a.y[(int64_t)col * a.units * 16 + unit * 16 + row] = f32_to_bf16_rne(sum);
        }
        buf ^= 1;
        filled = 0;
      }
    }
    r = rn;
    b = bn;
    return r < r1;
  };
  uint4 W0[kTiles], W1[kTiles];
  uint2 S0[kTiles], S1[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) load(i, W0[i], S0[i]);
  advance();
#pragma unroll
  for (int i = 0; i < kTiles; ++i) load(i, W1[i], S1[i]);
  advance();
  if constexpr (kKeepX) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) load_x(0, i, X[i][0], X[i][1]);
  }
  while (step(W0, S0) && step(W1, S1)) {
  }
}

template <int kTiles, bool kKeepX, bool kFull>
cudaError_t start(const Q4Args& a, int grid, cudaStream_t s) {
  constexpr int kSmem = 2 * kGroup * kWarps * 32 * (int)sizeof(float4);
  static OncePerDevice ready;
  const cudaError_t e = ready.run([] {
    return cudaFuncSetAttribute(k_q4_proj<kTiles, kKeepX, kFull>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(k_q4_proj<kTiles, kKeepX, kFull>, dim3(grid), kThreads, kSmem, s, a);
}

}  // namespace

cudaError_t launch_q4_project(const void* tiles, int rows, int K, const uint16_t* x, int R,
                              uint16_t* y, cudaStream_t s) {
  Q4Args a{};
  a.tiles = static_cast<const uint8_t*>(tiles);
  a.units = rows / 16;
  a.Tk = K / 64;
  a.R = R;
  a.x = x;
  a.y = y;
  // As many warps along K as there are tiles for them (8 instead of 16 at K = 4096: 79 against 61
  // us for 129,280 rows, 4.5 against 3.8 for 4096), and batches no longer than a warp's share (4
  // tiles instead of 2 at K = 2048: 29.7 against 18.8 us for 65,536 rows). Where a share is one
  // batch the activations are kept (4 tiles, K = 4096: read again 82 us, kept 61).
  while (a.wk_log < 4 && (2 << a.wk_log) <= a.Tk) ++a.wk_log;
  const int wu = kWarps >> a.wk_log, per_warp = (a.Tk + (1 << a.wk_log) - 1) >> a.wk_log;
  const int rounds = (a.units + wu - 1) / wu;
  const int grid = rounds < device_sm_count() ? rounds : device_sm_count();
  a.batches = (per_warp + 3) / 4;
  if (a.wk_log < 4) return start<2, true, false>(a, grid, s);   // (at most two tiles per warp)
  if (per_warp <= 2) return start<2, true, true>(a, grid, s);
  if (per_warp <= 4) return start<4, true, true>(a, grid, s);
  return start<4, false, true>(a, grid, s);
}

}  // namespace dsmoe
