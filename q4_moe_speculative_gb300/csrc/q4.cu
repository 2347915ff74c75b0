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
// k_q4_proj: 16 warps; kWk of them split a unit's (16 rows') K tiles, tile kt to warp
// kt mod kWk, and 16 / kWk units run side by side (short K). A warp's tiles of a unit come in
// batches of kTiles. When one batch is all of them the activation fragments stay in
// registers for the whole call (kKeepX); else they are read again through L1. The warps'
// partials meet in shared memory, added in warp order, rounded once. Nothing depends on R.
// Memory-bound: rows x K x 9/16 bytes.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace dsmoe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;

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
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += scales x (block of 16 rows x 32 values) x X: the K order of the two MMAs is
// (8w + {0, 4} | 8w + {1, 5}) and (8w + {2, 6} | 8w + {3, 7}) for lane w of a row.
__device__ __forceinline__ void block_mma(uint32_t lo, uint32_t hi, uint32_t scales,
                                          const uint4& X, float (&acc)[4]) {
  float d[4] = {0.f, 0.f, 0.f, 0.f};
  mma16816(d, nibble_pair(lo), nibble_pair(hi), nibble_pair(lo >> 4), nibble_pair(hi >> 4), X.x,
           X.y);
  mma16816(d, nibble_pair(lo >> 8), nibble_pair(hi >> 8), nibble_pair(lo >> 12),
           nibble_pair(hi >> 12), X.z, X.w);
  const float s0 = f16_bits_to_f32((uint16_t)scales), s1 = f16_bits_to_f32((uint16_t)(scales >> 16));
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

template <int kTiles, bool kKeepX>
__global__ void __launch_bounds__(kThreads, 1) k_q4_proj(const __grid_constant__ Q4Args a) {
  __shared__ float4 part[2][kWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q = lane & 3;
  const int wk = 1 << a.wk_log, wu = kWarps >> a.wk_log;      // warps along K, units side by side
  const int my_k = warp & (wk - 1), my_u = warp >> a.wk_log;
  const int rounds = (a.units + wu - 1) / wu;
  const int r0 = (int)((int64_t)blockIdx.x * rounds / gridDim.x);
  const int r1 = (int)((int64_t)(blockIdx.x + 1) * rounds / gridDim.x);
  pdl_trigger();
  pdl_wait();

  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 W[kTiles], Wn[kTiles];
  uint2 S[kTiles], Sn[kTiles];
  // batch b of round r into (w, s): tiles behind the row's end have scale 0
  auto load = [&](int r, int b, uint4(&w)[kTiles], uint2(&s)[kTiles]) {
    const int unit = r * wu + my_u;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int kt = ((b * kTiles + i) << a.wk_log) + my_k;
      w[i] = none;
      s[i] = make_uint2(0u, 0u);
      if (r < r1 && unit < a.units && kt < a.Tk) {
        const uint8_t* t = a.tiles + ((int64_t)unit * a.Tk + kt) * kQ4TileBytes;
        w[i] = ldg_once(t + 16 * lane);
        s[i] = ldg_once8(t + 512 + 8 * g);
      }
    }
  };
  auto load_x = [&](int b, int i, uint4& x0, uint4& x1) {
    const int kt = ((b * kTiles + i) << a.wk_log) + my_k;
    x0 = x1 = none;
    if (g < a.R && kt < a.Tk) {
      const uint4* src =
          reinterpret_cast<const uint4*>(a.x + (int64_t)g * a.Tk * 64 + kt * 64 + 8 * q);
      x0 = x_pairs(__ldg(src));
      x1 = x_pairs(__ldg(src + 4));
    }
  };
  uint4 X[kKeepX ? kTiles : 1][2];
  load(r0, 0, W, S);
  if constexpr (kKeepX) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) load_x(0, i, X[i][0], X[i][1]);
  }
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  int r = r0, b = 0, par = 0;
  while (r < r1) {
    const bool unit_ends = b + 1 == a.batches;
    const int rn = unit_ends ? r + 1 : r, bn = unit_ends ? 0 : b + 1;
    load(rn, bn, Wn, Sn);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      uint4 x0, x1;
      if constexpr (kKeepX) x0 = X[i][0], x1 = X[i][1];
      else load_x(b, i, x0, x1);
      block_mma(W[i].x, W[i].y, S[i].x, x0, acc);
      block_mma(W[i].z, W[i].w, S[i].y, x1, acc);
    }
    if (unit_ends) {
      part[par][warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      // (the slots written two rounds ago were read before the last barrier)
      __syncthreads();
      for (int o = tid; o < wu * 128; o += kThreads) {
        const int row = o & 15, col = (o >> 4) & 7, u = o >> 7, unit = r * wu + u;
        const int at = ((row & 7) * 4 + (col >> 1)) * 4 + (row >> 3) * 2 + (col & 1);
        if (col >= a.R || unit >= a.units) continue;
        float sum = 0.f;
        for (int w = 0; w < wk; ++w)
          sum = __fadd_rn(sum, reinterpret_cast<const float*>(part[par][u * wk + w])[at]);
        a.y[(int64_t)col * a.units * 16 + unit * 16 + row] = f32_to_bf16_rne(sum);
      }
      par ^= 1;
    }
    r = rn;
    b = bn;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) W[i] = Wn[i], S[i] = Sn[i];
  }
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
  // as many warps along K as there are tiles for them
  while (a.wk_log < 4 && (2 << a.wk_log) <= a.Tk) ++a.wk_log;
  const int wu = kWarps >> a.wk_log, per_warp = (a.Tk + (1 << a.wk_log) - 1) >> a.wk_log;
  const int rounds = (a.units + wu - 1) / wu;
  const int grid = rounds < device_sm_count() ? rounds : device_sm_count();
  a.batches = (per_warp + 3) / 4;
  if (per_warp <= 2) {
    a.batches = 1;
    return launch_pdl(k_q4_proj<2, true>, dim3(grid), kThreads, 0, s, a);
  }
  if (per_warp <= 4) return launch_pdl(k_q4_proj<4, true>, dim3(grid), kThreads, 0, s, a);
  return launch_pdl(k_q4_proj<4, false>, dim3(grid), kThreads, 0, s, a);
}

}  // namespace dsmoe
