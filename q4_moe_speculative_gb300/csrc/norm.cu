// norm.cu — what stands between two blocks of a layer, in one pass over the rows: a block's output
// normed, gated and scaled onto the residual stream, and the norm of the next block's input
// (arithmetic in include/dsmoe.h).
//
// k_block_norm: a row belongs to one warp, or to one CTA of up to 1024 threads; every thread holds
// its values of the row in registers (kChunks chunks of 8, neighbouring threads neighbouring
// chunks), so that x and y are read once and x_out and h written once, whatever is normed. The two
// sums of squares (y's, then the new x's, which needs the first) are shuffles and one exchange
// through shared memory each. Bound by bytes.
#include "common.cuh"
#include "kernels.h"

namespace dsmoe {
namespace {

struct NormArgs {
  BlockNormProblem p;
  int chunks;      // of 8 values in a row
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ uint4 load16(const uint16_t* p, int64_t chunk) {
  return reinterpret_cast<const uint4*>(p)[chunk];
}

// Sum over the row's threads; every one gets it. `sums`: one word per warp of the CTA.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (!kWarpRow) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    v = lane < warps ? sums[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}
__device__ __forceinline__ float inverse_rms(float squares, int H, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(squares, (float)H), eps)));
}

template <bool kFp32, int kChunks, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : (kChunks == 4 ? 512 : 1024))
    k_block_norm(const NormArgs a) {
  __shared__ float sums[2][32];
  const BlockNormProblem& p = a.p;
  const int row_threads = kWarpRow ? 32 : blockDim.x;
  const int at = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarpRow ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  if (kWarpRow && row >= p.T) return;
  float x[kChunks][8], y[kChunks][8];
  uint4 raw_y[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = at + i * row_threads;
    raw_y[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    if (c >= a.chunks) continue;
    if (p.y) raw_y[i] = load16(p.y + row * p.y_stride, c);
    if constexpr (kFp32) {
      const float4* const from =
          reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + row * p.x_stride) + 2 * c;
      const float4 lo = from[0], hi = from[1];
      x[i][0] = lo.x, x[i][1] = lo.y, x[i][2] = lo.z, x[i][3] = lo.w;
      x[i][4] = hi.x, x[i][5] = hi.y, x[i][6] = hi.z, x[i][7] = hi.w;
    } else {
      unpack8(load16(static_cast<const uint16_t*>(p.x) + row * p.x_stride, c), x[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) unpack8(raw_y[i], y[i]);
  float post = 1.f;
  if (p.post_weight) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __fmaf_rn(y[i][e], y[i][e], s);
    post = inverse_rms(row_sum<kWarpRow>(s, sums[0]), p.H, p.eps);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = at + i * row_threads;
    if (c >= a.chunks) continue;
    if (p.y) {
      float w[8];
      if (p.post_weight) {
        unpack8(load16(p.post_weight, c), w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[i][e] = __fmul_rn(__fmul_rn(y[i][e], post), __fadd_rn(w[e], p.weight_offset));
      }
      if (p.gate) {
        unpack8(load16(p.gate + row * p.gate_stride, c), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] = __fmul_rn(y[i][e], w[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[i][e] = __fmaf_rn(x[i][e], p.x_scale, __fmul_rn(y[i][e], p.y_scale));
    }
    if (p.x_out) {
      if constexpr (kFp32) {
        float4* const to = reinterpret_cast<float4*>(static_cast<float*>(p.x_out) + row * p.H) + 2 * c;
        to[0] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        to[1] = make_float4(x[i][4], x[i][5], x[i][6], x[i][7]);
      } else {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.x_out) + row * p.H)[c] = pack8(x[i]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __fmaf_rn(x[i][e], x[i][e], s);
  }
  if (!p.weight) return;
  const float pre = inverse_rms(row_sum<kWarpRow>(s, sums[1]), p.H, p.eps);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = at + i * row_threads;
    if (c >= a.chunks) continue;
    float w[8];
    unpack8(load16(p.weight, c), w);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = __fmul_rn(__fmul_rn(x[i][e], pre), __fadd_rn(w[e], p.weight_offset));
    reinterpret_cast<uint4*>(p.h_out + row * p.H)[c] = pack8(w);
  }
}

template <bool kFp32, int kChunks>
cudaError_t start(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.chunks + kChunks - 1) / kChunks + 31) / 32 * 32;
  if (threads == 32)
    return launch_pdl(k_block_norm<kFp32, kChunks, true>, dim3((a.p.T + 7) / 8), 256, 0, s, a);
  return launch_pdl(k_block_norm<kFp32, kChunks, false>, dim3(a.p.T), threads, 0, s, a);
}

template <bool kFp32>
cudaError_t choose(const NormArgs& a, cudaStream_t s) {
  // few rows: a chunk per thread, so that a row's latency is one load's; more: four
  if (a.p.T <= 2 * device_sm_count() && a.chunks <= 1024) return start<kFp32, 1>(a, s);
  return a.chunks <= 2048 && a.p.T <= 2 * device_sm_count() ? start<kFp32, 2>(a, s)
                                                            : start<kFp32, 4>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormProblem& p, cudaStream_t s) {
  const NormArgs a{p, p.H / 8};
  return p.fp32 ? choose<true>(a, s) : choose<false>(a, s);
}

}  // namespace dsmoe
