// norm.cu — what stands between two blocks of a layer, in one pass over the rows: a block's output
// normed, gated and scaled onto the residual stream, and the norm of the next block's input
// (arithmetic in include/dsmoe.h).
//
// k_block_norm: a row belongs to one warp, or to one CTA of up to 1024 threads; every thread holds
// its values of the row in registers (kChunks chunks of 8, neighbouring threads neighbouring
// chunks), so that x and y are read once and x_out and h written once, whatever is normed. The two
// sums of squares (y's, then the new x's, which needs the first) are shuffles and one exchange
// through shared memory each. CTAs walk over the rows, the next row's loads in flight while a row's
// sums are waited for. Bound by bytes.
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

// A thread's values of a row as they come.
template <bool kFp32, int kChunks>
struct Raw {
  uint4 x[kChunks * (kFp32 ? 2 : 1)], y[kChunks], gate[kChunks];
};

template <bool kFp32, int kChunks, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 512)
    k_block_norm(const __grid_constant__ NormArgs a) {
  __shared__ float sums[2][32];
  const BlockNormProblem& p = a.p;
  const int row_threads = kWarpRow ? 32 : blockDim.x;
  const int at = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * (kWarpRow ? 8 : 1);
  int64_t row = kWarpRow ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  pdl_trigger();
  auto there = [&](int i) { return at + i * row_threads < a.chunks; };
  Raw<kFp32, kChunks> raw;
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = at + i * row_threads;
      if (!there(i)) continue;
      if constexpr (kFp32) {
        const uint4* const from =
            reinterpret_cast<const uint4*>(static_cast<const float*>(p.x) + row * p.x_stride) + 2 * c;
        raw.x[2 * i] = from[0];
        raw.x[2 * i + 1] = from[1];
      } else {
        raw.x[i] = load16(static_cast<const uint16_t*>(p.x) + row * p.x_stride, c);
      }
      if (p.y) raw.y[i] = load16(p.y + row * p.y_stride, c);
      if (p.gate && p.gate_stride) raw.gate[i] = load16(p.gate + row * p.gate_stride, c);
    }
  };
  if (kWarpRow && row >= p.T) return;
  // (zeros where there is nothing, for the sums; what all rows share stays in registers)
  uint4 weight[kChunks], post_weight[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    raw.y[i] = raw.gate[i] = weight[i] = post_weight[i] = make_uint4(0u, 0u, 0u, 0u);
    raw.x[i] = raw.x[kFp32 ? kChunks + i : i] = raw.y[i];
  }
  load(row);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = at + i * row_threads;
    if (!there(i)) continue;
    if (p.weight) weight[i] = load16(p.weight, c);
    if (p.post_weight) post_weight[i] = load16(p.post_weight, c);
    if (p.gate && !p.gate_stride) raw.gate[i] = load16(p.gate, c);
  }
  for (;; row += step) {
    float x[kChunks][8], y[kChunks][8], w[8];
    uint4 gate[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if constexpr (kFp32) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 v = raw.x[2 * i + e];
          x[i][4 * e] = __uint_as_float(v.x), x[i][4 * e + 1] = __uint_as_float(v.y);
          x[i][4 * e + 2] = __uint_as_float(v.z), x[i][4 * e + 3] = __uint_as_float(v.w);
        }
      } else {
        unpack8(raw.x[i], x[i]);
      }
      unpack8(raw.y[i], y[i]);
      gate[i] = raw.gate[i];
    }
    // the next row is on its way while this one's sums are waited for
    const bool more = row + step < p.T;
    if (more) load(row + step);
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
      if (!there(i)) continue;
      if (p.y) {
        if (p.post_weight) {
          unpack8(post_weight[i], w);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[i][e] = __fmul_rn(__fmul_rn(y[i][e], post), __fadd_rn(w[e], p.weight_offset));
        }
        if (p.gate) {
          unpack8(gate[i], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] = __fmul_rn(y[i][e], w[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[i][e] = __fmaf_rn(x[i][e], p.x_scale, __fmul_rn(y[i][e], p.y_scale));
      }
      if (p.x_out) {
        if constexpr (kFp32) {
          float4* const to =
              reinterpret_cast<float4*>(static_cast<float*>(p.x_out) + row * p.H) + 2 * c;
          to[0] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
          to[1] = make_float4(x[i][4], x[i][5], x[i][6], x[i][7]);
        } else {
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.x_out) + row * p.H)[c] = pack8(x[i]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __fmaf_rn(x[i][e], x[i][e], s);
    }
    if (p.weight) {
      const float pre = inverse_rms(row_sum<kWarpRow>(s, sums[1]), p.H, p.eps);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (!there(i)) continue;
        unpack8(weight[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = __fmul_rn(__fmul_rn(x[i][e], pre), __fadd_rn(w[e], p.weight_offset));
        reinterpret_cast<uint4*>(p.h_out + row * p.H)[at + i * row_threads] = pack8(w);
      }
    }
    if (!more) return;
    // (a sum's words are read before they are written again: by the other sum's barrier, or here)
    if (!kWarpRow && !(p.weight && p.post_weight)) __syncthreads();
  }
}

template <bool kFp32, int kChunks, bool kWarpRow>
cudaError_t launch(const NormArgs& a, int threads, cudaStream_t s) {
  const auto kernel = k_block_norm<kFp32, kChunks, kWarpRow>;
  const int rows = kWarpRow ? 8 : 1;
  const int64_t need = ((int64_t)a.p.T + rows - 1) / rows, sms = device_sm_count();
  int64_t grid = need;
  if (need > sms) {   // as many CTAs as fit, each with several rows
    static std::atomic<int> fit[33] = {};   // by warps
    int n = fit[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
      const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
      if (e != cudaSuccess) return e;
      if (n < 1) n = 1;
      fit[threads / 32].store(n, std::memory_order_relaxed);
    }
    if (need > sms * n) grid = sms * n;
  }
  return launch_pdl(kernel, dim3((unsigned)grid), threads, 0, s, a);
}

template <bool kFp32, int kChunks>
cudaError_t start(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.chunks + kChunks - 1) / kChunks + 31) / 32 * 32;
  return threads == 32 ? launch<kFp32, kChunks, true>(a, 256, s)
                       : launch<kFp32, kChunks, false>(a, threads, s);
}

template <bool kFp32>
cudaError_t choose(const NormArgs& a, cudaStream_t s) {
  return a.chunks <= 1024 ? start<kFp32, 2>(a, s) : start<kFp32, 4>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormProblem& p, cudaStream_t s) {
  const NormArgs a{p, p.H / 8};
  return p.fp32 ? choose<true>(a, s) : choose<false>(a, s);
}

}  // namespace dsmoe
