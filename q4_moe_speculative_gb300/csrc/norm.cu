// norm.cu — what stands between two blocks of a layer, in one pass over the rows: a block's output
// normed, gated and scaled onto the residual stream, and the norm of the next block's input
// (arithmetic in include/dsmoe.h).
//
// k_block_norm: a row belongs to 8, 16 or 32 lanes of a warp, or to one CTA of up to 512 threads; every
// thread holds its values of the row in registers (kChunks chunks of 8, neighbouring threads
// neighbouring chunks), so that x and y are read once and x_out and h written once, whatever is
// normed. The two sums of squares (y's, then the new x's, which needs the first) are shuffles and,
// for a CTA's row, one exchange through shared memory each. CTAs walk over the rows, the next row's
// loads in flight while a row's sums are waited for: in registers, and for rows above 8192 values,
// whose own take them all, in shared memory.
//
// Bound by bytes, the smallest calls by latency. Measured (bf16, both norms): 6 rows of 4096 2.3 us;
// 16,384 x 4096 91 us, 5.9 TB/s (89% of the copy rate); 8192 x 8192 93 us; 4096 x 16,384 97 us,
// 5.5 TB/s; 4096 x 12,000 83 us, 4.7 TB/s; 32,768 x 256 12.4 us; 65,536 x 64 7.3 us.
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
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* sums) {
#pragma unroll
  for (int o = (kLanes ? kLanes : 32) / 2; o > 0; o >>= 1)
    v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (kLanes == 0) {
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

__device__ __forceinline__ void cp_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from)
               : "memory");
}

// A thread's values of a row as they come.
template <bool kFp32, int kChunks>
struct Raw {
  uint4 x[kChunks * (kFp32 ? 2 : 1)], y[kChunks], gate[kChunks];
};

// kLanes: of a row within a warp, or 0: the CTA has a row.
template <bool kFp32, int kChunks, int kLanes>
__global__ void __launch_bounds__(kLanes ? 256 : 512)
    k_block_norm(const __grid_constant__ NormArgs a) {
  constexpr int kUnit = kLanes ? kLanes : 1;
  constexpr int kRows = kLanes ? 256 / kUnit : 1;    // of a CTA at a time
  // the weights, and the next row's values on their way, in registers; else the latter in shared memory
  constexpr bool kHold = kChunks <= 2;
  __shared__ float sums[2][32];
  const BlockNormProblem& p = a.p;
  const int row_threads = kLanes ? kLanes : blockDim.x;
  const int at = kLanes ? threadIdx.x % kUnit : threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + (kLanes ? threadIdx.x / kUnit : 0);
  pdl_wait();
  pdl_trigger();
  auto there = [&](int i) { return at + i * row_threads < a.chunks; };
  Raw<kFp32, kChunks> raw;
  // (a thread's own vectors, at its place in rows of blockDim.x)
  extern __shared__ uint4 room[];
  auto slot = [&](int j) { return room + j * blockDim.x + threadIdx.x; };
  auto copy = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = at + i * row_threads;
      if (!there(i)) continue;
      if constexpr (kFp32) {
        const float* const from = static_cast<const float*>(p.x) + row * p.x_stride + 8 * c;
        cp_async16(slot(i), from);
        cp_async16(slot(kChunks * 3 + i), from + 4);
      } else {
        cp_async16(slot(i), static_cast<const uint16_t*>(p.x) + row * p.x_stride + 8 * c);
      }
      if (p.y) cp_async16(slot(kChunks + i), p.y + row * p.y_stride + 8 * c);
      if (p.gate && p.gate_stride)
        cp_async16(slot(kChunks * 2 + i), p.gate + row * p.gate_stride + 8 * c);
    }
  };
  auto take = [&] {
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (!there(i)) continue;
      if constexpr (kFp32) {
        raw.x[2 * i] = *slot(i);
        raw.x[2 * i + 1] = *slot(kChunks * 3 + i);
      } else {
        raw.x[i] = *slot(i);
      }
      if (p.y) raw.y[i] = *slot(kChunks + i);
      if (p.gate && p.gate_stride) raw.gate[i] = *slot(kChunks * 2 + i);
    }
    __syncthreads();   // (what has been read may be overwritten)
  };
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
  // (a warp's rows together: where there is none, zeros, and nothing is written)
  if (kLanes && row - (threadIdx.x & 31) / kUnit >= p.T) return;
  // zeros where there is nothing, for the sums; what all rows share stays in registers
  uint4 weight[kChunks], post_weight[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    raw.y[i] = raw.gate[i] = weight[i] = post_weight[i] = make_uint4(0u, 0u, 0u, 0u);
    raw.x[i] = raw.x[kFp32 ? kChunks + i : i] = raw.y[i];
  }
  if constexpr (!kHold) copy(row);
  else if (!kLanes || row < p.T) load(row);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = at + i * row_threads;
    if (!there(i)) continue;
    if (kHold && p.weight) weight[i] = load16(p.weight, c);
    if (kHold && p.post_weight) post_weight[i] = load16(p.post_weight, c);
    if (p.gate && !p.gate_stride) raw.gate[i] = load16(p.gate, c);
  }
  for (;; row += step) {
    float x[kChunks][8], y[8], w[8];
    if constexpr (!kHold) take();
    const Raw<kFp32, kChunks> now = raw;
    // the next row is on its way while this one's sums are waited for
    const bool valid = !kLanes || row < p.T;
    const bool more = kLanes ? __any_sync(0xffffffffu, row + step < p.T) : row + step < p.T;
    if (kLanes ? row + step < p.T : more) {
      if constexpr (kHold) load(row + step);
      else copy(row + step);
    }
    float post = 1.f;
    if (p.post_weight) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        unpack8(now.y[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __fmaf_rn(y[e], y[e], s);
      }
      post = inverse_rms(row_sum<kLanes>(s, sums[0]), p.H, p.eps);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = at + i * row_threads;
      if (!there(i)) continue;
      if constexpr (kFp32) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 v = now.x[2 * i + e];
          x[i][4 * e] = __uint_as_float(v.x), x[i][4 * e + 1] = __uint_as_float(v.y);
          x[i][4 * e + 2] = __uint_as_float(v.z), x[i][4 * e + 3] = __uint_as_float(v.w);
        }
      } else {
        unpack8(now.x[i], x[i]);
      }
      if (p.y) {
        unpack8(now.y[i], y);
        if (p.post_weight) {
          unpack8(kHold ? post_weight[i] : load16(p.post_weight, c), w);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = __fmul_rn(__fmul_rn(y[e], post), __fadd_rn(w[e], p.weight_offset));
        }
        if (p.gate) {
          unpack8(now.gate[i], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(y[e], w[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[i][e] = __fmaf_rn(x[i][e], p.x_scale, __fmul_rn(y[e], p.y_scale));
      }
      if (p.x_out && valid) {
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
      const float pre = inverse_rms(row_sum<kLanes>(s, sums[1]), p.H, p.eps);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (!there(i) || !valid) continue;
        unpack8(kHold ? weight[i] : load16(p.weight, at + i * row_threads), w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = __fmul_rn(__fmul_rn(x[i][e], pre), __fadd_rn(w[e], p.weight_offset));
        reinterpret_cast<uint4*>(p.h_out + row * p.H)[at + i * row_threads] = pack8(w);
      }
    }
    if (!more) return;
    // (a sum's words are read before they are written again: by the other sum's barrier, or here)
    if (!kLanes && !(p.weight && p.post_weight)) __syncthreads();
  }
}

template <bool kFp32, int kChunks, int kLanes>
cudaError_t launch(const NormArgs& a, int threads, cudaStream_t s) {
  const auto kernel = k_block_norm<kFp32, kChunks, kLanes>;
  const int rows = kLanes ? threads / kLanes : 1;
  const int smem = kChunks <= 2 ? 0 : threads * kChunks * (kFp32 ? 64 : 48);
  if (smem) {
    static OncePerDevice ready;
    const cudaError_t e = ready.run([&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  512 * kChunks * (kFp32 ? 64 : 48));
    });
    if (e != cudaSuccess) return e;
  }
  const int64_t need = ((int64_t)a.p.T + rows - 1) / rows, sms = device_sm_count();
  int64_t grid = need;
  if (need > sms) {   // as many CTAs as fit, each with several rows
    static std::atomic<int> fit[33] = {};   // by warps
    int n = fit[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
      const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
      if (e != cudaSuccess) return e;
      if (n < 1) n = 1;
      fit[threads / 32].store(n, std::memory_order_relaxed);
    }
    if (need > sms * n) grid = sms * n;
  }
  return launch_pdl(kernel, dim3((unsigned)grid), threads, smem, s, a);
}

// Two chunks a thread: with one, twice the threads share a row's barriers (16,384 x 4096: 123 against
// 91 us); with four and their copies in shared memory, less is in flight (103 us), but rows above
// 8192 values need more than two (4096 x 16,384 with the next row's in registers: spills, 159 against
// 97 us), and of 9000 three (75 against 84 us). One chunk where a row fits a warp, in as few
// lanes as it fills: 65,536 x 64 27 us with 32 lanes, 7.3 with 8; 32,768 x 256 15.2 with two chunks,
// 12.4 with one.
template <bool kFp32>
cudaError_t choose(const NormArgs& a, cudaStream_t s) {
  const int threads = (a.chunks + 63) / 64 * 32;   // of two chunks
  if (a.chunks <= 8) return launch<kFp32, 1, 8>(a, 256, s);
  if (a.chunks <= 16) return launch<kFp32, 1, 16>(a, 256, s);
  if (a.chunks <= 32) return launch<kFp32, 1, 32>(a, 256, s);
  if (threads == 32) return launch<kFp32, 2, 32>(a, 256, s);
  if (threads <= 512) return launch<kFp32, 2, 0>(a, threads, s);
  if (a.chunks <= 1536) return launch<kFp32, 3, 0>(a, (a.chunks + 95) / 96 * 32, s);
  return launch<kFp32, 4, 0>(a, (a.chunks + 127) / 128 * 32, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormProblem& p, cudaStream_t s) {
  const NormArgs a{p, p.H / 8};
  return p.fp32 ? choose<true>(a, s) : choose<false>(a, s);
}

}  // namespace dsmoe
