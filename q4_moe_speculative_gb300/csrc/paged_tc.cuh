// paged_tc.cuh — what the tcgen05 kernels of the attention over the paged cache share: copies,
// arrivals and operand descriptors.
#pragma once
#include "paged.cuh"
#include "sm100.cuh"

namespace dsmoe {
namespace paged {

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// What this thread may read of memory, copies that it begins may as well.
__device__ __forceinline__ void fence_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
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

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace paged
}  // namespace dsmoe
