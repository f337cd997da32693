// Device-side building blocks of the 8-bit kernels, beside device.cuh.
#pragma once

#include "device.cuh"

namespace svdq {

// maximum that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Smallest scale of a block of 128: a block of zeros has a scale whose
// reciprocal is finite.
constexpr float kFp8MinScale = 0x1p-126f;

// D[tmem] (+)= A[smem] * B[smem], E4M3 x E4M3 -> fp32, K = 32 per instruction.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of an E4M3 x E4M3 -> fp32 product of m x n.
constexpr uint32_t f8_idesc(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One arrival on an mbarrier of the cluster by the lane(s) with `on`, as a
// predicated instruction rather than a branch. It hands over tensor memory
// alone: the loads from it have returned (tcgen05.wait::ld) and the tcgen05
// fences order what follows, so the default scope (the CTA) will do. A release
// at cluster scope in the drain's inner loop waits for every earlier access of
// the warp (it was that loop's largest stall: 8192^3 took 1.04 ms, 0.55 without).
__device__ __forceinline__ void mbar_arrive_if(bool on, uint32_t cluster_addr) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr), "r"((uint32_t)on)
      : "memory");
}

// Whether phase `parity` of `bar` has completed, without holding the warp until
// it has (mbar_try_wait may).
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// `bytes` from p on into L2 (both multiples of 16). L2 is the point of coherence
// of device memory: a prefetch ahead of the wait for the previous kernel can
// never make a later load see an older value.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// two fp32 -> bf16x2 (round to nearest even); `lo` in bits 0..15
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A wait that runs out sends its kernel to the end. What is in flight by then
// (copies, MMAs, stores of the cluster's other CTAs into this one) has to land
// before shared memory and tensor memory are given up. That takes microseconds
// and has this limit of its own, however short the waits' limit was set.
constexpr unsigned long long kLandNs = 100000000ull;

// The same for copies whose barrier is another CTA's, which cannot be waited for.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < kLandNs) __nanosleep(1000);
}

// Register shares of a warpgroup (all four warps execute it).
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace svdq
