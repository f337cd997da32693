// The 8-bit form of activations, with or without a root-mean-square norm and
// the residual's addition ahead of it (svdq_fp8_norm_quantize,
// svdq_fp8_quantize_act):
//   r = bf16(x + residual);  v = r / sqrt(mean(r^2) + eps) * w
//   per 128 columns: scale = max(max|v| / 448, 2^-126), code = e4m3(v / scale)
// One CTA per row.
#include "device.cuh"
#include "kernels.h"

namespace svdq {
namespace {

constexpr int kThreadsA = 256;

// maximum that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float value(const Fp8ActArgs& a, size_t m, int k) {
  const float x = bf16_bits_to_f32(a.x[m * (size_t)a.ldx + k]);
  if (!a.residual) return x;
  const uint32_t r = f32_to_bf16_bits(x + bf16_bits_to_f32(a.residual[m * (size_t)a.ldr + k]));
  return bf16_bits_to_f32(r);
}

// sum over the row of (up * r)^2
__device__ __forceinline__ float row_squares(const Fp8ActArgs& a, size_t m, float up, float* part) {
  float ss = 0.f;
  for (int k = threadIdx.x; k < a.K; k += kThreadsA) {
    const float r = up * value(a, m, k);
    ss = fmaf(r, r, ss);
  }
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.f;
  for (int i = 0; i < kThreadsA / 32; ++i) ss += part[i];
  return ss;
}

__global__ void __launch_bounds__(kThreadsA) fp8_act_kernel(Fp8ActArgs a) {
  __shared__ float part[kThreadsA / 32];
  const size_t m = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float inv = 1.f;
  if (a.weight) {
    float ss = row_squares(a, m, 1.f, part), up = 1.f;
    // squares of bf16 values can pass fp32's range at both ends: such a row
    // is summed again, scaled by a power of two
    if (ss > 0x1p120f)
      up = 0x1p-64f;
    else if (ss < 0x1p-80f && a.eps < 0x1p-60f)
      up = 0x1p64f;
    if (up != 1.f) ss = row_squares(a, m, up, part);
    inv = up * rsqrtf(ss / (float)a.K + up * up * a.eps);
  }
  const int G = (a.K + 127) / 128;
  for (int g = warp; g < G; g += kThreadsA / 32) {
    float v[4], am = 0.f;
    for (int j = 0; j < 4; ++j) {
      const int k = g * 128 + 4 * lane + j;
      v[j] = 0.f;
      if (k < a.K) {
        const float r = value(a, m, k);
        v[j] = a.weight ? r * inv * bf16_bits_to_f32(a.weight[k]) : r;
        if (a.residual_out) a.residual_out[m * (size_t)a.ldo + k] = (uint16_t)f32_to_bf16_bits(r);
      }
      am = max_nan(am, fabsf(v[j]));
    }
    for (int o = 16; o; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    const float scale = max_nan(am / 448.0f, 1.17549435e-38f);
    for (int j = 0; j < 4; ++j) {
      const int k = g * 128 + 4 * lane + j;
      if (k < a.K) a.codes[m * (size_t)a.K + k] = (uint8_t)cvt_e4m3(v[j] / scale);
    }
    if (lane == 0) a.scales[(size_t)g * a.M + m] = scale;
  }
}

}  // namespace

cudaError_t launch_fp8_act(const Fp8ActArgs& a, cudaStream_t s) {
  fp8_act_kernel<<<(unsigned)a.M, kThreadsA, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
