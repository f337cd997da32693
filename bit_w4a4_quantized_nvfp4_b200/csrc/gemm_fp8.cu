// The 8-bit GEMM (svdq_fp8_linear):
//   y[m,n] = sum_g sx[g,m] sw[n/128,g] sum_{k in g} qx[m,k] qw[n,k] + bias[n]
// with E4M3 codes and fp32 scales per 128 columns of K. A 64 x 64 output tile
// per CTA, the operands converted to fp32 in shared memory.
#include "device.cuh"
#include "kernels.h"

namespace svdq {
namespace {

__global__ void __launch_bounds__(256) gemm_fp8_kernel(Fp8GemmArgs a) {
  __shared__ float sx[32][65], sw[32][65];
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int G = (a.K + 127) / 128;
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int r = i >> 5, k = i & 31;
      const bool in = k0 + k < a.K;
      sx[k][r] = in && m0 + r < a.M ? e4m3_to_f32(a.x_codes[(size_t)(m0 + r) * a.K + k0 + k]) : 0.f;
      sw[k][r] = in && n0 + r < a.N ? e4m3_to_f32(a.w_codes[(size_t)(n0 + r) * a.K + k0 + k]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sx[k][ty + 16 * i], sw[k][tx + 16 * j], part[i][j]);
    __syncthreads();
    if (k0 % 128 == 96 || k0 + 32 >= a.K) {
      const int g = k0 / 128;
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty + 16 * i;
        const float s = m < a.M ? a.x_scales[(size_t)g * a.M + m] : 0.f;
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + tx + 16 * j;
          if (n < a.N) acc[i][j] = fmaf(s * a.w_scales[(size_t)(n / 128) * G + g], part[i][j], acc[i][j]);
          part[i][j] = 0.f;
        }
      }
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      const float y = acc[i][j] + (a.bias ? bf16_bits_to_f32(a.bias[n]) : 0.f);
      if (a.out_f32)
        static_cast<float*>(a.y)[(size_t)m * a.N + n] = y;
      else
        static_cast<uint16_t*>(a.y)[(size_t)m * a.N + n] = (uint16_t)f32_to_bf16_bits(y);
    }
}

}  // namespace

cudaError_t launch_fp8_linear(const Fp8GemmArgs& a, cudaStream_t s) {
  const dim3 grid((a.N + 63) / 64, (a.M + 63) / 64);
  gemm_fp8_kernel<<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
