// Rotary positions (svdq_rope_apply, svdq_rope_tables): pair i of a head at
// row m turns by t = pos[m, axis[i]] * freq[i], cos and sin times factor.
//
// t is formed in 64 bits, since a position of a long context times a
// frequency near 1 leaves fp32 too few bits behind the whole turns. The whole
// turns are taken off by Cody and Waite's reduction: t - n * 2pi with 2pi in
// two parts and fused multiply-adds, so that the remainder keeps its bits;
// cos and sin of the remainder are fp32.
#include "device.cuh"
#include "kernels.h"

namespace svdq {
namespace {

// 2 pi as the nearest double and the rest of it (the next 53 bits)
constexpr double kTwoPi = 6.283185307179586477;
constexpr double kTwoPiRest = 2.449293598294706414e-16;

__device__ __forceinline__ void rope_turn(long long pos, double freq, float factor, float& c, float& s) {
  const double t = (double)pos * freq;
  const double n = rint(t * (1.0 / kTwoPi));
  const double r = fma(-n, kTwoPiRest, fma(-n, kTwoPi, t));
  float cs, sn;
  sincospif((float)(r * (2.0 / kTwoPi)), &sn, &cs);
  c = cs * factor;
  s = sn * factor;
}

__device__ __forceinline__ long long rope_position(const RopeArgs& a, size_t m, int i) {
  const int x = a.axis ? a.axis[i] : 0;
  return a.pos[m * a.axes + (x >= 0 && x < a.axes ? x : 0)];
}

__global__ void __launch_bounds__(256) rope_tables_kernel(RopeArgs a, float* __restrict__ cos_t,
                                                          float* __restrict__ sin_t) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (size_t)a.M * a.pairs) return;
  const size_t m = i / a.pairs;
  const int p = (int)(i % a.pairs);
  rope_turn(rope_position(a, m, p), a.freq[p], a.factor, cos_t[i], sin_t[i]);
}

__global__ void __launch_bounds__(256) rope_apply_kernel(RopeArgs a) {
  __shared__ float cs[kRopeMaxPairs], sn[kRopeMaxPairs];
  const size_t m = blockIdx.x;
  for (int i = threadIdx.x; i < a.pairs; i += 256)
    rope_turn(rope_position(a, m, i), a.freq[i], a.factor, cs[i], sn[i]);
  __syncthreads();
  const uint16_t* x = a.x + m * (size_t)a.ldx;
  uint16_t* y = a.y + m * (size_t)a.ldy;
  for (int j = threadIdx.x; j < a.heads * a.pairs; j += 256) {
    const int h = j / a.pairs, i = j % a.pairs;
    const int p = h * a.head_dim + (a.half ? i : 2 * i), q = a.half ? p + a.pairs : p + 1;
    const float u = bf16_bits_to_f32(x[p]), v = bf16_bits_to_f32(x[q]);
    y[p] = (uint16_t)f32_to_bf16_bits(fmaf(u, cs[i], -v * sn[i]));
    y[q] = (uint16_t)f32_to_bf16_bits(fmaf(u, sn[i], v * cs[i]));
  }
  if (x == y) return;
  const int rest = a.head_dim - 2 * a.pairs;
  for (int j = threadIdx.x; j < a.heads * rest; j += 256) {
    const int p = j / rest * a.head_dim + 2 * a.pairs + j % rest;
    y[p] = x[p];
  }
}

}  // namespace

cudaError_t launch_rope_tables(const RopeArgs& a, float* cos_t, float* sin_t, cudaStream_t s) {
  const size_t n = (size_t)a.M * a.pairs;
  rope_tables_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, cos_t, sin_t);
  return cudaGetLastError();
}

cudaError_t launch_rope_apply(const RopeArgs& a, cudaStream_t s) {
  rope_apply_kernel<<<(unsigned)a.M, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
