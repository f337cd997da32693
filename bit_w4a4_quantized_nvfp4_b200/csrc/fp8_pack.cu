// Offline pack of an 8-bit weight (svdq_fp8_pack_weight): W fp32 [K, N] ->
// E4M3 codes [N, K] with one fp32 scale per 128 x 128 block. One CTA per
// block: it finds the block's largest magnitude (a first pass over W), then
// turns the block through shared memory so that both the reads (along N) and
// the writes (along K) are contiguous. Not on a timed path.
#include "fp8.cuh"
#include "kernels.h"

namespace svdq {
namespace {

constexpr int kThreadsP = 256;

__global__ void __launch_bounds__(kThreadsP) fp8_pack_kernel(int K, int N, const float* __restrict__ W,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ float part[kThreadsP / 32];
  __shared__ uint8_t tile[128][132];  // [n][k]; the pitch spreads a column's writes over the banks
  const int k0 = blockIdx.x * 128, n0 = blockIdx.y * 128;
  const int nk = min(128, K - k0), nn = min(128, N - n0);
  float am = 0.f;
  for (int i = threadIdx.x; i < 128 * 128; i += kThreadsP) {
    const int k = i >> 7, n = i & 127;
    if (k < nk && n < nn) am = max_nan(am, fabsf(W[(size_t)(k0 + k) * N + n0 + n]));
  }
  for (int o = 16; o; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = am;
  __syncthreads();
  am = part[0];
  for (int i = 1; i < kThreadsP / 32; ++i) am = max_nan(am, part[i]);
  const float scale = max_nan(am / 448.0f, kFp8MinScale);
  for (int i = threadIdx.x; i < 128 * 128; i += kThreadsP) {
    const int k = i >> 7, n = i & 127;
    if (k < nk && n < nn) tile[n][k] = (uint8_t)cvt_e4m3(W[(size_t)(k0 + k) * N + n0 + n] / scale);
  }
  __syncthreads();
  // K and the block's start are multiples of 16: rows go out in 4-byte words
  for (int i = threadIdx.x; i < 128 * 32; i += kThreadsP) {
    const int n = i >> 5, k = 4 * (i & 31);
    if (n < nn && k < nk)
      *reinterpret_cast<uint32_t*>(codes + (size_t)(n0 + n) * K + k0 + k) =
          *reinterpret_cast<const uint32_t*>(&tile[n][k]);
  }
  if (threadIdx.x == 0) scales[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = scale;
}

}  // namespace

cudaError_t launch_fp8_pack(int K, int N, const float* W, uint8_t* codes, float* scales, cudaStream_t s) {
  const dim3 grid((K + 127) / 128, (N + 127) / 128);
  fp8_pack_kernel<<<grid, kThreadsP, 0, s>>>(K, N, W, codes, scales);
  return cudaGetLastError();
}

}  // namespace svdq
