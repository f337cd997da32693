// The 8-bit form of activations, with or without a root-mean-square norm and
// the residual's addition ahead of it (svdq_fp8_norm_quantize,
// svdq_fp8_quantize_act):
//   r = bf16(x + residual);  v = r / sqrt(mean(r^2) + eps) * w
//   per 128 columns: scale = max(max|v| / 448, 2^-126), code = e4m3(v / scale)
// Bound by HBM: 3 bytes an element, 7 with a residual.
//
// A lane holds 8 consecutive columns (16 bytes of bf16), so 16 lanes are one
// block of 128: its largest magnitude is four shuffles. v stays in fp32 from
// the norm to its one rounding to E4M3 (no bf16 in between, which would round
// twice); the residual's sum is rounded to bf16 first, since that is the
// value the next layer reads.
//
// Norm: a row belongs to tpr threads (a power of two of warps) and stays in
// their registers; CTAs are persistent, hold the norm weight in registers
// and load their next row while the current one is reduced. Without the norm
// blocks are independent: a warp takes four pieces of 256 columns at a time.
#include "fp8.cuh"
#include "kernels.h"

namespace svdq {
namespace {

// largest magnitude of 8 values; a NaN among them stays
__device__ __forceinline__ float absmax8(const float (&v)[8]) {
  float a = max_nan(fabsf(v[0]), fabsf(v[1])), b = max_nan(fabsf(v[2]), fabsf(v[3]));
  const float c = max_nan(fabsf(v[4]), fabsf(v[5])), d = max_nan(fabsf(v[6]), fabsf(v[7]));
  a = max_nan(a, b);
  b = max_nan(c, d);
  return max_nan(a, b);
}

// the same over the 16 lanes of a block, and the block's scale
__device__ __forceinline__ float block_scale(float am) {
#pragma unroll
  for (int o = 8; o; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  return max_nan(am * (1.0f / 448.0f), kFp8MinScale);
}

// 8 codes of v / scale (as v times the rounded reciprocal: half a step of
// fp32 more, against half a step of E4M3)
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float rcp) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r.x)
      : "f"(v[0] * rcp), "f"(v[1] * rcp), "f"(v[2] * rcp), "f"(v[3] * rcp));
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r.y)
      : "f"(v[4] * rcp), "f"(v[5] * rcp), "f"(v[6] * rcp), "f"(v[7] * rcp));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// ------------------------------------------------------------------ norm
constexpr int kMaxWarps = 16;

template <int VPT, bool RES>
__global__ void __launch_bounds__(512) fp8_norm_kernel(const Fp8ActArgs a, int tpr) {
  __shared__ float part[2][kMaxWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpc = blockDim.x / tpr, mr = threadIdx.x / tpr, tid = threadIdx.x % tpr;
  const int wpr = tpr / 32, w0 = mr * wpr;
  const int nv = a.K / 8;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (threadIdx.x == 0) launch_dependents();
  // every input may be the previous kernel's output, every output may still
  // be read by it
  grid_dependency_wait();

  // registers for the weight and the next row: up to 4 vectors a thread
  constexpr bool kAhead = VPT <= 4;
  auto weight = [&](int j) {
    const int i = j * tpr + tid;
    return i < nv ? __ldg(reinterpret_cast<const uint4*>(a.weight) + i) : zero;
  };
  uint4 wv[VPT];
  if (kAhead) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) wv[j] = weight(j);
  }
  // a barrier of the row's threads
  auto row_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + mr), "r"(tpr) : "memory"); };
  uint4 xn[VPT], rn[VPT];
  auto fetch = [&](long long m) {
    const uint4* xp = reinterpret_cast<const uint4*>(a.x + (size_t)m * (size_t)a.ldx);
    const uint4* rp = reinterpret_cast<const uint4*>(a.residual + (size_t)m * (size_t)a.ldr);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * tpr + tid;
      const bool in = m < a.M && i < nv;
      xn[j] = in ? xp[i] : zero;
      if (RES) rn[j] = in ? rp[i] : zero;
    }
  };
  const long long step = (long long)gridDim.x * rpc;
  long long m = (long long)blockIdx.x * rpc + mr;
  if (kAhead) fetch(m);
  int par = 0;
  for (long long base = (long long)blockIdx.x * rpc; base < a.M; base += step, m += step, par ^= 1) {
    if (!kAhead) fetch(m);
    uint4 r[VPT];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float v[8];
      unpack8(xn[j], v);
      if (RES) {
        float u[8];
        unpack8(rn[j], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += u[i];
        r[j] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
        unpack8(r[j], v);
      } else {
        r[j] = xn[j];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    }
    if (RES && m < a.M) {
      uint4* op = reinterpret_cast<uint4*>(a.residual_out + (size_t)m * (size_t)a.ldo);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (j * tpr + tid < nv) op[j * tpr + tid] = r[j];
    }
    if (kAhead) fetch(m + step);
    // the row's sum: lanes, then its warps in order (two buffers: a warp may
    // be a row ahead of the slowest)
    auto row_sum = [&](float s, float* buf) {
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (wpr == 1) return s;
      if (lane == 0) buf[warp] = s;
      row_sync();
      s = 0.f;
      for (int i = 0; i < wpr; ++i) s += buf[w0 + i];
      return s;
    };
    ss = row_sum(ss, part[par]);
    float up = 1.f;
    // squares of bf16 values can pass fp32's range at both ends: such a row is
    // summed again, scaled by a power of two
    if (ss > 0x1p120f || (ss < 0x1p-80f && a.eps < 0x1p-60f && m < a.M)) {
      up = ss > 0x1p120f ? 0x1p-64f : 0x1p64f;
      float s2 = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float v[8];
        unpack8(r[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s2 = fmaf(up * v[i], up * v[i], s2);
      }
      if (wpr > 1) row_sync();   // the first sums have been read
      ss = row_sum(s2, part[par]);
    }
    const float inv = up * rsqrtf(ss / (float)a.K + up * up * a.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * tpr + tid;
      float v[8], w[8];
      unpack8(r[j], v);
      unpack8(kAhead ? wv[j] : weight(j), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * inv * w[k];
      const float scale = block_scale(i < nv ? absmax8(v) : 0.f);
      const uint2 c = codes8(v, __frcp_rn(scale));
      if (m < a.M && i < nv) {
        *reinterpret_cast<uint2*>(a.codes + (size_t)m * a.K + 8 * (size_t)i) = c;
        if ((lane & 15) == 0) a.scales[(size_t)(i / 16) * a.M + m] = scale;
      }
    }
  }
}

// -------------------------------------------------------------- no norm
constexpr int kPieces = 4;   // pieces of 256 columns a warp loads at once

__global__ void __launch_bounds__(256) fp8_quant_kernel(const Fp8ActArgs a, int per_row, long long pieces) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) launch_dependents();
  grid_dependency_wait();
  const long long p0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPieces;
  uint4 x[kPieces];
  long long row[kPieces];
  int col[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const long long p = p0 + u;
    row[u] = p / per_row;
    col[u] = (int)(p - row[u] * per_row) * 256 + 8 * lane;
    const bool in = p < pieces && col[u] < a.K;
    if (!in) col[u] = -1;
    x[u] = in ? *reinterpret_cast<const uint4*>(a.x + (size_t)row[u] * (size_t)a.ldx + col[u])
              : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    float v[8];
    unpack8(x[u], v);
    const float scale = block_scale(absmax8(v));
    const uint2 c = codes8(v, __frcp_rn(scale));
    if (col[u] >= 0) {
      *reinterpret_cast<uint2*>(a.codes + (size_t)row[u] * a.K + col[u]) = c;
      if ((lane & 15) == 0) a.scales[(size_t)(col[u] / 128) * a.M + row[u]] = scale;
    }
  }
}

cudaError_t launch_pdl(const void* fn, unsigned grid, int block, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int VPT>
cudaError_t launch_norm(const Fp8ActArgs& a, int tpr, int num_sms, cudaStream_t s) {
  Fp8ActArgs args = a;
  const int block = tpr < 256 ? 256 : tpr, rpc = block / tpr;
  const long long ctas = ((long long)a.M + rpc - 1) / rpc, most = (long long)num_sms * (1024 / block);
  void* ptrs[] = {&args, &tpr};
  const void* fn = a.residual ? reinterpret_cast<const void*>(fp8_norm_kernel<VPT, true>)
                              : reinterpret_cast<const void*>(fp8_norm_kernel<VPT, false>);
  return launch_pdl(fn, (unsigned)(ctas < most ? ctas : most), block, s, ptrs);
}

}  // namespace

cudaError_t launch_fp8_act(const Fp8ActArgs& a, int num_sms, cudaStream_t s) {
  if (!a.weight) {
    Fp8ActArgs args = a;
    int per_row = (a.K + 255) / 256;
    long long pieces = (long long)a.M * per_row;
    void* ptrs[] = {&args, &per_row, &pieces};
    return launch_pdl(reinterpret_cast<const void*>(fp8_quant_kernel), (unsigned)((pieces + 8 * kPieces - 1) / (8 * kPieces)),
                      256, s, ptrs);
  }
  // threads of a row: a power of two of warps, up to 8 vectors of 8 columns each
  const int nv = a.K / 8;
  int vpt = a.M <= 2 * num_sms ? 1 : 2, tpr = 32;
  while (tpr < 512 && tpr * vpt < nv) tpr *= 2;
  while (tpr * vpt < nv) vpt *= 2;
  switch (vpt) {
    case 1: return launch_norm<1>(a, tpr, num_sms, s);
    case 2: return launch_norm<2>(a, tpr, num_sms, s);
    case 4: return launch_norm<4>(a, tpr, num_sms, s);
    default: return launch_norm<8>(a, tpr, num_sms, s);
  }
}

}  // namespace svdq
