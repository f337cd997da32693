// The 8-bit form of activations, with or without a root-mean-square norm and
// the residual's addition ahead of it (svdq_fp8_norm_quantize,
// svdq_fp8_quantize_act):
//   r = bf16(x + residual);  v = r / sqrt(mean(r^2) + eps) * w
//   per 128 columns: scale = max(max|v| / 448, 2^-126), code = e4m3(v / scale)
// Bound by HBM: 3 bytes an element, 7 with a residual. Measured from HBM
// (launches in a row over three sets of inputs): norm + residual 4608 x 4096
// 21.1 us, 6.3 TB/s, 0.97 of the measured copy rate (20.4 us at that rate); 8192
// x 8192 67.9 us; norm alone 4608 x 12288 29.3 us, 0.90; without the norm 4608 x
// 12288 28.3 us, 0.93. What is left of the norm's is the columns' arithmetic,
// some ten instructions each.
//
// A load is 8 consecutive columns (16 bytes of bf16); a block of 128 is 16 of
// them, held by 16 lanes, or by 4 with four loads each: its largest magnitude is
// four shuffles, or two. v stays in fp32 from the norm to its one rounding to
// E4M3 (no bf16 in between, which would round twice); the residual's sum is
// rounded to bf16 first, since that is the value the next layer reads.
//
// Norm: one pass, a row to a warp or several. Without the norm blocks are
// independent: a warp takes two pieces of 256 columns at a time.
#include "fp8.cuh"
#include "kernels.h"

namespace svdq {
namespace {

// largest magnitude of three / of 8 values; a NaN among them stays
__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float absmax8(const float2 (&v)[4]) {
  return absmax3(absmax3(v[0].x, v[0].y, v[1].x), absmax3(v[1].y, v[2].x, v[2].y), absmax3(v[3].x, v[3].y, 0.f));
}

// the same over the LANES lanes of a block
template <int LANES>
__device__ __forceinline__ float block_max(float am) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  return am;
}
__device__ __forceinline__ float scale_of(float am) { return max_nan(am * (1.0f / 448.0f), kFp8MinScale); }

__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 8 codes of v * f. f is a rounded reciprocal, which with the product is off
// by under 2^-22, against half a step of E4M3, 2^-4.
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float f) {
  uint32_t r[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 a = __fmul2_rn(v[2 * h], make_float2(f, f)), b = __fmul2_rn(v[2 * h + 1], make_float2(f, f));
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r[h])
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  }
  return make_uint2(r[0], r[1]);
}

__device__ __forceinline__ void unpack8(const uint4 q, float2 (&v)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// ------------------------------------------------------------------ norm
// A block's codes do not depend on the row's norm: with t = r w the block's v
// is t / rms, its largest magnitude max|t| / rms, and v / scale = 448 t /
// max|t|. So one pass over the row writes r and the codes and leaves only
// max|t| of each block behind; the scales follow once the row's sum is known,
// and nothing of the row has to be held.
// A: vectors of 8 columns a thread has in flight. They belong to one block, so
// 16 / A lanes share a block and its maximum and factor come once for all A
// (norm alone 4608 x 12288 29.7 us; 33.0 with a block's vectors in 16 lanes).
template <bool RES, int A>
__global__ void __launch_bounds__(512, 2) fp8_norm_kernel(const Fp8ActArgs a, int wpr, float inv_k) {
  constexpr int kLanes = 16 / A;
  __shared__ float part[2][16];
  extern __shared__ float block_am[];   // [warps][2 A * steps]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mr = warp / wpr, w0 = mr * wpr, tpr = 32 * wpr;
  const int tid = threadIdx.x - 32 * w0;
  const int nv = a.K / 8, steps = (nv + A * tpr - 1) / (A * tpr);
  const long long m = (long long)blockIdx.x * ((blockDim.x >> 5) / wpr) + mr;
  float* am_w = block_am + 2 * A * steps * warp;
  // this thread's vectors of a step: vector u of them is kLanes u further
  auto at = [&](int j) { return ((j * wpr + warp - w0) * 2 * A + lane / kLanes) * 16 + lane % kLanes; };
  if (threadIdx.x == 0) launch_dependents();
  // (the last CTA's rows past M take the barriers below and write nothing)
  const bool live = m < a.M;
  // Each row's first columns are on their way to L2 while the previous kernel
  // ends (norm + residual 4608 x 4096, a row a warp, 22.9 us, 24.0 without; 512
  // x 4096 4.4 against 5.0; more than 2 KB a warp is slower at many rows).
  if (tid == 0 && live) {
    const uint32_t bytes = (uint32_t)min(2048 * wpr, 2 * a.K);
    prefetch_l2(a.x + (size_t)m * (size_t)a.ldx, bytes);
    if (RES) prefetch_l2(a.residual + (size_t)m * (size_t)a.ldr, bytes);
  }
  // every input may be the previous kernel's output, every output may still
  // be read by it
  grid_dependency_wait();
  const uint4* xp = reinterpret_cast<const uint4*>(a.x + (size_t)m * (size_t)a.ldx);
  const uint4* qp = reinterpret_cast<const uint4*>(a.residual + (size_t)m * (size_t)a.ldr);
  uint4* op = reinterpret_cast<uint4*>(a.residual_out + (size_t)m * (size_t)a.ldo);
  const uint4* wp = reinterpret_cast<const uint4*>(a.weight);
  uint2* cp = reinterpret_cast<uint2*>(a.codes + (size_t)m * a.K);

  float2 ss2 = make_float2(0.f, 0.f);
  float least = 0x1p127f;   // the smallest max|t| of a block that is not all zeros
  bool odd = false;         // a block whose products need the definition's order
  for (int j = 0; j < steps; ++j) {
    const int i0 = at(j);
    uint4 r[A], q[A], w[A];
    // whole steps (all but a row's last) load without conditions
    const bool whole = live && (j * wpr + warp - w0 + 1) * 32 * A <= nv;
    if (whole) {
#pragma unroll
      for (int u = 0; u < A; ++u) {
        r[u] = xp[i0 + u * kLanes];
        if (RES) q[u] = qp[i0 + u * kLanes];
        w[u] = __ldg(wp + i0 + u * kLanes);
      }
    } else {
#pragma unroll
      for (int u = 0; u < A; ++u) {
        const bool in = live && i0 + u * kLanes < nv;
        r[u] = in ? xp[i0 + u * kLanes] : make_uint4(0u, 0u, 0u, 0u);
        if (RES) q[u] = in ? qp[i0 + u * kLanes] : make_uint4(0u, 0u, 0u, 0u);
        w[u] = in ? __ldg(wp + i0 + u * kLanes) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    float2 v[A][4];
    float am = 0.f;
#pragma unroll
    for (int u = 0; u < A; ++u) {
      float2 g[4];
      unpack8(r[u], v[u]);
      if (RES) {
        unpack8(q[u], g);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][k] = __fadd2_rn(v[u][k], g[k]);
        r[u] = make_uint4(pack_bf16x2(v[u][0].x, v[u][0].y), pack_bf16x2(v[u][1].x, v[u][1].y),
                          pack_bf16x2(v[u][2].x, v[u][2].y), pack_bf16x2(v[u][3].x, v[u][3].y));
        if (whole || (live && i0 + u * kLanes < nv)) op[i0 + u * kLanes] = r[u];
        unpack8(r[u], v[u]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) ss2 = __ffma2_rn(v[u][k], v[u][k], ss2);
      unpack8(w[u], g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[u][k] = __fmul2_rn(v[u][k], g[k]);
      am = max_nan(am, absmax8(v[u]));
    }
    am = block_max<kLanes>(am);
    const bool some = am != 0.f;
    least = some ? fminf(least, am) : least;
    odd = odd || (some && !(am >= 0x1p-100f && am < 0x1p127f));
    const float f = some ? 448.0f * rcp(am) : 0.f;
#pragma unroll
    for (int u = 0; u < A; ++u)
      if (whole || (live && i0 + u * kLanes < nv)) cp[i0 + u * kLanes] = codes8(v[u], f);
    if (lane % kLanes == 0) am_w[2 * A * j + lane / kLanes] = am;
  }
  // the row's sum: lanes, then its warps (the same order whatever the timing)
  auto row_sum = [&](float s, float* buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (wpr == 1) return s;
    if (lane == 0) buf[warp] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + mr), "r"(tpr) : "memory");
    s = lane < wpr ? buf[w0 + lane] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return __shfl_sync(0xffffffffu, s, 0);
  };
  // r once more, for the paths that are hardly ever taken (with a residual as
  // this thread has just stored it)
  auto again = [&](int i, float2 (&v)[4]) {
    unpack8(live && i < nv ? (RES ? op[i] : xp[i]) : make_uint4(0u, 0u, 0u, 0u), v);
  };
  float ss = row_sum(ss2.x + ss2.y, part[0]), up = 1.f;
  // squares of bf16 values can pass fp32's range at both ends: such a row is
  // summed again, scaled by a power of two. Downwards by 2^80: 32768 squares of
  // the largest value, 2^128, then add up to 2^111, and the columns that count
  // in such a row, 2^52 and above, still have squares of 2^-56. Upwards by 2^80:
  // the smallest value, 2^-133, squares to 2^-106, a sum below 2^-80 stays below
  // 2^80, eps below 2^-60 below 2^100.
  if (ss > 0x1p120f || (ss < 0x1p-80f && a.eps < 0x1p-60f)) {
    up = ss > 0x1p120f ? 0x1p-80f : 0x1p80f;
    float s2 = 0.f;
    for (int j = 0; j < steps; ++j)
      for (int u = 0; u < A; ++u) {
        float2 v[4];
        again(at(j) + u * kLanes, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s2 = fmaf(up * v[k].x, up * v[k].x, s2);
          s2 = fmaf(up * v[k].y, up * v[k].y, s2);
        }
      }
    ss = row_sum(s2, part[1]);
  }
  const float root = rsqrtf(fmaf(ss, inv_k, up * a.eps * up)), inv = up * root;
  __syncwarp();
  for (int l = lane; l < 2 * A * steps; l += 32) {
    const int g = (l / (2 * A) * wpr + warp - w0) * 2 * A + l % (2 * A);
    const float top = am_w[l] * inv;   // max|v|
    if (live && g * 16 < nv) a.scales[(size_t)g * a.M + m] = scale_of(top);
    // Past fp32; or zeros that may be products r w below 2^-150, which count
    // where 1 / rms brings them past the smallest code of the smallest scale,
    // 2^-136 (with an eps of 2^-27 or more never; at 1e-12 a batch of nothing but
    // zeros takes 25.7 us at 4608 x 4096, 11.3 at 1e-6)
    odd = odd || top > 0x1.fffffep127f || (live && g * 16 < nv && am_w[l] == 0.f && inv > 0x1.8p13f);
  }
  if (__any_sync(0xffffffffu, odd || least * inv * (1.0f / 448.0f) < kFp8MinScale || inv > 0x1p100f)) {
    // the smallest scale, NaN, infinities, values, products r w or a factor
    // 1 / rms out of fp32's range: the warp's blocks by the definition, v first
    // (in 64 bits: of r, 1 / rms and w any two may leave fp32)
    const double inv64 = (double)up * (double)root;
    __syncwarp();   // the scales above, from other lanes, come before these
    for (int j = 0; j < steps; ++j) {
      const int i0 = at(j);
      float2 v[A][4];
      float am = 0.f;
#pragma unroll
      for (int u = 0; u < A; ++u) {
        float2 g[4];
        const int i = i0 + u * kLanes;
        again(i, v[u]);
        unpack8(i < nv ? __ldg(wp + i) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[u][k] = make_float2((float)(v[u][k].x * inv64 * g[k].x), (float)(v[u][k].y * inv64 * g[k].y));
        am = max_nan(am, absmax8(v[u]));
      }
      const float scale = scale_of(block_max<kLanes>(am));
#pragma unroll
      for (int u = 0; u < A; ++u) {
        const int i = i0 + u * kLanes;
        if (live && i < nv) {
          cp[i] = codes8(v[u], rcp(scale));
          if (i % 16 == 0) a.scales[(size_t)(i / 16) * a.M + m] = scale;
        }
      }
    }
  }
}

// -------------------------------------------------------------- no norm
// kPieces: pieces of 256 columns a warp loads at once. Two leave 30 registers, so
// the SM is full of warps (4608 x 12288 28.2 us; one 35.1, four 33.3); with few
// pieces one each (512 x 4096 2.1 us against 2.3, 800 x 4096 3.0 against 3.2, but
// 1200 x 4096 4.3 against 3.9). The wait for the previous kernel stands behind
// the index arithmetic (512 x 4096, two pieces: 2.4 us, 2.6 ahead of it).
template <int kPieces>
__global__ void __launch_bounds__(256) fp8_quant_kernel(const Fp8ActArgs a, int per_row, long long pieces) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) launch_dependents();
  const long long p0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPieces;
  // one division a thread (in 32 bits where the count allows), then steps
  long long r0 = pieces >> 31 ? p0 / per_row : (long long)((uint32_t)p0 / (uint32_t)per_row);
  int c0 = (int)(p0 - r0 * per_row);
  uint4 x[kPieces];
  long long row[kPieces];
  int col[kPieces];
  grid_dependency_wait();
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    row[u] = r0;
    col[u] = c0 * 256 + 8 * lane;
    const bool in = p0 + u < pieces && col[u] < a.K;
    if (!in) col[u] = -1;
    if (++c0 == per_row) {
      c0 = 0;
      ++r0;
    }
    x[u] = in ? *reinterpret_cast<const uint4*>(a.x + (size_t)row[u] * (size_t)a.ldx + col[u])
              : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    float2 v[4];
    unpack8(x[u], v);
    const float scale = scale_of(block_max<16>(absmax8(v)));
    const uint2 c = codes8(v, rcp(scale));
    if (col[u] >= 0) {
      *reinterpret_cast<uint2*>(a.codes + (size_t)row[u] * a.K + col[u]) = c;
      if ((lane & 15) == 0) a.scales[(size_t)(col[u] / 128) * a.M + row[u]] = scale;
    }
  }
}

cudaError_t launch_pdl(const void* fn, unsigned grid, int block, int smem, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

Fp8ActPlan fp8_act_plan(int M, int K, bool norm, bool residual, int num_sms) {
  if (!norm) {
    const long long pieces = (long long)M * ((K + 255) / 256);
    return Fp8ActPlan{pieces <= 96ll * num_sms ? 1 : 2, 1, 1};
  }
  // Warps of a row: one where there are rows enough to fill the SMs (no
  // barrier, the least work beside the columns), more for fewer rows, but no
  // more than the row has columns for. With a residual a thread has at most four
  // vectors, unless more warps would leave lanes idle: memory takes few long
  // streams better than many (in turn on one card: 8192 x 8192 68.4 us, 71.4 with
  // eight, 76.6 with a row a warp; 4608 x 4096 20.9, 21.3, 23.2; 1200 x 8192 12.4
  // against 15.0; but 1024 x 8192 10.8 against 10.2). Without one it is the other
  // way round (4608 x 12288 29.7, 37.1 with eight).
  const int nv = K / 8;
  auto lanes = [nv](int w) { return (nv + 64 * w - 1) / (64 * w) * 64 * w; };   // steps come in twos
  int wpr = 1;
  while (wpr < 16 && wpr * 32 < nv &&
         ((long long)M * wpr < 24ll * num_sms || (residual && nv > 4 * 32 * wpr && lanes(2 * wpr) <= lanes(wpr))))
    wpr *= 2;
  // Vectors in flight: four, two where each brings the residual's along (in 64
  // registers four of those spill), fewer where the last step would be idle for
  // more than an eighth.
  auto padded = [&](int A) { return (nv + 32 * A * wpr - 1) / (32 * A * wpr) * (32 * A * wpr); };
  int A = residual ? 2 : 4;
  while (A > 1 && 8 * padded(A) > 9 * padded(1)) A /= 2;
  return Fp8ActPlan{A, wpr, padded(A) / (32 * A * wpr)};
}

cudaError_t launch_fp8_act(const Fp8ActArgs& a, int num_sms, cudaStream_t s) {
  const Fp8ActPlan pl = fp8_act_plan(a.M, a.K, a.weight != nullptr, a.residual != nullptr, num_sms);
  Fp8ActArgs args = a;
  if (!a.weight) {
    int per_row = (a.K + 255) / 256;
    long long pieces = (long long)a.M * per_row;
    void* ptrs[] = {&args, &per_row, &pieces};
    const int n = pl.loads;
    const void* fn = n == 1 ? reinterpret_cast<const void*>(fp8_quant_kernel<1>)
                            : reinterpret_cast<const void*>(fp8_quant_kernel<2>);
    return launch_pdl(fn, (unsigned)((pieces + 8 * n - 1) / (8 * n)), 256, 0, s, ptrs);
  }
  int wpr = pl.warps;
  const int A = pl.loads, warps = wpr < 8 ? 8 : wpr, rpc = warps / wpr;
  float inv_k = (float)(1.0 / a.K);
  void* ptrs[] = {&args, &wpr, &inv_k};
  const void* fn = a.residual ? (A == 1 ? reinterpret_cast<const void*>(fp8_norm_kernel<true, 1>)
                                        : reinterpret_cast<const void*>(fp8_norm_kernel<true, 2>))
                   : A == 1 ? reinterpret_cast<const void*>(fp8_norm_kernel<false, 1>)
                   : A == 2 ? reinterpret_cast<const void*>(fp8_norm_kernel<false, 2>)
                            : reinterpret_cast<const void*>(fp8_norm_kernel<false, 4>);
  return launch_pdl(fn, (unsigned)(((long long)a.M + rpc - 1) / rpc), 32 * warps, warps * 2 * A * pl.steps * 4, s,
                    ptrs);
}

}  // namespace svdq
