// Rotary positions (svdq_rope_apply, svdq_rope_tables): pair i of a head at
// row m turns by t = pos[m, axis[i]] * freq[i], cos and sin times factor.
//
// t is formed in 64 bits, since a position of a long context times a
// frequency near 1 leaves fp32 too few bits behind the whole turns. The whole
// turns are taken off by Cody and Waite's reduction: t - n * 2pi with 2pi in
// two parts and fused multiply-adds, so that the remainder keeps its bits;
// cos and sin of the remainder are fp32.
//
// Bound by HBM: the heads are read and written once, 16 bytes a load. A CTA
// has a few rows (or, while rows are few, a piece of one), loads its first
// columns, then forms its rows' cos and sin once in shared memory for all
// heads, so the angles' arithmetic runs under the loads. Measured: 16384 rows of
// 64 heads of 128, half layout, whole heads, 78.9 us (6.8 TB/s, 1.05 of the
// measured copy rate); interleaved with half of each head rotated 79.4 us.
// Tables are bound by the functions' arithmetic: 65536 x 64 in 14.4 us.
#include "fp8.cuh"
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

__global__ void __launch_bounds__(256) rope_tables_kernel(const RopeArgs a, float* __restrict__ cos_t,
                                                          float* __restrict__ sin_t) {
  if (threadIdx.x == 0) launch_dependents();
  grid_dependency_wait();
  // row and pair advance by a fixed stride: no division in the loop
  const long long stride = (long long)gridDim.x * 256, first = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long dm = stride / a.pairs;
  const int dp = (int)(stride - dm * a.pairs);
  long long m = first / a.pairs;
  int p = (int)(first - m * a.pairs);
  while (m < a.M) {
    float c, s;
    rope_turn(rope_position(a, (size_t)m, p), a.freq[p], a.factor, c, s);
    cos_t[m * a.pairs + p] = c;
    sin_t[m * a.pairs + p] = s;
    m += dm;
    p += dp;
    if (p >= a.pairs) {
      p -= a.pairs;
      ++m;
    }
  }
}

constexpr int kThreadsO = 256;
// Units a thread has in flight: two (16384 x 8 x 128 half 12.7 us, one 13.6,
// four 16.0; 4096 x 128 heads interleaved 41.7, 43.7, 41.7), or one where a CTA
// has a single row or piece without two for each thread (4608 x 48 x 128 half
// 19.3 us against 20.3, 512 x 48 x 128 4.4 against 4.6).
constexpr int kUnits = 2;
// What of a row is brought to L2 ahead of its loads (16384 x 64 x 128 interleaved
// 79.4 us, 87.8 without, half 78.9 against 82.7; 4096 x 128 heads 41.7 us, 43.0
// with 16 KB; 64 KB makes 256 heads slower, 89 against 83).
constexpr int kAheadBytes = 32 * 1024;
constexpr int kMaxAngles = 4096;     // cos and sin of a CTA's rows (32 KB)

// How a row is cut into units: `uph` of each head (interleaved: 8 columns of 4
// pairs each, those past the last pair passed through; half: `rot`, V columns
// and their partners), then, half and not in place, `rest` of each head's other
// columns, rw columns each. (Not head by head: a warp that had both kinds took
// 96 us at 16384 x 64 x 128 with half of each head rotated, 81 so.)
struct RopePlan {
  int rows, chunks;        // rows of a CTA; pieces of a row (one of the two is 1)
  int upr, uph, rot, rest, rw;
  int first;               // a row's units ahead of the rest's
  unsigned long long uph_magic, upr_magic, rest_magic;   // ceil(2^40 / d): u / d for u < 2^20
};
__device__ __forceinline__ int div_magic(int u, unsigned long long magic) {
  return (int)(((unsigned long long)u * magic) >> 40);
}

template <int N>
__device__ __forceinline__ void load_cols(const uint16_t* p, uint32_t (&r)[4]) {
  if constexpr (N == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else if constexpr (N == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x; r[1] = v.y;
  } else if constexpr (N == 2) {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void store_cols(uint16_t* p, const uint32_t (&r)[4]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
  else if constexpr (N == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
  else if constexpr (N == 2)
    *reinterpret_cast<uint32_t*>(p) = r[0];
  else
    *p = (uint16_t)r[0];
}
__device__ __forceinline__ float col(const uint32_t* r, int k) {
  return __uint_as_float(k & 1 ? r[k >> 1] & 0xFFFF0000u : r[k >> 1] << 16);
}

// V: columns of a load. Interleaved V = 8 (pairs past the last are passed
// through); half V = 8, 4 or 1 as the number of pairs divides. U: units in flight.
template <bool HALF, int V, int U>
__global__ void __launch_bounds__(kThreadsO) rope_apply_kernel(const RopeArgs a, const RopePlan pl) {
  extern __shared__ __align__(16) float turn[];   // [rows][pairs] cos, then sin
  const int P = a.pairs;
  const long long m0 = (long long)(blockIdx.x / pl.chunks) * pl.rows;
  const int rows = (int)min((long long)pl.rows, (long long)a.M - m0);
  const int chunk = (int)(blockIdx.x % pl.chunks), per = (pl.upr + pl.chunks - 1) / pl.chunks;
  const int u0 = chunk * per, u1 = pl.chunks > 1 ? min(pl.upr, u0 + per) : rows * pl.upr;
  float* cs = turn;
  float* sn = turn + pl.rows * P;
  if (threadIdx.x == 0) launch_dependents();
  // rows of 1 KB or more (below, the prefetches cost more than they bring) are
  // on their way to L2 while the previous kernel ends
  if ((int)threadIdx.x < rows && pl.chunks == 1 && a.heads * a.head_dim >= 512)
    prefetch_l2(a.x + (size_t)(m0 + threadIdx.x) * (size_t)a.ldx, (uint32_t)min(kAheadBytes, 2 * a.heads * a.head_dim));
  // every input may be the previous kernel's output, y may still be read by it
  grid_dependency_wait();

  bool angles = false;
  for (int ub = u0; ub < u1; ub += kThreadsO * U) {
    uint32_t lo[U][4], hi[U][4];
    int row[U], col0[U], unit[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = ub + k * kThreadsO + (int)threadIdx.x;
      unit[k] = -1;
      if (u >= u1) continue;
      row[k] = pl.chunks > 1 ? 0 : div_magic(u, pl.upr_magic);
      const int ur = u - row[k] * pl.upr;
      int h;
      if (HALF && ur >= pl.first) {
        h = div_magic(ur - pl.first, pl.rest_magic);
        unit[k] = pl.rot + ur - pl.first - h * pl.rest;
      } else {
        h = div_magic(ur, pl.uph_magic);
        unit[k] = ur - h * pl.uph;
      }
      col0[k] = h * a.head_dim;
      const uint16_t* xp = a.x + (size_t)(m0 + row[k]) * (size_t)a.ldx + col0[k];
      if (!HALF) {
        load_cols<V>(xp + V * unit[k], lo[k]);
      } else if (unit[k] < pl.rot) {
        load_cols<V>(xp + V * unit[k], lo[k]);
        load_cols<V>(xp + V * unit[k] + P, hi[k]);
      } else if (pl.rw == 8) {   // (units past the rotated ones: not in place)
        load_cols<8>(xp + 2 * P + 8 * (unit[k] - pl.rot), lo[k]);
      } else {
        load_cols<2>(xp + 2 * P + 2 * (unit[k] - pl.rot), lo[k]);
      }
    }
    if (!angles) {
      for (int i = threadIdx.x; i < rows * P; i += kThreadsO) {
        const int r = i / P, p = i - r * P;
        rope_turn(rope_position(a, (size_t)(m0 + r), p), a.freq[p], a.factor, cs[i], sn[i]);
      }
      __syncthreads();
      angles = true;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (unit[k] < 0) continue;
      const float* c = cs + row[k] * P;
      const float* s = sn + row[k] * P;
      uint16_t* yp = a.y + (size_t)(m0 + row[k]) * (size_t)a.ldy + col0[k];
      if constexpr (!HALF) {
        const int p0 = V / 2 * unit[k];
        if (P % 4 == 0) {
          if (p0 < P) {
            const float4 ct = *reinterpret_cast<const float4*>(c + p0), st = *reinterpret_cast<const float4*>(s + p0);
            const float cv[4] = {ct.x, ct.y, ct.z, ct.w}, sv[4] = {st.x, st.y, st.z, st.w};
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float u = col(lo[k], 2 * i), v = col(lo[k], 2 * i + 1);
              lo[k][i] = pack_bf16x2(fmaf(u, cv[i], -v * sv[i]), fmaf(u, sv[i], v * cv[i]));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            if (p0 + i >= P) break;
            const float u = col(lo[k], 2 * i), v = col(lo[k], 2 * i + 1), ct = c[p0 + i], st = s[p0 + i];
            lo[k][i] = pack_bf16x2(fmaf(u, ct, -v * st), fmaf(u, st, v * ct));
          }
        }
        store_cols<V>(yp + V * unit[k], lo[k]);
      } else if (unit[k] < pl.rot) {
        const int p0 = V * unit[k];
        float o[V], w[V], cv[V], sv[V];
        if constexpr (V >= 4) {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const float4 ct = *reinterpret_cast<const float4*>(c + p0 + i);
            const float4 st = *reinterpret_cast<const float4*>(s + p0 + i);
            cv[i] = ct.x; cv[i + 1] = ct.y; cv[i + 2] = ct.z; cv[i + 3] = ct.w;
            sv[i] = st.x; sv[i + 1] = st.y; sv[i + 2] = st.z; sv[i + 3] = st.w;
          }
        } else {
          cv[0] = c[p0];
          sv[0] = s[p0];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u = col(lo[k], i), v = col(hi[k], i), ct = cv[i], st = sv[i];
          o[i] = fmaf(u, ct, -v * st);
          w[i] = fmaf(u, st, v * ct);
        }
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          lo[k][i / 2] = V == 1 ? f32_to_bf16_bits(o[i]) : pack_bf16x2(o[i], o[i + 1 < V ? i + 1 : i]);
          hi[k][i / 2] = V == 1 ? f32_to_bf16_bits(w[i]) : pack_bf16x2(w[i], w[i + 1 < V ? i + 1 : i]);
        }
        store_cols<V>(yp + p0, lo[k]);
        store_cols<V>(yp + p0 + P, hi[k]);
      } else if (pl.rw == 8) {
        store_cols<8>(yp + 2 * P + 8 * (unit[k] - pl.rot), lo[k]);
      } else {
        store_cols<2>(yp + 2 * P + 2 * (unit[k] - pl.rot), lo[k]);
      }
    }
  }
}

cudaError_t launch_rope(const void* fn, unsigned grid, int smem, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreadsO);
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

cudaError_t launch_rope_tables(const RopeArgs& a, float* cos_t, float* sin_t, int num_sms, cudaStream_t s) {
  const long long blocks = ((long long)a.M * a.pairs + 255) / 256, most = 8ll * num_sms;
  RopeArgs args = a;
  void* ptrs[] = {&args, &cos_t, &sin_t};
  return launch_rope(reinterpret_cast<const void*>(rope_tables_kernel), (unsigned)(blocks < most ? blocks : most), 0, s,
                     ptrs);
}

cudaError_t launch_rope_apply(const RopeArgs& a, int num_sms, cudaStream_t s) {
  const bool inplace = a.x == a.y;
  const int P = a.pairs;
  const int v = !a.half ? 8 : P % 8 == 0 ? 8 : P % 4 == 0 ? 4 : 1;
  RopePlan pl;
  pl.rw = (2 * P) % 8 == 0 ? 8 : 2;
  if (a.half) {
    pl.rot = P / v;
    pl.uph = pl.rot;
    pl.rest = inplace ? 0 : (a.head_dim - 2 * P) / pl.rw;
  } else {
    pl.rest = 0;
    pl.rot = (2 * P + 7) / 8;
    pl.uph = inplace ? pl.rot : a.head_dim / 8;
  }
  pl.first = pl.uph * a.heads;
  pl.upr = pl.first + pl.rest * a.heads;
  // rows of a CTA: as many as give each thread its units, within the angles'
  // room, and no more than leave every SM four CTAs; where that is one row and
  // there are fewer rows than that, a row is cut into pieces of one unit a
  // thread (each piece forms the row's angles again)
  const long long spread = (long long)a.M / (4 * num_sms);
  long long rows = kThreadsO * kUnits / pl.upr;
  if (rows > kMaxAngles / P) rows = kMaxAngles / P;
  if (rows > spread) rows = spread;
  pl.rows = rows < 1 ? 1 : (int)rows;
  pl.chunks = spread < 1 ? (pl.upr + kThreadsO - 1) / kThreadsO : 1;
  if ((long long)a.M * pl.chunks > 8ll * num_sms) pl.chunks = 1;
  pl.uph_magic = ((1ull << 40) + pl.uph - 1) / pl.uph;
  pl.rest_magic = pl.rest ? ((1ull << 40) + pl.rest - 1) / pl.rest : 0;
  pl.upr_magic = ((1ull << 40) + pl.upr - 1) / pl.upr;
  const long long grid = ((long long)a.M + pl.rows - 1) / pl.rows * pl.chunks;
  RopeArgs args = a;
  void* ptrs[] = {&args, &pl};
  const bool one = pl.chunks > 1 || (pl.rows == 1 && pl.upr < kThreadsO * kUnits);
  auto pick = [&](auto two_units, auto one_unit) { return reinterpret_cast<const void*>(one ? one_unit : two_units); };
  const void* fn = !a.half  ? pick(rope_apply_kernel<false, 8, kUnits>, rope_apply_kernel<false, 8, 1>)
                   : v == 8 ? pick(rope_apply_kernel<true, 8, kUnits>, rope_apply_kernel<true, 8, 1>)
                   : v == 4 ? pick(rope_apply_kernel<true, 4, kUnits>, rope_apply_kernel<true, 4, 1>)
                            : pick(rope_apply_kernel<true, 1, kUnits>, rope_apply_kernel<true, 1, 1>);
  return launch_rope(fn, (unsigned)grid, pl.rows * P * 8, s, ptrs);
}

}  // namespace svdq
