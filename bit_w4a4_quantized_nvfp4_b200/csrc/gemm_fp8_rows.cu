// The 8-bit GEMM (svdq_fp8_linear) for few rows: one token of a decoding
// step up to a few hundred. It reads every weight once, so it is bound by HBM
// (N K bytes) until the rows' products take longer than the weights' way in.
//
// The operands change places: 128 weight rows are the M of a tcgen05.mma, T
// tokens (16 .. 128) its N, so a handful of tokens fills the tensor cores as
// well as it can. One CTA has a 128-column x T-token tile of y and a part of K;
// the CTAs of a cluster share the tile and split K (S of them), so that few
// column tiles still keep all SMs reading. At the end every CTA sends its
// partial sums of token t to CTA t mod S of its cluster, which adds them in
// the order of the ranks (the result does not depend on timing), adds the bias
// and rounds once.
//
//   warp 0      TMA producer: per K block the 128 x 128 weight tile and the
//               T x 128 activation tile, 128B-swizzled
//   warp 1      tensor memory, MMA issuer: per block one product into one of
//               kBufs accumulators
//   others      drain, one warp per lane quadrant (two, with half the tokens
//               each, above 32): a thread is a weight row; its sums, each times
//               its token's scale (the block's weight scale multiplied in when
//               the scales are brought into shared memory, ahead of the loop)
#include "fp8.cuh"
#include "kernels.h"

namespace svdq {
namespace {

constexpr int kMaxSplit = 8;           // portable cluster size

// Tokens of a tile that each CTA of a split adds, a multiple of 4.
__host__ __device__ constexpr int join_tokens(int tile, int split) { return ((tile + split - 1) / split + 3) / 4 * 4; }

template <int T>
struct CfgR {
  static constexpr int kDrainWarps = T > 32 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kDrainWarps;
  static constexpr int kHT = T / (kDrainWarps / 4);   // tokens of a drain thread
  static constexpr int kWBytes = 128 * 128, kXBytes = T * 128;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kBufs = T > 64 ? 2 : 4;
  static constexpr uint32_t kTmemCols = T * kBufs < 32 ? 32 : T * kBufs;
  static constexpr int kCtas = T <= 32 ? 2 : 1;   // CTAs per SM
  static constexpr int kScaleFloats = T <= 32 ? 4096 : 8192;   // scales of a CTA's part of K: blocks x T
  // partial sums: split x the tokens a CTA adds x 128 rows, at the worst split
  static constexpr int red_tokens() {
    int most = 0;
    for (int s = 2; s <= kMaxSplit; s = T > 64 ? 2 * s : s + 1)   // at 128 tokens powers of two alone
      most = s * join_tokens(T, s) > most ? s * join_tokens(T, s) : most;
    return most;
  }
  static constexpr int kRedBytes = red_tokens() * 128 * 4;
  static constexpr int kFixed = kScaleFloats * 4 + kRedBytes + 512 + 1024;
  static constexpr int kFit = ((T <= 32 ? 113 : 226) * 1024 - kFixed) / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
};

struct ParamsR {
  const float* x_scales;
  const float* w_scales;
  const uint16_t* bias;
  void* y;
  int M, N, G, split;
  int out_f32;
  unsigned* err;
  unsigned long long wait_ns;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// 16 bytes into the shared memory of a CTA of the cluster, counted on that
// CTA's mbarrier when they have landed
__device__ __forceinline__ void st_async_f32x4(uint32_t addr, uint32_t bar, float a, float b, float c, float d) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2,%3,%4,%5}, [%1];" ::"r"(addr),
               "r"(bar), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}

template <int T>
__global__ void __launch_bounds__(CfgR<T>::kThreads, CfgR<T>::kCtas)
gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const ParamsR p) {
  using C = CfgR<T>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_align<1024>(smem_raw);
  float* scl = reinterpret_cast<float*>(stages + S * C::kStageBytes);   // [blocks][T]
  float* red = scl + C::kScaleFloats;                                     // [split][tokens / 4][128][4]
  uint64_t* full = reinterpret_cast<uint64_t*>(red + C::kRedBytes / 4);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_free = acc_full + C::kBufs;
  uint64_t* mma_done = acc_free + C::kBufs;
  uint64_t* joined = mma_done + 1;
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(joined + 1);
  volatile uint32_t* left = tmem_ptr + 1;   // whether the producer or the MMA warp has given up

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % p.split, tn = (int)blockIdx.x / p.split;
  const int n0 = tn * 128, m0 = (int)blockIdx.y * T;
  const int kb0 = (int)((long long)p.G * rank / p.split), kb1 = (int)((long long)p.G * (rank + 1) / p.split);
  const int nkb = kb1 - kb0;
  const int tv = min(T, p.M - m0);            // tokens of the tile
  // With a split, CTA j of the cluster adds tokens j * per .. of the tile; all
  // its CTAs send it their sums of them, in groups of four tokens
  const int per = join_tokens(T, p.split);
  const int groups = min(per / 4, (max(tv - rank * per, 0) + 3) / 4);   // this CTA's

  if (threadIdx.x == 0) {
    *left = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_free[b], C::kDrainWarps);
    }
    mbar_init(mma_done, 1);
    mbar_init(joined, 1);
    fence_mbar_init();
    if (p.split > 1 && groups > 0) mbar_expect_tx(joined, (uint32_t)(p.split * groups) * 128 * 16);
    // weights are hardly ever the previous kernel's output: their way to L2
    // may begin before it ends (a prefetch only moves data closer). At up to 32
    // tokens three blocks more than the stages hold (1 x 12288 x 4096 9.1 us,
    // 9.7 with the stages' own), at more the stages' own (64 x 4096 x 4096 7.4,
    // 7.6 with two more); prefetches that go on in the loop were slower.
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    for (int k = 0; k < nkb && k < S + (T <= 32 ? 3 : 0); ++k) tma_prefetch_l2_2d(&tm_w, (kb0 + k) * 128, n0);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(tmem_ptr, C::kTmemCols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  // (its wait, ahead of the first write to another CTA's shared memory, tells
  // that every CTA of the cluster has started)
  cluster_arrive();
  // every input may be the previous kernel's output, y may still be read by it
  if (threadIdx.x == 0) launch_dependents();
  grid_dependency_wait();

  int issued = 0;   // blocks (thread 0)
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      for (; issued < nkb; ++issued) {
        const int k = issued, s = k % S;
        if (k >= S && !mbar_wait(&empty[s], ((k / S) - 1) & 1, p.wait_ns, p.err)) {
          *left = 1;
          break;
        }
        uint8_t* st = stages + s * C::kStageBytes;
        mbar_expect_tx(&full[s], C::kStageBytes);
        tma_load_2d(st, &tm_w, &full[s], (kb0 + k) * 128, n0);
        tma_load_2d(st + C::kWBytes, &tm_x, &full[s], (kb0 + k) * 128, m0);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // descriptors of stage 0; a stage further is kStageBytes further, a K
    // step of 32 bytes 2 (addresses are in units of 16 bytes)
    const uint64_t a0 = make_sdesc(smem_u32(stages), 16, 1024, kLayoutSw128);
    const uint64_t b0 = make_sdesc(smem_u32(stages) + C::kWBytes, 16, 1024, kLayoutSw128);
    uint32_t s = 0, sph = 0, b = 0, bph = 1;
    for (int k = 0; k < nkb; ++k) {
      // both barriers tested at once: the tests' latencies are a good part of
      // a block's time here
      const bool rf = mbar_try_wait(&acc_free[b], bph);
      const bool rs = mbar_try_wait(&full[s], sph);
      if (!__all_sync(0xffffffffu, rs && rf) && !(warp_wait(&full[s], sph, p.wait_ns, p.err) &&
                                                  warp_wait(&acc_free[b], bph, p.wait_ns, p.err))) {
        if (lane == 0) *left = 1;
        break;
      }
      tc_fence_after();
      const uint64_t da = a0 + (uint64_t)(s * (C::kStageBytes >> 4)), db = b0 + (uint64_t)(s * (C::kStageBytes >> 4));
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f8(tmem + T * b, da + 2 * j, db + 2 * j, f8_idesc(128, T), j > 0 ? 1u : 0u);
        tc_commit(&acc_full[b]);
        tc_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == (uint32_t)S) {
        s = 0;
        sph ^= 1;
      }
      if (++b == (uint32_t)C::kBufs) {
        b = 0;
        bph ^= 1;
      }
    }
    // every MMA issued has completed before tensor memory is freed
    if (elect_one()) tc_commit(mma_done);
    __syncwarp();
    (void)warp_wait(mma_done, 0, kLandNs, p.err);
  }

  constexpr int HT = C::kHT;
  const int t0 = (warp - 2) / 4 * HT;         // this drain warp's tokens
  float2 acc[HT / 2];
  if (warp >= 2) {
    // ------------------------------------------------------------ drain
    constexpr int kD = 32 * C::kDrainWarps;
    const int dt = threadIdx.x - 64;
    const float* swp = p.w_scales + (size_t)tn * p.G + kb0;
    const float* sxp = p.x_scales + (size_t)kb0 * p.M + m0;
    // eight loads of each kind in flight
    for (int i0 = dt; i0 < nkb * T; i0 += 8 * kD) {
      float a[8], b[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kD, k = i / T, t = i % T;
        const bool in = k < nkb && t < tv;
        a[u] = in ? __ldg(sxp + (size_t)k * p.M + t) : 0.f;
        b[u] = in ? __ldg(swp + k) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * kD < nkb * T) scl[i0 + u * kD] = a[u] * b[u];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kD) : "memory");
#pragma unroll
    for (int i = 0; i < HT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    const uint32_t tq = tmem + t0 + ((uint32_t)(32 * (warp & 3)) << 16);
    for (int k = 0; k < nkb; ++k) {
      const int b = k % C::kBufs;
      if (!warp_wait(&acc_full[b], (k / C::kBufs) & 1, p.wait_ns, p.err)) break;
      tc_fence_after();
      const float4* sv = reinterpret_cast<const float4*>(scl + k * T + t0);
      uint32_t v[2][16];
      tmem_ld16(tq + T * b, v[0]);
#pragma unroll
      for (int c = 0; c < HT / 16; ++c) {
        tmem_ld_wait();
        tmem_regs_ready(v[c & 1]);
        if (c + 1 < HT / 16) {
          tmem_ld16(tq + T * b + 16 * (c + 1), v[(c + 1) & 1]);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_free[b]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 s = sv[4 * c + i];
          const uint32_t* w = v[c & 1] + 4 * i;
          acc[8 * c + 2 * i] = __ffma2_rn(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])),
                                          make_float2(s.x, s.y), acc[8 * c + 2 * i]);
          acc[8 * c + 2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])),
                                              make_float2(s.z, s.w), acc[8 * c + 2 * i + 1]);
        }
      }
    }
  }

  // ---------------------------------------------------------------- output
  const int r = 32 * (warp & 3) + lane, n = n0 + r;   // drain threads: weight row of the tile, column of y
  const float bias = warp >= 2 && n < p.N && p.bias ? bf16_bits_to_f32(p.bias[n]) : 0.f;
  auto put = [&](int t, float v) {
    const size_t at = (size_t)(m0 + t) * p.N + n;
    if (p.out_f32)
      static_cast<float*>(p.y)[at] = v + bias;
    else
      static_cast<uint16_t*>(p.y)[at] = (uint16_t)f32_to_bf16_bits(v + bias);
  };
  if (p.split == 1) {
    if (warp >= 2 && n < p.N) {
#pragma unroll
      for (int t = 0; t < HT; ++t)
        if (t0 + t < tv) put(t0 + t, t & 1 ? acc[t / 2].y : acc[t / 2].x);
    }
  }
  __syncwarp();
  cluster_wait();
  if (p.split > 1 && warp >= 2) {
    // Sent with a count of bytes rather than between two cluster barriers: a
    // CTA that adds nothing is done here, the others wait for their bytes alone
    // (1 x 1024 x 1024 2.7 us, 3.0 with the barriers; 64 x 4096 x 4096 7.4 both)
#pragma unroll
    for (int t = 0; t < HT; t += 4)
      if (t0 + t < tv) {
        const uint32_t to = (uint32_t)((t0 + t) / per);
        const int at = (t0 + t) % per / 4;
        st_async_f32x4(mapa_shared(smem_u32(red + ((rank * (per / 4) + at) * 128 + r) * 4), to),
                       mapa_shared(smem_u32(joined), to), acc[t / 2].x, acc[t / 2].y, acc[t / 2 + 1].x,
                       acc[t / 2 + 1].y);
      }
    // (a CTA whose wait runs out stays until the others' late stores have come)
    const bool whole = groups == 0 || mbar_wait_cluster(joined, 0, p.wait_ns, p.err);
    if (!whole && !mbar_wait_cluster(joined, 0, p.wait_ns, nullptr)) (void)mbar_wait_cluster(joined, 0, kLandNs, nullptr);
    if (groups > 0 && __all_sync(0xffffffffu, whole) && n < p.N) {
      for (int u = (warp - 2) / 4; u < groups; u += C::kDrainWarps / 4) {
        const int t = rank * per + 4 * u;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < p.split; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(red + ((i * (per / 4) + u) * 128 + r) * 4);
          v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        put(t, v.x);
        if (t + 1 < tv) put(t + 1, v.y);
        if (t + 2 < tv) put(t + 2, v.z);
        if (t + 3 < tv) put(t + 3, v.w);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // Where the producer's wait ran out, or the MMA warp's, which then leaves
  // blocks that it never waited for, the copies issued land before the CTA exits
  if (threadIdx.x == 0 && *left)
    for (int j = max(0, issued - S); j < issued; ++j) (void)mbar_wait(&full[j % S], (j / S) & 1, kLandNs, nullptr);
}

template <int T>
cudaError_t launch_rows_t(const Fp8GemmArgs& a, int split, cudaStream_t s) {
  using C = CfgR<T>;
  static_assert(C::kStages >= 3 && (2 * C::kStages + 2 * C::kBufs + 3) * 8 <= 512, "shared-memory plan");
  // (228 KB on an SM, 1 KB of it taken by each CTA)
  static_assert(C::kSmem + kProbeMmaSmem > 226 * 1024, "no SM shared with the tensor-core probe");
  CUtensorMap tm_w, tm_x;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_tmap_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w_codes, a.K, a.N, a.K, 128, 128, sw) ||
      !make_tmap_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x_codes, a.K, a.M, a.K, 128, T, sw))
    return cudaErrorInvalidValue;
  ParamsR p;
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.bias = a.bias;
  p.y = a.y;
  p.M = a.M; p.N = a.N;
  p.G = (a.K + 127) / 128;
  p.split = split;
  p.out_f32 = a.out_f32;
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  auto kern = gemm_fp8_rows_kernel<T>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + 127) / 128 * split), (unsigned)((a.M + T - 1) / T));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, tm_w, tm_x, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

// Of 148 SMs, those on which clusters of a size find room at one CTA an SM (a
// cluster stays within a processing cluster of 16 to 20 SMs). A device with
// another number of SMs would have other figures: these are scaled, unmeasured.
constexpr int kRoom[kMaxSplit + 1] = {0, 148, 148, 135, 132, 130, 132, 105, 120};

// Up to 32 tokens the tile is as wide as they are and two CTAs fit on an SM; K is
// split as far as fills seven quarters of the SMs (5120 columns of K 4096, 40
// tiles: split by 6 5.8 us, 3 6.2, 2 7.6, but 7, 280 CTAs, 7.9; 9216 columns: 3
// 8.3, 2 8.9, 4, 288 CTAs, 10.9), while a CTA keeps four blocks (2048 x 4096, 16
// blocks: 5 3.8 us, 8 4.4) or there is an SM for each (1024 x 1024: 8 2.6, 2 3.0).
// Above, the plan is the one with the least estimated time, in microseconds:
//   this kernel     waves (a + c blocks) + 1.2 with a split
//   the pair kernel 5.2 + waves (1.7 + 0.41 blocks)
// where a wave is one CTA (pair) per SM and blocks the K blocks of a CTA.
// Measured at N = 4096 with 8, 32 and 64 blocks: T = 64 5.9, 12.3, 20.7 us
// (a = 3.8, c = 0.265), T = 128 8.0, 15.6, 26.4 (5.4, 0.33), the pair kernel
// 10.1, 20.3, 33.4; three waves of it at 8 and 32 blocks 19.3, 47.2. So M = 512,
// N = K = 4096 comes here (in turn on one card 16.6 us against 20.3), M = 512 with
// N = 12288 does not (33.6 on the pair kernel, three waves here). Splits of any
// number help here too (64 x 4096 x 5120: by 3 8.1 us, by 2 9.9; 77 x 2064 x 1000:
// by 6 4.9, by 4 5.2).
bool fp8_rows_plan(const Fp8GemmArgs& a, int* tokens, int* split) {
  const int G = (a.K + 127) / 128;
  const long long tn = (a.N + 127) / 128;
  auto up = [](long long x, long long y) { return (x + y - 1) / y; };
  if (a.M <= 32) {
    const int T = a.M <= 16 ? 16 : 32;
    int S = 1;
    for (int t = 2; t <= kMaxSplit && t <= G; ++t)
      if (4 * t * tn <= 7ll * a.num_sms && (up(G, t) >= 4 || t * tn <= a.num_sms)) S = t;
    if (up(G, S) * T > CfgR<16>::kScaleFloats) return false;
    *tokens = T;
    *split = S;
    return true;
  }
  const double pair = 5.2 + (double)up(up(a.M, 256) * up(a.N, 256), a.num_sms / 2) * (1.7 + 0.41 * G);
  double best = pair;
  for (int T : {64, 128}) {
    const long long tiles = tn * up(a.M, T);
    for (int S = 1; S <= kMaxSplit && S <= G; S = T > 64 ? 2 * S : S + 1) {
      if (up(G, S) * T > CfgR<64>::kScaleFloats || up(a.M, T) > 65535) continue;
      const double blocks = (double)up(G, S), waves = (double)up(tiles * S, (long long)a.num_sms * kRoom[S] / 148);
      const double t = waves * (T == 64 ? 3.8 + 0.265 * blocks : 5.4 + 0.33 * blocks) + (S > 1 ? 1.2 : 0.0);
      if (t < best) {
        best = t;
        *tokens = T;
        *split = S;
      }
    }
  }
  return best < pair;
}

cudaError_t launch_fp8_rows(const Fp8GemmArgs& a, int tokens, int split, cudaStream_t s) {
  switch (tokens) {
    case 16: return launch_rows_t<16>(a, split, s);
    case 32: return launch_rows_t<32>(a, split, s);
    case 64: return launch_rows_t<64>(a, split, s);
    default: return launch_rows_t<128>(a, split, s);
  }
}

}  // namespace svdq
