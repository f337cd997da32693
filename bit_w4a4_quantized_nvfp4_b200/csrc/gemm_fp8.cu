// The 8-bit GEMM (svdq_fp8_linear) for many rows:
//   y[m,n] = sum_g (sx[g,m] sw[n/128,g]) sum_{k in g} qx[m,k] qw[n,k] + bias[n]
//
// A block's product is one accumulator of the tensor cores; the scales are
// fp32 and differ from block to block of 128 along K, so a block's sums leave
// tensor memory before a later block may use their place, and are added,
// scaled, to sums in registers. That drain (one fused multiply-add for every
// 128 products) is the second bound beside the MMA rate: 32,768 sums per SM
// and K block of 512 MMA cycles.
//
// Persistent, warp-specialised CTA pairs (cluster of 2, cta_group::2), each
// with a 256 x 256 tile of y:
//   warp 0       TMA producer (both CTAs): per K block this CTA's 128 rows of A
//                and 2 x 64 rows of B, 128-byte rows, 128B-swizzled
//   warps 1, 3   MMA issuers (leader CTA), one for each 128-column half of the
//                tile: per K block a product of 256 x 128 x 128 into one of the
//                half's two accumulators
//   warp 2       tensor-memory allocation, then the output copies (bf16)
//   warps 4..11  drain (both CTAs), two warps per lane quadrant, one for each
//                column half: a thread is a row, its 128 sums stay in registers
//                over the whole K loop. A half is one 128-wide weight block, so
//                a K block has one combined scale per thread. At the end bias,
//                rounding, TMA store through staging.
// Why this shape:
//   - 256 x 256 per pair is what tensor memory holds twice (4 x 128 columns) and
//     keeps the operands at 64 bytes per SM and cycle; L2 was seen to deliver
//     some 50, so a smaller tile would wait for its operands.
//   - Hand-overs cost more than the columns do. A barrier test takes some 140
//     cycles beside the MMAs' shared-memory reads, an accumulator's way from
//     the issuer through the drain and back several hundred. So a drain warp
//     has one hand-over per K block (128 columns; units of 64 columns, two
//     hand-overs, took 496 us at 8192^3 where this took 463), the next block's
//     barrier is tested ahead, the issuers test both their barriers at once, and
//     each half has its own issuer and its own two accumulators, so that one
//     half's hand-over runs under the other's MMAs (one issuer with N = 256
//     products and two accumulators for both halves: 478 against 469).
//   - A tile's end is short: the drain stages its columns and goes on, warp 2
//     issues the copies (a warp waits 1000 cycles to issue its own), and the
//     next tile's scales are loaded ahead (4608 x 1024 x 9216 with bias 62 us, 58
//     so, in turn on one card). Output straight from the registers, 32 bytes a
//     store, was slower than the staging (522 us against 510 at 8192^3): a
//     thread's stores are rows apart.
// Measured: 8192^3 443 to 465 us by card (2.36 to 2.48 PFLOP/s; the measured bf16
// rate is 1.65 in bursts, so 0.71 to 0.75 of twice that), 4608 x 4096 x 12288 198
// to 207 us (2.24 to 2.34), 1024 x 4096 x 4096 21.4 us. The large ones run into the
// 1000 W limit: the SMs go down to 1.35 GHz, and back to back for a second 8192^3
// takes 523 us (2.10 PFLOP/s, 1.5 times the bf16 rate under the same limit). A
// copy of an earlier version (463 us) without the drain's arithmetic and loads
// took 425 us at the same power: what bounds it is energy, the operands' way to
// the SMs and the products themselves.
#include "fp8.cuh"
#include "kernels.h"

namespace svdq {
namespace {

constexpr int BM = 128, BN = 256, BK = 128;   // rows per CTA, columns per pair, bytes of K per stage
constexpr int kStages = 5;
constexpr int kABytes = BM * BK;
constexpr int kBBytes = (BN / 2) * BK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kDrainWarps = 8;
constexpr int kThreads = 128 + 32 * kDrainWarps;
constexpr int kSlots = 2, kSlotBytes = 32 * 128;   // output staging per drain warp (the bf16 columns)
constexpr uint32_t kTmemCols = 512;
constexpr int UN = 128;                        // columns of a unit: one accumulator
constexpr uint32_t kIdesc = f8_idesc(2 * BM, UN);
constexpr int kGroupM = 8;                     // row tiles that share their column tiles in time
// shares of the 384 x 168 registers of a launch: 256 x 216 + 128 x 72
constexpr int kDrainRegs = 216, kOtherRegs = 72;
static_assert(256 * kDrainRegs + 128 * kOtherRegs <= kThreads * 168, "register shares");

struct Smem {
  uint8_t stage[kStages][kStageBytes];
  uint8_t out[kDrainWarps][kSlots][kSlotBytes];
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[4], acc_free[4], mma_done;
  uint64_t out_ready[kDrainWarps], out_free;
  uint32_t tmem_base;
  uint32_t left;   // whether the producer or an issuer has given up (leader)
};

struct Params {
  const float* x_scales;
  const float* w_scales;
  const uint16_t* bias;
  int M, N, G;
  int tiles_m, tiles_n;    // 256-row and 256-column tiles
  int out_f32;
  unsigned* err;
  unsigned long long wait_ns;
};

// bias of 8 columns from n on (n % 8 == 0, n + 8 <= N)
__device__ __forceinline__ uint4 bias8(const Params& p, int n) {
  const uint32_t* b = reinterpret_cast<const uint32_t*>(p.bias + n);
  return make_uint4(__ldg(b), __ldg(b + 1), __ldg(b + 2), __ldg(b + 3));
}

// Tiles in groups of kGroupM tile rows, down the rows first: the tiles in
// work at one time span about as many rows as columns, so that both operands
// are read from L2 rather than HBM.
__device__ __forceinline__ void tile_at(int t, const Params& p, int& tm, int& tn) {
  const int per = kGroupM * p.tiles_n;
  const int g = t / per, r = t % per;
  const int rows = min(kGroupM, p.tiles_m - g * kGroupM);
  tm = g * kGroupM + r % rows;
  tn = r / rows;
}

// The leader's producer and issuers at the end of their loops.
__device__ __forceinline__ void issuers_done() { asm volatile("bar.sync 1, 96;" ::: "memory"); }

// kHold: the early test of the next block's barrier may hold the warp until the
// barrier turns (try_wait) or only looks (test_wait). Looking is faster while a
// pair has few K blocks to do (21.6 us against 24.7 at 1024 x 4096 x 4096, 53.9
// against 57.0 at 4608 x 1024 x 9216 with bias); in long runs holding is (454 us
// against 469 at 8192^3, 202 against 207 at 4608 x 4096 x 12288): the halves'
// drains then fall into step. At 2048 x 4096 x 12288, 192 blocks a pair, holding
// takes 98.2 us, looking 99.5.
constexpr int kHoldBlocks = 256;

template <bool kHold>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_fp8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ CUtensorMap tm_y, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_align<1024>(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int num_tiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    sm.left = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 2);   // both issuers
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_free[b], kDrainWarps);   // a half's four warps of both CTAs
    }
    mbar_init(&sm.mma_done, 2);
    for (int e = 0; e < kDrainWarps; ++e) mbar_init(&sm.out_ready[e], 1);
    mbar_init(&sm.out_free, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_y);
  }
  if (warp == 2) {
    __syncwarp();
    tmem_alloc_pair(&sm.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // every input may be the previous kernel's output, y may still be read by it
  if (threadIdx.x == 0) launch_dependents();
  grid_dependency_wait();

  if (warp < 4) {
    regs_dec<kOtherRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t it = 0;
      if (lane == 0) {
        bool ok = true;
        for (int tile = pair; tile < num_tiles && ok; tile += npairs) {
          int tm, tn;
          tile_at(tile, p, tm, tn);
          const int row0 = tm * 256 + (int)rank * BM;
          const int col0 = tn * BN + (int)rank * (UN / 2);   // this CTA's half of each unit's columns
          for (int kb = 0; kb < p.G; ++kb, ++it) {
            const int s = it % kStages;
            if (!mbar_wait(&sm.empty[s], ((it / kStages) & 1) ^ 1, p.wait_ns, p.err)) { ok = false; break; }
            uint8_t* st = sm.stage[s];
            const uint32_t fb = mapa_shared(smem_u32(&sm.full[s]), 0);
            if (leader) mbar_expect_tx(&sm.full[s], 2 * kStageBytes);
            tma_load_2d_pair(st, &tm_a, fb, kb * BK, row0);
            tma_load_2d_pair(st + kABytes, &tm_b, fb, kb * BK, col0);
            tma_load_2d_pair(st + kABytes + kBBytes / 2, &tm_b, fb, kb * BK, col0 + UN);
          }
        }
        if (!ok) {
          sm.left = 1;
          if (!leader) let_copies_land();   // (they count on the leader's barriers)
        }
      }
      __syncwarp();
      // Where the leader's producer or an issuer gave up (it then leaves blocks
      // that it never waited for), the copies issued land before the pair exits.
      // Both CTAs' count on the leader's barriers; a block that one of them did
      // not issue never turns its barrier, so copies past it have their time.
      if (leader) {
        issuers_done();
        if (lane == 0 && sm.left) {
          for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
            if (!mbar_wait(&sm.full[j % kStages], (j / kStages) & 1, kLandNs, nullptr)) break;
          let_copies_land();
        }
      }
    } else if ((warp == 1 || warp == 3) && leader) {
      // ---------------------------------------------------------- MMA issuers
      const int h = warp >> 1;
      // descriptors of stage 0; a stage further is kStageBytes further, a K
      // step of 32 bytes 2 (addresses are in units of 16 bytes)
      const uint64_t a0 = make_sdesc(smem_u32(sm.stage[0]), 16, 1024, kLayoutSw128);
      const uint64_t b0 = make_sdesc(smem_u32(sm.stage[0]) + kABytes + h * (kBBytes / 2), 16, 1024, kLayoutSw128);
      uint32_t s = 0, sph = 0;   // stage and its phase
      uint32_t aph = 3;          // phases of the half's two accumulators, a bit each
      bool ok = true;
      for (int tile = pair; tile < num_tiles && ok; tile += npairs) {
        for (int kb = 0; kb < p.G; ++kb) {
          const uint32_t j = kb & 1, b = 2 * j + h;
          // both barriers tested at once: a test takes some 140 cycles
          const bool rf = mbar_try_wait(&sm.acc_free[b], (aph >> j) & 1);
          const bool rs = mbar_try_wait(&sm.full[s], sph);
          if (!__all_sync(0xffffffffu, rs && rf) &&
              !(warp_wait(&sm.full[s], sph, p.wait_ns, p.err) &&
                warp_wait(&sm.acc_free[b], (aph >> j) & 1, p.wait_ns, p.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = a0 + (uint64_t)(s * (kStageBytes >> 4)), db = b0 + (uint64_t)(s * (kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8_pair(tmem + UN * b, da + 2 * k, db + 2 * k, kIdesc, k > 0 ? 1u : 0u);
            tc_commit_pair(&sm.acc_full[b], 0x3);
            tc_commit_pair(&sm.empty[s], 0x3);
          }
          __syncwarp();
          aph ^= 1u << j;
          if (++s == kStages) {
            s = 0;
            sph ^= 1;
          }
        }
      }
      if (!ok && lane == 0) sm.left = 1;
      // every MMA issued has completed before tensor memory is freed
      if (elect_one()) tc_commit_pair(&sm.mma_done, 0x1);
      __syncwarp();
      (void)warp_wait(&sm.mma_done, 0, kLandNs, p.err);
      issuers_done();
    } else if (warp == 2 && !p.out_f32) {
      // ---------------------------------------------------------- output copies
      uint32_t tl = 0;
      bool ok = true;
      for (int tile = pair; tile < num_tiles && ok; tile += npairs, ++tl) {
        int tm, tn;
        tile_at(tile, p, tm, tn);
        for (int e = 0; e < kDrainWarps; ++e) {
          if (!warp_wait(&sm.out_ready[e], tl & 1, p.wait_ns, p.err)) { ok = false; break; }
          const int m = tm * 256 + (int)rank * BM + 32 * (e & 3), n = tn * BN + UN * (e >> 2);
          if (lane == 0) {
            if (m < p.M && n < p.N) tma_store_2d(&tm_y, sm.out[e][0], n, m);
            if (m < p.M && n + 64 < p.N) tma_store_2d(&tm_y, sm.out[e][1], n + 64, m);
            bulk_commit();
          }
          __syncwarp();
        }
        if (lane == 0) {
          bulk_wait_read<0>();
          mbar_arrive(&sm.out_free);
        }
        __syncwarp();
      }
      if (lane == 0) bulk_wait<0>();
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ drain
    regs_inc<kDrainRegs>();
    const int q = warp & 3, e = warp - 4, h = e >> 2;
    const uint32_t tq = tmem + UN * h + ((uint32_t)(32 * q) << 16);   // accumulator 0 of the half; 1 is 2 UN on
    const uint32_t freeb = mapa_shared(smem_u32(&sm.acc_free[h]), 0);
    uint32_t ph[2] = {0, 0};                                          // the two accumulators' phases
    // A tile's row and columns for this warp, and its first two K blocks'
    // scales, loaded ahead of the previous tile's output. (Rows and columns past
    // the end are not stored: any scale will do.) Later blocks' scales are
    // loaded two blocks ahead of their use: beside the tiles' loads a read of L2
    // can take longer than one block.
    int row0 = 0, n0 = 0;
    const float *sxp = nullptr, *swp = nullptr;
    float sx[2], sw[2];
    auto open = [&](int tile) {
      int tm, tn;
      tile_at(tile, p, tm, tn);
      row0 = tm * 256 + (int)rank * BM + 32 * q;
      n0 = tn * BN + UN * h;
      sxp = p.x_scales + min(row0 + lane, p.M - 1);
      swp = p.w_scales + (size_t)min(n0 / 128, (p.N - 1) / 128) * p.G;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int kb = min(j, p.G - 1);
        sx[j] = __ldg(sxp + (size_t)kb * p.M);
        sw[j] = __ldg(swp + kb);
      }
    };
    bool ok = true;
    uint32_t tl = 0;   // tiles done
    open(pair);
    for (int tile = pair; tile < num_tiles && ok; tile += npairs, ++tl) {
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      // The sums of consecutive K blocks are read as one stream of 16-column
      // steps: the next step's load is in flight during this step's
      // multiply-adds, across blocks too. The next block's barrier is tested
      // ahead, since a test takes some 150 cycles beside the MMAs' shared-memory
      // reads. Two blocks a turn, so that accumulators and
      // barriers are fixed addresses: in the few instructions between two
      // blocks every one counts.
      if (!warp_wait(&sm.acc_full[h], ph[0], p.wait_ns, p.err)) break;
      tc_fence_after();
      uint32_t v[2][16];
      tmem_ld16(tq, v[0]);
#pragma unroll 1
      for (int kb0 = 0; kb0 < p.G && ok; kb0 += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int kb = kb0 + j;
          if (kb >= p.G) break;
          const float s = sx[j] * sw[j];
          const float2 s2 = make_float2(s, s);
          ph[j] ^= 1;
          uint32_t ready = 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_ld_wait();
            tmem_regs_ready(v[c & 1]);
            if (c < 7) {
              tmem_ld16(tq + 2 * UN * j + 16 * (c + 1), v[(c + 1) & 1]);
            } else {
              tc_fence_before();
              mbar_arrive_if(lane == 0, freeb + 16 * j);
              if (kb + 1 < p.G) {
                if (!__all_sync(0xffffffffu, ready) &&
                    !warp_wait(&sm.acc_full[2 * (j ^ 1) + h], ph[j ^ 1], p.wait_ns, p.err)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                tmem_ld16(tq + 2 * UN * (j ^ 1), v[0]);
              }
            }
            if (c == 1) {
              const int kn = min(kb + 2, p.G - 1);
              sx[j] = __ldg(sxp + (size_t)kn * p.M);
              sw[j] = __ldg(swp + kn);
            }
            if (c == 4)
              ready = kHold ? mbar_try_wait(&sm.acc_full[2 * (j ^ 1) + h], ph[j ^ 1])
                            : mbar_test_wait(&sm.acc_full[2 * (j ^ 1) + h], ph[j ^ 1]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[8 * c + i] = __ffma2_rn(
                  make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), s2, acc[8 * c + i]);
          }
          if (!ok) break;
        }
      }
      if (!ok) break;
      // ---- output: 128 columns in pieces of 128 bytes a row
      const int m = row0, nt = n0;
      if (tile + npairs < num_tiles) open(tile + npairs);
      if (p.out_f32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = nt + 32 * c;
          uint8_t* buf = sm.out[e][c % kSlots];
          if (lane == 0) bulk_wait_read<kSlots - 1>();
          __syncwarp();
          uint4 b8;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            float2 lo = acc[16 * c + 2 * u], hi = acc[16 * c + 2 * u + 1];
            // the bias of 8 columns serves two of the 16-byte pieces
            if (u % 2 == 0) b8 = p.bias && n + 4 * u < p.N ? bias8(p, n + 4 * u) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t b0 = u % 2 ? b8.z : b8.x, b1 = u % 2 ? b8.w : b8.y;
            lo.x += bf16_bits_to_f32(b0 & 0xFFFFu);
            lo.y += bf16_bits_to_f32(b0 >> 16);
            hi.x += bf16_bits_to_f32(b1 & 0xFFFFu);
            hi.y += bf16_bits_to_f32(b1 >> 16);
            *reinterpret_cast<float4*>(buf + lane * 128 + ((u ^ (lane & 7)) * 16)) = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m < p.M && n < p.N) tma_store_2d(&tm_y, buf, n, m);
            bulk_commit();
          }
        }
      } else {
        // both pieces, then one fence; warp 2 issues the copies (a warp that
        // issues its own waits 1000 cycles a tile for it)
        if (tl > 0 && !warp_wait(&sm.out_free, (tl - 1) & 1, p.wait_ns, p.err)) { ok = false; break; }
#pragma unroll
        for (int c = 0; c < kSlots; ++c) {
          const int n = nt + 64 * c;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint4 b8 = make_uint4(0u, 0u, 0u, 0u);
            if (p.bias && n + 8 * u < p.N) b8 = bias8(p, n + 8 * u);
            const uint32_t bw[4] = {b8.x, b8.y, b8.z, b8.w};
            uint32_t w4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 a = acc[32 * c + 4 * u + k];
              w4[k] = pack_bf16x2(a.x + bf16_bits_to_f32(bw[k] & 0xFFFFu), a.y + bf16_bits_to_f32(bw[k] >> 16));
            }
            *reinterpret_cast<uint4*>(sm.out[e][c] + lane * 128 + ((u ^ (lane & 7)) * 16)) =
                make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.out_ready[e]);
      }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  __syncwarp();  // the cluster barrier is .aligned: every warp reconverges first
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  __syncwarp();
  cluster_sync();
}

}  // namespace

bool fp8_pair_holds(const Fp8GemmArgs& a) {
  const long long tiles = (long long)((a.M + 255) / 256) * ((a.N + BN - 1) / BN), pairs = a.num_sms / 2;
  return (tiles + pairs - 1) / pairs * ((a.K + 127) / 128) >= kHoldBlocks;   // K blocks of a pair
}

cudaError_t launch_fp8_linear(const Fp8GemmArgs& a, cudaStream_t s) {
  int tokens, split;
  if (fp8_rows_plan(a, &tokens, &split)) return launch_fp8_rows(a, tokens, split, s);
  CUtensorMap tm_a, tm_b, tm_y;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = make_tmap_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x_codes, a.K, a.M, a.K, BK, BM, sw) &&
            make_tmap_2d(&tm_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w_codes, a.K, a.N, a.K, BK, UN / 2, sw);
  if (a.out_f32)
    ok = ok && make_tmap_2d(&tm_y, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.y, a.N, a.M, (uint64_t)a.N * 4, 32, 32, sw);
  else
    ok = ok && make_tmap_2d(&tm_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.y, a.N, a.M, (uint64_t)a.N * 2, 64, 32, sw);
  if (!ok) return cudaErrorInvalidValue;
  Params p;
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.bias = a.bias;
  p.M = a.M; p.N = a.N;
  p.G = (a.K + 127) / 128;
  p.tiles_m = (a.M + 255) / 256;
  p.tiles_n = (a.N + BN - 1) / BN;
  p.out_f32 = a.out_f32;
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  const size_t smem = sizeof(Smem) + 1024;
  const int tiles = p.tiles_m * p.tiles_n, pairs = a.num_sms / 2;
  auto kern = fp8_pair_holds(a) ? gemm_fp8_kernel<true> : gemm_fp8_kernel<false>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (tiles < pairs ? tiles : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, tm_y, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svdq
