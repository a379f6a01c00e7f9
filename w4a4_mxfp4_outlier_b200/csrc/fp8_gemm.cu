// Matrix product of e4m3 operands with one float32 scale per block of 128:
//
//   Y[t, n] = sum_kb  sa[kb, t] * sb[n / 128, kb] * sum_{p in kb} a[t, p] w[n, p]
//
// The inner sums (128 products) run on the tensor cores (tcgen05 kind::f8f6f4)
// into tensor memory; the scales are any float32 numbers, which the tensor
// cores' own block scales (powers of two) cannot hold, so the outer sum is
// done by the epilogue warps in float32 registers: for every K block they read
// the block's partial sums from tensor memory and add them, scaled.  Two
// accumulator buffers in tensor memory let the tensor cores work on the next K
// block meanwhile.
//
// Three kernels:
//  * fp8_gemm_pair_kernel: CTA pairs (cta_group::2), 256 tokens x 256 channels
//    per tile, persistent.
//  * fp8_gemm_few_kernel: for few tokens, where reading the weight is the
//    work, and for small products: the weight rows are the MMA's M (128 per CTA),
//    the tokens its N (16 .. 64), and the CTAs of a cluster split K and join
//    their sums through distributed shared memory, in the order of the ranks.
//  * fp8_gemm_mid_kernel: where tiles of 256 x 256 would leave most SMs idle:
//    128 tokens x 256 channels per CTA, K split and joined in the same way.
// Every wait is bounded, as in the other kernels of the library.
#include <atomic>
#include <cuda.h>

#include "fp8_device.cuh"
#include "fp8_internal.h"
#include "fp8_rules.h"

namespace w4a4 {

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
constexpr int F_THREADS = 224;                // weights, MMA, 4 epilogue, activations
constexpr int F_W_BYTES = 128 * 128;          // weight rows x bytes of one K block
constexpr int F_BUFS = 4;                     // accumulators in tensor memory
constexpr int F_PER_SM = 2;                   // CTAs that run on an SM

template <int N>
struct FewSmem {
  // about 90 KB in flight, two CTAs per SM (so that the next kernel's are
  // already there when this one's leave; 1 token, 5120 -> 13824: 16.8 us, with
  // one CTA of 195 KB per SM 19.3)
  static constexpr int kStageBytes = F_W_BYTES + N * 128;
  static constexpr int kStages = N <= 32 ? 5 : 4;
  // An accumulator buffer is reused F_BUFS K blocks later, after the epilogue
  // has read the scales of the first, so F_BUFS slots more than stages are enough.
  static constexpr int kSaSlots = kStages + F_BUFS;
  uint8_t stage[kStages][kStageBytes];
  alignas(16) float sa[kSaSlots][N];
  float sb[kSaSlots];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t sa_full[kSaSlots];
  uint64_t acc_full[F_BUFS];
  uint64_t acc_empty[F_BUFS];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
  static_assert(N * 512 <= kStages * kStageBytes, "the sums fit the ring");
};

template <int N>
__global__ void __launch_bounds__(F_THREADS, F_PER_SM)
    fp8_gemm_few_kernel(const __grid_constant__ CUtensorMap tm_w,
                        const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ Fp8GemmArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using Smem = FewSmem<N>;
  constexpr int NST = Smem::kStages;
  constexpr int TCOLS = F_BUFS * (N == 48 ? 64 : N);    // a power of two
  static_assert(F_PER_SM * TCOLS <= 512 && F_PER_SM * (sizeof(Smem) + 2048) <= 228 * 1024,
                "F_PER_SM CTAs fit an SM");
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile uint32_t* abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int C = static_cast<int>(gridDim.z);              // cluster = CTAs along z, one K range each
  const int rank = static_cast<int>(blockIdx.z);
  const int n0 = blockIdx.x * 128;
  const int t0 = blockIdx.y * N;
  const int nt = args.T - t0 < N ? args.T - t0 : N;       // tokens of the tile
  const int kb0 = static_cast<int>(static_cast<int64_t>(args.nkb) * rank / C);
  const int kb1 = static_cast<int>(static_cast<int64_t>(args.nkb) * (rank + 1) / C);
  const int nk = kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 2);                       // weights, activations
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < Smem::kSaSlots; ++s) mbar_init(&sm.sa_full[s], 1);
    for (int b = 0; b < F_BUFS; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 4);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0u;
    fence_barrier_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    // ============================ weights =================================
    uint32_t issued = 0;
    for (int i = 0; i < nk; ++i) {
      const int s = i % NST;
      if (i >= NST && !warp_wait_bounded(&sm.empty[s], ((i / NST) & 1) ^ 1u, abort_flag,
                                         DEVERR_TIMEOUT_PRODUCER))
        break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&sm.full[s], F_W_BYTES);
        tma_load_2d(sm.stage[s], &tm_w, &sm.full[s], (kb0 + i) * 128, n0);
      }
      __syncwarp();
      issued = i + 1;
    }
    if (issued != 0 && *abort_flag) spin_ns(200000);   // copies in flight land before teardown
    __syncwarp();
  } else if (warp == 6) {
    // ============================ activations =============================
    // (a warp of its own: one warp's copies for weights and activations take
    // some 500 cycles a K block to issue)
    const uint32_t sa_bytes = static_cast<uint32_t>((nt + 3) & ~3) * 4u;
    WarpRun sb(args.sb + static_cast<int64_t>(blockIdx.x) * args.nkb + kb0, nk);
    for (int i = 0; i < nk; ++i) {
      const int s = i % NST;
      const int q = i % Smem::kSaSlots;
      const float sbi = sb.get(i);
      if (i >= NST && !warp_wait_bounded(&sm.empty[s], ((i / NST) & 1) ^ 1u, abort_flag,
                                         DEVERR_TIMEOUT_PRODUCER))
        break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&sm.full[s], N * 128);
        if (!args.no_acts) tma_load_2d(sm.stage[s] + F_W_BYTES, &tm_x, &sm.full[s], (kb0 + i) * 128, t0);
        sm.sb[q] = sbi;
        mbar_arrive_expect_tx(&sm.sa_full[q], sa_bytes);
        bulk_load(sm.sa[q], args.sa + (kb0 + i) * args.ld_sa + t0, sa_bytes, &sm.sa_full[q]);
      }
      __syncwarp();
    }
    if (*abort_flag) spin_ns(200000);
    __syncwarp();
  } else if (warp == 1) {
    // ============================ MMA issuer ==============================
    const uint64_t dw0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]));
    const uint64_t dx0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]) + F_W_BYTES);
    for (int i = 0; i < nk; ++i) {
      const int s = i % NST;
      const uint32_t b = i % F_BUFS;
      if (!warp_wait_bounded(&sm.acc_empty[b], ((i / F_BUFS) & 1) ^ 1u, abort_flag, DEVERR_TIMEOUT_MMA))
        break;
      if (!warp_wait_bounded(&sm.full[s], (i / NST) & 1u, abort_flag, DEVERR_TIMEOUT_MMA)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t so = static_cast<uint64_t>(s * (Smem::kStageBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8(tmem + b * N, dw0 + so + 2 * kk, dx0 + so + 2 * kk, idesc_f8(128, N), kk != 0);
        tc_commit(&sm.empty[s]);
        tc_commit(&sm.acc_full[b]);
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(&sm.drain);
    __syncwarp();
    mbar_wait_bounded(&sm.drain, 0u, nullptr, DEVERR_TIMEOUT_MMA);
    __syncwarp();
  } else {
    // ============================ epilogue ================================
    const int sp = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * sp) << 16);
    float2 acc[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    for (int i = 0; i < nk; ++i) {
      const int q = i % Smem::kSaSlots;
      const uint32_t b = i % F_BUFS;
      if (!warp_wait_bounded(&sm.sa_full[q], (i / Smem::kSaSlots) & 1u, abort_flag,
                             DEVERR_TIMEOUT_EPILOGUE) ||
          !warp_wait_bounded(&sm.acc_full[b], (i / F_BUFS) & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE))
        break;
      const float sb = sm.sb[q];
      tc_fence_after();
      constexpr int CH = N % 32 != 0 ? 16 : 32;
#pragma unroll
      for (int c = 0; c < N / CH; ++c) {
        uint32_t r[CH];
        tmem_ld_now(taddr + b * N + c * CH, r);
#pragma unroll
        for (int j = 0; j < CH / 4; ++j) {
          const float4 s4 = *reinterpret_cast<const float4*>(&sm.sa[q][c * CH + 4 * j]);
          float2& a0 = acc[c * CH / 2 + 2 * j];
          float2& a1 = acc[c * CH / 2 + 2 * j + 1];
          a0 = __ffma2_rn(make_float2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])),
                          make_float2(s4.x * sb, s4.y * sb), a0);
          a1 = __ffma2_rn(make_float2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                          make_float2(s4.z * sb, s4.w * sb), a1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
    }
    // this CTA's sums, [token][channel], over the ring: the last accumulator is
    // complete, so every tile has arrived and been read
    if (*abort_flag == 0u) {
      float* red = reinterpret_cast<float*>(sm.stage[0]) + 32 * sp + lane;
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        red[(2 * j) * 128] = acc[j].x;
        red[(2 * j + 1) * 128] = acc[j].y;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TCOLS);
  }
  __syncwarp();
  cluster_sync_all();
  if (*abort_flag == 0u) {
    // CTA r of the cluster joins tokens r, r + C, ...: the ranks' sums in order
    const uint32_t red = smem_u32(sm.stage[0]);
    for (int i = threadIdx.x; i < ((nt - rank + C - 1) / C) * 64; i += F_THREADS) {
      const int t = rank + (i >> 6) * C, c = 2 * (i & 63);
      if (n0 + c >= args.d_out) continue;                  // d_out is even
      float2 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = r < C ? ld_cluster_f32x2(mapa_shared(red + 4u * (t * 128 + c), r)) : make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 1; r < 8; ++r) {
        v[0].x += v[r].x;
        v[0].y += v[r].y;
      }
      const int64_t at = (t0 + t) * args.ldy + n0 + c;
      if (args.y_f32) {
        *reinterpret_cast<float2*>(static_cast<float*>(args.Y) + at) = v[0];
      } else {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(args.Y) + at) =
            __floats2bfloat162_rn(v[0].x, v[0].y);
      }
    }
  }
  __syncwarp();
  cluster_sync_all();          // no CTA leaves while another reads its sums
}

template <int kRegs>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---------------------------------------------------------------------------
// K split over a cluster
// ---------------------------------------------------------------------------
constexpr int H_STAGES = 4;
constexpr int H_X_BYTES = 128 * 128;                  // 128 token rows
constexpr int H_STAGE_BYTES = 3 * H_X_BYTES;          // and 256 weight rows
constexpr int H_THREADS = 384;                        // producer, MMA, 2 idle, 8 epilogue warps
constexpr int H_EPI_WARPS = 8;
constexpr int H_GROUP_M = 16;
constexpr int H_SA_GROUP = 8;
constexpr int H_MAX_C = 5;                            // CTAs of a cluster

struct MidSmem {
  uint8_t stage[H_STAGES][H_STAGE_BYTES];
  // scales of the 128 tokens, for groups of 8 K blocks in turn
  alignas(16) float sa[2][H_SA_GROUP][128];
  uint64_t sa_full[2];
  uint64_t sa_empty[2];
  uint64_t full[H_STAGES];
  uint64_t empty[H_STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
  static_assert(128 * 256 * 4 <= H_STAGES * H_STAGE_BYTES, "the sums fit the ring");
};

__global__ void __launch_bounds__(H_THREADS, 1)
    fp8_gemm_mid_kernel(const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ CUtensorMap tm_w,
                        const __grid_constant__ Fp8GemmArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  MidSmem& sm = *reinterpret_cast<MidSmem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile uint32_t* abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int C = static_cast<int>(gridDim.z);              // cluster = CTAs along z, one K range each
  const int rank = static_cast<int>(blockIdx.z);
  int tm, tn;
  tile_coords<H_GROUP_M>(blockIdx.x, args.tiles_m, args.tiles_n, tm, tn);
  const int m0 = tm * 128, n0 = tn * 256;
  const int rows = args.T - m0 < 128 ? args.T - m0 : 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(args.nkb) * rank / C);
  const int nk = static_cast<int>(static_cast<int64_t>(args.nkb) * (rank + 1) / C) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < H_STAGES; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.sa_full[s], 1);
      mbar_init(&sm.sa_empty[s], H_EPI_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], H_EPI_WARPS);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0u;
    fence_barrier_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();
  pdl_launch_dependents();

  if (warp < 4) {
    // the launch's 384 x 168 registers: 128 x 56 here, 256 x 224 for the epilogue
    setmaxnreg_dec<56>();
    if (warp == 0) {
      // ============================ TMA producer ==========================
      uint32_t issued = 0, s = 0, ph = 0;
      const uint32_t sa_bytes = static_cast<uint32_t>((rows + 3) & ~3) * 4u;
      for (int i = 0; i < nk; ++i) {
        if (i % H_SA_GROUP == 0) {
          const uint32_t grp = i / H_SA_GROUP, q = grp & 1u;
          if (grp >= 2 && !warp_wait_bounded(&sm.sa_empty[q], ((grp >> 1) & 1u) ^ 1u, abort_flag,
                                             DEVERR_TIMEOUT_PRODUCER))
            break;
          if (elect_one()) {
            const int n = nk - i < H_SA_GROUP ? nk - i : H_SA_GROUP;
            mbar_arrive_expect_tx(&sm.sa_full[q], sa_bytes * n);
            for (int j = 0; j < n; ++j)
              bulk_load(sm.sa[q][j], args.sa + (kb0 + i + j) * args.ld_sa + m0, sa_bytes, &sm.sa_full[q]);
          }
          __syncwarp();
          issued = 1;
        }
        if (i >= H_STAGES && !warp_wait_bounded(&sm.empty[s], ph ^ 1u, abort_flag, DEVERR_TIMEOUT_PRODUCER))
          break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.full[s], H_STAGE_BYTES);
          if (!args.no_acts) tma_load_2d(sm.stage[s], &tm_x, &sm.full[s], (kb0 + i) * 128, m0);
          tma_load_2d(sm.stage[s] + H_X_BYTES, &tm_w, &sm.full[s], (kb0 + i) * 128, n0);
        }
        __syncwarp();
        if (++s == H_STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (issued != 0 && *abort_flag) spin_ns(200000);   // copies in flight land before teardown
      __syncwarp();
    } else if (warp == 1) {
      // ============================ MMA issuer ============================
      constexpr uint32_t ID = idesc_f8(128, 256);
      const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]));
      const uint64_t db0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]) + H_X_BYTES);
      uint32_t s = 0, ph = 0;
      uint64_t soff = 0;
      for (int i = 0; i < nk; ++i) {
        const uint32_t b = i & 1;
        if (!warp_wait_bounded(&sm.full[s], ph, abort_flag, DEVERR_TIMEOUT_MMA) ||
            !warp_wait_bounded(&sm.acc_empty[b], ((i >> 1) & 1u) ^ 1u, abort_flag, DEVERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + 256u * b;
          mma_f8(d, da0 + soff + 0, db0 + soff + 0, ID, 0u);
          mma_f8(d, da0 + soff + 2, db0 + soff + 2, ID, 1u);
          mma_f8(d, da0 + soff + 4, db0 + soff + 4, ID, 1u);
          mma_f8(d, da0 + soff + 6, db0 + soff + 6, ID, 1u);
          tc_commit(&sm.acc_full[b]);
          tc_commit(&sm.empty[s]);
        }
        __syncwarp();
        soff += H_STAGE_BYTES >> 4;
        if (++s == H_STAGES) {
          s = 0;
          ph ^= 1u;
          soff = 0;
        }
      }
      if (elect_one()) tc_commit(&sm.drain);
      __syncwarp();
      mbar_wait_bounded(&sm.drain, 0u, nullptr, DEVERR_TIMEOUT_MMA);
      __syncwarp();
    }
    __syncwarp();
    cluster_sync_all();
  } else {
    // ============================ epilogue ================================
    // Each warp owns 32 rows (its lanes) x 128 columns: 128 sums a lane.
    setmaxnreg_inc<224>();
    const int ew = warp - 4;
    const int sp = warp & 3;
    const int half = ew >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * sp) << 16) + 128 * half;
    const int nblk = tn * 2 + half;
    // (a block past d_out reads nothing; rows past T have any scale, and are not stored)
    WarpRun sbr(args.sb + static_cast<int64_t>(nblk) * args.nkb + kb0, nblk * 128 < args.d_out ? nk : 0);
    float2 acc[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
    // A wait that fails (it ends in bounded time, and all later ones then fail
    // at once) also raises abort_flag, which is looked at behind the loop.
    for (int i = 0; i < nk; ++i) {
      const uint32_t grp = i / H_SA_GROUP, q = grp & 1u, b = i & 1;
      const int qi = i % H_SA_GROUP;
      if (qi == 0)
        mbar_wait_bounded(&sm.sa_full[q], (grp >> 1) & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
      const float m = sm.sa[q][qi][32 * sp + lane] * sbr.get(i);
      mbar_wait_bounded(&sm.acc_full[b], (i >> 1) & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
      __syncwarp();
      tc_fence_after();
      if (qi == H_SA_GROUP - 1) mbar_arrive_lane0(&sm.sa_empty[q], lane);   // (all lanes have read theirs)
      const float2 m2 = make_float2(m, m);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[64];
        tmem_ld_now(taddr + 256u * b + 64 * c, r);
        if (c == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          acc[32 * c + j] = __ffma2_rn(
              make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), m2, acc[32 * c + j]);
      }
    }
    __syncwarp();
    // This CTA's sums over its own ring (its last accumulator is complete, so
    // every tile has arrived and been read): [8 columns][half of them][row][4].
    // Each rank then joins its share of the tile.  Pulling the others' sums costs
    // less than their pushing them did (128 tokens, 5120 -> 5120: 15.1 us, 16.4).
    const uint32_t ring = smem_u32(sm.stage[0]);
    const int row = 32 * sp + lane;
    if (*abort_flag == 0u && row < rows) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int u = 16 * half + v;
        const uint32_t at = ring + 4096u * u + 16u * row;
        st_shared_f32x4(at, acc[4 * v], acc[4 * v + 1]);
        st_shared_f32x4(at + 2048u, acc[4 * v + 2], acc[4 * v + 3]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    if (*abort_flag == 0u) {
      // pieces of 8 rows (8 lanes) x 8 columns, the ranks' sums in order
      const int pieces = 32 * ((rows + 7) >> 3);
      const int end = pieces * (rank + 1) / C;
      for (int i = pieces * rank / C + 4 * ew + (lane >> 3); i < end; i += 4 * H_EPI_WARPS) {
        const int r = 8 * (i >> 5) + (lane & 7), col = n0 + 8 * (i & 31);
        if (r >= rows || col >= args.d_out) continue;      // d_out is a multiple of 16
        const uint32_t at = ring + 4096u * (i & 31) + 16u * r;
        float4 v[H_MAX_C][2];
#pragma unroll
        for (int k = 0; k < H_MAX_C; ++k)
          if (k < C) {
            const uint32_t from = mapa_shared(at, k);
            v[k][0] = ld_cluster_f32x4(from);
            v[k][1] = ld_cluster_f32x4(from + 2048u);
          }
        float4 x = v[0][0], y = v[0][1];
#pragma unroll
        for (int k = 1; k < H_MAX_C; ++k)
          if (k < C) {
            const float4 a = v[k][0], b = v[k][1];
            x.x += a.x; x.y += a.y; x.z += a.z; x.w += a.w;
            y.x += b.x; y.y += b.y; y.z += b.z; y.w += b.w;
          }
        const int64_t out = static_cast<int64_t>(m0 + r) * args.ldy + col;
        if (args.y_f32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(args.Y) + out);
          o[0] = x;
          o[1] = y;
        } else {
          const __nv_bfloat162 p[4] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w),
                                       __floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.Y) + out) =
              *reinterpret_cast<const uint4*>(p);
        }
      }
    }
  }

  __syncwarp();
  cluster_sync_all();          // no CTA leaves while another reads its sums
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// CTA pairs
// ---------------------------------------------------------------------------
constexpr int Q_STAGES = 6;
constexpr int Q_HALF = 128 * 128;                     // own 128 rows of A, and of B
constexpr int Q_STAGE_BYTES = 2 * Q_HALF;
constexpr int Q_THREADS = 384;                        // producer, MMA, 2 idle, 8 epilogue warps
constexpr int Q_EPI_WARPS = 8;
constexpr int Q_GROUP_M = 16;
constexpr int Q_SA_GROUP = 8;

struct Fp8PairSmem {
  uint8_t stage[Q_STAGES][Q_STAGE_BYTES];
  alignas(1024) uint8_t epi[Q_EPI_WARPS][2][1024];
  // scales of the CTA's own 128 tokens, for groups of 8 K blocks in turn
  alignas(16) float sa[2][Q_SA_GROUP][128];
  uint64_t sa_full[2];
  uint64_t sa_empty[2];
  uint64_t full[Q_STAGES];      // leader's counts the bytes of both CTAs
  uint64_t empty[Q_STAGES];     // both CTAs: MMA commit, multicast
  uint64_t acc_full[2];         // both CTAs: MMA commit, multicast
  uint64_t acc_empty[2];        // leader: epilogue warps of both CTAs
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

template <bool kF32>
__global__ void __launch_bounds__(Q_THREADS, 1)
    fp8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ CUtensorMap tm_w,
                         const __grid_constant__ CUtensorMap tm_y,
                         const __grid_constant__ Fp8GemmArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Fp8PairSmem& sm = *reinterpret_cast<Fp8PairSmem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile uint32_t* abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();          // 0 = leader
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;
  const int ntiles = args.tiles_m * args.tiles_n;
  const int nkb = args.nkb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Q_STAGES; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.sa_full[s], 1);
      mbar_init(&sm.sa_empty[s], Q_EPI_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * Q_EPI_WARPS);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0u;
    fence_barrier_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_y);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sm.tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();
  pdl_launch_dependents();

  if (warp < 4) {
    // the launch's 384 x 168 registers: 128 x 56 here, 256 x 224 for the epilogue
    setmaxnreg_dec<56>();
    if (warp == 0) {
      // ============================ TMA producer (both CTAs) ==============
      uint32_t issued = 0, it = 0, s = 0, ph = 0, grp = 0;
      bool ok = true;
      for (int t = pair; t < ntiles && ok; t += npairs) {
        int tm, tn;
        tile_coords<Q_GROUP_M>(t, args.tiles_m, args.tiles_n, tm, tn);
        const int m_rows = tm * 256 + 128 * static_cast<int>(rank);
        const int n_rows = tn * 256 + 128 * static_cast<int>(rank);
        const int rows = args.T - m_rows < 128 ? args.T - m_rows : 128;
        const uint32_t sa_bytes = rows > 0 ? static_cast<uint32_t>((rows + 3) & ~3) * 4u : 0u;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          if (kb % Q_SA_GROUP == 0) {
            const uint32_t q = grp & 1u;
            if (grp >= 2 && !warp_wait_bounded(&sm.sa_empty[q], ((grp >> 1) & 1u) ^ 1u, abort_flag,
                                               DEVERR_TIMEOUT_PRODUCER)) {
              ok = false;
              break;
            }
            if (elect_one()) {
              const int n = nkb - kb < Q_SA_GROUP ? nkb - kb : Q_SA_GROUP;
              mbar_arrive_expect_tx(&sm.sa_full[q], sa_bytes * n);
              if (sa_bytes)
                for (int i = 0; i < n; ++i)
                  bulk_load(sm.sa[q][i], args.sa + (kb + i) * args.ld_sa + m_rows, sa_bytes,
                            &sm.sa_full[q]);
            }
            __syncwarp();
            ++grp;
          }
          if (it >= Q_STAGES &&
              !warp_wait_bounded(&sm.empty[s], ph ^ 1u, abort_flag, DEVERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            const uint32_t full_leader = mapa_shared(smem_u32(&sm.full[s]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * Q_STAGE_BYTES);
            if (!args.no_acts) tma_load_2d_pair(sm.stage[s], &tm_x, full_leader, kb * 128, m_rows);
            tma_load_2d_pair(sm.stage[s] + Q_HALF, &tm_w, full_leader, kb * 128, n_rows);
          }
          __syncwarp();
          issued = it + 1;
          if (++s == Q_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (lane == 0 && *abort_flag) {
        if (rank == 0) {
          const uint32_t first = issued > Q_STAGES ? issued - Q_STAGES : 0;
          for (uint32_t i = first; i < issued; ++i)
            mbar_wait_bounded(&sm.full[i % Q_STAGES], (i / Q_STAGES) & 1u, nullptr,
                              DEVERR_TIMEOUT_PRODUCER);
        }
        spin_ns(50000);   // scales, and the peer CTA's copies, which land on the leader's barriers
      }
      __syncwarp();
    } else if (rank == 0 && warp == 1) {
      // ============================ MMA issuer (leader) ===================
      constexpr uint64_t STAGE_DESC = Q_STAGE_BYTES >> 4;
      constexpr uint32_t ID = idesc_f8(256, 256);
      const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]));
      const uint64_t db0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]) + Q_HALF);
      uint32_t s = 0, ph = 0, g = 0;
      uint64_t soff = 0;
      bool ok = true;
      for (int t = pair; t < ntiles && ok; t += npairs) {
        for (int kb = 0; kb < nkb; ++kb, ++g) {
          const uint32_t b = g & 1u;
          if (!warp_wait_bounded(&sm.full[s], ph, abort_flag, DEVERR_TIMEOUT_MMA) ||
              !warp_wait_bounded(&sm.acc_empty[b], ((g >> 1) & 1u) ^ 1u, abort_flag,
                                 DEVERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + 256u * b;
            mma_f8_pair(d, da0 + soff + 0, db0 + soff + 0, ID, 0u);
            mma_f8_pair(d, da0 + soff + 2, db0 + soff + 2, ID, 1u);
            mma_f8_pair(d, da0 + soff + 4, db0 + soff + 4, ID, 1u);
            mma_f8_pair(d, da0 + soff + 6, db0 + soff + 6, ID, 1u);
            tc_commit_pair_multicast(&sm.acc_full[b], 0x3);
            tc_commit_pair_multicast(&sm.empty[s], 0x3);
          }
          __syncwarp();
          if (++s == Q_STAGES) {
            s = 0;
            ph ^= 1u;
            soff = 0;
          } else {
            soff += STAGE_DESC;
          }
        }
      }
      if (elect_one()) tc_commit_pair(&sm.drain);
      __syncwarp();
      mbar_wait_bounded(&sm.drain, 0u, nullptr, DEVERR_TIMEOUT_MMA);
      __syncwarp();
    }
  } else {
    // ============================ epilogue (both CTAs) ====================
    // Each warp owns 32 rows (its lanes) x 128 columns: 128 sums a lane.
    setmaxnreg_inc<224>();
    const int ew = warp - 4;
    const int sp = warp & 3;
    const int half = ew >> 2;
    const uint32_t acc_empty_leader = mapa_shared(smem_u32(&sm.acc_empty[0]), 0);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * sp) << 16) + 128 * half;
    const uint32_t stg = smem_u32(sm.epi[ew]);
    uint32_t g = 0, buf = 0, grp = 0;
    for (int t = pair; t < ntiles; t += npairs) {
      int tm, tn;
      tile_coords<Q_GROUP_M>(t, args.tiles_m, args.tiles_n, tm, tn);
      const int row0 = tm * 256 + 128 * static_cast<int>(rank) + 32 * sp;
      const int nblk = tn * 2 + half;
      // (a block past d_out reads nothing; rows past T have any scale, and are not stored)
      WarpRun sbr(args.sb + static_cast<int64_t>(nblk) * nkb, nblk * 128 < args.d_out ? nkb : 0);
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
      // What bounds the kernel: these warps.  A K block takes 744 cycles (T = 16384,
      // 13824 -> 5120; and a tile's end 3700 more, so 803 with the 40 K blocks of
      // T = 4096, 5120 -> 13824), its MMAs 512.  Delays of 100, 200, 400 cycles
      // before the arrival below cost 136, 218, 406 cycles a K block, all of
      // them; in the issuer, between its looks and its MMAs, 37, 92, 268.  With one
      // addition in eight a K block takes 590: the additions (330 at 100 FMAs per
      // cycle and SM) are half hidden, the rest is the chain of one warp (look,
      // scale, load, load, arrival), of which a scheduler has two to run.  The power
      // limit holds the SMs at 1.47 and 1.56 GHz meanwhile.  Measured and no
      // faster: 16 warps of 64 columns (268 us, this 260), MMAs of 128 columns with a
      // buffer pair per half (267), 32-column loads (262 to 276), scalar FMAs
      // (283), the next block's loads before the last additions (299), the
      // issuer's looks ahead of its MMAs (276).  A wait that fails (it ends in
      // bounded time, and all later ones then fail at once) only clears `ok`,
      // which is looked at once per tile.
      bool ok = true;
      float m = 0.f;
      // scale of K block kb, and its sums complete
      auto next_block = [&](int kb, uint32_t gk) {
        const uint32_t q = grp & 1u;
        const int qi = kb % Q_SA_GROUP;
        if (qi == 0)
          ok &= mbar_wait_bounded(&sm.sa_full[q], (grp >> 1) & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
        m = sm.sa[q][qi][32 * sp + lane] * sbr.get(kb);
        ok &= mbar_wait_bounded(&sm.acc_full[gk & 1u], (gk >> 1) & 1u, abort_flag,
                                DEVERR_TIMEOUT_EPILOGUE);
        __syncwarp();
        tc_fence_after();
        if (qi == Q_SA_GROUP - 1 || kb + 1 == nkb) {     // (all lanes have read their scale)
          mbar_arrive_lane0(&sm.sa_empty[q], lane);
          ++grp;
        }
      };
      for (int kb = 0; kb < nkb; ++kb, ++g) {
        const uint32_t b = g & 1u;
        const uint32_t ta = taddr + 256u * b;
        next_block(kb, g);
        const float2 m2 = make_float2(m, m);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[64];
          tmem_ld_now(ta + 64 * c, r);
          if (c == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(acc_empty_leader + 8u * b);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            acc[32 * c + j] = __ffma2_rn(
                make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), m2, acc[32 * c + j]);
        }
      }
      if (__any_sync(0xFFFFFFFFu, !ok)) break;
      // Y through staging blocks of 16 rows x 64 bytes (64-byte swizzle), as
      // the dual-branch GEMM stores it: 32 bf16 or 16 f32 columns a block,
      // two blocks in turn
      constexpr int CB = kF32 ? 16 : 32;                   // columns per block
#pragma unroll
      for (int c = 0; c < 128 / CB; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if constexpr (kF32) {
            const float2 v = acc[8 * c + (j >> 1)];
            p[j] = __float_as_uint((j & 1) ? v.y : v.x);
          } else {
            const float2 v = acc[16 * c + j];
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(v.x, v.y);
            p[j] = *reinterpret_cast<const uint32_t*>(&b2);
          }
        }
        const int col = tn * 256 + 128 * half + CB * c;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t blk = stg + 1024u * buf;
          buf ^= 1u;
          // the store before the last one has read its block
          if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
          if ((lane >> 4) == hh) {
            const uint32_t rl = static_cast<uint32_t>(lane & 15);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q)
              st_shared_v4(blk + rl * 64u + 16u * (q ^ ((rl >> 1) & 3u)), p[4 * q], p[4 * q + 1],
                           p[4 * q + 2], p[4 * q + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
            tma_store_2d(&tm_y, blk, col, row0 + 16 * hh);
            bulk_commit_group();
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) bulk_wait_group0();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();          // the pair's MMAs, copies and remote arrivals are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Clusters of c CTAs of the few-token kernel that run at once, for every c of
// kFewSplits, once per device.
template <int N>
static cudaError_t few_fits(const int** fits) {
  static int cached[64][kFewMaxSplit + 1] = {{0}};
  static std::atomic<int> filled[64];        // (threads that fill it at once write the same numbers)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int* n = cached[dev];
  *fits = n;
  if (filled[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const size_t smem = sizeof(FewSmem<N>) + 1024;
  e = cudaFuncSetAttribute(fp8_gemm_few_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(F_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int counted = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&counted, fp8_gemm_few_kernel<N>, F_THREADS, smem);
  if (e != cudaSuccess) return e;
  for (const int c : kFewSplits) {
    attr[0].val.clusterDim.z = static_cast<unsigned>(c);
    cfg.gridDim = dim3(148, 1, c);
    int fit = 0;
    e = cudaOccupancyMaxActiveClusters(&fit, fp8_gemm_few_kernel<N>, &cfg);
    if (e != cudaSuccess) return e;
    n[c] = fp8_clusters_that_fit(fit, counted, F_PER_SM);
  }
  filled[dev].store(1, std::memory_order_release);
  return cudaSuccess;
}

// Clusters of C CTAs of the mid kernel that run at once (C = 2 .. 5: 74, 45, 33, 26);
// 0 on an error.
static int mid_capacity(int C) {
  static int cached[64][H_MAX_C + 1] = {{0}};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev][C] > 0) return cached[dev][C];
  const size_t smem = sizeof(MidSmem) + 1024;
  if (cudaFuncSetAttribute(fp8_gemm_mid_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(148, 1, C);
  cfg.blockDim = dim3(H_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(C);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fp8_gemm_mid_kernel, &cfg) != cudaSuccess) return 0;
  cached[dev][C] = n;
  return n;
}

static int fp8_pair_capacity() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] > 0) return cached[dev];
  const size_t smem = sizeof(Fp8PairSmem) + 1024;
  if (cudaFuncSetAttribute(fp8_gemm_pair_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess ||
      cudaFuncSetAttribute(fp8_gemm_pair_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * 148, 1, 1);
  cfg.blockDim = dim3(Q_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0, n2 = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fp8_gemm_pair_kernel<false>, &cfg) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n2, fp8_gemm_pair_kernel<true>, &cfg) != cudaSuccess)
    return 0;
  cached[dev] = n < n2 ? n : n2;
  return cached[dev];
}

// Token counts up to the first take the few-token kernel, and so do products of
// few tiles of 128 channels x 64 tokens, which it can split six or eight ways at once
// (linear(), us, without this rule and with it: 128 x 1024 x 1024 9.6, 7.5;
// 128 x 4096 x 1024 12.5, 10.1; 384 x 7168 x 512 15.8, 14.5; 128 x 2048 x 2048,
// 32 tiles, 11.2, 10.6; above 32 tiles 192 x 2048 x 2048 11.7, 14.4).
constexpr int64_t kFp8FewMaxT = 64;
constexpr int64_t kFp8FewMaxTiles = 32;

cudaError_t plan_fp8_gemm(const uint8_t* aq, const float* sa, int64_t ld_sa, int64_t T, int64_t d_in,
                          int64_t d_out, const uint8_t* wq, const float* wscale, void* Y, int64_t ldy,
                          bool f32, Fp8GemmPlan* p) {
  memset(p, 0, sizeof(*p));
  p->empty = T == 0;
  if (p->empty) return cudaSuccess;
  p->f32 = f32;
  Fp8GemmArgs& a = p->a;
  a.sa = sa;
  a.sb = wscale;
  a.Y = Y;
  a.ld_sa = ld_sa;
  a.ldy = ldy;
  a.T = static_cast<int>(T);
  a.d_out = static_cast<int>(d_out);
  a.nkb = static_cast<int>((d_in + kFp8Block - 1) / kFp8Block);
  a.y_f32 = f32 ? 1 : 0;
  a.no_acts = (host_fault_mask() & FAULT_FP8_SKIP_ACTS) != 0u;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int tn = static_cast<int>((d_out + 127) / 128);
  if (T <= kFp8FewMaxT || tn * ((T + 63) / 64) <= kFp8FewMaxTiles) {
    const int N = T <= 16 ? 16 : T <= 32 ? 32 : T <= 48 ? 48 : 64;
    const int* fits = nullptr;
    const cudaError_t e = N == 16   ? few_fits<16>(&fits)
                          : N == 32 ? few_fits<32>(&fits)
                          : N == 48 ? few_fits<48>(&fits)
                                    : few_fits<64>(&fits);
    if (e != cudaSuccess) return e;
    p->few = N;
    p->smem = 1024 + (N == 16   ? sizeof(FewSmem<16>)
                      : N == 32 ? sizeof(FewSmem<32>)
                      : N == 48 ? sizeof(FewSmem<48>)
                                : sizeof(FewSmem<64>));
    const int ty = static_cast<int>((T + N - 1) / N);
    // (T = 1, 5120 -> 5120, 40 tiles: 1 16.2, 2 10.7, 3 9.0, 4 8.8, 6 8.2, 8 11.5 us)
    const int C = fp8_few_split(static_cast<int64_t>(tn) * ty, a.nkb, fits);
    p->cluster = C;
    p->grid = dim3(tn, ty, C);
    if (!make_tmap(&p->tm_w, wq, u8, 1, d_in, d_out, d_in, 128) ||
        !make_tmap(&p->tm_x, aq, u8, 1, d_in, T, d_in, N))
      return cudaErrorInvalidValue;
    return cudaSuccess;
  }
  a.tiles_m = static_cast<int>((T + 127) / 128);
  a.tiles_n = static_cast<int>((d_out + 255) / 256);
  // Where the tiles leave SMs idle, K is split over the CTAs of a cluster, as far
  // as all clusters run at once.  The join costs 2 us (two CTAs, few rows) to 6 us
  // (five, 128 rows), a K block 0.43 us in either kernel, so the split has to
  // spare some.  linear(), us, pair kernel and this one (CTAs of a cluster):
  // 128 x 5120 x 5120 23.3, 15.1 (5); 256 x 5120 x 5120 24.4, 19.8 (3);
  // 300 x 5120 x 5120 25.0, 22.5 (2); 128 x 13824 x 5120 52.1, 25.0 (5);
  // 384 x 13824 x 6144 58.5, 42.1 (2); 128 x 2048 x 5120 13.1, 12.2 (5);
  // 128 x 1024 x 1024, which spares 6 blocks, 9.6, 10.4.
  const int64_t mid_tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
  int C = 1;
  for (int c = 2; c <= H_MAX_C; ++c)
    if (mid_tiles <= mid_capacity(c)) C = c;
  if (a.nkb - (a.nkb + C - 1) / C >= 12) {
    p->mid = true;
    p->cluster = C;
    p->grid = dim3(static_cast<unsigned>(mid_tiles), 1, C);
    p->smem = sizeof(MidSmem) + 1024;
    if (!make_tmap(&p->tm_x, aq, u8, 1, d_in, T, d_in, 128) ||
        !make_tmap(&p->tm_w, wq, u8, 1, d_in, d_out, d_in, 256))
      return cudaErrorInvalidValue;
    return cudaSuccess;
  }
  const int cap = fp8_pair_capacity();
  if (cap <= 0) return cudaErrorInvalidConfiguration;
  a.tiles_m = static_cast<int>((T + 255) / 256);
  a.tiles_n = static_cast<int>((d_out + 255) / 256);
  const int64_t ntiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
  if (ntiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  p->grid = dim3(static_cast<unsigned>(2 * (ntiles < cap ? ntiles : cap)));
  p->smem = sizeof(Fp8PairSmem) + 1024;
  const int eb = f32 ? 4 : 2;
  if (!make_tmap(&p->tm_x, aq, u8, 1, d_in, T, d_in, 128) ||
      !make_tmap(&p->tm_w, wq, u8, 1, d_in, d_out, d_in, 128) ||
      !make_tmap(&p->tm_y, Y, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                 eb, d_out, T, static_cast<uint64_t>(ldy) * eb, 16, 64 / eb, false,
                 CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

cudaError_t run_fp8_gemm(const Fp8GemmPlan& p, cudaStream_t stream) {
  if (p.empty) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.grid;
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + static_cast<unsigned>(pdl_attrs(&attr[1]));
  if (p.few) {
    cfg.blockDim = dim3(F_THREADS, 1, 1);
    attr[0].val.clusterDim.z = static_cast<unsigned>(p.cluster);
    void (*k)(CUtensorMap, CUtensorMap, Fp8GemmArgs) =
        p.few == 16   ? fp8_gemm_few_kernel<16>
        : p.few == 32 ? fp8_gemm_few_kernel<32>
        : p.few == 48 ? fp8_gemm_few_kernel<48>
                      : fp8_gemm_few_kernel<64>;
    return cudaLaunchKernelEx(&cfg, k, p.tm_w, p.tm_x, p.a);
  }
  if (p.mid) {
    cfg.blockDim = dim3(H_THREADS, 1, 1);
    attr[0].val.clusterDim.z = static_cast<unsigned>(p.cluster);
    return cudaLaunchKernelEx(&cfg, fp8_gemm_mid_kernel, p.tm_x, p.tm_w, p.a);
  }
  cfg.blockDim = dim3(Q_THREADS, 1, 1);
  attr[0].val.clusterDim.x = 2;
  return cudaLaunchKernelEx(&cfg, p.f32 ? fp8_gemm_pair_kernel<true> : fp8_gemm_pair_kernel<false>,
                            p.tm_x, p.tm_w, p.tm_y, p.a);
}

}  // namespace w4a4
