// A whole mixture-of-experts layer for a few tokens (T <= 64) in two kernels:
//
//   l[t, e] = sum_j x[t, j] r[e, j];  E_t = the top_k experts of largest l
//   w[t, e] = exp(l[t, e]) / sum exp(l[t, .])  over E_t (renorm) or all experts
//   h[t, e] = silu(G_e x_t) * (U_e x_t)   or   gelu(U_e x_t)
//   y[t]    = sum_{e in E_t} w[t, e] D_e h[t, e]
//
// with x and h quantised to e4m3 per token and 128 columns, G, U, D in e4m3
// with one float32 scale per 128 x 128 tile, sums in float32.
//
// With few tokens the layer is the reading of the chosen experts' weights.
//  * moe_route_kernel: router logits, selection, quantisation of x.
//  * moe_experts_kernel: persistent, one CTA per SM.  All CTAs take work units
//    from one counter: first the units of the up projections, then those of the
//    down projections, in an order that lets the first down units find the
//    blocks of h they need complete; a unit is two tiles of 128 weight rows over
//    a range of K.  The roles of a CTA run ahead of each other: weight tiles of
//    the following units, down units included, are fetched while h is still
//    being made, and a finishing warp group takes a unit's sums from shared
//    memory (a few columns: little beside the weights) while the next unit's are
//    made: for an up unit the activation and the e4m3 codes of h, for a down
//    unit float32 sums to the workspace.  Where K of an up unit is split (few
//    units), the last range to arrive adds the ranges in their order; y is summed
//    at the end by all CTAs, in the order of selection: results do not depend on
//    timing.
//    A unit of the down projection waits until its range of its expert's h is
//    complete.  All up units were taken, by running CTAs that wait for nothing,
//    before the first down unit is: the wait ends however few CTAs of the grid
//    run at once.
//
// Measured (back to back, three sets of weights in turn): 64 tokens, 64 experts
// of 5120 x 1536, 8 chosen: 292 us, 5.2 TB/s of the weights met; 16 tokens, 128
// experts of 2048 x 768, 8 chosen: 75 us, 5.2 TB/s; 1 token, 2 of 8 experts of
// 5120 x 13824: 80 us, 5.3 TB/s; 1 token, 6 of 64 experts of 2048 x 1024: 26 us,
// of which the router takes 5.5 and the chain route -> up -> down -> y the rest
// (about ten round trips to memory one after the other).
// What brought it there: the finishing warps beside the epilogue (64 tokens 787
// -> 305 us; before, the memory idled while a unit was finished, and the sums of
// y were made by whichever CTA ended a tile's units, mostly the same one); eight
// epilogue warps (300 -> 274); order of the units and flags per block of h (1
// token, 2 of 8 experts: 84 -> 79).
#include <cuda.h>

#include "fp8_device.cuh"
#include "fp8_internal.h"

namespace w4a4 {

constexpr int kMoeMaxT = 64;
constexpr int kMoeMaxE = 512;
constexpr int kMoeMaxK = 16;
constexpr int kMoeMaxSplit = 8;

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------
constexpr int R_CTAS = 8;          // cluster: the experts are split over its CTAs
constexpr int R_WARPS = 8;         // warps for the logits; four more quantise x meanwhile
constexpr int R_THREADS = 32 * (R_WARPS + 4);

__device__ __forceinline__ void st_cluster_f64(uint32_t cluster_addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(cluster_addr), "d"(v) : "memory");
}

// the two halves of cluster_sync_all
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// acc0 += x . w0 and, where there are two experts, acc1 += x . w1 over 8 columns,
// in four sums each (a chain of 64-bit FMAs waits for each one's result).  The
// selection is the layer's one discontinuous step: two logits closer than a
// float32 sum's rounding would change places, and with them whole experts.  So
// logits are summed in 64 bits, where the products of bf16 numbers are exact
// and their sums nearly always are.  Layer, us, against float32 sums: 1 token, 6 of
// 64 experts of 2048 x 1024 25.8, 25.7; 16 tokens, 8 of 128 of 2048 x 768 74.2,
// 75.2; 64 tokens, 16 of 512 of 2048 x 256 220, 236; the router alone for 64 tokens,
// 64 experts of 5120 columns 15, 24.  The conversions bound it there: moving the bits
// into a double's fields instead took 18, but the layer with 4 tokens 41.7 for 40.0.
__device__ __forceinline__ void dot8(const uint4& x, const uint4& w0, const uint4& w1, bool two,
                                     double (&acc0)[4], double (&acc1)[4]) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, as[4] = {w0.x, w0.y, w0.z, w0.w},
                 bs[4] = {w1.x, w1.y, w1.z, w1.w};
  double lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = bf16_lo_to_f32(xs[i]);
    hi[i] = bf16_hi_to_f32(xs[i]);
    acc0[i] = fma(lo[i], static_cast<double>(bf16_lo_to_f32(as[i])), acc0[i]);
    acc0[i] = fma(hi[i], static_cast<double>(bf16_hi_to_f32(as[i])), acc0[i]);
  }
  if (two) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc1[i] = fma(lo[i], static_cast<double>(bf16_lo_to_f32(bs[i])), acc1[i]);
      acc1[i] = fma(hi[i], static_cast<double>(bf16_hi_to_f32(bs[i])), acc1[i]);
    }
  }
}

template <int n>
struct Steps {
  static constexpr int value = n;
};

// One cluster per token (four tokens to a cluster read less and took longer: 16
// tokens, 128 experts of 2048 columns, 13 against 6 us).  A warp takes two
// experts at a time over a range of the width (its lanes split it, 16 bytes
// each; the width is split where there are fewer pairs of experts than warps);
// the sums go to the shared memory of the cluster's first CTA, which adds the
// ranges in order and selects.
// U: steps of 256 columns whose loads are in flight together.  Four take 96
// registers, one CTA per SM, which is enough for few tokens; two take 68.  Layer,
// us, with U = 4 and 2: 1 token, 64 experts 25.7, 26.4; 9 tokens, 64 experts 52.0,
// 52.4; 16 tokens, 128 experts 77.0, 75.2; 24 tokens, 32 experts 97.2, 95.6.
constexpr int R_FEW_TOKENS = 12;
template <int U>
__global__ void __launch_bounds__(R_THREADS) moe_route_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ double part[kMoeMaxE];            // [split][expert]: more than one split only where E <= 64
  __shared__ double logits[kMoeMaxE];
  __shared__ alignas(16) uint32_t key[kMoeMaxE], key_lo[kMoeMaxE];
  __shared__ uint16_t chosen[kMoeMaxK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int t = static_cast<int>(blockIdx.x / R_CTAS);
  const int epc = (a.E + R_CTAS - 1) / R_CTAS;               // experts per CTA
  const int pairs = (epc + 1) / 2;
  const int splits = pairs > 4 ? 1 : pairs > 2 ? 2 : pairs > 1 ? 4 : 8;
  cluster_arrive();                    // (waited for before the first remote store)
  pdl_wait();
  pdl_launch_dependents();

  if (warp >= R_WARPS) {
    // counters of the next kernel, and x, four tokens by every fourth cluster:
    // one half-warp per block of 128 columns
    const int tid = threadIdx.x - 32 * R_WARPS;
    for (int i = blockIdx.x * 128 + tid; i < a.ncounters; i += gridDim.x * 128) a.counters[i] = 0;
    const int nb = (a.d + kFp8Block - 1) / kFp8Block;
    const int odd = (tid >> 4) & 1;
    if (t % 4 == 0)
      for (int kb = rank * 8 + (tid >> 4); kb - odd < nb; kb += R_CTAS * 8)
        fp8_quant_rows4(a.X, a.T, a.d, a.ldx, a.xq, a.xs, a.ld_x, t, kb);
    __syncwarp();
    cluster_wait();
  } else {
    const int e_end = (rank + 1) * epc < a.E ? (rank + 1) * epc : a.E;
    const int split = warp % splits;
    const int steps = (a.d + 255) / 256;
    const int s_lo = steps * split / splits, s_hi = steps * (split + 1) / splits;
    const int c_end = 256 * s_hi < a.d ? 256 * s_hi : a.d;
    const __nv_bfloat16* xr = a.X + t * a.ldx;
    bool waited = false;
    for (int e0 = rank * epc + 2 * (warp / splits); e0 < e_end; e0 += 2 * (R_WARPS / splits)) {
      const bool two = e0 + 1 < e_end;
      const __nv_bfloat16* r0 = a.router + static_cast<int64_t>(e0) * a.d;
      const __nv_bfloat16* r1 = two ? r0 + a.d : r0;
      double sum0[4] = {0.0, 0.0, 0.0, 0.0}, sum1[4] = {0.0, 0.0, 0.0, 0.0};
      auto step = [&](int c0, auto count) {     // `count` steps: all their loads, then the sums
        constexpr int n = decltype(count)::value;
        uint4 w0[n], w1[n], x[n];
#pragma unroll
        for (int u = 0; u < n; ++u) {
          w0[u] = *reinterpret_cast<const uint4*>(r0 + c0 + 256 * u);
          w1[u] = *reinterpret_cast<const uint4*>(r1 + c0 + 256 * u);
          x[u] = *reinterpret_cast<const uint4*>(xr + c0 + 256 * u);
        }
#pragma unroll
        for (int u = 0; u < n; ++u) dot8(x[u], w0[u], w1[u], two, sum0, sum1);
      };
      int c = 256 * s_lo + 8 * lane;
      for (; c + 256 * (U - 1) < c_end; c += 256 * U) step(c, Steps<U>());
      for (; c < c_end; c += 256) step(c, Steps<1>());
      __syncwarp();
      double acc0 = (sum0[0] + sum0[1]) + (sum0[2] + sum0[3]);
      double acc1 = (sum1[0] + sum1[1]) + (sum1[2] + sum1[3]);
      if (!waited) cluster_wait();
      waited = true;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        acc0 += __shfl_xor_sync(0xFFFFFFFFu, acc0, o);
        acc1 += __shfl_xor_sync(0xFFFFFFFFu, acc1, o);
      }
      if (lane == 0) {
        const uint32_t at = mapa_shared(smem_u32(&part[split * a.E + e0]), 0);
        st_cluster_f64(at, acc0);
        if (two) st_cluster_f64(at + 8u, acc1);
      }
      __syncwarp();
    }
    if (!waited) cluster_wait();
  }
  __syncwarp();
  cluster_sync_all();
  if (rank != 0) return;

  // Selection: every expert's place is the number of those before it.  Keys
  // order as the logits do; NaN comes last.  Their upper halves (20 bits behind
  // the first) decide nearly always; the rest is looked at where two are equal.
  const int e4 = (a.E + 3) & ~3;
  for (int e = threadIdx.x; e < e4; e += R_THREADS) {
    double l = 0.0;
    unsigned long long k = 0ull;       // (past the last expert: behind all)
    if (e < a.E) {
      for (int s = 0; s < splits; ++s) l += part[s * a.E + e];
      const unsigned long long b = __double_as_longlong(l);
      k = l != l ? 1ull << 32 : (b >> 63) ? ~b : (b | 1ull << 63);
    }
    logits[e] = l;
    key[e] = static_cast<uint32_t>(k >> 32);
    key_lo[e] = static_cast<uint32_t>(k);
  }
  __syncthreads();
  // four lanes to an expert, each counts a quarter of the others
  for (int i = threadIdx.x; (i & ~31) < 4 * a.E; i += R_THREADS) {
    const int e = i >> 2;
    const uint32_t k = e < a.E ? key[e] : 0u;
    int before = 0, same = 0;
#pragma unroll 4
    for (int j = 4 * (i & 3); j < e4; j += 16) {
      const uint4 o = *reinterpret_cast<const uint4*>(&key[j]);
      before += (o.x > k) + (o.y > k) + (o.z > k) + (o.w > k);
      same += (o.x == k) + (o.y == k) + (o.z == k) + (o.w == k);
    }
    __syncwarp();
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
    same += __shfl_xor_sync(0xFFFFFFFFu, same, 1);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
    same += __shfl_xor_sync(0xFFFFFFFFu, same, 2);
    if ((i & 3) == 0 && e < a.E && before < a.top_k) {
      if (same > 1) {
        const uint32_t lo = key_lo[e];
        for (int j = 0; j < a.E; ++j)
          before += key[j] == k && (key_lo[j] > lo || (key_lo[j] == lo && j < e));
      }
      if (before < a.top_k) chosen[before] = static_cast<uint16_t>(e);
    }
  }
  __syncthreads();
  if (warp != 0) return;
  const double lmax = logits[chosen[0]];
  const int e = lane < a.top_k ? chosen[lane] : 0;
  const float ex = lane < a.top_k ? expf(static_cast<float>(logits[e] - lmax)) : 0.f;
  float lsum = ex;
  if (!a.renorm) {
    lsum = 0.f;
    for (int j = lane; j < a.E; j += 32) lsum += expf(static_cast<float>(logits[j] - lmax));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, o);
  if (lane < a.top_k) {
    const int at = t * a.top_k + lane;
    const float w = ex / lsum;
    a.ids[at] = e;
    a.wts[at] = w;
    if (a.ids_out) a.ids_out[at] = e;
    if (a.wts_out) a.wts_out[at] = w;
  }
}

// ---------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------
// How many ranges K is split into: the fewest K blocks for the CTA with the most
// units, a unit counted as one more than its own, and `join` more where the
// ranges have to be joined; split only for a gain of a tenth.  One warp, the
// same result in all lanes.
__device__ __forceinline__ int moe_split(int units, int nkb, int most, int ctas, int join) {
  const int s = static_cast<int>(threadIdx.x & 31) + 1;
  auto cost = [&](int n) {
    return ((units * n + ctas - 1) / ctas) * ((nkb + n - 1) / n + 1) + (n > 1 ? join : 0);
  };
  const int c = s <= most && s <= nkb ? cost(s) : 0x3FFFFFF;
  const uint32_t best = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(c) * 32u + s - 1);
  const int c1 = __shfl_sync(0xFFFFFFFFu, c, 0);
  return 10 * static_cast<int>(best >> 5) < 9 * c1 ? static_cast<int>(best & 31u) + 1 : 1;
}

constexpr int M_THREADS = 512;     // weights, MMA, activations, idle, 8 epilogue, 4 finishing warps
constexpr int M_W_BYTES = 2 * 128 * 128;
constexpr int M_BUFS = 4;          // pairs of accumulators in tensor memory
constexpr int M_UNITS = 4;         // units between the producer and the epilogue
constexpr int M_CONSUMERS = 14;    // warps that read a unit: all but weights and idle

struct MoeUnit {
  int kind;          // 0: up, 1: down, 2: no more
  int ex;            // index of the expert among those with tokens
  int blk;           // up: unit of d_ff rows; down: 256 columns of y
  int split;
};

template <int N>
struct MoeSmem {
  static constexpr int kStageBytes = M_W_BYTES + N * 128;
  static constexpr int kStages = N == 64 ? 3 : 5;
  static constexpr int kSaSlots = kStages + M_BUFS;      // as in the few-token product
  uint8_t stage[kStages][kStageBytes];
  float sums[N][256];                               // a unit's sums, by pair and tile row
  alignas(16) float sa[kSaSlots][N];
  float2 sb[kSaSlots];                              // scales of the two weight tiles
  uint64_t mask[kMoeMaxE];                          // tokens of each expert
  uint16_t act_e[kMoeMaxE];                         // experts with tokens
  uint16_t off[kMoeMaxE];                           // by expert: its first row among the pairs
  uint16_t row_of[kMoeMaxT * kMoeMaxK];             // (token, choice) -> row
  uint32_t amax[2][4][4];
  MoeUnit unit[M_UNITS];
  uint64_t unit_full[M_UNITS];
  uint64_t unit_empty[M_UNITS];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t sa_full[kSaSlots];
  uint64_t acc_full[M_BUFS];
  uint64_t acc_empty[M_BUFS];
  uint64_t sums_full;
  uint64_t sums_empty;
  uint64_t drain;
  int n_act, s_up, s_dn;
  int last;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

// The barrier of the 128 finishing threads.  Named barriers are instructions of
// whole warps, and single lanes have work of their own before many of them.
__device__ __forceinline__ void finish_sync() {
  __syncwarp();
  named_bar_sync(1, 128);
}
// The same, which also tells all of them whether any had a non-zero pred.
__device__ __forceinline__ bool finish_any(uint32_t pred) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(pred), "r"(1u), "r"(128u)
      : "memory");
  return r != 0;
}

// global-memory writes of other SMs, seen through a counter, become visible to
// this SM's TMA loads (and the reverse)
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Waits until *p >= target; bounded like the barrier waits.
__device__ __forceinline__ bool counter_wait_bounded(const int* p, int target,
                                                     volatile uint32_t* abort, uint32_t err_bit) {
  if (ld_acquire(p) >= target) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(p) >= target) return true;
    if ((it & 15u) == 0) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > *static_cast<volatile uint64_t*>(&g_wait_limit_ns)) {
        atomicOr(&g_device_error, err_bit);
        *abort = 1u;
        return false;
      }
    }
  }
}

__device__ __forceinline__ float moe_silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }
__device__ __forceinline__ float moe_gelu(float y) {
  const float u = 0.7978845608028654f * (y + 0.044715f * y * y * y);
  return y / (1.0f + expf(-2.0f * u));
}

// After all 128 finishing threads' writes: counts one arrival; true for all of
// them if it was the last of `all`, whose earlier writes they may then read.
__device__ __forceinline__ bool moe_last_arrival(int* counter, int all, int* last, int tid) {
  finish_sync();
  if (tid == 0) {
    __threadfence();
    *last = atomicAdd(counter, 1) == all - 1;
    __threadfence();
  }
  finish_sync();
  return *last != 0;
}

// One block of 128 hidden rows of one expert, all its pairs, by the 128
// finishing threads: the activation and the e4m3 codes with their scale.  The
// sums are this CTA's own in shared memory (`own`, rows at `second` where there
// is no gate), or, with K split, the ranges' in the workspace, added in order.
template <bool kGated>
__device__ __forceinline__ void moe_finish_h(const MoeArgs& a, uint32_t (&amax)[2][4][4], int off, int m,
                                             int blk, int splits, const float* own, int second, int tid) {
  const int row = blk * 128 + tid;
  const bool in = row < a.ff;
  const int64_t stride = static_cast<int64_t>(kGated ? 2 : 1) * a.ff;      // floats per pair
  int buf = 0;
  for (int p0 = 0; p0 < m; p0 += 4, buf ^= 1) {
    float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
    if (own != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (in && p0 + i < m) {
          g[i] = own[(p0 + i) * 256];
          u[i] = kGated ? own[(p0 + i) * 256 + 128] : own[(p0 + i) * 256 + second];
        }
      }
    } else {
#pragma unroll 2
      for (int s = 0; s < splits; ++s) {
        const float* ps = a.part_up + (static_cast<int64_t>(s) * a.pairs + off + p0) * stride + row;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (in && p0 + i < m) {
            if constexpr (kGated) {
              g[i] += __ldcg(ps + i * stride);
              u[i] += __ldcg(ps + i * stride + a.ff);
            } else {
              u[i] += __ldcg(ps + i * stride);
            }
          }
        }
      }
    }
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = kGated ? moe_silu_mul(g[i], u[i]) : moe_gelu(u[i]);
      const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h[i]) & 0x7FFFFFFFu);
      if ((tid & 31) == 0) amax[buf][i][tid >> 5] = w;
    }
    finish_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p0 + i < m) {
        const uint32_t eb = f8_scale_exp(max(max(amax[buf][i][0], amax[buf][i][1]),
                                             max(amax[buf][i][2], amax[buf][i][3])));
        const int64_t r = off + p0 + i;
        if (in) {
          const uint32_t c = eb == 0u ? 0u : cvt_e4m3x4(h[i] * f8_inv_scale(eb), 0.f, 0.f, 0.f);
          a.hq[r * a.ff + row] = static_cast<uint8_t>(c);
        }
        if (tid == 0) a.hs[static_cast<int64_t>(blk) * a.pairs + r] = f8_scale(eb);
      }
    }
  }
}

// y: the weighted sum of the chosen experts' outputs, in the order of selection,
// over the ranges of K in order.  Thread i of `threads` over the whole grid takes
// every `threads`-th pair of columns.
__device__ __forceinline__ void moe_combine(const MoeArgs& a, const uint16_t* row_of, int splits, int i,
                                            int threads) {
  const int half = a.d / 2;
  const int64_t range = a.pairs * a.d;
  for (; i < a.T * half; i += threads) {
    const int t = i / half, col = 2 * (i - t * half);
    float2 y = make_float2(0.f, 0.f);
    for (int j0 = 0; j0 < a.top_k; j0 += 8) {
      float2 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int s = 0; s < splits; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j < a.top_k) {
            const int64_t r = row_of[t * a.top_k + j0 + j];
            const float2 w = __ldcg(reinterpret_cast<const float2*>(a.part_dn + s * range + r * a.d + col));
            v[j].x += w.x;
            v[j].y += w.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j < a.top_k) {
          const float wt = a.wts[t * a.top_k + j0 + j];
          y.x = fmaf(wt, v[j].x, y.x);
          y.y = fmaf(wt, v[j].y, y.y);
        }
      }
    }
    const int64_t at = t * a.ldy + col;
    if (a.y_f32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.Y) + at) = y;
    else
      *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.Y) + at) =
          __floats2bfloat162_rn(y.x, y.y);
  }
}

template <int N, bool kGated>
__global__ void __launch_bounds__(M_THREADS, 1)
    moe_experts_kernel(const __grid_constant__ CUtensorMap tm_gate,
                       const __grid_constant__ CUtensorMap tm_up,
                       const __grid_constant__ CUtensorMap tm_down,
                       const __grid_constant__ CUtensorMap tm_xq,
                       const __grid_constant__ CUtensorMap tm_hq, const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using Smem = MoeSmem<N>;
  constexpr int NST = Smem::kStages;
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile uint32_t* abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nkb_d = (a.d + 127) / 128, nkb_f = (a.ff + 127) / 128;
  const int up_units = kGated ? nkb_f : (nkb_f + 1) / 2;         // per expert
  const int dn_tiles = (a.d + 255) / 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 2);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < Smem::kSaSlots; ++s) mbar_init(&sm.sa_full[s], 1);
    for (int b = 0; b < M_BUFS; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 8);
    }
    for (int u = 0; u < M_UNITS; ++u) {
      mbar_init(&sm.unit_full[u], 1);
      mbar_init(&sm.unit_empty[u], M_CONSUMERS);
    }
    mbar_init(&sm.sums_full, 8);
    mbar_init(&sm.sums_empty, 4);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0u;
    fence_barrier_init();
    if (kGated) prefetch_tmap(&tm_gate);
    prefetch_tmap(&tm_up);
    prefetch_tmap(&tm_down);
    prefetch_tmap(&tm_xq);
    prefetch_tmap(&tm_hq);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 2 * M_BUFS * N);
    tmem_relinquish();
  }
  for (int e = threadIdx.x; e < a.E; e += M_THREADS) sm.mask[e] = 0ull;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();
  pdl_launch_dependents();

  // The tokens of each expert as a bit mask (a token chooses an expert once at
  // most), the experts that have any in ascending order, and the rows of their
  // (token, expert) pairs: expert by expert, tokens ascending, each expert's
  // first row a multiple of 4 so that its scales start on 16 bytes.
  int first_unit = 0;
  if (threadIdx.x == 0) first_unit = atomicAdd(a.ticket, 1);
  const int npairs = a.T * a.top_k;
  for (int p = threadIdx.x; p < npairs; p += M_THREADS)
    atomicOr(reinterpret_cast<unsigned long long*>(&sm.mask[a.ids[p]]), 1ull << (p / a.top_k));
  __syncthreads();
  if (warp == 0) {
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int m = e < a.E ? __popcll(sm.mask[e]) : 0;
      const uint32_t any = __ballot_sync(0xFFFFFFFFu, m != 0);
      int inc = (m + 3) & ~3;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      if (m != 0) {
        const int at = n + __popc(any & ((1u << lane) - 1u));
        sm.act_e[at] = static_cast<uint16_t>(e);
        sm.off[e] = static_cast<uint16_t>(rows + inc - ((m + 3) & ~3));
      }
      n += __popc(any);
      rows += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    const int ctas = static_cast<int>(gridDim.x);
    const int su = moe_split(n * up_units, nkb_d, a.most_up, ctas, 8);
    const int sd = moe_split(n * dn_tiles, nkb_f, a.most_dn, ctas, 0);
    if (lane == 0) {
      sm.n_act = n;
      sm.s_up = su;
      sm.s_dn = sd;
    }
  }
  __syncthreads();
  const int n_act = sm.n_act, s_up = sm.s_up, s_dn = sm.s_dn;
  for (int p = threadIdx.x; p < npairs; p += M_THREADS) {
    const int e = a.ids[p], t = p / a.top_k;
    sm.row_of[p] = static_cast<uint16_t>(sm.off[e] + __popcll(sm.mask[e] & ((1ull << t) - 1ull)));
  }
  __syncthreads();
  const int n_up = n_act * up_units * s_up;
  const int n_all = n_up + dn_tiles * n_act * s_dn;
  auto kb_lo = [](int nkb, int s, int splits) { return nkb * s / splits; };

  if (warp == 0) {
    // ================== weights (and the order of the units) ==============
    int next = __shfl_sync(0xFFFFFFFFu, first_unit, 0);
    uint32_t it = 0, u = 0;
    bool ok = true;
    while (ok) {
      const int cur = next;
      const int us = static_cast<int>(u % M_UNITS);
      if (u >= M_UNITS && !warp_wait_bounded(&sm.unit_empty[us], ((u / M_UNITS) & 1u) ^ 1u, abort_flag,
                                             DEVERR_TIMEOUT_PRODUCER))
        break;
      MoeUnit un;
      if (cur < n_up) {
        un.kind = 0;
        const int c = cur / s_up;
        un.split = cur - c * s_up;
        un.ex = s_dn > 1 ? c % n_act : c / up_units;
        un.blk = s_dn > 1 ? c / n_act : c % up_units;
      } else if (cur < n_all) {
        const int v = cur - n_up;
        un.kind = 1;
        const int c = v / dn_tiles;
        un.blk = v - c * dn_tiles;
        un.split = c / n_act;
        un.ex = c - un.split * n_act;
      } else {
        un.kind = 2;
        un.split = un.ex = un.blk = 0;
      }
      if (lane == 0) {
        sm.unit[us] = un;
        mbar_arrive(&sm.unit_full[us]);
        if (un.kind != 2) next = atomicAdd(a.ticket, 1);     // used after this unit's tiles
      }
      __syncwarp();
      if (un.kind == 2) break;
      ++u;
      const int e = sm.act_e[un.ex];
      const int nkb = un.kind == 0 ? nkb_d : nkb_f;
      const int splits = un.kind == 0 ? s_up : s_dn;
      const int kb1 = kb_lo(nkb, un.split + 1, splits);
      for (int kb = kb_lo(nkb, un.split, splits); kb < kb1; ++kb, ++it) {
        const int s = static_cast<int>(it % NST);
        if (it >= NST && !warp_wait_bounded(&sm.empty[s], ((it / NST) & 1u) ^ 1u, abort_flag,
                                            DEVERR_TIMEOUT_PRODUCER)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* st = sm.stage[s];
          mbar_arrive_expect_tx(&sm.full[s], M_W_BYTES);
          if (un.kind == 1) {
            tma_load_3d(st, &tm_down, &sm.full[s], kb * 128, un.blk * 256, e);
            tma_load_3d(st + 128 * 128, &tm_down, &sm.full[s], kb * 128, un.blk * 256 + 128, e);
          } else if (kGated) {
            tma_load_3d(st, &tm_gate, &sm.full[s], kb * 128, un.blk * 128, e);
            tma_load_3d(st + 128 * 128, &tm_up, &sm.full[s], kb * 128, un.blk * 128, e);
          } else {
            tma_load_3d(st, &tm_up, &sm.full[s], kb * 128, un.blk * 256, e);
            tma_load_3d(st + 128 * 128, &tm_up, &sm.full[s], kb * 128, un.blk * 256 + 128, e);
          }
        }
        __syncwarp();
      }
      next = __shfl_sync(0xFFFFFFFFu, next, 0);
    }
    if (*abort_flag) spin_ns(200000);          // copies in flight land before teardown
    __syncwarp();
  } else if (warp == 2) {
    // ======================== activations =================================
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t u = 0; ok; ++u) {
      const int us = static_cast<int>(u % M_UNITS);
      if (!warp_wait_bounded(&sm.unit_full[us], (u / M_UNITS) & 1u, abort_flag, DEVERR_TIMEOUT_PRODUCER))
        break;
      const MoeUnit un = sm.unit[us];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[us]);
      if (un.kind == 2) break;
      const int nkb = un.kind == 0 ? nkb_d : nkb_f;
      const int splits = un.kind == 0 ? s_up : s_dn;
      const int off = un.kind == 0 ? 0 : sm.off[sm.act_e[un.ex]];
      const int cols = un.kind == 0 ? a.T : __popcll(sm.mask[sm.act_e[un.ex]]);
      const uint32_t sa_bytes = static_cast<uint32_t>((cols + 3) & ~3) * 4u;
      const float* sa = un.kind == 0 ? a.xs : a.hs + off;
      const int64_t ld = un.kind == 0 ? a.ld_x : a.pairs;
      // the two tiles' scales; a second tile without rows takes the first one's
      const int e = sm.act_e[un.ex];
      const float *sb0, *sb1;
      if (un.kind == 1) {
        sb0 = a.down_s + (static_cast<int64_t>(e) * nkb_d + 2 * un.blk) * nkb_f;
        sb1 = 2 * un.blk + 1 < nkb_d ? sb0 + nkb_f : sb0;
      } else if (kGated) {
        sb0 = a.gate_s + (static_cast<int64_t>(e) * nkb_f + un.blk) * nkb_d;
        sb1 = a.up_s + (static_cast<int64_t>(e) * nkb_f + un.blk) * nkb_d;
      } else {
        sb0 = a.up_s + (static_cast<int64_t>(e) * nkb_f + 2 * un.blk) * nkb_d;
        sb1 = 2 * un.blk + 1 < nkb_f ? sb0 + nkb_d : sb0;
      }
      const int k0 = kb_lo(nkb, un.split, splits), k1 = kb_lo(nkb, un.split + 1, splits);
      WarpRun r0(sb0 + k0, k1 - k0), r1(sb1 + k0, k1 - k0);
      if (un.kind == 1) {
        bool got = true;
        for (int kb = k0 + lane; kb < k1 && got; kb += 32)
          got = counter_wait_bounded(a.ready + un.ex * nkb_f + kb, 1, abort_flag, DEVERR_TIMEOUT_PRODUCER);
        if (!__all_sync(0xFFFFFFFFu, got)) break;
        // every lane acquired other blocks' flags, one lane issues all copies: the
        // vote alone does not order the one behind the others
        __syncwarp();
        fence_proxy_async_global();
      }
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = static_cast<int>(it % NST);
        const int q = static_cast<int>(it % Smem::kSaSlots);
        if (it >= NST && !warp_wait_bounded(&sm.empty[s], ((it / NST) & 1u) ^ 1u, abort_flag,
                                            DEVERR_TIMEOUT_PRODUCER)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.full[s], N * 128);
          if (!a.no_acts)
            tma_load_2d(sm.stage[s] + M_W_BYTES, un.kind == 0 ? &tm_xq : &tm_hq, &sm.full[s], kb * 128,
                        off);
          bulk_load(sm.sa[q], sa + kb * ld, sa_bytes, &sm.sa_full[q]);
        }
        __syncwarp();
        const float2 sb2 = make_float2(r0.get(kb - k0), r1.get(kb - k0));
        if (elect_one()) {
          sm.sb[q] = sb2;
          mbar_arrive_expect_tx(&sm.sa_full[q], sa_bytes);
        }
        __syncwarp();
      }
    }
    if (*abort_flag) spin_ns(200000);
    __syncwarp();
  } else if (warp == 1) {
    // ============================ MMA issuer ==============================
    const uint64_t dw0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]));
    const uint64_t dw1 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]) + 128 * 128);
    const uint64_t dx0 = sdesc_kmajor_sw128(smem_u32(sm.stage[0]) + M_W_BYTES);
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t u = 0; ok; ++u) {
      const int us = static_cast<int>(u % M_UNITS);
      if (!warp_wait_bounded(&sm.unit_full[us], (u / M_UNITS) & 1u, abort_flag, DEVERR_TIMEOUT_MMA))
        break;
      const MoeUnit un = sm.unit[us];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[us]);
      if (un.kind == 2) break;
      const int nkb = un.kind == 0 ? nkb_d : nkb_f;
      const int splits = un.kind == 0 ? s_up : s_dn;
      const int nk = kb_lo(nkb, un.split + 1, splits) - kb_lo(nkb, un.split, splits);
      for (int i = 0; i < nk; ++i, ++it) {
        const int s = static_cast<int>(it % NST);
        const uint32_t b = it % M_BUFS;
        if (!warp_wait_bounded(&sm.acc_empty[b], ((it / M_BUFS) & 1u) ^ 1u, abort_flag, DEVERR_TIMEOUT_MMA) ||
            !warp_wait_bounded(&sm.full[s], (it / NST) & 1u, abort_flag, DEVERR_TIMEOUT_MMA)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t so = static_cast<uint64_t>(s * (Smem::kStageBytes >> 4));
          const uint32_t d0 = tmem + b * 2 * N;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_f8(d0, dw0 + so + 2 * kk, dx0 + so + 2 * kk, idesc_f8(128, N), kk != 0);
            mma_f8(d0 + N, dw1 + so + 2 * kk, dx0 + so + 2 * kk, idesc_f8(128, N), kk != 0);
          }
          tc_commit(&sm.empty[s]);
          tc_commit(&sm.acc_full[b]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(&sm.drain);
    __syncwarp();
    mbar_wait_bounded(&sm.drain, 0u, nullptr, DEVERR_TIMEOUT_MMA);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ============================ epilogue ================================
    // Four warps for each of the two tiles: add the K blocks' partial sums in
    // registers and hand a unit's sums on.  (With four for both, 64 columns took
    // them 1700 cycles a K block, more than its weights take to come.)
    const int h = (warp - 4) >> 2;
    const int sp = warp & 3;
    const int tid = 32 * sp + lane;                    // the tile row of this thread
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * sp) << 16) + h * N;
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t u = 0; ok; ++u) {
      const int us = static_cast<int>(u % M_UNITS);
      if (!warp_wait_bounded(&sm.unit_full[us], (u / M_UNITS) & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE))
        break;
      const MoeUnit un = sm.unit[us];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[us]);
      if (un.kind == 2) break;
      const uint64_t mk = sm.mask[sm.act_e[un.ex]];
      const int nkb = un.kind == 0 ? nkb_d : nkb_f;
      const int splits = un.kind == 0 ? s_up : s_dn;
      const int nk = kb_lo(nkb, un.split + 1, splits) - kb_lo(nkb, un.split, splits);
      float2 acc[N / 2];
#pragma unroll
      for (int j = 0; j < N / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      for (int i = 0; i < nk; ++i, ++it) {
        const int q = static_cast<int>(it % Smem::kSaSlots);
        const uint32_t b = it % M_BUFS;
        if (!warp_wait_bounded(&sm.sa_full[q], (it / Smem::kSaSlots) & 1u, abort_flag,
                               DEVERR_TIMEOUT_EPILOGUE) ||
            !warp_wait_bounded(&sm.acc_full[b], (it / M_BUFS) & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float sb = h ? sm.sb[q].y : sm.sb[q].x;
        const float2 sb2 = make_float2(sb, sb);
        constexpr int CH = N < 32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < N / CH; ++c) {
          uint32_t r[CH];
          tmem_ld_now(taddr + b * 2 * N + CH * c, r);
#pragma unroll
          for (int j = 0; j < CH / 4; ++j) {
            const float4 s4 = *reinterpret_cast<const float4*>(&sm.sa[q][CH * c + 4 * j]);
            float2& a0 = acc[CH / 2 * c + 2 * j];
            float2& a1 = acc[CH / 2 * c + 2 * j + 1];
            a0 = __ffma2_rn(make_float2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])),
                            __fmul2_rn(make_float2(s4.x, s4.y), sb2), a0);
            a1 = __ffma2_rn(make_float2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                            __fmul2_rn(make_float2(s4.z, s4.w), sb2), a1);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
      }
      if (!ok || !warp_wait_bounded(&sm.sums_empty, (u & 1u) ^ 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE))
        break;
      // up: the columns are all tokens, those of this expert are kept; down: the
      // columns are the expert's pairs, then others'
      const uint64_t keep = un.kind == 0 ? mk : ~0ull >> (64 - __popcll(mk));
      float* p = &sm.sums[0][128 * h + tid];
#pragma unroll
      for (int c = 0; c < N; ++c) {
        if ((keep >> c) & 1ull) {
          *p = (c & 1) ? acc[c >> 1].y : acc[c >> 1].x;
          p += 256;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.sums_full);
    }
  } else if (warp >= 12) {
    // ============================ finishing ===============================
    // What follows a unit's sums, while the next unit's are made.  The four
    // warps agree at their barriers on whether one of them gave up
    // (finish_any), so none is left waiting for another.
    const int tid = threadIdx.x - 384;
    for (uint32_t u = 0;; ++u) {
      const int us = static_cast<int>(u % M_UNITS);
      bool ok = warp_wait_bounded(&sm.unit_full[us], (u / M_UNITS) & 1u, abort_flag,
                                  DEVERR_TIMEOUT_EPILOGUE);
      if (finish_any(!ok)) break;
      const MoeUnit un = sm.unit[us];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[us]);
      if (un.kind == 2) break;
      ok = warp_wait_bounded(&sm.sums_full, u & 1u, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
      if (finish_any(!ok)) break;
      const int e = sm.act_e[un.ex];
      const int off = sm.off[e];
      const int m = __popcll(sm.mask[e]);
      const float* own = &sm.sums[0][tid];
      if (un.kind == 0) {
        bool finish = true;
        if (s_up > 1) {
          // this range's sums to the workspace; the last range to arrive goes on
          const int r0 = (kGated ? un.blk : 2 * un.blk) * 128 + tid;
          const int64_t stride = static_cast<int64_t>(kGated ? 2 : 1) * a.ff;
          const int64_t second_at = kGated ? a.ff : 128;
          const bool in0 = r0 < a.ff, in1 = kGated ? in0 : r0 + 128 < a.ff;
          float* p = a.part_up + (static_cast<int64_t>(un.split) * a.pairs + off) * stride + r0;
          for (int i = 0; i < m; ++i, p += stride) {
            if (in0) __stcg(p, own[i * 256]);
            if (in1) __stcg(p + second_at, own[i * 256 + 128]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sums_empty);
          finish = moe_last_arrival(a.up_done + un.ex * up_units + un.blk, s_up, &sm.last, tid);
        }
        if (finish) {
          const float* src = s_up > 1 ? nullptr : own;
          if constexpr (kGated) {
            moe_finish_h<true>(a, sm.amax, off, m, un.blk, s_up, src, 0, tid);
          } else {
            moe_finish_h<false>(a, sm.amax, off, m, 2 * un.blk, s_up, src, 0, tid);
            finish_sync();
            if (2 * un.blk + 1 < nkb_f)
              moe_finish_h<false>(a, sm.amax, off, m, 2 * un.blk + 1, s_up, src, 128, tid);
          }
          if (s_up == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.sums_empty);
          }
          fence_proxy_async_global();
          finish_sync();
          if (tid == 0) {
            __threadfence();
            int* flag = a.ready + un.ex * nkb_f + (kGated ? un.blk : 2 * un.blk);
            atomicExch(flag, 1);
            if (!kGated && 2 * un.blk + 1 < nkb_f) atomicExch(flag + 1, 1);
          }
        }
      } else {
        const int r0 = un.blk * 256 + tid;
        const bool in0 = r0 < a.d, in1 = r0 + 128 < a.d;
        float* p = a.part_dn + (static_cast<int64_t>(un.split) * a.pairs + off) * a.d + r0;
        for (int i = 0; i < m; ++i, p += a.d) {
          if (in0) __stcg(p, own[i * 256]);
          if (in1) __stcg(p + 128, own[i * 256 + 128]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sums_empty);
        finish_sync();
        if (tid == 0) {
          __threadfence();
          atomicAdd(a.dn_done, 1);
        }
      }
    }
    // y, once all down units are done: every CTA a share.  (Like the wait for h,
    // this one is for units that running CTAs have taken.)
    bool done = *abort_flag == 0u;
    if (done && tid == 0)
      done = counter_wait_bounded(a.dn_done, dn_tiles * n_act * s_dn, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
    if (!finish_any(!done))
      moe_combine(a, sm.row_of, s_dn, blockIdx.x * 128 + tid, gridDim.x * 128);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * M_BUFS * N);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// A stack of matrices of e4m3 codes in boxes of 128 x 128.
static bool make_tmap_stack(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t n) {
  PFN_encodeTiled enc = get_encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {cols, rows, n};
  cuuint64_t strides[2] = {cols, cols * rows};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace, from the sizes alone (no device query: the same on every device).
MoeLayout moe_layout(int64_t T, int64_t d, int64_t ff, int64_t E, int64_t top_k, bool gated) {
  MoeLayout l;
  constexpr int kCtas = 148;
  const int64_t P = T * top_k;
  l.pairs = round_up(P + 3 * (E < P ? E : P), 4);
  l.ld_x = round_up(T, 4);
  const int64_t nkb_d = (d + 127) / 128, nkb_f = (ff + 127) / 128;
  const int64_t up_units = gated ? nkb_f : (nkb_f + 1) / 2, dn_tiles = (d + 255) / 256;
  // at least top_k experts have tokens; more splits than two per CTA gain nothing
  auto most = [&](int64_t units, int64_t nkb) {
    int64_t s = (2 * kCtas + top_k * units - 1) / (top_k * units);
    s = s < kMoeMaxSplit ? s : kMoeMaxSplit;
    return s < nkb ? s : nkb;
  };
  l.most_up = static_cast<int>(most(up_units, nkb_d));
  l.most_dn = static_cast<int>(most(dn_tiles, nkb_f));
  const int64_t nE = E < P ? E : P;
  l.up_done = 0;
  l.ready = l.up_done + nE * up_units;
  l.dn_done = l.ready + nE * nkb_f;
  l.ticket = l.dn_done + 1;
  l.ncounters = l.ticket + 1;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t p = at;
    at += static_cast<size_t>(round_up(bytes, 1024));
    return p;
  };
  l.xq = take(T * d);
  l.xs = take(nkb_d * l.ld_x * 4);
  l.ids = take(P * 4);
  l.wts = take(P * 4);
  l.hq = take(l.pairs * ff);
  l.hs = take(nkb_f * l.pairs * 4);
  l.part_up = take(l.most_up * l.pairs * (gated ? 2 : 1) * ff * 4);
  l.part_dn = take(l.most_dn * l.pairs * d * 4);
  l.counters = take(l.ncounters * 4);
  l.total = at;
  return l;
}

template <int N, bool kGated>
static cudaError_t moe_attr() {
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(moe_experts_kernel<N, kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(MoeSmem<N>) + 1024));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = 1;
  return e;
}

template <int N, bool kGated>
static cudaError_t run_moe_experts(const MoePlan& p, cudaStream_t stream) {
  return launch_pdl(moe_experts_kernel<N, kGated>, dim3(p.ctas), dim3(M_THREADS),
                    sizeof(MoeSmem<N>) + 1024, stream, p.tm_gate, p.tm_up, p.tm_down, p.tm_xq, p.tm_hq,
                    p.a);
}

cudaError_t plan_moe(const MoeArgs& a, int64_t E, const uint8_t* gate, const uint8_t* up,
                     const uint8_t* down, bool gated, MoePlan* p) {
  memset(p, 0, sizeof(*p));
  p->a = a;
  p->a.no_acts = (host_fault_mask() & FAULT_FP8_SKIP_ACTS) != 0u;
  p->gated = gated;
  p->n = a.T <= 16 ? 16 : a.T <= 32 ? 32 : 64;
  p->ctas = device_num_sms();
  if (p->ctas <= 0) return cudaErrorInvalidDevice;
  cudaError_t e = gated ? (p->n == 16 ? moe_attr<16, true>() : p->n == 32 ? moe_attr<32, true>() : moe_attr<64, true>())
                        : (p->n == 16 ? moe_attr<16, false>() : p->n == 32 ? moe_attr<32, false>() : moe_attr<64, false>());
  if (e != cudaSuccess) return e;
  if ((gated && !make_tmap_stack(&p->tm_gate, gate, a.d, a.ff, E)) ||
      !make_tmap_stack(&p->tm_up, up, a.d, a.ff, E) || !make_tmap_stack(&p->tm_down, down, a.ff, a.d, E) ||
      !make_tmap(&p->tm_xq, a.xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d, a.T, a.d, p->n) ||
      !make_tmap(&p->tm_hq, a.hq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.ff, a.pairs, a.ff, p->n))
    return cudaErrorInvalidValue;
  if (!gated) p->tm_gate = p->tm_up;
  return cudaSuccess;
}

cudaError_t run_moe(const MoePlan& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(R_CTAS * p.a.T));
  cfg.blockDim = dim3(R_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R_CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + static_cast<unsigned>(pdl_attrs(&attr[1]));
  void (*route)(MoeArgs) = p.a.T <= R_FEW_TOKENS ? moe_route_kernel<4> : moe_route_kernel<2>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, route, p.a);
  if (e != cudaSuccess) return e;
  if (p.gated)
    return p.n == 16 ? run_moe_experts<16, true>(p, stream)
                     : p.n == 32 ? run_moe_experts<32, true>(p, stream) : run_moe_experts<64, true>(p, stream);
  return p.n == 16 ? run_moe_experts<16, false>(p, stream)
                   : p.n == 32 ? run_moe_experts<32, false>(p, stream) : run_moe_experts<64, false>(p, stream);
}

}  // namespace w4a4
