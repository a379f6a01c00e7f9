// Internal declarations of the 8-bit floating point operators.
#pragma once

#include "w4a4_internal.h"

namespace w4a4 {

// Failure-detection test hook (w4a4_test_fault), beside the prep producer's bit:
// the products and the expert kernel copy no activation tiles, so that the waits
// for them run out.  Seen by the host, which hands it to the kernels as an argument.
enum : uint32_t { FAULT_FP8_SKIP_ACTS = 1u << 2 };
uint32_t host_fault_mask();       // the mask last given to w4a4_test_fault

cudaError_t launch_fp8_quant_act(const void* X, int64_t T, int64_t d, int64_t ldx, uint8_t* q,
                                 float* scale, int64_t ld_scale, cudaStream_t stream);
cudaError_t launch_fp8_pack_weight(const void* W, int64_t ldw, int64_t rows, int64_t cols,
                                   int64_t experts, uint8_t* q, float* scale, cudaStream_t stream);

struct Fp8GemmArgs {
  const float* sa;          // [nkb][ld_sa]
  const float* sb;          // [ceil(d_out / 128)][nkb]
  void* Y;
  int64_t ld_sa, ldy;
  int T, d_out, nkb, y_f32;
  int no_acts;              // failure-detection test hook: copy no activation tiles
  int tiles_m, tiles_n;     // not the few-token kernel
};

// plan: tensor maps, tile choice (host only); run: the launch.
struct Fp8GemmPlan {
  CUtensorMap tm_x, tm_w, tm_y;
  Fp8GemmArgs a;
  dim3 grid;
  size_t smem;
  int few;                  // 0: pair kernel; else tokens per tile of the few-token kernel
  int cluster;
  bool mid;                 // K split over a cluster
  bool f32, empty;
};
cudaError_t plan_fp8_gemm(const uint8_t* aq, const float* sa, int64_t ld_sa, int64_t T, int64_t d_in,
                          int64_t d_out, const uint8_t* wq, const float* wscale, void* Y, int64_t ldy,
                          bool f32, Fp8GemmPlan* p);
cudaError_t run_fp8_gemm(const Fp8GemmPlan& p, cudaStream_t stream);

// The expert layer.  Pairs are (token, chosen expert), in rows sorted by expert.
struct MoeArgs {
  const __nv_bfloat16* X;
  const __nv_bfloat16* router;      // [E, d]
  int64_t ldx, ldy;
  void* Y;
  int32_t* ids_out;                 // optional, the caller's
  float* wts_out;
  const float *gate_s, *up_s, *down_s;
  // workspace
  uint8_t* xq;                      // [T, d]
  float* xs;                        // [blocks of d][ld_x]
  int32_t* ids;                     // [T, top_k]
  float* wts;
  uint8_t* hq;                      // [pairs, ff]
  float* hs;                        // [blocks of ff][pairs]
  float* part_up;                   // [split][pairs][gate, up][ff]
  float* part_dn;                   // [split][pairs][d]
  int32_t* counters;                // all of the following, zeroed by the router
  int32_t *up_done, *ready, *dn_done, *ticket;
  int64_t ld_x, pairs;
  int T, d, ff, E, top_k, renorm, y_f32, ncounters, most_up, most_dn;
  int no_acts;                      // failure-detection test hook: copy no activation tiles
};
struct MoeLayout {
  int64_t pairs, ld_x, up_done, ready, dn_done, ticket, ncounters;
  int most_up, most_dn;
  size_t xq, xs, ids, wts, hq, hs, part_up, part_dn, counters, total;
};
MoeLayout moe_layout(int64_t T, int64_t d, int64_t ff, int64_t E, int64_t top_k, bool gated);
struct MoePlan {
  CUtensorMap tm_gate, tm_up, tm_down, tm_xq, tm_hq;
  MoeArgs a;
  int n, ctas;
  bool gated;
};
cudaError_t plan_moe(const MoeArgs& a, int64_t E, const uint8_t* gate, const uint8_t* up,
                     const uint8_t* down, bool gated, MoePlan* p);
cudaError_t run_moe(const MoePlan& p, cudaStream_t stream);

}  // namespace w4a4
