// C-ABI entry points of the 8-bit floating point operators (declared in
// include/w4a4.h): argument validation, workspace layout and launches.
#include "fp8_internal.h"
#include "w4a4.h"

namespace w4a4 {

constexpr int64_t kFp8MaxT = (int64_t(1) << 31) - 256;

static w4a4_status fp8_check_dims(int64_t d_in, int64_t d_out) {
  if (d_in <= 0 || d_out <= 0) return W4A4_ERR_INVALID_ARG;
  if (d_in % 16 != 0 || d_out % 16 != 0 || d_in > 65535 || d_out > (int64_t(1) << 30))
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  return W4A4_OK;
}

static w4a4_status fp8_check_weight(const w4a4_fp8_weight* w) {
  if (w == nullptr) return W4A4_ERR_INVALID_ARG;
  const w4a4_status st = fp8_check_dims(w->d_in, w->d_out);
  if (st != W4A4_OK) return st;
  if (w->experts < 1 || w->q == nullptr || w->scale == nullptr) return W4A4_ERR_INVALID_ARG;
  if (w->experts > 65535) return W4A4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(w->q) || (reinterpret_cast<uintptr_t>(w->scale) & 3u) != 0)
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  return W4A4_OK;
}

static w4a4_status fp8_check_quant(const void* X, int64_t T, int64_t d, int64_t ldx, const uint8_t* q,
                                   const float* scale, int64_t ld_scale) {
  if (T < 0 || d <= 0 || ldx < d || ld_scale < round_up(T, 4)) return W4A4_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > 65535 || ldx % 8 != 0 || ld_scale % 4 != 0 || T > kFp8MaxT)
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return W4A4_OK;
  if (X == nullptr || q == nullptr || scale == nullptr) return W4A4_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(q) || !aligned16(scale)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  return W4A4_OK;
}

static w4a4_status fp8_check_gemm(const uint8_t* a, const float* scale_a, int64_t ld_scale, int64_t T,
                                  const w4a4_fp8_weight* w, const void* Y, int64_t ldy) {
  const w4a4_status st = fp8_check_weight(w);
  if (st != W4A4_OK) return st;
  if (w->experts != 1 || T < 0 || ldy < w->d_out || ld_scale < round_up(T, 4))
    return W4A4_ERR_INVALID_ARG;
  if (T > kFp8MaxT || ldy % 8 != 0 || ld_scale % 4 != 0) return W4A4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return W4A4_OK;
  if (a == nullptr || scale_a == nullptr || Y == nullptr) return W4A4_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(scale_a) || !aligned16(Y)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  return W4A4_OK;
}

struct Fp8Workspace {
  size_t scale, total;
  int64_t ld_scale;
};
static Fp8Workspace fp8_workspace(int64_t T, int64_t d_in) {
  Fp8Workspace w;
  w.ld_scale = round_up(T, 4);
  w.scale = static_cast<size_t>(round_up(T * d_in, 1024));
  w.total = w.scale + static_cast<size_t>(
                          round_up((d_in + kFp8Block - 1) / kFp8Block * w.ld_scale * 4, 1024));
  return w;
}

static w4a4_status moe_check(const w4a4_fp8_experts* m, int64_t T) {
  if (m == nullptr || T < 0) return W4A4_ERR_INVALID_ARG;
  if (m->act != W4A4_MOE_GELU && m->act != W4A4_MOE_SILU_GATED) return W4A4_ERR_INVALID_ARG;
  w4a4_status st = fp8_check_weight(&m->up);
  if (st != W4A4_OK) return st;
  st = fp8_check_weight(&m->down);
  if (st != W4A4_OK) return st;
  const int64_t d = m->up.d_in, ff = m->up.d_out, E = m->up.experts;
  if (m->down.d_in != ff || m->down.d_out != d || m->down.experts != E) return W4A4_ERR_INVALID_ARG;
  if (m->act == W4A4_MOE_SILU_GATED) {
    st = fp8_check_weight(&m->gate);
    if (st != W4A4_OK) return st;
    if (m->gate.d_in != d || m->gate.d_out != ff || m->gate.experts != E) return W4A4_ERR_INVALID_ARG;
  }
  if (m->router == nullptr || m->top_k < 1 || m->top_k > E) return W4A4_ERR_INVALID_ARG;
  if (T > kMoeMaxT || E > kMoeMaxE || m->top_k > kMoeMaxK || ff > 65535 || d > 65535 ||
      !aligned16(m->router))
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  return W4A4_OK;
}

}  // namespace w4a4

using namespace w4a4;

extern "C" {

w4a4_status w4a4_fp8_quant_act(const void* X, int64_t T, int64_t d, int64_t ldx, uint8_t* q,
                               float* scale, int64_t ld_scale, void* stream) {
  const w4a4_status st = fp8_check_quant(X, T, d, ldx, q, scale, ld_scale);
  if (st != W4A4_OK || T == 0) return st;
  return from_cuda(
      launch_fp8_quant_act(X, T, d, ldx, q, scale, ld_scale, static_cast<cudaStream_t>(stream)));
}

w4a4_status w4a4_fp8_pack_weight(const void* W, int64_t ldw, const w4a4_fp8_weight* w, void* stream) {
  const w4a4_status st = fp8_check_weight(w);
  if (st != W4A4_OK) return st;
  if (W == nullptr || ldw < w->d_in) return W4A4_ERR_INVALID_ARG;
  // grid y: tiles of 128 rows
  if (ldw % 8 != 0 || !aligned16(W) || w->d_out > int64_t(65535) * kFp8Block)
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  return from_cuda(launch_fp8_pack_weight(W, ldw, w->d_out, w->d_in, w->experts, w->q, w->scale,
                                          static_cast<cudaStream_t>(stream)));
}

w4a4_status w4a4_fp8_gemm(const uint8_t* a, const float* scale_a, int64_t ld_scale, int64_t T,
                          const w4a4_fp8_weight* w, void* Y, int64_t ldy, int y_f32, void* stream) {
  const w4a4_status st = fp8_check_gemm(a, scale_a, ld_scale, T, w, Y, ldy);
  if (st != W4A4_OK || T == 0) return st;
  Fp8GemmPlan p;
  cudaError_t e = plan_fp8_gemm(a, scale_a, ld_scale, T, w->d_in, w->d_out, w->q, w->scale, Y, ldy,
                                y_f32 != 0, &p);
  if (e == cudaSuccess) e = run_fp8_gemm(p, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

w4a4_status w4a4_fp8_workspace_size(int64_t T, int64_t d_in, size_t* bytes) {
  if (bytes == nullptr || T < 0) return W4A4_ERR_INVALID_ARG;
  const w4a4_status st = fp8_check_dims(d_in, 16);
  if (st != W4A4_OK) return st;
  if (T > kFp8MaxT) return W4A4_ERR_UNSUPPORTED_SHAPE;
  *bytes = fp8_workspace(T, d_in).total;
  return W4A4_OK;
}

w4a4_status w4a4_fp8_linear(const void* X, int64_t T, int64_t ldx, const w4a4_fp8_weight* w,
                            void* workspace, size_t ws_bytes, void* Y, int64_t ldy, int y_f32,
                            void* stream) {
  w4a4_status st = fp8_check_weight(w);
  if (st != W4A4_OK) return st;
  if (w->experts != 1 || T < 0 || ldx < w->d_in || ldy < w->d_out) return W4A4_ERR_INVALID_ARG;
  if (T > kFp8MaxT) return W4A4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return W4A4_OK;
  const Fp8Workspace ws = fp8_workspace(T, w->d_in);
  if (workspace == nullptr || ws_bytes < ws.total) return W4A4_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  uint8_t* q = static_cast<uint8_t*>(workspace);
  float* scale = reinterpret_cast<float*>(q + ws.scale);
  st = fp8_check_quant(X, T, w->d_in, ldx, q, scale, ws.ld_scale);
  if (st != W4A4_OK) return st;
  st = fp8_check_gemm(q, scale, ws.ld_scale, T, w, Y, ldy);
  if (st != W4A4_OK) return st;
  Fp8GemmPlan p;
  cudaError_t e = plan_fp8_gemm(q, scale, ws.ld_scale, T, w->d_in, w->d_out, w->q, w->scale, Y, ldy,
                                y_f32 != 0, &p);
  if (e != cudaSuccess) return W4A4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = launch_fp8_quant_act(X, T, w->d_in, ldx, q, scale, ws.ld_scale, s);
  if (e == cudaSuccess) e = run_fp8_gemm(p, s);
  return from_cuda(e);
}

w4a4_status w4a4_fp8_moe_workspace_size(const w4a4_fp8_experts* m, int64_t T, size_t* bytes) {
  if (bytes == nullptr) return W4A4_ERR_INVALID_ARG;
  const w4a4_status st = moe_check(m, T);
  if (st != W4A4_OK) return st;
  *bytes = moe_layout(T, m->up.d_in, m->up.d_out, m->up.experts, m->top_k,
                      m->act == W4A4_MOE_SILU_GATED).total;
  return W4A4_OK;
}

w4a4_status w4a4_fp8_moe(const void* X, int64_t T, int64_t ldx, const w4a4_fp8_experts* m,
                         void* workspace, size_t ws_bytes, void* Y, int64_t ldy, int y_f32,
                         int32_t* ids, float* weights, void* stream) {
  const w4a4_status st = moe_check(m, T);
  if (st != W4A4_OK) return st;
  const int64_t d = m->up.d_in, ff = m->up.d_out, E = m->up.experts;
  const bool gated = m->act == W4A4_MOE_SILU_GATED;
  if (ldx < d || ldy < d) return W4A4_ERR_INVALID_ARG;
  if (ldx % 8 != 0 || ldy % 8 != 0) return W4A4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return W4A4_OK;
  const MoeLayout l = moe_layout(T, d, ff, E, m->top_k, gated);
  if (X == nullptr || Y == nullptr || workspace == nullptr || ws_bytes < l.total)
    return W4A4_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(ids) & 3u) != 0 || (reinterpret_cast<uintptr_t>(weights) & 3u) != 0)
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  MoeArgs a = {};
  a.X = static_cast<const __nv_bfloat16*>(X);
  a.router = static_cast<const __nv_bfloat16*>(m->router);
  a.ldx = ldx;
  a.ldy = ldy;
  a.Y = Y;
  a.ids_out = ids;
  a.wts_out = weights;
  a.gate_s = m->gate.scale;
  a.up_s = m->up.scale;
  a.down_s = m->down.scale;
  a.xq = base + l.xq;
  a.xs = reinterpret_cast<float*>(base + l.xs);
  a.ids = reinterpret_cast<int32_t*>(base + l.ids);
  a.wts = reinterpret_cast<float*>(base + l.wts);
  a.hq = base + l.hq;
  a.hs = reinterpret_cast<float*>(base + l.hs);
  a.part_up = reinterpret_cast<float*>(base + l.part_up);
  a.part_dn = reinterpret_cast<float*>(base + l.part_dn);
  a.counters = reinterpret_cast<int32_t*>(base + l.counters);
  a.up_done = a.counters + l.up_done;
  a.ready = a.counters + l.ready;
  a.dn_done = a.counters + l.dn_done;
  a.ticket = a.counters + l.ticket;
  a.ld_x = l.ld_x;
  a.pairs = l.pairs;
  a.T = static_cast<int>(T);
  a.d = static_cast<int>(d);
  a.ff = static_cast<int>(ff);
  a.E = static_cast<int>(E);
  a.top_k = static_cast<int>(m->top_k);
  a.renorm = m->renorm != 0;
  a.y_f32 = y_f32 != 0;
  a.ncounters = static_cast<int>(l.ncounters);
  a.most_up = l.most_up;
  a.most_dn = l.most_dn;
  MoePlan p;
  cudaError_t e = plan_moe(a, E, m->gate.q, m->up.q, m->down.q, gated, &p);
  if (e == cudaSuccess) e = run_moe(p, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

}  // extern "C"
