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
                                y_f32 != 0, false, &p);
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
                                y_f32 != 0, pdl_enabled(), &p);
  if (e != cudaSuccess) return W4A4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = launch_fp8_quant_act(X, T, w->d_in, ldx, q, scale, ws.ld_scale, s);
  if (e == cudaSuccess) e = run_fp8_gemm(p, s);
  return from_cuda(e);
}

}  // extern "C"
