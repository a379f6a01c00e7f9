// e4m3 quantisers with one float32 scale per block of 128.
//
//   s = 2^e, e = max(-126, min{ e : max|x| <= 448 * 2^e }),  c = e4m3_rn(x / s)
//
// over 128 consecutive columns of one token (activations) or a 128 x 128 tile
// (weights).  s is a power of two, so x / s is exact (a product with 2^-e)
// and each element is rounded once; an e4m3 value has its own exponent, so a
// scale that is not the exact amax / 448 costs no precision except for the
// smallest elements of a block, which lose at most one bit of the subnormal
// range.  A block holding an infinity or a NaN has scale NaN and codes 0:
// every output of the product that reads it is NaN, and no other.
//
// Both kernels move each byte once and are bound by memory (launch latency
// below some tens of MB).
#include "fp8_device.cuh"
#include "fp8_internal.h"

namespace w4a4 {

// The codes of one block's 128 values, 8 per lane of a half-warp (every lane of
// the warp takes part), and their scale.
__device__ __forceinline__ float fp8_quant_half_warp(const uint4& v, uint2& codes) {
  // magnitudes of bf16 pairs compare as 16-bit integers, infinities and NaN above all
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                        __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const uint32_t eb = f8_scale_exp(max(m & 0xFFFFu, m >> 16) << 16);
  codes = make_uint2(0u, 0u);
  if (eb != 0u) {
    const float inv = f8_inv_scale(eb);
    codes.x = cvt_e4m3x4(bf16_lo_to_f32(v.x) * inv, bf16_hi_to_f32(v.x) * inv,
                         bf16_lo_to_f32(v.y) * inv, bf16_hi_to_f32(v.y) * inv);
    codes.y = cvt_e4m3x4(bf16_lo_to_f32(v.z) * inv, bf16_hi_to_f32(v.z) * inv,
                         bf16_lo_to_f32(v.w) * inv, bf16_hi_to_f32(v.w) * inv);
  }
  return f8_scale(eb);
}

// One half-warp per (4 rows, one block): 16 lanes x 16 bytes cover a row's
// 128 columns, the four rows' loads are independent, and the four scales of
// consecutive tokens leave as one 16-byte store (scale is [blocks][ld_scale],
// ld_scale a multiple of 4 and at least T rounded up to 4).  Called by whole
// warps; a half-warp with kb outside [0, nb) only takes part in the shuffles.
__device__ __forceinline__ void fp8_quant_rows4(const __nv_bfloat16* __restrict__ X, int64_t T, int d,
                                                int64_t ldx, uint8_t* __restrict__ q,
                                                float* __restrict__ scale, int64_t ld_scale,
                                                int64_t t0, int kb) {
  const int hl = threadIdx.x & 15;
  const int nb = (d + kFp8Block - 1) / kFp8Block;
  const int col = kb * kFp8Block + 8 * hl;
  const bool in = kb < nb && col < d;
  uint4 v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v[r] = make_uint4(0u, 0u, 0u, 0u);
    if (in && t0 + r < T) v[r] = __ldcs(reinterpret_cast<const uint4*>(X + (t0 + r) * ldx + col));
  }
  float sc[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint2 c;
    sc[r] = fp8_quant_half_warp(v[r], c);
    if (in && t0 + r < T) *reinterpret_cast<uint2*>(q + (t0 + r) * d + col) = c;
  }
  if (hl == 0 && kb < nb)
    *reinterpret_cast<float4*>(scale + kb * ld_scale + t0) =
        make_float4(sc[0], t0 + 1 < T ? sc[1] : 0.f, t0 + 2 < T ? sc[2] : 0.f, t0 + 3 < T ? sc[3] : 0.f);
}

__global__ void __launch_bounds__(256) fp8_quant_act_kernel(const __nv_bfloat16* __restrict__ X,
                                                            int64_t T, int d, int64_t ldx,
                                                            uint8_t* __restrict__ q,
                                                            float* __restrict__ scale,
                                                            int64_t ld_scale) {
  pdl_wait();
  pdl_launch_dependents();
  fp8_quant_rows4(X, T, d, ldx, q, scale, ld_scale, static_cast<int64_t>(blockIdx.x) * 4,
                  static_cast<int>(blockIdx.y * (blockDim.x >> 4) + (threadIdx.x >> 4)));
}

cudaError_t launch_fp8_quant_act(const void* X, int64_t T, int64_t d, int64_t ldx, uint8_t* q,
                                 float* scale, int64_t ld_scale, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const int64_t nb = (d + kFp8Block - 1) / kFp8Block;
  const int64_t gy = (nb + 15) / 16;
  int64_t hws = (nb + gy - 1) / gy;
  hws += hws & 1;                      // whole warps
  return launch_pdl(fp8_quant_act_kernel,
                    dim3(static_cast<unsigned>((T + 3) / 4), static_cast<unsigned>(gy)),
                    dim3(static_cast<unsigned>(16 * hws)), 0, stream,
                    static_cast<const __nv_bfloat16*>(X), T, static_cast<int>(d), ldx, q, scale,
                    ld_scale);
}

// One block per 128 x 128 tile of a weight (grid z: matrices of a stack):
// the tile stays in registers between its maximum and its codes.
__global__ void __launch_bounds__(256) fp8_pack_weight_kernel(const __nv_bfloat16* __restrict__ W,
                                                              int rows, int cols, int64_t ldw,
                                                              uint8_t* __restrict__ q,
                                                              float* __restrict__ scale) {
  __shared__ uint32_t red[8];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t e = blockIdx.z;
  const int c0 = blockIdx.x * kFp8Block + 8 * (threadIdx.x & 15);
  const int r0 = blockIdx.y * kFp8Block + (threadIdx.x >> 4);
  const __nv_bfloat16* we = W + e * rows * ldw;
  uint8_t* qe = q + e * rows * static_cast<int64_t>(cols);
  uint4 v[8];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && c0 < cols)
      v[i] = *reinterpret_cast<const uint4*>(we + static_cast<int64_t>(r) * ldw + c0);
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                             __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, red[i]);
  const uint32_t eb = f8_scale_exp(max(m & 0xFFFFu, m >> 16) << 16);
  const float inv = f8_inv_scale(eb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r < rows && c0 < cols) {
      uint32_t a = 0u, b = 0u;
      if (eb != 0u) {
        a = cvt_e4m3x4(bf16_lo_to_f32(v[i].x) * inv, bf16_hi_to_f32(v[i].x) * inv,
                       bf16_lo_to_f32(v[i].y) * inv, bf16_hi_to_f32(v[i].y) * inv);
        b = cvt_e4m3x4(bf16_lo_to_f32(v[i].z) * inv, bf16_hi_to_f32(v[i].z) * inv,
                       bf16_lo_to_f32(v[i].w) * inv, bf16_hi_to_f32(v[i].w) * inv);
      }
      *reinterpret_cast<uint2*>(qe + static_cast<int64_t>(r) * cols + c0) = make_uint2(a, b);
    }
  }
  if (threadIdx.x == 0)
    scale[(e * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = f8_scale(eb);
}

cudaError_t launch_fp8_pack_weight(const void* W, int64_t ldw, int64_t rows, int64_t cols,
                                   int64_t experts, uint8_t* q, float* scale, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((cols + kFp8Block - 1) / kFp8Block),
                  static_cast<unsigned>((rows + kFp8Block - 1) / kFp8Block),
                  static_cast<unsigned>(experts));
  return launch_pdl(fp8_pack_weight_kernel, grid, dim3(256), 0, stream,
                    static_cast<const __nv_bfloat16*>(W), static_cast<int>(rows),
                    static_cast<int>(cols), ldw, q, scale);
}

}  // namespace w4a4
