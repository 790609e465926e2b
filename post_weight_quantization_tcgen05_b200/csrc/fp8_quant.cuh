// The e4m3 quantiser of one block, shared by the kernels that write e4m3 codes.
//
// A block's absolute maximum a gives the stored scale s = fp32(a / 448) and the factor
// r = fp32(448 / a); a code is the e4m3 value next to fp32(x r) (ties to even, saturating).  The
// product by r replaces a division by s in every element; the two differ by at most two roundings
// of fp32, which moves a code only where x / s lies within 2^-23 of a tie.  a == 0 gives s = 0 and
// zero codes; 0 < a < 2^-100 takes a = 2^-100, so that r stays finite.  The maximum is taken over
// the bit patterns of |x|, which order NaN above infinity above every number: a block that holds
// either gets a non-finite scale, and all of it dequantises to NaN or infinity, never to a
// plausible number.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"

namespace hq {

constexpr int kFp8Block = 128;  // columns (and, for weights, rows) of one scale

inline int64_t fp8_pitch(int64_t K) { return ceil_div(K, 16) * 16; }  // bytes of a row of codes

__device__ __forceinline__ uint32_t fp8_abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// scale and factor of a block from the bits of its absolute maximum
__device__ __forceinline__ void fp8_scale(uint32_t amax_bits, float& scale, float& factor) {
  float a = __uint_as_float(amax_bits);
  if (amax_bits == 0) {
    scale = 0.f;
    factor = 0.f;
    return;
  }
  if (a < 0x1p-100f) a = 0x1p-100f;  // false for NaN
  scale = __fdiv_rn(a, 448.f);
  factor = __fdiv_rn(448.f, a);
}

// 16 codes (in memory order) of 16 values
__device__ __forceinline__ uint4 fp8_codes16(const float (&v)[16], float factor) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * factor, v[4 * i + 1] * factor), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * factor, v[4 * i + 3] * factor),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 consecutive values row[col .. col + 15] as fp32, zero at and past column K.  `vec`: the base is
// 16-byte aligned and so is every row (16-byte loads).
__device__ __forceinline__ void fp8_load16(const __nv_bfloat16* row, int64_t col, int64_t K, bool vec, float (&v)[16]) {
  if (vec && col + 16 <= K) {
    const uint4* p = reinterpret_cast<const uint4*>(row + col);
    const uint4 a = __ldg(p), b = __ldg(p + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = col + i < K ? __bfloat162float(row[col + i]) : 0.f;
}

__device__ __forceinline__ void fp8_load16(const float* row, int64_t col, int64_t K, bool vec, float (&v)[16]) {
  if (vec && col + 16 <= K) {
    const float4* p = reinterpret_cast<const float4*>(row + col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldg(p + i);
      v[4 * i] = a.x;
      v[4 * i + 1] = a.y;
      v[4 * i + 2] = a.z;
      v[4 * i + 3] = a.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = col + i < K ? row[col + i] : 0.f;
}

__device__ __forceinline__ uint32_t fp8_amax16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, fp8_abs_bits(v[i]));
  return m;
}

// One lane's 16 values of a 1 x 128 block that 8 consecutive lanes hold together: codes, and the
// block's scale (the same in all 8 lanes).  All 32 lanes call it.
__device__ __forceinline__ uint4 fp8_quantise_row16(const float (&v)[16], float& scale) {
  uint32_t m = fp8_amax16(v);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  float factor;
  fp8_scale(m, scale, factor);
  return fp8_codes16(v, factor);
}

}  // namespace hq
