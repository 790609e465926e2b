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

// Whether the rows of K values from X on start at 16-byte boundaries.
template <typename T>
inline bool fp8_aligned(const void* X, int64_t K) {
  return aligned(X, 16) && K * static_cast<int64_t>(sizeof(T)) % 16 == 0;
}

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

// 16 consecutive values of a matrix [begin, end) as they lie in memory, so that the loads of several can
// be on their way at once: load, then align, then values.  Where they do not start at a 16-byte boundary
// the aligned 16-byte pieces that hold them are loaded, one more than at a boundary, and align shifts
// them down (by words, then by half a word).  Pieces that would reach outside the matrix, and a row's
// last values (`left` < 16), are read one by one; values past `left` are zero.  kAligned: every row starts
// at a 16-byte boundary (fewer registers: fp32 weights 66 us instead of 92 us at 17408 x 5120).
template <typename T, bool kAligned>
struct Raw16 {
  static constexpr int kWords = 16 * sizeof(T) / 4;  // 8 (bf16) or 16 (fp32)
  static constexpr int kMore = kAligned ? 0 : 4;
  uint32_t w[kWords + kMore];
  uint32_t off;  // bytes past the boundary

  __device__ __forceinline__ void load(const T* begin, const T* end, const T* p, int64_t left) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    off = kAligned ? 0 : static_cast<uint32_t>(at & 15);
    const uint4* q = reinterpret_cast<const uint4*>(at - off);
    if (left >= 16 && (kAligned || (at - off >= reinterpret_cast<uintptr_t>(begin) &&
                                    at - off + 4 * kWords + (off != 0 ? 16 : 0) <= reinterpret_cast<uintptr_t>(end)))) {
#pragma unroll
      for (int i = 0; i < (kWords + kMore) / 4; ++i) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (i < kWords / 4 || off != 0) a = __ldg(q + i);
        w[4 * i] = a.x;
        w[4 * i + 1] = a.y;
        w[4 * i + 2] = a.z;
        w[4 * i + 3] = a.w;
      }
      return;
    }
    off = 0;
#pragma unroll
    for (int i = 0; i < kWords + kMore; ++i) w[i] = 0;
    if (left <= 0) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i >= left) continue;
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(__ldg(p + i));
      else
        w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p) + i)) << (16 * (i & 1));
    }
  }

  __device__ __forceinline__ void align() {
    if constexpr (!kAligned) {
      if (off == 0) return;
#pragma unroll
      for (int i = 0; i < kWords + 3; ++i) w[i] = (off & 4) ? w[i + 1] : w[i];
#pragma unroll
      for (int i = 0; i < kWords + 1; ++i) w[i] = (off & 8) ? w[i + 2] : w[i];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = (off & 2) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
      }
    }
  }

  __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 4)
        v[i] = __uint_as_float(w[i]);
      else
        v[i] = __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
  }
};

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
