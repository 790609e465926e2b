// Quantisation to e4m3 with one fp32 scale per block: 1 x 128 for activations (rows), 128 x 128
// for weights.  One pass over the input: a block's values stay in registers between its maximum
// and its codes.  A lane holds 16 consecutive values, so that its codes leave in one 16-byte
// store and 8 lanes cover a row of a block.
#include "common.cuh"
#include "fp8_quant.cuh"
#include "kernels.cuh"

namespace hq {

// Rows: a warp takes 512 columns (four blocks) of one row, the 8 warps of a CTA 8 consecutive
// rows, so that the scales, stored [block][row], leave in 32-byte pieces.
constexpr int kFp8RowsPerCta = 8;
constexpr int kFp8ColsPerWarp = 512;

template <typename TX>
__global__ void __launch_bounds__(32 * kFp8RowsPerCta)
    fp8_rows_kernel(const TX* __restrict__ X, int64_t M, int64_t K, int64_t pitch, bool vec,
                    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_launch_dependents();  // a product launched behind this kernel may set itself up meanwhile
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kFp8RowsPerCta + (threadIdx.x >> 5);
  if (row >= M) return;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * kFp8ColsPerWarp + lane * 16;
  float v[16];
  fp8_load16(X + row * K, col, K, vec, v);
  float scale;
  const uint4 c = fp8_quantise_row16(v, scale);
  if (col < pitch && HQ_IN_BOUNDS(col + 16 <= pitch)) *reinterpret_cast<uint4*>(codes + row * pitch + col) = c;
  if ((lane & 7) == 0 && col < K) scales[(col / kFp8Block) * M + row] = scale;
}

// Weights: a CTA takes one 128 x 128 block; a thread holds 16 columns of 4 rows 32 apart.
template <typename TX>
__global__ void __launch_bounds__(256)
    fp8_blocks_kernel(const TX* __restrict__ W, int64_t N, int64_t K, int64_t pitch, bool vec,
                      uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t warp_max[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int64_t col = kb * kFp8Block + (threadIdx.x & 7) * 16;
  const int64_t row0 = nb * kFp8Block + (threadIdx.x >> 3);
  float v[4][16];
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = row0 + 32 * p;
    fp8_load16(W + (e * N + (row < N ? row : 0)) * K, col, row < N ? K : 0, vec, v[p]);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) m = max(m, fp8_amax16(v[p]));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
  float scale, factor;
  fp8_scale(m, scale, factor);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = row0 + 32 * p;
    if (row < N && col < pitch && HQ_IN_BOUNDS(col + 16 <= pitch))
      *reinterpret_cast<uint4*>(codes + (e * N + row) * pitch + col) = fp8_codes16(v[p], factor);
  }
  if (threadIdx.x == 0) scales[(e * gridDim.y + nb) * gridDim.x + kb] = scale;
}

template <typename TX>
static bool fp8_vec(const void* X, int64_t K) {
  return aligned(X, 16) && (K * static_cast<int64_t>(sizeof(TX))) % 16 == 0;
}

template <typename TX>
static hq_status fp8_rows_typed(const void* X, int64_t M, int64_t K, uint8_t* codes, float* scales, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(M, kFp8RowsPerCta)), static_cast<unsigned>(ceil_div(K, kFp8ColsPerWarp)));
  fp8_rows_kernel<TX><<<grid, 32 * kFp8RowsPerCta, 0, s>>>(static_cast<const TX*>(X), M, K, fp8_pitch(K),
                                                           fp8_vec<TX>(X, K), codes, scales);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

hq_status launch_fp8_rows(const void* X, int x_dtype, int64_t M, int64_t K, uint8_t* codes, float* scales,
                          cudaStream_t s) {
  if (M == 0) return HQ_OK;
  return x_dtype == HQ_BF16 ? fp8_rows_typed<__nv_bfloat16>(X, M, K, codes, scales, s)
                            : fp8_rows_typed<float>(X, M, K, codes, scales, s);
}

template <typename TX>
static hq_status fp8_blocks_typed(const void* W, int64_t E, int64_t N, int64_t K, uint8_t* codes, float* scales,
                                  cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(K, kFp8Block)), static_cast<unsigned>(ceil_div(N, kFp8Block)),
                  static_cast<unsigned>(E));
  fp8_blocks_kernel<TX><<<grid, 256, 0, s>>>(static_cast<const TX*>(W), N, K, fp8_pitch(K), fp8_vec<TX>(W, K), codes,
                                             scales);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

hq_status launch_fp8_blocks(const void* W, int w_dtype, int64_t E, int64_t N, int64_t K, uint8_t* codes, float* scales,
                            cudaStream_t s) {
  return w_dtype == HQ_BF16 ? fp8_blocks_typed<__nv_bfloat16>(W, E, N, K, codes, scales, s)
                            : fp8_blocks_typed<float>(W, E, N, K, codes, scales, s);
}

}  // namespace hq
