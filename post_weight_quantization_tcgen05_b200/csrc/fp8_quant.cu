// Quantisation to e4m3 with one fp32 scale per block: 1 x 128 for activations (rows), 128 x 128
// for weights.  One pass over the input: a block's values stay in registers between its maximum
// and its codes.  A lane holds 16 consecutive values, so that its codes leave in one 16-byte
// store and 8 lanes cover a row of a block.  Bound by DRAM.  On the device: rows 16384 x 5120 bf16
// 40.3 us (6.3 TB/s), fp32 64 us (6.6 TB/s), bf16 rows that start at no 16-byte boundary 56 us (4.5 TB/s:
// five loads instead of four and the shifts); weights 17408 x 5120 bf16 42.5 us (6.3 TB/s), fp32 66 us.
#include "common.cuh"
#include "fp8_quant.cuh"
#include "kernels.cuh"

namespace hq {

// Rows: a warp takes 512 columns (four blocks) of two rows, both on their way at once; the 8 warps of a
// CTA 16 consecutive rows, so that the scales, stored [block][row], leave in 32-byte pieces.
constexpr int kFp8RowsPerCta = 16;
constexpr int kFp8ColsPerWarp = 512;

template <bool kAligned, typename TX>
__global__ void __launch_bounds__(256, kAligned && sizeof(TX) == 2 ? 6 : 4)
    fp8_rows_kernel(const TX* __restrict__ X, int64_t M, int64_t K, int64_t pitch, uint8_t* __restrict__ codes,
                    float* __restrict__ scales) {
  pdl_launch_dependents();  // a product launched behind this kernel may set itself up meanwhile
  const int lane = threadIdx.x & 31;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kFp8RowsPerCta + (threadIdx.x >> 5);
  const int64_t col = static_cast<int64_t>(blockIdx.y) * kFp8ColsPerWarp + lane * 16;
  Raw16<TX, kAligned> raw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (row0 + 8 * i < M) raw[i].load(X, X + M * K, X + (row0 + 8 * i) * K + col, K - col);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = row0 + 8 * i;
    if (row >= M) break;  // the whole warp
    float v[16], scale;
    raw[i].align();
    raw[i].values(v);
    const uint4 c = fp8_quantise_row16(v, scale);
    if (col < pitch && HQ_IN_BOUNDS(col + 16 <= pitch)) *reinterpret_cast<uint4*>(codes + row * pitch + col) = c;
    if ((lane & 7) == 0 && col < K) scales[(col / kFp8Block) * M + row] = scale;
  }
}

// Weights: a CTA takes one 128 x 128 block; a thread holds 16 columns of 4 rows 32 apart, kept as they
// lie in memory (half the registers of bf16, twice the CTAs on an SM).
template <bool kAligned, typename TX>
__global__ void __launch_bounds__(256, sizeof(TX) == 2 ? 3 : 2)
    fp8_blocks_kernel(const TX* __restrict__ W, int64_t N, int64_t K, int64_t pitch, uint8_t* __restrict__ codes,
                      float* __restrict__ scales) {
  __shared__ uint32_t warp_max[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int64_t col = kb * kFp8Block + (threadIdx.x & 7) * 16;
  const int64_t row0 = nb * kFp8Block + (threadIdx.x >> 3);
  const TX* const end = W + gridDim.z * N * K;
  Raw16<TX, kAligned> raw[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = row0 + 32 * p;
    raw[p].load(W, end, W + (e * N + (row < N ? row : 0)) * K + col, row < N ? K - col : 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float v[16];
    raw[p].align();
    raw[p].values(v);
    m = max(m, fp8_amax16(v));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
  float scale, factor;
  fp8_scale(m, scale, factor);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = row0 + 32 * p;
    float v[16];
    raw[p].values(v);
    if (row < N && col < pitch && HQ_IN_BOUNDS(col + 16 <= pitch))
      *reinterpret_cast<uint4*>(codes + (e * N + row) * pitch + col) = fp8_codes16(v, factor);
  }
  if (threadIdx.x == 0) scales[(e * gridDim.y + nb) * gridDim.x + kb] = scale;
}

template <typename TX>
static hq_status fp8_rows_typed(const void* X, int64_t M, int64_t K, uint8_t* codes, float* scales, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(M, kFp8RowsPerCta)), static_cast<unsigned>(ceil_div(K, kFp8ColsPerWarp)));
  const auto kernel = fp8_aligned<TX>(X, K) ? fp8_rows_kernel<true, TX> : fp8_rows_kernel<false, TX>;
  kernel<<<grid, 256, 0, s>>>(static_cast<const TX*>(X), M, K, fp8_pitch(K), codes, scales);
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
  const auto kernel = fp8_aligned<TX>(W, K) ? fp8_blocks_kernel<true, TX> : fp8_blocks_kernel<false, TX>;
  kernel<<<grid, 256, 0, s>>>(static_cast<const TX*>(W), N, K, fp8_pitch(K), codes, scales);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

hq_status launch_fp8_blocks(const void* W, int w_dtype, int64_t E, int64_t N, int64_t K, uint8_t* codes, float* scales,
                            cudaStream_t s) {
  return w_dtype == HQ_BF16 ? fp8_blocks_typed<__nv_bfloat16>(W, E, N, K, codes, scales, s)
                            : fp8_blocks_typed<float>(W, E, N, K, codes, scales, s);
}

}  // namespace hq
