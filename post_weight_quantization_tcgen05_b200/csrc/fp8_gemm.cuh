// What the kernels of the e4m3 product share: their arguments and the tiles of the experts' rows.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8_quant.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace hq {
namespace fp8 {

constexpr int kSMs = 148;
constexpr int kBK = kFp8Block;  // columns of a pipeline stage: one scale block
constexpr int kBand = 16;       // row tiles of a band (the order of the tiles)

struct Tile {
  int e, m0, m1, n0;  // expert, rows m0 .. m1 - 1, first column
};
struct GemmArgs {
  void* Y;
  int rows;             // rows of A and Y
  int N, K;
  int kblocks, nblocks;  // ceil(K / 128), ceil(N / 128)
  const float* a_scales;  // [kblocks][rows]
  const float* w_scales;  // [E][nblocks][kblocks]
  const int* offsets;     // [E + 1] row ranges of the experts (NULL: one matrix for all rows)
  int E;
  int y_aligned;          // rows of Y are 16-byte aligned (its tensor map is valid)
  int* status;
  // read by the kernels' kTimeout variants only, which run the test of the timeout path (as arguments
  // of every call they cost 0.1 to 0.2 us: 384 x 5120 x 5120 17.67 -> 17.87 us)
  long long wait_limit;  // cycles a pipeline wait may take before the CTA gives up
  int withhold_stage;    // -1, or a ring stage whose first release the MMA issuer skips
};

// An expert's rows.  Offsets are device data: a range outside [0, rows] is cut to it and an inverted
// one is empty, so no row index leaves Y.
__device__ __forceinline__ void expert_range(const GemmArgs& a, int e, int& r0, int& r1) {
  if (a.offsets == nullptr) {
    r0 = 0;
    r1 = a.rows;
    return;
  }
  r0 = min(max(a.offsets[e], 0), a.rows);
  r1 = min(max(a.offsets[e + 1], r0), a.rows);
}

template <bool kTimeout>
__device__ __forceinline__ long long wait_limit(const GemmArgs& a) {
  return kTimeout ? a.wait_limit : kWaitLimitCycles;
}

// All threads: fills start[0 .. E] with tiles of BM rows; valid after the next barrier.  Ranges that do
// not overlap have rows / BM + E tiles at most; the sums stop there, so that offsets that name rows again
// and again leave no index outside 32 bits, and no more tiles than the launch allows for.
template <int BM>
__device__ __forceinline__ void expert_tiles(const GemmArgs& a, int* start) {
  if (a.offsets == nullptr) {  // one matrix for all rows
    if (threadIdx.x == 0) {
      start[0] = 0;
      start[1] = (a.rows + BM - 1) / BM;
    }
    return;
  }
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    int r0, r1;
    expert_range(a, e, r0, r1);
    start[e + 1] = (r1 - r0 + BM - 1) / BM;
  }
  if (threadIdx.x == 0) start[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = (a.E + 31) / 32, e0 = threadIdx.x * per;
    const int most = a.rows / BM + a.E;
    int sum = 0;
    for (int e = e0; e < e0 + per && e < a.E; ++e) sum = min(sum + start[e + 1], most);
    int before = sum;
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, off);
      if (static_cast<int>(threadIdx.x) >= off) before = min(before + y, most);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);  // the lanes before this one
    if (threadIdx.x == 0) before = 0;
    for (int e = e0; e < e0 + per && e < a.E; ++e) {
      before = min(before + start[e + 1], most);
      start[e + 1] = before;
    }
  }
}

// Tile t, in bands of kBand row tiles, inside a band column by column, so that the tiles in flight
// share their operands through L2.
template <int BM, int BN>
__device__ __forceinline__ Tile tile_at(const GemmArgs& a, const int* start, int t) {
  const int tiles_m = start[a.E], tiles_n = (a.N + BN - 1) / BN;
  const int per_band = kBand * tiles_n;
  const int band = t / per_band;
  const int in_band = t - band * per_band;
  const int h = min(kBand, tiles_m - band * kBand);
  const int mt = band * kBand + in_band % h;
  int lo = 0, hi = a.E - 1;  // the last expert whose first row tile is at or before mt
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (start[mid] <= mt)
      lo = mid;
    else
      hi = mid - 1;
  }
  // experts without rows share their successor's start: the search ends at the last of them, which
  // is the one with rows
  int r0, r1;
  expert_range(a, lo, r0, r1);
  Tile x;
  x.e = lo;
  x.m0 = r0 + (mt - start[lo]) * BM;
  x.m1 = min(r1, x.m0 + BM);
  x.n0 = in_band / h * BN;
  return x;
}

// Tiles of bm rows x bn columns at most: an expert's rows may leave one partial row tile each.
inline int64_t most_tiles(const Fp8Gemm& p, int64_t bm, int64_t bn) {
  return (p.rows / bm + (p.offsets != nullptr ? p.E : 1)) * ceil_div(p.N, bn);
}

// The kernel arguments and the tensor maps of both operands, boxes of box_a and box_w rows.
inline hq_status gemm_args(const Fp8Gemm& p, int64_t tiles, uint32_t box_a, uint32_t box_w, GemmArgs& a,
                           CUtensorMap& map_a, CUtensorMap& map_w) {
  const int64_t kblocks = ceil_div(p.K, kFp8Block);
  if (tiles * kblocks > 0x7FFFFFFF) return HQ_ERR_UNSUPPORTED;  // the kernels count blocks in 32 bits
  const uint64_t pitch = static_cast<uint64_t>(fp8_pitch(p.K));
  a.Y = p.Y;
  a.rows = static_cast<int>(p.rows);
  a.N = static_cast<int>(p.N);
  a.K = static_cast<int>(p.K);
  a.kblocks = static_cast<int>(kblocks);
  a.nblocks = static_cast<int>(ceil_div(p.N, kFp8Block));
  a.a_scales = p.a_scales;
  a.w_scales = p.w_scales;
  a.offsets = p.offsets;
  a.E = static_cast<int>(p.E);
  a.y_aligned = aligned(p.Y, 16) && p.N * (p.y_dtype == HQ_F32 ? 4 : 2) % 16 == 0;
  a.status = p.status;
  a.wait_limit = p.wait_limit;
  a.withhold_stage = p.withhold_stage;
  if (!make_tmap_2d(&map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.a_codes, static_cast<uint64_t>(p.K),
                    static_cast<uint64_t>(p.rows), pitch, kBK, box_a) ||
      !make_tmap_2d(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w_codes, static_cast<uint64_t>(p.K),
                    static_cast<uint64_t>(p.E * p.N), pitch, kBK, box_w))
    return HQ_ERR_CUDA;
  return HQ_OK;
}

// Launches a product's kernel: `cluster` CTAs to a cluster, and, after the kernel that quantises its
// rows, as its dependent (the kernel calls pdl_wait before it touches codes or scales of A).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_product(const Fp8Gemm& p, void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem,
                                  unsigned cluster, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (p.chained) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// fp8_gemm_few.cu: for few rows, in tiles of 16 or 64.  With p.X (few_quantises(p), tiles of 16) the
// rows are quantised by the kernel itself.
bool few_quantises(const Fp8Gemm& p);
hq_status gemm_few(const Fp8Gemm& p, int tile_rows, cudaStream_t s);

}  // namespace fp8
}  // namespace hq
