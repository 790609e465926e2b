// Y = A W^T on e4m3 codes with block scales: A rows have one fp32 scale per 128 columns, W one per
// 128 x 128 block, so
//   Y[m, n] = sum_b sa[b, m] sw[n / 128, b] sum_{k in block b} A[m, k] W[n, k],
// for one weight matrix, or for the rows of every expert with that expert's matrix.
//
// The inner sum is exact to the tensor core's fp32 accumulation (kind::f8f6f4, four MMAs of 32
// columns); it leaves TMEM after every block of 128 columns, is scaled by sa sw and added in fp32
// registers.  So the accumulator restarts at every block, and the epilogue warps read and scale
// one while the tensor core fills the other (two accumulators).
//
// One CTA per SM walks 128 x 128 tiles of Y; warp 0 loads 128 x 128 e4m3 boxes of A and W by TMA
// (128-byte swizzle, K-major) into a ring of 32 KB stages, one stage per scale block; warp 1 issues
// the MMAs; warps 2-9 (two per TMEM lane quadrant, 64 columns each) scale, add and store.  Columns
// at and past K read as zeros (the tensor map's extent is K, not the row pitch), as do rows past
// the operands' ends.  A tile of an expert that ends inside it computes rows of the next expert as
// well (against the wrong matrix) and does not store them.
//
// Every wait is bounded: on expiry the CTA records HQ_ERR_TIMEOUT, waits (bounded) for its
// in-flight TMA and MMA work, frees TMEM and returns.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8_quant.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace hq {
namespace {

constexpr int kBM = 128, kBN = 128, kBK = kFp8Block;
constexpr int kStages = 6;
constexpr int kStageBytes = (kBM + kBN) * kBK;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kSMs = 148;
constexpr int kBand = 16;  // tile rows of a band (the order of the tiles)

struct GemmArgs {
  void* Y;
  int rows;             // rows of A and Y
  int N, K;
  int kblocks, nblocks;  // ceil(K / 128), ceil(N / 128)
  const float* a_scales;  // [kblocks][rows]
  const float* w_scales;  // [E][nblocks][kblocks]
  const int* offsets;     // [E + 1] row ranges of the experts (NULL: one matrix for all rows)
  int E;
  int* status;
};

// Row tiles before each expert: start[e], with start[E] the total.  Offsets are device data: a
// range outside [0, rows] is cut to it and an inverted one is empty, so no row index leaves Y.
__device__ __forceinline__ void expert_range(const GemmArgs& a, int e, int& r0, int& r1) {
  if (a.offsets == nullptr) {
    r0 = 0;
    r1 = a.rows;
    return;
  }
  r0 = min(max(a.offsets[e], 0), a.rows);
  r1 = min(max(a.offsets[e + 1], r0), a.rows);
}

// All threads: fills start[0 .. E].
__device__ __forceinline__ void expert_tiles(const GemmArgs& a, int* start) {
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    int r0, r1;
    expert_range(a, e, r0, r1);
    start[e + 1] = (r1 - r0 + kBM - 1) / kBM;
  }
  if (threadIdx.x == 0) start[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = (a.E + 31) / 32, e0 = threadIdx.x * per;
    int sum = 0;
    for (int e = e0; e < e0 + per && e < a.E; ++e) sum += start[e + 1];
    int before = sum;
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, off);
      if (static_cast<int>(threadIdx.x) >= off) before += y;
    }
    before -= sum;
    for (int e = e0; e < e0 + per && e < a.E; ++e) {
      before += start[e + 1];
      start[e + 1] = before;
    }
  }
}

struct Tile {
  int e, m0, m1, n0;  // expert, its rows m0 .. m1 - 1 of this tile, first column
};

// Tiles in bands of kBand row tiles, inside a band column by column, so that the tiles in flight
// share their operands through L2.
__device__ __forceinline__ Tile tile_at(const GemmArgs& a, const int* start, int tiles_n, int64_t t) {
  const int tiles_m = start[a.E];
  const int64_t per_band = static_cast<int64_t>(kBand) * tiles_n;
  const int band = static_cast<int>(t / per_band);
  const int in_band = static_cast<int>(t - band * per_band);
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
  x.m0 = r0 + (mt - start[lo]) * kBM;
  x.m1 = min(r1, x.m0 + kBM);
  x.n0 = in_band / h * kBN;
  return x;
}

template <typename TY>
__device__ __forceinline__ void store_row(TY* y, int col, int N, bool vec, const float (&acc)[64]);

template <>
__device__ __forceinline__ void store_row<float>(float* y, int col, int N, bool vec, const float (&acc)[64]) {
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    if (vec && col + i + 4 <= N) {
      *reinterpret_cast<float4*>(y + col + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + i + k < N) y[col + i + k] = acc[i + k];
    }
  }
}

template <>
__device__ __forceinline__ void store_row<__nv_bfloat16>(__nv_bfloat16* y, int col, int N, bool vec,
                                                         const float (&acc)[64]) {
#pragma unroll
  for (int i = 0; i < 64; i += 8) {
    if (vec && col + i + 8 <= N) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[i + 2 * k], acc[i + 2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(y + col + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + i + k < N) y[col + i + k] = __float2bfloat16_rn(acc[i + k]);
    }
  }
}

constexpr int kSmem = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/ + (kMaxExperts + 1) * 4;

template <typename TY>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW, GemmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* accf = empty + kStages;  // [2] accumulator filled
  uint64_t* acce = accf + 2;         // [2] accumulator drained
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* start = reinterpret_cast<int*>(smem + kStages * kStageBytes + 256);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&accf[a], 1);
      ptx::mbar_init(&acce[a], kEpiWarps);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 2 * kBN);
    ptx::tmem_relinquish();
  }
  expert_tiles(args, start);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles_n = (args.N + kBN - 1) / kBN;
  const int64_t tiles = static_cast<int64_t>(start[args.E]) * tiles_n;

  auto fail = [&]() {
    *abort_flag = 1;
    record_status(args.status, HQ_ERR_TIMEOUT);
  };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    ptx::prefetch_tensormap(&mapA);
    ptx::prefetch_tensormap(&mapW);
    int g = 0;  // stages issued by this CTA
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile x = tile_at(args, start, tiles_n, t);
      const int w_row = x.e * args.N + x.n0;
      for (int k = 0; k < args.kblocks; ++k, ++g) {
        const int s = g % kStages;
        if (g >= kStages && !ptx::mbar_wait(&empty[s], ((g / kStages) - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + s * kStageBytes;
        (void)HQ_IN_BOUNDS(x.m0 < args.rows && x.n0 < args.N && k * kBK < args.K);
        ptx::mbar_arrive_expect_tx(&full[s], kStageBytes);
        ptx::tma_load_2d(sa, &mapA, k * kBK, x.m0, &full[s]);
        ptx::tma_load_2d(sa + kBM * kBK, &mapW, k * kBK, w_row, &full[s]);
      }
    }
    if (!ok) {
      fail();
      // let the copies already issued land before the CTA's shared memory goes away
      const int first = g > kStages ? g - kStages : 0;
      for (int k = first; k < g; ++k) ptx::mbar_wait(&full[k % kStages], (k / kStages) & 1, nullptr);
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kIdesc = ptx::idesc(ptx::kFmtE4M3, kBM, kBN, false, false);
    bool ok = true;
    int g = 0;  // blocks issued (stage g % kStages, accumulator g & 1)
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      for (int k = 0; k < args.kblocks; ++k, ++g) {
        const int s = g % kStages, acc = g & 1;
        if ((g >= 2 && !ptx::mbar_wait(&acce[acc], ((g >> 1) - 1) & 1, abort_flag)) ||
            !ptx::mbar_wait(&full[s], (g / kStages) & 1, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t dacc = tmem + static_cast<uint32_t>(acc * kBN);
        const uint32_t sa = ptx::smem_u32(smem + s * kStageBytes);
        const uint32_t sb = sa + kBM * kBK;
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk) {
          // K-major rows of 128 bytes, 8-row groups 1 KB apart (SBO); an MMA takes 32 bytes of each row
          const uint64_t ad = ptx::sdesc_sw128(sa + kk * 32, 16, 1024);
          const uint64_t bd = ptx::sdesc_sw128(sb + kk * 32, 16, 1024);
          ptx::mma_f8(dacc, ad, bd, kIdesc, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit(&empty[s]);
        ptx::mma_commit(&accf[acc]);
      }
    }
    if (!ok) {
      fail();
      ptx::mma_commit(drain);
      ptx::mbar_wait(drain, 0, nullptr);
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;         // TMEM lane quadrant this warp may access
    const int h = (warp - 2) >> 2;  // which 64-column half of the tile
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const bool vec = (reinterpret_cast<uintptr_t>(args.Y) & 15) == 0 && (args.N * static_cast<int64_t>(sizeof(TY))) % 16 == 0;
    bool ok = true;
    int g = 0;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile x = tile_at(args, start, tiles_n, t);
      const int row = x.m0 + q * 32 + lane;
      const bool live = row < x.m1;
      const float* sa = args.a_scales + row;  // + k * rows
      const float* sw = args.w_scales + (static_cast<int64_t>(x.e) * args.nblocks + x.n0 / kFp8Block) * args.kblocks;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      for (int k = 0; k < args.kblocks; ++k, ++g) {
        const float scale = live ? __ldg(sa + static_cast<int64_t>(k) * args.rows) * __ldg(sw + k) : 0.f;
        const int b = g & 1;
        if (!ptx::mbar_wait(&accf[b], (g >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        uint32_t r0[32], r1[32];
        const uint32_t from = tmem + lane_off + static_cast<uint32_t>(b * kBN + h * 64);
        ptx::tmem_ld32_nowait(from, r0);
        ptx::tmem_ld32_nowait(from + 32, r1);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&acce[b]);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          acc[i] = fmaf(scale, __uint_as_float(r0[i]), acc[i]);
          acc[32 + i] = fmaf(scale, __uint_as_float(r1[i]), acc[32 + i]);
        }
      }
      if (ok && live && HQ_IN_BOUNDS(row >= 0 && row < args.rows))
        store_row<TY>(static_cast<TY*>(args.Y) + static_cast<int64_t>(row) * args.N, x.n0 + h * 64, args.N, vec, acc);
    }
    if (!ok) fail();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 2 * kBN);
  }
}

template <typename TY>
hq_status run_gemm(const Fp8Gemm& p, cudaStream_t s) {
  CUtensorMap map_a, map_w;
  const uint64_t pitch = static_cast<uint64_t>(fp8_pitch(p.K));
  if (!make_tmap_2d(&map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.a_codes, static_cast<uint64_t>(p.K),
                    static_cast<uint64_t>(p.rows), pitch, kBK, kBM) ||
      !make_tmap_2d(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w_codes, static_cast<uint64_t>(p.K),
                    static_cast<uint64_t>(p.E * p.N), pitch, kBK, kBN))
    return HQ_ERR_CUDA;
  HQ_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<TY>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  GemmArgs a{};
  a.Y = p.Y;
  a.rows = static_cast<int>(p.rows);
  a.N = static_cast<int>(p.N);
  a.K = static_cast<int>(p.K);
  a.kblocks = static_cast<int>(ceil_div(p.K, kFp8Block));
  a.nblocks = static_cast<int>(ceil_div(p.N, kFp8Block));
  a.a_scales = p.a_scales;
  a.w_scales = p.w_scales;
  a.offsets = p.offsets;
  a.E = static_cast<int>(p.E);
  a.status = p.status;
  // an expert's rows may leave one partial row tile each
  const int64_t most = (p.rows / kBM + (p.offsets != nullptr ? p.E : 1)) * ceil_div(p.N, kBN);
  const int grid = static_cast<int>(most < kSMs ? most : kSMs);
  fp8_gemm_kernel<TY><<<grid, kThreads, kSmem, s>>>(map_a, map_w, a);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

}  // namespace

hq_status launch_fp8_gemm(const Fp8Gemm& p, cudaStream_t s) {
  if (p.rows == 0) return HQ_OK;
  return p.y_dtype == HQ_F32 ? run_gemm<float>(p, s) : run_gemm<__nv_bfloat16>(p, s);
}

}  // namespace hq
