// The e4m3 product for few rows (a serving step), bound by reading the weights, and for few tiles.  The
// mathematics and the scaling after every block of 128 columns are those of fp8_gemm.cu, with the operands
// exchanged: 128 rows of W are the MMA's 128 rows, BT rows of A (16 or 64) its columns.  A block's accumulator is
// then BT columns of tensor memory, so 256 of them hold 16 or 4 accumulators and the hand-over to the
// epilogue, several hundred cycles, never holds up the loads; a stage takes 16 KB of W and 2 or 8 KB
// of A, and two CTAs on an SM keep 10 stages on their way.
//
// Where there are fewer tiles than CTAs the GPU holds, a cluster of up to 8 CTAs shares a tile, each
// taking a part of the K blocks.  At the end each leaves its sums in shared memory, and every CTA adds
// up the parts of some of the tile's rows of A, in the order of the CTAs, and stores them: no workspace,
// no second launch, the same result every time.
//
// Of hq_fp8_linear's activations, one to four rows are quantised here, where a CTA's part of K is 16
// blocks at most: the warps of a CTA turn the blocks of its part into codes in shared memory while the first
// weights are on their way.  Every tile's CTAs repeat that, but it reads little and saves a launch, which
// costs the host as long as the kernel takes.  Other rows (one of 17408 x 5120, whose 136 tiles leave two
// CTAs to each, 20 blocks a CTA) are quantised by a kernel of their own and this one launched as its
// dependent, with the first weights loaded meanwhile: for 16 rows of 5120 11.0 us against 13.2 us.
//
// hq_fp8_linear on the device, weights rotated through 1.2 GB so that all come from DRAM: 1 x 5120 x 5120
// 10.2 us, 1 x 17408 x 5120 and 1 x 5120 x 17408 19.3 us, 24 x 17408 x 5120 22 us; experts, 512 rows of
// 2560 x 5120, 39 of 48 of which have rows, 85 us (511 MB of weights, 6.0 TB/s).  All of these are about
// 6 us and the weights at 6.5 TB/s: the 6 us are the launch, the set-up (0.8 us before the first load), 3 us
// to the first weights and, where K is split, 1.2 us of the cluster's sums.  Experts' tiles do not split K:
// one token's 8 experts of 768 x 2048 take 11 us, of 2560 x 5120 23 us (4.6 TB/s).
//
// Per CTA: warp 0 loads, warp 1 issues the MMAs, warp 2 leaves the products of the scales in shared
// memory, warps 4-7 (one TMEM lane quadrant each) scale and add: a thread holds one row of W, that is a
// column of Y, for the BT rows of A.  Neighbouring lanes store neighbouring columns.
//
// Every wait is bounded, as in fp8_gemm.cu.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8_gemm.cuh"

namespace hq {
namespace fp8 {
namespace {

constexpr int kRows = 128;  // rows of W of a tile
constexpr int kEpiWarps = 4;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kCtasPerSM = 2;
constexpr int kTmemCols = 256;  // of the SM's 512
constexpr int kMaxSplit = 8;
// blocks whose scales are kept, handed over and given back by halves; loads run kFetch blocks ahead
constexpr int kScales = 8, kScaleHalf = kScales / 2;
constexpr int kFetch = kScaleHalf;
constexpr int kPlaces = 16;
static_assert(kPlaces > kScales + kFetch, "a tile's place is overwritten after the epilogue read it");

constexpr int kPanel = 16;  // blocks of A that a CTA quantises and keeps

template <int BT, bool kQuantise>
struct Shared {
  float scales[kQuantise ? kPanel : kScales][BT];
  Tile places[kPlaces];
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t accf[kTmemCols / BT];
  uint64_t acce[kTmemCols / BT];
  uint64_t scf[2], sce[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int start[kMaxExperts + 1];
};

template <int BT, bool kQuantise>
struct Few {
  static_assert(!kQuantise || BT == 16, "16 rows are quantised");
  static constexpr int kStageBytes = kRows * kBK + (kQuantise ? 0 : BT * kBK);
  static constexpr int kStages = BT < 64 && !kQuantise ? 5 : 4;
  static constexpr int kPanelBytes = kQuantise ? kPanel * BT * kBK : 0;
  static constexpr int kAccs = kTmemCols / BT;
  static constexpr int kSmem =
      kStages * kStageBytes + kPanelBytes + 1024 /*align*/ + static_cast<int>(sizeof(Shared<BT, kQuantise>));
  static_assert(kStages <= 8 && kSmem <= 232448 / kCtasPerSM - 1024, "two CTAs on an SM");
  static_assert(kRows * BT * 4 <= kStages * kStageBytes, "a tile's sums fit into the stages");
};

// grid: CTAs in clusters of `split`; cluster c takes tiles c, c + clusters, ...  TX: uint8_t (A's codes
// and scales are read), or the type of the activations X, which are quantised here; then BT == 16, there
// is a tile for every cluster, and a CTA's part of K has at most kPanel blocks.
template <int BT, typename TY, typename TX, bool kTimeout>
__global__ void __launch_bounds__(kThreads, kCtasPerSM)
    fp8_gemm_few_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW,
                        GemmArgs args, int split, const TX* __restrict__ X) {
  constexpr bool kQuantise = !std::is_same<TX, uint8_t>::value;
  using F = Few<BT, kQuantise>;
  constexpr int kStages = F::kStages, kStageBytes = F::kStageBytes, kAccs = F::kAccs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* panel = smem + kStages * kStageBytes;  // A's codes, if quantised here: 2 KB a block
  Shared<BT, kQuantise>& sh = *reinterpret_cast<Shared<BT, kQuantise>*>(panel + F::kPanelBytes);
  volatile int* abort_flag = &sh.abort;
  const long long limit = wait_limit<kTimeout>(args);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;

  // barriers by the lanes of warp 0: one after the other they take longer than the rest of the set-up
  if (warp == 0) {
    if (lane < kStages) {
      ptx::mbar_init(&sh.full[lane], 1);
      ptx::mbar_init(&sh.empty[lane], 1);
    }
    if (lane < kAccs) {
      ptx::mbar_init(&sh.accf[lane], 1);
      ptx::mbar_init(&sh.acce[lane], kEpiWarps);
    }
    if (lane < 2) {
      ptx::mbar_init(&sh.scf[lane], 1);
      ptx::mbar_init(&sh.sce[lane], kEpiWarps);
    }
    if (lane == 0) {
      ptx::mbar_init(&sh.drain, 1);
      sh.abort = 0;
      if (!kQuantise) ptx::prefetch_tensormap(&mapA);
      ptx::prefetch_tensormap(&mapW);
    }
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  expert_tiles<BT>(args, sh.start);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int tiles = sh.start[args.E] * ((args.N + kRows - 1) / kRows);
  const int first = blockIdx.x / split, step = gridDim.x / split;
  const int own = tiles > first ? (tiles - 1 - first) / step + 1 : 0;
  // this CTA's part of the K blocks, the same for every tile
  const int k0 = static_cast<int>(static_cast<int64_t>(rank) * args.kblocks / split);
  const int kn = static_cast<int>(static_cast<int64_t>(rank + 1) * args.kblocks / split) - k0;
  const int blocks = own * kn;  // they follow one another across tiles

  auto fail = [&]() {
    *abort_flag = 1;
    record_status(args.status, HQ_ERR_TIMEOUT);
  };

  bool ok = true;
  if constexpr (kQuantise) {
    // ------------------------------------------------------------ quantisation of A
    // Warp 0 starts the first weights on their way, the others take A: 8 lanes a block of 128 columns of
    // a row, 16 columns a lane.  16-byte part p of row r is kept at place p ^ (r % 8), as a TMA load with
    // the 128-byte swizzle would.
    const Tile x = tile_at<BT, kRows>(args, sh.start, own > 0 ? first : 0);
    if (warp == 0) {
      if (lane == 0) {
        sh.places[0] = x;
        for (int g = 0; g < kStages && g < blocks; ++g) {
          ptx::mbar_arrive_expect_tx(&sh.full[g], kRows * kBK);
          ptx::tma_load_2d(smem + g * kStageBytes, &mapW, (k0 + g) * kBK, x.n0, &sh.full[g]);
        }
      }
    } else {
      const float* sw = args.w_scales + static_cast<int64_t>(x.n0 / kFp8Block) * args.kblocks + k0;
      const int live = (x.m1 - x.m0) * blocks, c = lane & 7;  // blocks of the rows that are there
      for (int u = (warp - 1) * 4 + (lane >> 3); u < blocks * BT; u += (kThreads - 32) / 8) {
        const int r = u / kn, k = u - r * kn;
        const int64_t col = static_cast<int64_t>(k0 + k) * kBK + c * 16;
        Raw16<TX, false> raw;
        raw.load(X, X + static_cast<int64_t>(args.rows) * args.K,
                 X + static_cast<int64_t>(u < live ? x.m0 + r : 0) * args.K + col, u < live ? args.K - col : 0);
        const float scale_w = u < live && c == 0 ? __ldg(sw + k) : 0.f;
        float v[16], scale;
        raw.align();
        raw.values(v);
        const uint4 codes = fp8_quantise_row16(v, scale);
        *reinterpret_cast<uint4*>(panel + k * (BT * kBK) + r * kBK + ((c ^ (r & 7)) << 4)) = codes;
        if (c == 0) sh.scales[k][r] = scale * scale_w;
      }
    }
    ptx::fence_async_smem();  // the codes, to the tensor core
    __syncthreads();
  }
  if (warp == 0 && ptx::elect_one()) {
    // ------------------------------------------------------------ TMA producer
    bool waited = false;
    int g = 0;
    for (int i = 0; i < own && ok; ++i) {
      const Tile x = tile_at<BT, kRows>(args, sh.start, first + i * step);
      (void)HQ_IN_BOUNDS(x.m0 < args.rows && x.n0 < args.N);
      for (int k = 0; k < kn; ++k, ++g) {
        const int s = g % kStages;
        if (kQuantise && g < kStages) continue;  // on its way
        if (g >= kStages && !ptx::mbar_wait(&sh.empty[s], ((g / kStages) - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
        uint8_t* sw = smem + s * kStageBytes;
        ptx::mbar_arrive_expect_tx(&sh.full[s], kStageBytes);
        // the weights were there before the kernel that quantises A started
        ptx::tma_load_2d(sw, &mapW, (k0 + k) * kBK, x.e * args.N + x.n0, &sh.full[s]);
        if constexpr (!kQuantise) {
          if (!waited && g + 1 < kStages && g + 1 < blocks) continue;
          if (!waited) {
            pdl_wait();
            waited = true;
            // A's boxes of the stages so far
            for (int b = 0; b < g; ++b) {
              const Tile t = tile_at<BT, kRows>(args, sh.start, first + b / kn * step);
              ptx::tma_load_2d(smem + b * kStageBytes + kRows * kBK, &mapA, (k0 + b % kn) * kBK, t.m0, &sh.full[b]);
            }
          }
          ptx::tma_load_2d(sw + kRows * kBK, &mapA, (k0 + k) * kBK, x.m0, &sh.full[s]);
        }
      }
    }
    if (!ok) {
      fail();
      // let the copies already issued land before shared memory goes away
      for (int k = g > kStages ? g - kStages : 0; k < g; ++k)
        ptx::mbar_wait(&sh.full[k % kStages], (k / kStages) & 1, nullptr);
    }
  } else if (warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kIdesc = ptx::idesc(ptx::kFmtE4M3, kRows, BT, false, false);
    for (int g = 0; g < blocks; ++g) {
      const int s = g % kStages, b = g % kAccs;
      if (!ptx::mbar_wait(&sh.full[s], (g / kStages) & 1, abort_flag, limit) ||
          (g >= kAccs && !ptx::mbar_wait(&sh.acce[b], ((g / kAccs) - 1) & 1, abort_flag, limit))) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t dacc = tmem + static_cast<uint32_t>(b * BT);
      const uint32_t sw = ptx::smem_u32(smem + s * kStageBytes);
      const uint32_t sa = kQuantise ? ptx::smem_u32(panel + g * (BT * kBK)) : sw + kRows * kBK;
#pragma unroll
      for (int kk = 0; kk < kBK / 32; ++kk)
        // K-major rows of 128 bytes, 8-row groups 1 KB apart (SBO); an MMA takes 32 bytes of each row
        ptx::mma_f8(dacc, ptx::sdesc_sw128(sw + kk * 32, 16, 1024), ptx::sdesc_sw128(sa + kk * 32, 16, 1024), kIdesc,
                    kk > 0 ? 1u : 0u);
      ptx::mma_commit(&sh.accf[b]);
      if (!kTimeout || g != args.withhold_stage || rank != 0) ptx::mma_commit(&sh.empty[s]);
    }
    if (!ok) {
      fail();
      ptx::mma_commit(&sh.drain);
      ptx::mbar_wait(&sh.drain, 0, nullptr);
    }
  } else if (!kQuantise && warp == 2) {
    // ------------------------------------------------------------ scales
    pdl_wait();
    constexpr int kPer = (BT + 31) / 32;  // rows of A a lane fetches
    float sa[kFetch][kPer], sw[kFetch];
    Tile x{};
    int k = kn, i = -1;  // the block to fetch: the first of the tile after tile i
    auto fetch = [&](int f, int g) {
      if (g >= blocks) return;
      if (k == kn) {
        k = 0;
        ++i;
        x = tile_at<BT, kRows>(args, sh.start, first + i * step);
        // its place is read by the epilogue after its first block's scales are announced, later
        if (lane == 0) sh.places[i % kPlaces] = x;
      }
      // not __ldg: the kernel that writes these scales may have run beside this one until pdl_wait
      const float* col = args.a_scales + static_cast<int64_t>(k0 + k) * args.rows;
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int row = x.m0 + r * 32 + lane;
        sa[f][r] = row < x.m1 ? __ldcg(col + row) : 0.f;
      }
      sw[f] = __ldg(args.w_scales + (static_cast<int64_t>(x.e) * args.nblocks + x.n0 / kFp8Block) * args.kblocks + k0 + k);
      ++k;
    };
#pragma unroll
    for (int f = 0; f < kFetch; ++f) fetch(f, f);
    for (int g0 = 0; g0 < blocks; g0 += kScaleHalf) {
      const int half = (g0 / kScaleHalf) & 1;
      if (g0 >= kScales) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh.sce[half], ((g0 / kScales) - 1) & 1, abort_flag, limit));
        if (!ok) break;
      }
#pragma unroll
      for (int f = 0; f < kFetch; ++f) {
        if (g0 + f >= blocks) break;
#pragma unroll
        for (int r = 0; r < kPer; ++r)
          if (r * 32 + lane < BT) sh.scales[(g0 + f) % kScales][r * 32 + lane] = sa[f][r] * sw[f];
        fetch(f, g0 + f + kFetch);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.scf[half]);
    }
    if (!ok) fail();
  }

  if (warp < 4) {
    if (split > 1) {
      // the other warps' share of the clusters' two meetings below
      __syncwarp();
      ptx::cluster_sync();
      ptx::cluster_sync_relaxed();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quadrant this warp may access
    const uint32_t tmem_w = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int n = q * 32 + lane;  // this thread's row of the tile's 128 of W
    constexpr int kStep = BT < 32 ? BT : 32;
    int g = 0, left = 0;
    for (int i = 0; i < own && ok; ++i) {
      float acc[BT];
#pragma unroll
      for (int c = 0; c < BT; ++c) acc[c] = 0.f;
      for (int k = 0; k < kn; ++k, ++g) {
        const int b = g % kAccs;
        // the warp goes on or gives up as one: a wait may run out for some of its lanes only
        ok = __all_sync(0xffffffffu,
                        (kQuantise || g % kScaleHalf != 0 ||
                         ptx::mbar_wait(&sh.scf[(g / kScaleHalf) & 1], (g / kScales) & 1, abort_flag, limit)) &&
                            ptx::mbar_wait(&sh.accf[b], (g / kAccs) & 1, abort_flag, limit));
        if (!ok) break;
        ptx::tc_fence_after();
        const float4* scale = reinterpret_cast<const float4*>(sh.scales[kQuantise ? g : g % kScales]);
        const uint32_t from = tmem_w + static_cast<uint32_t>(b * BT);
        if (k == 0) left = sh.places[i % kPlaces].m1 - sh.places[i % kPlaces].m0;
#pragma unroll
        for (int c = 0; c < BT; c += kStep) {
          if (c >= left) break;  // rows that the tile does not have
          uint32_t r[kStep];
          if constexpr (kStep == 16)
            ptx::tmem_ld16_nowait(from + c, r);
          else
            ptx::tmem_ld32_nowait(from + c, r);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kStep; j += 4) {
            const float4 sc = scale[(c + j) / 4];
            ptx::fma2(acc[c + j], acc[c + j + 1], sc.x, sc.y, r[j], r[j + 1]);
            ptx::fma2(acc[c + j + 2], acc[c + j + 3], sc.z, sc.w, r[j + 2], r[j + 3]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        ptx::mbar_arrive_cluster(ptx::smem_u32(&sh.acce[b]), lane == 0);
        if (!kQuantise && g % kScaleHalf == kScaleHalf - 1)
          ptx::mbar_arrive_cluster(ptx::smem_u32(&sh.sce[(g / kScaleHalf) & 1]), lane == 0);
      }
      if (!ok) break;
      const Tile x = sh.places[i % kPlaces];
      const int col = x.n0 + n;
      if (split == 1) {
        TY* y = static_cast<TY*>(args.Y) + static_cast<int64_t>(x.m0) * args.N + col;
        if (col < args.N && HQ_IN_BOUNDS(x.m0 >= 0 && x.m1 <= args.rows)) {
#pragma unroll
          for (int c = 0; c < BT; ++c)
            if (c < left) y[static_cast<int64_t>(c) * args.N] = static_cast<TY>(acc[c]);
        }
      } else {
        // one tile per cluster: its blocks' operands have been used, the stages are free
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < BT; ++c) part[c * kRows + n] = acc[c];
      }
    }
    if (!ok) fail();
    if (split > 1) {
      // both meetings are of whole warps, which columns at and past N have split by the second
      __syncwarp();
      ptx::cluster_sync();  // every part is in its CTA's shared memory
      if (ok && own > 0) {
        const Tile x = sh.places[0];
        const int col = x.n0 + n, left = x.m1 - x.m0;
        const float* part = reinterpret_cast<const float*>(smem);
        if (col < args.N && HQ_IN_BOUNDS(x.m0 >= 0 && x.m1 <= args.rows)) {
          TY* y = static_cast<TY*>(args.Y) + static_cast<int64_t>(x.m0) * args.N + col;
          for (int c = rank; c < left; c += split) {
            float v[kMaxSplit];
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
              v[r] = r < split ? ptx::ld_cluster_f32(ptx::mapa(part + c * kRows + n, r)) : 0.f;
            float sum = v[0];
#pragma unroll
            for (int r = 1; r < kMaxSplit; ++r)
              if (r < split) sum += v[r];
            y[static_cast<int64_t>(c) * args.N] = static_cast<TY>(sum);
          }
        }
      }
      __syncwarp();
      ptx::cluster_sync_relaxed();  // no CTA leaves while another reads its part
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr int kSlots = kSMs * kCtasPerSM;

// How many clusters of `split` CTAs the current device holds at once, asked once: a cluster lies within
// one GPC, so it depends on how many SMs each of the chip's GPCs has (40 clusters of 7 did not fit at
// once although their 280 CTAs are fewer than 296, and 5120 x 5120 took 15.8 us instead of 9.9).  Asked of
// the variant that takes most shared memory, so that all variants of a tile height split alike and their
// sums are the same; the device is assumed to be like the first one asked.  The runtime counts one CTA an
// SM for kernels that allocate tensor memory; two of these run there (240 CTAs in clusters of 6 were seen
// at once, 272 of 2), so its count is taken up by that.  Where two did not run, clusters would wait for one
// another: slower, with the same result.  0: not known.
template <int BT>
int clusters_at_once(int split) {
  using TX = typename std::conditional<BT == 16, __nv_bfloat16, uint8_t>::type;
  static std::atomic<int> known[kMaxSplit + 1];
  int n = known[split].load(std::memory_order_relaxed);
  if (n > 0) return n;
  const auto kernel = fp8_gemm_few_kernel<BT, __nv_bfloat16, TX, false>;
  constexpr int kSmem = Few<BT, BT == 16>::kSmem;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int counted = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&counted, kernel, kThreads, kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (counted == 1) n *= kCtasPerSM;
  known[split].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs to a tile: as many as leave all tiles' clusters on the GPU at once, where the number of tiles is
// known (one weight).
template <int BT>
int pick_split(const Fp8Gemm& p) {
  const int64_t tiles = ceil_div(p.rows, BT) * ceil_div(p.N, kRows);
  if (p.offsets != nullptr || tiles * 2 > kSlots) return 1;
  for (int n = static_cast<int>(std::min<int64_t>({kMaxSplit, kSlots / tiles, ceil_div(p.K, kFp8Block)})); n > 1; --n)
    if (tiles <= clusters_at_once<BT>(n)) return n;
  return 1;
}

template <int BT, typename TY, typename TX, bool kTimeout = false>
hq_status run_few(const Fp8Gemm& p, cudaStream_t s) {
  const int64_t most = most_tiles(p, BT, kRows);
  CUtensorMap map_a, map_w;
  GemmArgs a{};
  const hq_status st = gemm_args(p, most, BT, kRows, a, map_a, map_w);
  if (st != HQ_OK) return st;
  constexpr int kSmem = Few<BT, !std::is_same<TX, uint8_t>::value>::kSmem;
  const auto kernel = fp8_gemm_few_kernel<BT, TY, TX, kTimeout>;
  HQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  const int split = pick_split<BT>(p);
  const int64_t clusters = split > 1 ? ceil_div(p.rows, BT) * ceil_div(p.N, kRows) : std::min<int64_t>(most, kSlots);
  HQ_LAUNCH_CHAINED(launch_product(p, kernel, static_cast<unsigned>(clusters * split), kThreads, kSmem,
                                   static_cast<unsigned>(split), s, map_a, map_w, a, split,
                                   static_cast<const TX*>(p.X)));
  return HQ_OK;
}

template <typename TY>
hq_status run_few_as(const Fp8Gemm& p, int tile_rows, cudaStream_t s) {
  if (tile_rows == 64) return run_few<64, TY, uint8_t>(p, s);
  if (p.X == nullptr) return run_few<16, TY, uint8_t>(p, s);
  return p.x_dtype == HQ_F32 ? run_few<16, TY, float>(p, s) : run_few<16, TY, __nv_bfloat16>(p, s);
}

}  // namespace

bool few_quantises(const Fp8Gemm& p) {
  return p.offsets == nullptr && p.rows <= 4 && ceil_div(p.N, kRows) <= kSlots &&
         ceil_div(ceil_div(p.K, kFp8Block), pick_split<16>(p)) <= kPanel;
}

hq_status gemm_few(const Fp8Gemm& p, int tile_rows, cudaStream_t s) {
  if (p.timeout) return tile_rows == 64 ? run_few<64, float, uint8_t, true>(p, s) : run_few<16, float, uint8_t, true>(p, s);
  return p.y_dtype == HQ_F32 ? run_few_as<float>(p, tile_rows, s) : run_few_as<__nv_bfloat16>(p, tile_rows, s);
}

}  // namespace fp8
}  // namespace hq
