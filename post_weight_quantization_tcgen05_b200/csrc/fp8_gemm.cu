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
// What bounds it: the hand-over of the accumulators.  Of a pair's block of 128 columns the MMAs alone, with
// their loads, take 675 cycles (8192 x 17408 x 5120: 412 us, 3.5 PFLOP/s; shared memory moves 64 KB a block
// and SM at 128 bytes a cycle); a signal from the MMAs to the epilogue or back takes about 400 cycles,
// reading an accumulator 400.  With two whole accumulators that came to 1040 cycles (645 us); handed over
// by halves of 128 columns the two halves' hand-overs overlap each other's MMAs, which then read A's
// operand twice: 605 to 634 us on a rested GPU, 2.3 to 2.4 PFLOP/s.  Under load the power limit lowers the
// clock: after two seconds of such calls 748 us at 1372 MHz (median of 61 samples), and 513 us at 1957 MHz
// on constant operands, which take less power; both are a million cycles, 840 to 855 a block.  What is left
// over the MMAs: the warps of the epilogue that share a quarter of the SM with a warp of another role take
// some 300 cycles a block longer, and the stores of a tile come on top (2000 cycles when its pieces went
// out one at a time; two at a time, and the scales by two warps, took 2 % off the whole).
//
// Two tilings of one kernel:
//   pair   : two CTAs (a cluster) compute a 256 x 256 tile with cta_group::2 MMAs, each of them 128
//            rows.  On one SM a 128 x 256 tile takes 48 KB of operands for every 512 cycles of
//            tensor work, more than L2 gives all SMs at once; in a pair each CTA loads its 128 rows
//            of A and half of the 256 rows of W, 32 KB, and the tensor cores read the other half
//            from the peer's shared memory.  For many rows.
//   single : one CTA, a 128 x 128 tile.  For some hundred rows, where more, smaller tiles keep more SMs
//            at work; few rows, and few tiles, go to fp8_gemm_few.cu.  Which of them runs is pick_impl's choice.
//
// One CTA per SM walks its tiles.  Warp 0 loads the operands by TMA (128 rows of A and 128 of W, in a
// pair 64 for each half of the tile's columns, by 128 columns; 128-byte swizzle, K-major) into a ring of
// 32 KB stages, one stage per scale block; warp 1 issues
// the MMAs (in a pair, the even CTA's for both); warps 2 and 3 fetch the scales some blocks ahead and
// leave their products, and each tile's place, in shared memory; warps 4-11 (two per TMEM lane
// quadrant, half of the tile's columns each) scale, add and store.  Columns at and past K read as
// zeros (the tensor map's extent is K, not the row pitch), as do rows past the operands' ends.  A
// tile of an expert that ends inside it computes rows of the next expert as well (against the wrong
// matrix) and does not store them.
//
// Every wait is bounded: on expiry the CTA records HQ_ERR_TIMEOUT, waits (bounded) for its
// in-flight TMA and MMA work, frees TMEM and returns; the CTAs of a pair meet at the end, so that
// neither leaves while the other may still signal into its shared memory.
#include <algorithm>
#include <atomic>

#include "fp8_gemm.cuh"

namespace hq {
namespace fp8 {
namespace {

constexpr int kRows = 128;      // rows of A, and of W, that one CTA loads for a stage
constexpr int kStages = 4;
constexpr int kStageBytes = 2 * kRows * kBK;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
// Blocks whose scales are kept.  They are handed over, and given back, by halves of the ring.
constexpr int kScales = 8, kScaleHalf = kScales / 2;
constexpr int kFetch = kScaleHalf;  // blocks that the loads of the scales run ahead of their writes
// Tiles whose places are kept: the scales are at most kScales blocks ahead of the epilogue, their loads
// kFetch more, and every block may be another tile's.
constexpr int kPlaces = 16;
static_assert(kPlaces > kScales + kFetch, "a tile's place is overwritten after the epilogue read it");
constexpr int kStoreBytes = 2 * 32 * 128;  // a warp's staging of output rows: two pieces of 32 x 128 bytes

// Shared memory after the stages and the staging (both 1024-byte aligned).
struct Shared {
  float scales[kScales][2][kRows];  // by half of the tile's columns, by row
  Tile places[kPlaces];
  uint64_t full[kStages];   // in a pair the even CTA's: both CTAs' loads
  uint64_t empty[kStages];
  uint64_t accf[2][2];      // accumulator filled, by half of its columns (one half in a single CTA)
  uint64_t acce[2][2];      // the same drained (in a pair the even CTA's: by both)
  uint64_t scf[2];          // scales of half the ring written
  uint64_t sce[2];          // scales of half the ring read
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int start[kMaxExperts + 1];  // row tiles before each expert
};
constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kStoreBytes + 1024 /*align*/ + static_cast<int>(sizeof(Shared));
static_assert(kSmem <= 232448, "shared memory of a CTA");

// Registers of the pair: 384 threads launch with 168 each; the epilogue's 256 hold 128 sums each and
// take 216, the other 128 keep 72: 256 * 216 + 128 * 72 = 384 * 168.
constexpr int kRegsLaunch = 168, kRegsEpi = 216, kRegsCtl = 72;
static_assert(kEpiWarps * 32 * kRegsEpi + 128 * kRegsCtl <= kThreads * kRegsLaunch, "register split");

// 16 bytes of output from fp32 sums.
__device__ __forceinline__ uint4 pack16(const float* v, float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float* v, __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's 32 rows x NC columns of Y, one row of sums a lane, through shared memory of its own in
// pieces of 32 rows x 128 bytes: a lane's own row would go out as 16-byte pieces of 32 different lines
// (measured 10,000 cycles for a 128 x 256 tile, the time of eleven blocks of the product; this way, a piece
// at a time, 2,000).
// Whole pieces leave by TMA stores, two at a time, which run on while the warp takes up the next tile; one
// that an expert's last row cuts, or unaligned rows of Y, by stores of the lanes, 8 a row.  16-byte part p
// of row r is kept at place p ^ (r % 8), the 128-byte swizzle of the tensor map.  Rows from `rows_left`
// on and columns from N on are not written.  The elected lane is always the same: it waits for its own
// stores.
template <int NC, typename TY>
__device__ __forceinline__ void store_rows(const GemmArgs& a, const CUtensorMap* map, uint8_t* stage, int row, int col,
                                           int rows_left, const float (&acc)[NC], int lane) {
  constexpr int kPer = 16 / sizeof(TY);  // columns of 16 bytes
  constexpr int kPiece = 8 * kPer;       // columns of a piece
  constexpr int kPieces = NC / kPiece;
  constexpr int kAtOnce = kPieces < 2 ? kPieces : 2;
  static_assert(kPieces % kAtOnce == 0 && kAtOnce * 32 * 128 <= kStoreBytes, "pieces of a turn");
  if (rows_left <= 0 || col >= a.N) return;
  const bool whole = a.y_aligned && rows_left >= 32;
  (void)HQ_IN_BOUNDS(row >= 0 && row + min(rows_left, 32) <= a.rows);
  if (whole) {
#pragma unroll
    for (int i = 0; i < kPieces; i += kAtOnce) {
      // the pieces before, which lay here, have been read by their stores
      if (ptx::elect_one()) ptx::bulk_wait_read<0>();
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int p = 0; p < 8; ++p)
          *reinterpret_cast<uint4*>(stage + u * (32 * 128) + lane * 128 + ((p ^ (lane & 7)) << 4)) =
              pack16(acc + (i + u) * kPiece + p * kPer, TY());
      ptx::fence_async_smem();
      __syncwarp();
      if (ptx::elect_one()) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
          if (col + (i + u) * kPiece < a.N) ptx::tma_store_2d(map, stage + u * (32 * 128), col + (i + u) * kPiece, row);
        ptx::bulk_commit();
      }
    }
    return;
  }
  if (ptx::elect_one()) ptx::bulk_wait_read<0>();
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = i * kPiece;
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p)
      *reinterpret_cast<uint4*>(stage + lane * 128 + ((p ^ (lane & 7)) << 4)) = pack16(acc + c + p * kPer, TY());
    __syncwarp();
    TY* out = static_cast<TY*>(a.Y) + static_cast<int64_t>(row) * a.N;
    if (a.y_aligned) {
      const int p = lane & 7;
      const int at = col + c + p * kPer;
      if (at < a.N)  // whole 16 bytes, as the rows are made of them
        for (int r = lane >> 3; r < rows_left && r < 32; r += 4)
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * a.N + at) =
              *reinterpret_cast<const uint4*>(stage + r * 128 + ((p ^ (r & 7)) << 4));
    } else {
      // 4 bytes a lane, a row at a time
      constexpr int kEach = 4 / sizeof(TY);
      const int at = col + c + lane * kEach;
      for (int r = 0; r < rows_left && r < 32; ++r) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        TY* o = out + static_cast<int64_t>(r) * a.N + at;
        if (at + kEach <= a.N && (reinterpret_cast<uintptr_t>(o) & 3) == 0) {
          *reinterpret_cast<uint32_t*>(o) = v;
        } else {
          const TY* e = reinterpret_cast<const TY*>(&v);
#pragma unroll
          for (int k = 0; k < kEach; ++k)
            if (at + k < a.N) o[k] = e[k];
        }
      }
    }
  }
}

template <bool kPair, typename TY, bool kTimeout>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW,
                    const __grid_constant__ CUtensorMap mapY, GemmArgs args) {
  constexpr int kBM = kPair ? 256 : 128, kBN = kPair ? 256 : 128;  // the tile
  constexpr int NC = kBN / 2;                                      // columns of an epilogue warp
  constexpr int kHalves = kPair ? 2 : 1;                           // accumulators handed over by halves
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stores = smem + kStages * kStageBytes;
  Shared& sh = *reinterpret_cast<Shared*>(stores + kEpiWarps * kStoreBytes);
  volatile int* abort_flag = &sh.abort;
  const long long limit = wait_limit<kTimeout>(args);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(ptx::cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&sh.full[s], 1);
      ptx::mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 4; ++b) {
      ptx::mbar_init(&sh.accf[b >> 1][b & 1], 1);
      ptx::mbar_init(&sh.acce[b >> 1][b & 1], kEpiWarps);  // of a pair: half the warps of two CTAs
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&sh.scf[s], 2);
      ptx::mbar_init(&sh.sce[s], kEpiWarps);
    }
    ptx::mbar_init(&sh.drain, 1);
    sh.abort = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      ptx::tmem_alloc_pair(&sh.tmem, 2 * kBN);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&sh.tmem, 2 * kBN);
      ptx::tmem_relinquish();
    }
  }
  expert_tiles<kBM>(args, sh.start);
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (kPair) ptx::cluster_sync();  // the peer's barriers exist before anything signals them
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int tiles = sh.start[args.E] * ((args.N + kBN - 1) / kBN);
  const int first = kPair ? blockIdx.x >> 1 : blockIdx.x, step = kPair ? gridDim.x >> 1 : gridDim.x;
  const int own = tiles > first ? (tiles - 1 - first) / step + 1 : 0;  // tiles of this CTA (or pair)
  const int blocks = own * args.kblocks;  // their blocks follow one another across tiles

  auto fail = [&]() {
    *abort_flag = 1;
    record_status(args.status, HQ_ERR_TIMEOUT);
  };
  if (warp < 4) {
    if constexpr (kPair) ptx::regs_dec<kRegsCtl>();
  }
  if (warp == 0 && ptx::elect_one()) {
    // ------------------------------------------------------------ TMA producer
    ptx::prefetch_tensormap(&mapA);
    ptx::prefetch_tensormap(&mapW);
    pdl_wait();
    int g = 0;  // stages issued by this CTA
    bool ok = true;
    for (int i = 0; i < own && ok; ++i) {
      const Tile x = tile_at<kBM, kBN>(args, sh.start, first + i * step);
      const int a_row = x.m0 + rank * kRows;
      const int w_row = x.e * args.N + x.n0 + rank * 64;
      (void)HQ_IN_BOUNDS(x.m0 < args.rows && x.n0 < args.N);
      for (int k = 0; k < args.kblocks; ++k, ++g) {
        const int s = g % kStages;
        if (g >= kStages && !ptx::mbar_wait(&sh.empty[s], ((g / kStages) - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + s * kStageBytes;
        if constexpr (kPair) {
          // the even CTA announces both CTAs' bytes; the odd one's may arrive before that, the phase
          // completes only after it
          if (rank == 0) ptx::mbar_arrive_expect_tx(&sh.full[s], 2 * kStageBytes);
          const uint32_t bar = ptx::mapa(&sh.full[s], 0);
          ptx::tma_load_2d_pair(sa, &mapA, k * kBK, a_row, bar);
          // 64 rows for each half of the tile's columns
          ptx::tma_load_2d_pair(sa + kRows * kBK, &mapW, k * kBK, w_row, bar);
          ptx::tma_load_2d_pair(sa + (kRows + 64) * kBK, &mapW, k * kBK, w_row + 128, bar);
        } else {
          ptx::mbar_arrive_expect_tx(&sh.full[s], kStageBytes);
          ptx::tma_load_2d(sa, &mapA, k * kBK, a_row, &sh.full[s]);
          ptx::tma_load_2d(sa + kRows * kBK, &mapW, k * kBK, w_row, &sh.full[s]);
        }
      }
    }
    if (!ok) {
      fail();
      // let the copies already issued land before shared memory goes away
      if (rank == 0)
        for (int k = g > kStages ? g - kStages : 0; k < g; ++k)
          ptx::mbar_wait(&sh.full[k % kStages], (k / kStages) & 1, nullptr);
    }
  } else if (warp == 1 && rank == 0 && ptx::elect_one()) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem), 16, 1024);
    constexpr uint32_t kIdesc = ptx::idesc(ptx::kFmtE4M3, kBM, kBN / kHalves, false, false);
    bool ok = true;
    for (int g = 0; g < blocks && ok; ++g) {
      const int s = g % kStages, b = g & 1;
      if (!ptx::mbar_wait(&sh.full[s], (g / kStages) & 1, abort_flag, limit)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (g >= 2 && !ptx::mbar_wait(&sh.acce[b][h], ((g >> 1) - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t dacc = tmem + static_cast<uint32_t>(b * kBN + h * 128);
        // K-major rows of 128 bytes, 8-row groups 1 KB apart (SBO); an MMA takes 32 bytes of each row
        const uint64_t sd = desc0 + static_cast<uint64_t>(s * (kStageBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk) {
          const uint64_t ad = sd + kk * 2, bd = sd + kk * 2 + ((kRows + h * 64) * kBK >> 4);
          if constexpr (kPair)
            ptx::mma_f8_pair(dacc, ad, bd, kIdesc, kk > 0 ? 1u : 0u);
          else
            ptx::mma_f8(dacc, ad, bd, kIdesc, kk > 0 ? 1u : 0u);
        }
        if constexpr (kPair)
          ptx::mma_commit_pair(&sh.accf[b][h]);
        else
          ptx::mma_commit(&sh.accf[b][h]);
      }
      if (!ok) break;
      if (kTimeout && g == args.withhold_stage) continue;
      if constexpr (kPair)
        ptx::mma_commit_pair(&sh.empty[s]);
      else
        ptx::mma_commit(&sh.empty[s]);
    }
    if (!ok) {
      fail();
      if constexpr (kPair)
        ptx::mma_commit_pair(&sh.drain);
      else
        ptx::mma_commit(&sh.drain);
      ptx::mbar_wait(&sh.drain, 0, nullptr);
    }
  } else if (warp == 2 || warp == 3) {
    // ------------------------------------------------------------ scales
    // Each warp has 64 of the rows; a lane fetches the scales of 2, kFetch blocks ahead of the block it
    // writes.  (One warp for all rows 1 % slower: it holds up the epilogue warps that it shares the issue
    // slots of a quarter of the SM with.)
    pdl_wait();
    const int r0 = (warp - 2) * 64 + lane;
    float sa[kFetch][2], sw[kFetch][2];
    Tile x{};
    int k = args.kblocks, i = -1;  // the block to fetch: the first of the tile after tile i
    auto fetch = [&](int f, int g) {
      if (g >= blocks) return;
      if (k == args.kblocks) {
        k = 0;
        ++i;
        x = tile_at<kBM, kBN>(args, sh.start, first + i * step);
        // its place is read by the epilogue after its first block's scales are announced, later
        if (threadIdx.x == 64) sh.places[i % kPlaces] = x;
      }
      // not __ldg: the kernel that writes these scales may have run beside this one until pdl_wait
      const float* col = args.a_scales + static_cast<int64_t>(k) * args.rows;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = x.m0 + rank * kRows + r0 + r * 32;
        sa[f][r] = row < x.m1 ? __ldcg(col + row) : 0.f;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int nb = (x.n0 + h * NC) / kFp8Block;
        sw[f][h] = nb < args.nblocks
                       ? __ldg(args.w_scales + (static_cast<int64_t>(x.e) * args.nblocks + nb) * args.kblocks + k)
                       : 0.f;
      }
      ++k;
    };
#pragma unroll
    for (int f = 0; f < kFetch; ++f) fetch(f, f);
    bool ok = true;
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
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) sh.scales[(g0 + f) % kScales][h][r0 + r * 32] = sa[f][r] * sw[f][h];
        fetch(f, g0 + f + kFetch);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.scf[half]);
    }
    if (!ok) fail();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    if constexpr (kPair) ptx::regs_inc<kRegsEpi>();
    // The time from "accumulator filled" to "drained" holds up the tensor core, as there are only two,
    // so it contains the loads from tensor memory and no more of the sums than free the registers for
    // them.  The last sums run while the next block's barriers are looked at.
    const int q = warp & 3;         // TMEM lane quadrant this warp may access
    const int h = (warp - 4) >> 2;  // which half of the tile's columns
    const uint32_t tmem_w = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * NC);
    uint8_t* stage = stores + (warp - 4) * kStoreBytes;
    const int half = kPair ? h : 0;
    const uint32_t acce = kPair ? ptx::mapa(&sh.acce[0][half], 0) : ptx::smem_u32(&sh.acce[0][half]);
    const uint32_t sce = ptx::smem_u32(&sh.sce[0]);
    const uint32_t scale_at = ptx::smem_u32(&sh.scales[0][h][q * 32 + lane]);
    bool ok = true, seen = false;  // seen: the block's accumulator has been seen filled
    int g = 0;
    for (int i = 0; i < own && ok; ++i) {
      float acc[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = 0.f;
      for (int k = 0; k < args.kblocks; ++k, ++g) {
        const int b = g & 1;
        // the warp goes on or gives up as one: a wait may run out for some of its lanes only
        if (g % kScaleHalf == 0) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh.scf[(g / kScaleHalf) & 1], (g / kScales) & 1, abort_flag, limit));
          if (!ok) break;
        }
        if (!__all_sync(0xffffffffu, seen)) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh.accf[b][half], (g >> 1) & 1, abort_flag, limit));
          if (!ok) break;
        }
        ptx::tc_fence_after();
        const uint32_t from = tmem_w + static_cast<uint32_t>(b * kBN);
        uint32_t r[2][32];
        ptx::tmem_ld32_nowait(from, r[0]);
        ptx::tmem_ld32_nowait(from + 32, r[1]);
        const float scale = ptx::lds32(scale_at + (g % kScales) * (2 * kRows * 4));
        auto add = [&](int c) {
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            ptx::fma2(acc[32 * c + j], acc[32 * c + j + 1], scale, r[c & 1][j], r[c & 1][j + 1]);
        };
        ptx::tmem_wait_ld();
        if constexpr (NC == 128) {
          add(0);
          ptx::tmem_ld32_nowait(from + 64, r[0]);
          add(1);
          ptx::tmem_ld32_nowait(from + 96, r[1]);
          ptx::tmem_wait_ld();
        }
        ptx::tc_fence_before();
        __syncwarp();
        ptx::mbar_arrive_cluster(acce + 16 * b, lane == 0);
        ptx::mbar_arrive_cluster(sce + 8 * ((g / kScaleHalf) & 1), lane == 0 && g % kScaleHalf == kScaleHalf - 1);
        seen = ptx::mbar_test(&sh.accf[b ^ 1][half], ((g + 1) >> 1) & 1);
        add(NC / 32 - 2);
        add(NC / 32 - 1);
      }
      if (!ok) break;
      const Tile x = sh.places[i % kPlaces];
      const int row = x.m0 + rank * kRows + q * 32;
      store_rows<NC, TY>(args, &mapY, stage, row, x.n0 + h * NC, x.m1 - row, acc, lane);
    }
    if (ptx::elect_one()) ptx::bulk_wait<0>();
    if (!ok) fail();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (kPair) ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (kPair)
      ptx::tmem_dealloc_pair(tmem, 2 * kBN);
    else
      ptx::tmem_dealloc(tmem, 2 * kBN);
  }
}

template <bool kPair, typename TY, bool kTimeout = false>
hq_status run_gemm(const Fp8Gemm& p, cudaStream_t s) {
  constexpr int kTile = kPair ? 256 : 128;
  const int64_t most = most_tiles(p, kTile, kTile);
  CUtensorMap map_a, map_w, map_y;
  GemmArgs a{};
  const hq_status st = gemm_args(p, most, kRows, kPair ? 64 : kRows, a, map_a, map_w);
  if (st != HQ_OK) return st;
  if (!a.y_aligned)
    map_y = map_a;  // not used
  else if (!make_tmap_2d(&map_y, sizeof(TY) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.Y,
                         static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.rows), p.N * sizeof(TY), 128 / sizeof(TY), 32))
    return HQ_ERR_CUDA;
  if constexpr (kPair) {
    // the epilogue's registers come out of those the CTA was launched with: with fewer it would wait for good
    static std::atomic<int> regs;
    if (regs.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes attr;
      HQ_CUDA_TRY(cudaFuncGetAttributes(&attr, fp8_gemm_kernel<kPair, TY, kTimeout>));
      regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < kRegsLaunch) return HQ_ERR_UNSUPPORTED;
  }
  HQ_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<kPair, TY, kTimeout>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  const int slots = kPair ? kSMs / 2 : kSMs;
  const unsigned grid = static_cast<unsigned>((most < slots ? most : slots) * (kPair ? 2 : 1));
  HQ_LAUNCH_CHAINED(launch_product(p, fp8_gemm_kernel<kPair, TY, kTimeout>, grid, kThreads, kSmem, kPair ? 2 : 1, s, map_a, map_w,
                                   map_y, a));
  return HQ_OK;
}

}  // namespace

hq_status gemm_single(const Fp8Gemm& p, cudaStream_t s) {
  if (p.timeout) return run_gemm<false, float, true>(p, s);
  return p.y_dtype == HQ_F32 ? run_gemm<false, float>(p, s) : run_gemm<false, __nv_bfloat16>(p, s);
}
hq_status gemm_pair(const Fp8Gemm& p, cudaStream_t s) {
  if (p.timeout) return run_gemm<true, float, true>(p, s);
  return p.y_dtype == HQ_F32 ? run_gemm<true, float>(p, s) : run_gemm<true, __nv_bfloat16>(p, s);
}

}  // namespace fp8

namespace {

// Up to 32 rows: the kernel that reads the weights once, in tiles of 16 (1 x 5120 x 5120: 9 us against
// 18 us of the single CTAs; 24 x 17408 x 5120: 20.1 us against 23.5 us with tiles of 64, the second tile's
// weights coming from L2).  Experts go by their average, as their sizes differ: tiles of 16 up to 24 rows
// (800 rows, 48 experts 2560 x 5120: 100 us against 109 us with tiles of 64; 2048 rows, 64 experts 164 us
// against 153 us), of 64 up to 48 (2048 rows: 153 us against 167 us of the single CTAs; 4096 218 us against
// 194 us).
// Else by what each would take, in units of 10 ns from timings.  A block of 128 columns takes a single CTA
// 0.32 us, a pair (four times the work) 0.47 us, in rounds of tiles over the SMs, and a launch 5 or 6 us
// around them: 384 x 5120 x 5120 18 us against 24 us, 768 31 us against 25 us, 1024 43 us either way, 2048
// 69 us against 61 us, 256 x 17408 x 5120 34 us against 26 us.  Those two do not split K, so few tiles leave
// SMs idle; the kernel for few rows does, and then takes as long as its loads, or as one CTA its part:
// 300 x 256 x 17408 14 and 15 us in tiles of 16 and 64 against 44 us of the single CTAs, 128 x 512 x 5120
// 9.2 and 9.3 us against 17 us, 256 x 1024 x 5120 14 and 13 us against 17 us, 64 x 5120 x 17408 25 us with
// 64 against 50 us; but 96 x 5120 x 5120 19 and 20 us against 17 us, 64 x 17408 x 5120 27 us with 64
// against 21 us.
int pick_impl(const Fp8Gemm& p) {
  const bool experts = p.offsets != nullptr;
  const int64_t each = ceil_div(p.rows, p.E);
  if (each <= (experts ? 24 : 32)) return kFp8Few16;
  if (experts && each <= 48) return kFp8Few64;
  // an expert's last tile is half full on average
  const int64_t m128 = experts ? p.rows / 128 + ceil_div(p.E, 2) : ceil_div(p.rows, 128);
  const int64_t m256 = experts ? p.rows / 256 + ceil_div(p.E, 2) : ceil_div(p.rows, 256);
  const int64_t blocks = ceil_div(p.K, kFp8Block), n128 = ceil_div(p.N, 128);
  const int64_t single = 500 + 32 * blocks * ceil_div(m128 * n128, fp8::kSMs);
  const int64_t pair = 600 + 47 * blocks * ceil_div(m256 * ceil_div(p.N, 256), fp8::kSMs / 2);
  int64_t best = std::min(single, pair);
  int impl = pair < single ? kFp8Pair : kFp8Single;
  if (experts) return impl;
  const auto few = [&](int64_t rows, int64_t launch, int64_t block, double per_thousand) {
    const int64_t tiles = ceil_div(p.rows, rows) * n128;
    const int64_t split = std::max<int64_t>(1, std::min<int64_t>(8, 2 * fp8::kSMs / tiles));
    const int64_t loads = static_cast<int64_t>(1e-3 * per_thousand * tiles * blocks);  // any size: no overflow
    return launch + std::max(block * ceil_div(blocks, split), loads);
  };
  const int64_t few16 = few(16, 600, 27, 165), few64 = few(64, 700, 45, 360);
  if (few16 < best) best = few16, impl = kFp8Few16;
  if (few64 < best) impl = kFp8Few64;
  return impl;
}

}  // namespace

hq_status launch_fp8_gemm(const Fp8Gemm& p, int impl, cudaStream_t s) {
  if (p.rows == 0) return HQ_OK;
  switch (impl == kFp8Auto ? pick_impl(p) : impl) {
    case kFp8Pair: return fp8::gemm_pair(p, s);
    case kFp8Single: return fp8::gemm_single(p, s);
    case kFp8Few64: return fp8::gemm_few(p, 64, s);
    default: return fp8::gemm_few(p, 16, s);
  }
}

// One to four rows are quantised by the CTAs that multiply them, each the blocks that it needs, where those
// fit into its shared memory (few_quantises): one launch.  Others are quantised once, by a kernel of their
// own.
hq_status launch_fp8_linear(Fp8Gemm p, uint8_t* codes, float* scales, cudaStream_t s) {
  if (p.rows == 0) return HQ_OK;
  const int impl = pick_impl(p);
  if (impl == kFp8Few16 && fp8::few_quantises(p)) return fp8::gemm_few(p, 16, s);
  const hq_status st = launch_fp8_rows(p.X, p.x_dtype, p.rows, p.K, codes, scales, s);
  if (st != HQ_OK) return st;
  p.X = nullptr;
  p.chained = true;
  return launch_fp8_gemm(p, impl, s);
}

}  // namespace hq
