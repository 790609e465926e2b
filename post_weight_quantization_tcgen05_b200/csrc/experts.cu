// Tokens laid out by expert and back: a stable counting sort of the router's choices, the copy of
// each token's row to its places (as it is, or quantised to e4m3 on the way), the weighted sum of
// the experts' outputs back in token order, and that sum's gradient.
//
// A choice is a flat index i = t * top + j into ids [T, top]; position[i] is its row in the sorted
// layout, or -1 for an id outside [0, E) (a dropped choice: nothing is read, written or counted for
// it).  Every kernel checks a position against the number of rows before it uses it, so that a
// wrong one is treated as dropped.
#include <algorithm>

#include "common.cuh"
#include "fp8_quant.cuh"
#include "kernels.cuh"

namespace hq {

// ---------------------------------------------------------------- sort
//
// The ids are cut into chunks, one per CTA.  expert_hist_kernel counts each chunk's ids by expert;
// expert_place_kernel gives every chunk its first row in each expert (the counts of the chunks
// before it and of the experts before), and ranks the ids inside it.  There each warp owns a
// contiguous part of the chunk and counts it first, so that its own first rows are known and the
// ranking runs without any exchange between warps: 32 ids at a time, a lane's rank among the equal
// ids of its warp comes from a match over the warp.  One chunk (up to kSortOneChunk ids) needs no
// counts from the others: one launch.  Integer counts only, so the order is the same every time.
// Bound by launches and the latency of its passes over shared memory, and for long lists by the
// scattered 4-byte stores of `order`.  On the device: 64 x 8 choices of 48 experts 3.2 us, 16384 x 8 of 64
// 7.6 us, 65536 x 8 21 us.
constexpr int kSortWarps = 16;
constexpr int kSortChunk = 2048;     // ids per CTA of a long list, at least
constexpr int kSortOneChunk = 4096;  // up to here one CTA sorts alone
constexpr int kSortBatch = 8;        // ids a lane loads at once
constexpr int kSortMaxCtas = 148;

struct SortSplit {
  int chunks;
  int64_t chunk;  // ids per chunk
};
static SortSplit sort_split(int64_t R) {
  if (R <= kSortOneChunk) return {1, R};
  int64_t chunk = ceil_div(R, kSortMaxCtas);
  if (chunk < kSortChunk) chunk = kSortChunk;
  return {static_cast<int>(ceil_div(R, chunk)), chunk};
}

size_t expert_sort_workspace(int64_t R, int64_t E) {
  const SortSplit sp = sort_split(R);
  return sp.chunks == 1 ? 256 : round_up(static_cast<size_t>(sp.chunks) * E * sizeof(int), 256);
}

// ids i, i + step, ... below `end` (-1 past it), all on their way at once
__device__ __forceinline__ void load_ids(const int* ids, int64_t i, int64_t end, int step, int (&id)[kSortBatch]) {
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) id[u] = i + u * step < end ? __ldg(ids + i + u * step) : -1;
}

__global__ void __launch_bounds__(32 * kSortWarps)
    expert_hist_kernel(const int* __restrict__ ids, int64_t R, int64_t chunk, int E, int* __restrict__ hist) {
  extern __shared__ int count[];
  pdl_launch_dependents();  // expert_place_kernel counts its own ids meanwhile
  for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = 0;
  __syncthreads();
  const int64_t i0 = blockIdx.x * chunk, i1 = min(R, i0 + chunk);
  int id[kSortBatch];
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortBatch * blockDim.x) {
    load_ids(ids, i, i1, blockDim.x, id);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u)
      if (static_cast<unsigned>(id[u]) < static_cast<unsigned>(E)) atomicAdd(&count[id[u]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[static_cast<int64_t>(blockIdx.x) * E + e] = count[e];
}

// Exclusive sum over the CTA's 512 threads of one int each; every thread calls it.
__device__ __forceinline__ int block_exclusive_sum(int v, int* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  return before + x - v;
}

// hist == nullptr: one chunk, whose own counts are the totals.
__global__ void __launch_bounds__(32 * kSortWarps)
    expert_place_kernel(const int* __restrict__ ids, int64_t R, int64_t chunk, int E, const int* __restrict__ hist,
                        int* __restrict__ offsets, int* __restrict__ order, int* __restrict__ position) {
  extern __shared__ int next[];  // [warps][E]: the next row of each expert for each warp's ids; then sums
  __shared__ int warp_sum[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t i0 = blockIdx.x * chunk, i1 = min(R, i0 + chunk);
  const int64_t part = (i1 - i0 + 32 * kSortWarps - 1) / (32 * kSortWarps) * 32;
  const int64_t w0 = min(i1, i0 + warp * part), w1 = min(i1, w0 + part);

  for (int k = threadIdx.x; k < kSortWarps * E; k += blockDim.x) next[k] = 0;
  __syncthreads();
  int id[kSortBatch];
  for (int64_t i = w0 + lane; i < w1; i += 32 * kSortBatch) {
    load_ids(ids, i, w1, 32, id);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u)
      if (static_cast<unsigned>(id[u]) < static_cast<unsigned>(E)) atomicAdd(&next[warp * E + id[u]], 1);
  }
  __syncthreads();

  // Sums over the chunks by groups of P lanes, so that an expert's counts are not read one after the
  // other: lane r of a group takes the chunks r, r + P, ...
  int* const sums = next + kSortWarps * E;  // [2][E]: all chunks', and those before this one
  if (hist != nullptr) {
    pdl_wait();
    int P = 32;
    while (P > 1 && P * E > static_cast<int>(blockDim.x)) P /= 2;
    const int r = threadIdx.x % P;
    for (int eb = 0; eb < E; eb += blockDim.x / P) {
      const int e = eb + threadIdx.x / P;
      int total = 0, before = 0;
      if (e < E) {
#pragma unroll 8
        for (int b = r; b < static_cast<int>(gridDim.x); b += P) {
          const int c = __ldcg(hist + static_cast<int64_t>(b) * E + e);
          if (b < static_cast<int>(blockIdx.x)) before += c;
          total += c;
        }
      }
      for (int off = P / 2; off > 0; off /= 2) {
        total += __shfl_xor_sync(0xffffffffu, total, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
      }
      if (e < E && r == 0) {
        sums[e] = total;
        sums[E + e] = before;
      }
    }
    __syncthreads();
  }

  int base = 0;  // rows of the experts handled so far
  for (int eb = 0; eb < E; eb += blockDim.x) {
    const int e = eb + threadIdx.x;
    int total = 0, before = 0;
    if (e < E) {
      if (hist != nullptr) {
        total = sums[e];
        before = sums[E + e];
      } else {
        for (int w = 0; w < kSortWarps; ++w) total += next[w * E + e];
      }
    }
    const int first = base + block_exclusive_sum(total, warp_sum);
    if (e < E) {
      int at = first + before;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = next[w * E + e];
        next[w * E + e] = at;
        at += c;
      }
      if (blockIdx.x == 0) {
        offsets[e] = first;
        if (e == E - 1) offsets[E] = first + total;
      }
    }
    // every warp's sums were read before any thread gets here, and are not written again until the
    // next call's first barrier
    for (int w = 0; w < kSortWarps; ++w) base += warp_sum[w];
    __syncthreads();
  }

  for (int64_t i0w = w0; i0w < w1; i0w += 32 * kSortBatch) {
    load_ids(ids, i0w + lane, w1, 32, id);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const int64_t i = i0w + 32 * u + lane;
      if (i - lane >= w1) break;  // the whole warp
      const bool kept = static_cast<unsigned>(id[u]) < static_cast<unsigned>(E);
      const unsigned same = __match_any_sync(0xffffffffu, kept ? id[u] : -1);
      const int rank = __popc(same & ((1u << lane) - 1u));
      int at = 0;
      if (kept) at = next[warp * E + id[u]] + rank;
      __syncwarp();
      if (kept && rank == __popc(same) - 1) next[warp * E + id[u]] = at + 1;
      __syncwarp();
      if (i < w1 && HQ_IN_BOUNDS(!kept || (at >= 0 && at < R))) {
        position[i] = kept ? at : -1;
        if (kept) order[at] = static_cast<int>(i);
      }
    }
  }
}

hq_status launch_expert_sort(const int* ids, int64_t R, int64_t E, int* offsets, int* order, int* position,
                             uint8_t* ws, cudaStream_t s) {
  const SortSplit sp = sort_split(R);
  const int e = static_cast<int>(E);
  int* hist = nullptr;
  if (sp.chunks > 1) {
    hist = reinterpret_cast<int*>(ws);
    expert_hist_kernel<<<sp.chunks, 32 * kSortWarps, E * sizeof(int), s>>>(ids, R, sp.chunk, e, hist);
    HQ_LAUNCH_CHECK();
  }
  constexpr size_t kPer = (kSortWarps + 2) * sizeof(int);
  HQ_CUDA_TRY(cudaFuncSetAttribute(expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kPer * kMaxExperts)));
  if (sp.chunks > 1) {
    HQ_LAUNCH_CHAINED(launch_chained(expert_place_kernel, dim3(sp.chunks), dim3(32 * kSortWarps), kPer * E, s, ids, R,
                                     sp.chunk, e, hist, offsets, order, position));
  } else {
    expert_place_kernel<<<1, 32 * kSortWarps, kPer * E, s>>>(ids, R, sp.chunk, e, nullptr, offsets, order, position);
    HQ_LAUNCH_CHECK();
  }
  return HQ_OK;
}

// ---------------------------------------------------------------- rows in vectors
//
// The row kernels below give each token a group of 32 .. 256 threads (as many as its row has vectors,
// in powers of two), and each thread a vector of values at a time: 16 bytes that lie together (Vec), or,
// where rows are not made of aligned 16-byte vectors, four values 32 apart (Loose), so that neighbouring
// lanes still read neighbouring values.  What bounds those is the loads on their way: with one value a
// thread 8192 x 8 rows of 5119 bf16 are summed in 500 us, with two in 218, four 202, eight (registers
// spill) 507; copied in 256, 218, 171, 168 us; the sum's gradient takes 553, 410, 356 us, four of them with
// two CTAs on an SM (three, which spill: 470 us).
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr bool kSpread = false;
  using Raw = uint4;
  __device__ __forceinline__ static void values(const Raw& a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static Raw pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // vector i of a row of K values
  __device__ __forceinline__ static Raw load(const __nv_bfloat16* row, int64_t i, int64_t) {
    return __ldg(reinterpret_cast<const uint4*>(row) + i);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* row, int64_t i, int64_t, const Raw& a) {
    *(reinterpret_cast<uint4*>(row) + i) = a;
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr bool kSpread = false;
  using Raw = float4;
  __device__ __forceinline__ static void values(const Raw& a, float (&v)[4]) {
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
  }
  __device__ __forceinline__ static Raw pack(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ static Raw load(const float* row, int64_t i, int64_t) {
    return __ldg(reinterpret_cast<const float4*>(row) + i);
  }
  __device__ __forceinline__ static void store(float* row, int64_t i, int64_t, const Raw& a) {
    *(reinterpret_cast<float4*>(row) + i) = a;
  }
};
template <typename T>
struct Loose {  // "vector" i: the values i / 32 * 32 kN + i % 32 + 32 u, those of them below K
  static constexpr int kN = 4;
  static constexpr bool kSpread = true;
  struct Raw {
    T v[kN];
  };
  __device__ __forceinline__ static void values(const Raw& a, float (&v)[kN]) {
#pragma unroll
    for (int u = 0; u < kN; ++u) v[u] = static_cast<float>(a.v[u]);
  }
  __device__ __forceinline__ static Raw pack(const float (&v)[kN]) {
    Raw a;
#pragma unroll
    for (int u = 0; u < kN; ++u) a.v[u] = static_cast<T>(v[u]);
    return a;
  }
  __device__ __forceinline__ static int64_t first(int64_t i) { return (i >> 5) * (32 * kN) + (i & 31); }
  __device__ __forceinline__ static Raw load(const T* row, int64_t i, int64_t K) {
    const int64_t at = first(i);
    Raw a;
#pragma unroll
    for (int u = 0; u < kN; ++u) a.v[u] = at + 32 * u < K ? __ldg(row + at + 32 * u) : static_cast<T>(0.f);
    return a;
  }
  __device__ __forceinline__ static void store(T* row, int64_t i, int64_t K, const Raw& a) {
    const int64_t at = first(i);
#pragma unroll
    for (int u = 0; u < kN; ++u)
      if (at + 32 * u < K) row[at + 32 * u] = a.v[u];
  }
};
// "vectors" of a row of K values
template <typename V>
__host__ __device__ __forceinline__ int64_t row_vectors(int64_t K) {
  return V::kSpread ? (K + 32 * V::kN - 1) / (32 * V::kN) * 32 : K / V::kN;
}

// Choices handled at once: their positions and weights are in registers, and their rows' loads on
// their way together.  C is 4 where a token has no more, else 8: fewer registers, more CTAs on an SM
// (8192 x 4 rows of 5120 bf16 102 -> 72 us, their gradient 153 -> 121 us, one row a token 85 -> 50 us).
template <int C>
struct Choices {
  int p[C];  // -1: dropped, or none
  float w[C];
  __device__ __forceinline__ void load(const int* position, const float* weights, int j0, int top, int64_t rows) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      p[j] = j0 + j < top ? __ldg(position + j0 + j) : -1;
      if (p[j] >= rows) p[j] = -1;
      if (p[j] < 0) p[j] = -1;
      w[j] = weights == nullptr ? 1.f : p[j] >= 0 ? __ldg(weights + j0 + j) : 0.f;
    }
  }
};

constexpr int kRowThreads = 256;
// threads per token: enough for one vector each, 32 .. 256
static int row_threads(int64_t vectors) {
  int t = 32;
  while (t < kRowThreads && t < vectors) t *= 2;
  return t;
}

// ---------------------------------------------------------------- dispatch

// rows[position[t, j]] = X[t]: a token's row is read once and stored to each of its places.  Bound by the
// stores: 8192 x 8 rows of 5120 bf16 125 us, 6.0 TB/s.
template <typename T, template <typename> class V>
__global__ void __launch_bounds__(kRowThreads)
    expert_dispatch_kernel(const T* __restrict__ X, int64_t tokens, int64_t K, const int* __restrict__ position, int top,
                           int64_t rows, int tpt, T* __restrict__ out) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / tpt) + threadIdx.x / tpt;
  if (t >= tokens) return;
  const int64_t vectors = row_vectors<V<T>>(K);
  const int* pos = position + t * top;
  constexpr int C = 8;
  Choices<C> c;
  c.load(pos, nullptr, 0, top, rows);
  for (int64_t i = blockIdx.y * tpt + threadIdx.x % tpt; i < vectors; i += tpt * gridDim.y) {
    const typename V<T>::Raw v = V<T>::load(X + t * K, i, K);
    for (int j0 = 0; j0 < top; j0 += C) {
      if (top > C) c.load(pos, nullptr, j0, top, rows);
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (c.p[j] >= 0) V<T>::store(out + static_cast<int64_t>(c.p[j]) * K, i, K, v);
    }
  }
}

// The same with the row quantised on the way: once per token, whatever the number of its places.
// A warp takes 512 columns of one token.  8192 x 8 rows of 5120 from bf16: 82 us, 5.2 TB/s (a row's codes
// of a warp are 512 bytes, its scales single words of four lines).
template <typename T>
__global__ void __launch_bounds__(256)
    expert_dispatch_fp8_kernel(const T* __restrict__ X, int64_t tokens, int64_t K, int64_t pitch,
                               const int* __restrict__ position, int top, int64_t rows, uint8_t* __restrict__ codes,
                               float* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * 512 + lane * 16;
  Raw16<T, false> raw;
  raw.load(X, X + tokens * K, X + t * K + col, K - col);
  float v[16], scale;
  raw.align();
  raw.values(v);
  const uint4 c = fp8_quantise_row16(v, scale);
  const int* pos = position + t * top;
  for (int j = 0; j < top; ++j) {
    const int p = __ldg(pos + j);
    if (p < 0 || p >= rows) continue;
    if (col < pitch && HQ_IN_BOUNDS(col + 16 <= pitch))
      *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(p) * pitch + col) = c;
    if ((lane & 7) == 0 && col < K) scales[(col / kFp8Block) * rows + p] = scale;
  }
}

// ---------------------------------------------------------------- combine

// Y[t] = sum_j w[t, j] rows[position[t, j]] in the order of j, summed in fp32 and rounded once.  Bound by
// reading the rows, eight of them on their way in every thread: 8192 x 8 of 5120 bf16 128 us, 5.9 TB/s.
template <typename T, template <typename> class V, int C>
__global__ void __launch_bounds__(kRowThreads, C == 8 ? 3 : V<T>::kSpread ? 4 : 5)
    expert_combine_kernel(const T* __restrict__ rows, int64_t nrows, int64_t K, const int* __restrict__ position,
                          const float* __restrict__ weights, int64_t tokens, int top, int tpt, T* __restrict__ Y) {
  constexpr int N = V<T>::kN;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / tpt) + threadIdx.x / tpt;
  if (t >= tokens) return;
  const int64_t vectors = row_vectors<V<T>>(K);
  const int* pos = position + t * top;
  const float* wt = weights != nullptr ? weights + t * top : nullptr;
  Choices<C> c;
  c.load(pos, wt, 0, top, nrows);
  for (int64_t i = blockIdx.y * tpt + threadIdx.x % tpt; i < vectors; i += tpt * gridDim.y) {
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    for (int j0 = 0; j0 < top; j0 += C) {
      if (top > C) c.load(pos, wt, j0, top, nrows);
      typename V<T>::Raw raw[C];
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (c.p[j] >= 0) raw[j] = V<T>::load(rows + static_cast<int64_t>(c.p[j]) * K, i, K);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (c.p[j] < 0) continue;
        float z[N];
        V<T>::values(raw[j], z);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = fmaf(c.w[j], z[k], acc[k]);
      }
    }
    V<T>::store(Y + t * K, i, K, V<T>::pack(acc));
  }
}

// The gradient of the combine: d_rows[p] = w[t, j] dY[t] and d_weights[t, j] = <dY[t], rows[p]>,
// p = position[t, j]; a dropped choice has d_weights 0.  Eight choices at a time, their dot products
// in registers; a token's threads add them up in a fixed order.  Bound by DRAM, half reads and half
// writes: 8192 x 8 rows of 5120 bf16 228 us, 6.25 TB/s.
template <typename T, template <typename> class V, int C>
__global__ void __launch_bounds__(kRowThreads, C == 4 ? 4 : V<T>::kSpread ? 2 : 3)
    expert_combine_backward_kernel(const T* __restrict__ dY, const T* __restrict__ rows, int64_t nrows, int64_t K,
                                   const int* __restrict__ position, const float* __restrict__ weights, int64_t tokens,
                                   int top, int tpt, T* __restrict__ d_rows, float* __restrict__ d_weights) {
  constexpr int N = V<T>::kN;
  __shared__ float part[kRowThreads / 32][C];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / tpt) + threadIdx.x / tpt;
  const bool live = t < tokens;  // all threads stay for the barriers
  const int64_t vectors = live ? row_vectors<V<T>>(K) : 0;
  for (int j0 = 0; j0 < top; j0 += C) {
    Choices<C> c;
    c.load(position + t * top, weights + t * top, j0, live ? top : 0, nrows);
    float dot[C] = {};
    for (int64_t i = threadIdx.x % tpt; i < vectors; i += tpt) {
      typename V<T>::Raw raw[C];
      const typename V<T>::Raw raw_g = V<T>::load(dY + t * K, i, K);
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (c.p[j] >= 0) raw[j] = V<T>::load(rows + static_cast<int64_t>(c.p[j]) * K, i, K);
      float g[N];
      V<T>::values(raw_g, g);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (c.p[j] < 0) continue;
        float z[N], d[N];
        V<T>::values(raw[j], z);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          dot[j] = fmaf(g[k], z[k], dot[j]);
          d[k] = c.w[j] * g[k];
        }
        V<T>::store(d_rows + static_cast<int64_t>(c.p[j]) * K, i, K, V<T>::pack(d));
      }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], off);
    }
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < C; ++j) part[warp][j] = dot[j];
    }
    __syncthreads();
    const int j = threadIdx.x % tpt;
    if (live && j < C && j0 + j < top) {
      float sum = 0.f;
      for (int k = 0; k < tpt / 32; ++k) sum += part[warp + k][j];
      d_weights[t * top + j0 + j] = sum;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- launches

static bool rows_vec(int64_t row_bytes, const void* a, const void* b, const void* c = nullptr, const void* d = nullptr) {
  return row_bytes % 16 == 0 && aligned(a, 16) && aligned(b, 16) && aligned(c, 16) && aligned(d, 16);
}

struct RowGrid {
  int tpt;
  unsigned ctas, parts;
};
// parts: CTAs that share a token's row where there are few tokens, so that a thread has fewer vectors one
// after the other (sum of 8 rows of 5120 bf16 for one token 4.2 -> 3.0 us, for 64 4.3 -> 3.2, of 17408 for
// one 8.5 -> 3.0; copy of one row to 8 places 3.5 -> 2.4 us).  Not for the gradient, whose dot products
// would have to be added up across CTAs.
static RowGrid row_grid(int64_t tokens, int64_t vectors) {
  const int tpt = row_threads(vectors);
  const int64_t ctas = ceil_div(tokens, kRowThreads / tpt);
  const int64_t parts = std::min(ceil_div(vectors, tpt), std::max<int64_t>(1, 4 * 148 / ctas));
  return {tpt, static_cast<unsigned>(ctas), static_cast<unsigned>(parts)};
}

template <typename T, template <typename> class V>
static void dispatch_as(const void* X, int64_t tokens, int64_t K, const int* position, int64_t top, void* out,
                        cudaStream_t s) {
  const RowGrid g = row_grid(tokens, row_vectors<V<T>>(K));
  expert_dispatch_kernel<T, V><<<dim3(g.ctas, g.parts), kRowThreads, 0, s>>>(static_cast<const T*>(X), tokens, K, position,
                                                              static_cast<int>(top), tokens * top, g.tpt,
                                                              static_cast<T*>(out));
}

template <typename T>
static void dispatch_typed(const void* X, int64_t tokens, int64_t K, const int* position, int64_t top, void* out,
                           cudaStream_t s) {
  if (rows_vec(K * sizeof(T), X, out))
    dispatch_as<T, Vec>(X, tokens, K, position, top, out, s);
  else
    dispatch_as<T, Loose>(X, tokens, K, position, top, out, s);
}

hq_status launch_expert_dispatch(const void* X, int x_dtype, int64_t tokens, int64_t K, const int* position, int64_t top,
                                 void* out, cudaStream_t s) {
  if (x_dtype == HQ_BF16)
    dispatch_typed<__nv_bfloat16>(X, tokens, K, position, top, out, s);
  else
    dispatch_typed<float>(X, tokens, K, position, top, out, s);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

hq_status launch_expert_dispatch_fp8(const void* X, int x_dtype, int64_t tokens, int64_t K, const int* position,
                                     int64_t top, uint8_t* codes, float* scales, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(tokens, 8)), static_cast<unsigned>(ceil_div(K, 512)));
  const int64_t rows = tokens * top;
  const int n = static_cast<int>(top);
  if (x_dtype == HQ_BF16)
    expert_dispatch_fp8_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(X), tokens, K, fp8_pitch(K),
                                                    position, n, rows, codes, scales);
  else
    expert_dispatch_fp8_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(X), tokens, K, fp8_pitch(K), position, n,
                                                    rows, codes, scales);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

template <typename T, template <typename> class V>
static void combine_as(const void* rows, int64_t K, const int* position, const float* weights, int64_t tokens,
                       int64_t top, void* Y, cudaStream_t s) {
  const RowGrid g = row_grid(tokens, row_vectors<V<T>>(K));
  const auto kernel = top <= 4 ? expert_combine_kernel<T, V, 4> : expert_combine_kernel<T, V, 8>;
  kernel<<<dim3(g.ctas, g.parts), kRowThreads, 0, s>>>(static_cast<const T*>(rows), tokens * top, K, position,
                                                             weights, tokens, static_cast<int>(top), g.tpt,
                                                             static_cast<T*>(Y));
}

template <typename T>
static void combine_typed(const void* rows, int64_t K, const int* position, const float* weights, int64_t tokens,
                          int64_t top, void* Y, cudaStream_t s) {
  if (rows_vec(K * sizeof(T), rows, Y))
    combine_as<T, Vec>(rows, K, position, weights, tokens, top, Y, s);
  else
    combine_as<T, Loose>(rows, K, position, weights, tokens, top, Y, s);
}

hq_status launch_expert_combine(const void* rows, int dtype, int64_t tokens, int64_t K, const int* position, int64_t top,
                                const float* weights, void* Y, cudaStream_t s) {
  if (dtype == HQ_BF16)
    combine_typed<__nv_bfloat16>(rows, K, position, weights, tokens, top, Y, s);
  else
    combine_typed<float>(rows, K, position, weights, tokens, top, Y, s);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

template <typename T, template <typename> class V>
static void combine_backward_as(const void* dY, const void* rows, int64_t K, const int* position, const float* weights,
                                int64_t tokens, int64_t top, void* d_rows, float* d_weights, cudaStream_t s) {
  const RowGrid g = row_grid(tokens, row_vectors<V<T>>(K));
  const auto kernel = top <= 4 ? expert_combine_backward_kernel<T, V, 4> : expert_combine_backward_kernel<T, V, 8>;
  kernel<<<g.ctas, kRowThreads, 0, s>>>(
      static_cast<const T*>(dY), static_cast<const T*>(rows), tokens * top, K, position, weights, tokens,
      static_cast<int>(top), g.tpt, static_cast<T*>(d_rows), d_weights);
}

template <typename T>
static void combine_backward_typed(const void* dY, const void* rows, int64_t K, const int* position,
                                   const float* weights, int64_t tokens, int64_t top, void* d_rows, float* d_weights,
                                   cudaStream_t s) {
  if (rows_vec(K * sizeof(T), dY, rows, d_rows))
    combine_backward_as<T, Vec>(dY, rows, K, position, weights, tokens, top, d_rows, d_weights, s);
  else
    combine_backward_as<T, Loose>(dY, rows, K, position, weights, tokens, top, d_rows, d_weights, s);
}

hq_status launch_expert_combine_backward(const void* dY, const void* rows, int dtype, int64_t tokens, int64_t K,
                                         const int* position, int64_t top, const float* weights, void* d_rows,
                                         float* d_weights, cudaStream_t s) {
  if (dtype == HQ_BF16)
    combine_backward_typed<__nv_bfloat16>(dY, rows, K, position, weights, tokens, top, d_rows, d_weights, s);
  else
    combine_backward_typed<float>(dY, rows, K, position, weights, tokens, top, d_rows, d_weights, s);
  HQ_LAUNCH_CHECK();
  return HQ_OK;
}

}  // namespace hq
