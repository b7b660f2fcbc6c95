// dispatch.hip -- rows to their experts and back.  Row n chose the experts ids[n][0 .. k);
// assignment a = n k + j goes to a place in the order of (expert, a): places[a], a stable
// counting sort; expert e then has the places offsets[e] .. offsets[e + 1].
//   dispatch          rows[places[a]] = x[n]            (places of none: zeros)
//   combine           y[n] = residual[n] + sum_j w[a] rows[places[a]]
//   combine_backward  drows[places[a]] = w[a] dy[n],  dw[a] = <dy[n], rows[places[a]]>
// and dispatch's gradient is a combine without weights.  An id outside [0, experts) goes
// nowhere: place -1.
//
// Memory bounds all but the plan, which is a chain of counts, barriers and scattered 4-byte
// stores.  131072 assignments of 32768 rows to 128 experts, 1024 columns, bf16: plan 17 us (27
// with its assignments and counts one at a time), dispatch 53 us (6.0 TB/s, as x's lines are read
// once), combine with weights and a residual 104 us (3.9 TB/s), without them 78 us (4.3 TB/s; the
// same with a thread for every chunk of the whole matrix), its gradients 105 us (5.5 TB/s; 121 us
// with one of a row's places at a time).  Combine waits for its loads in 82% of its waves' time: a
// row's places come before its rows, and a thread's chunks one after the other.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "layers.hpp"

using namespace tbe;

namespace {

constexpr int kMaxExperts = 2048;
constexpr int64_t kTile = 2048;      // assignments a workgroup, or more:
constexpr int64_t kMostTiles = 256;  // every workgroup reads all tiles' counts
constexpr int kAtATime = 8;          // assignments a lane that are on their way together

struct PlanArgs {
  const void* ids;
  int32_t index64, experts;
  int64_t n;        // assignments
  int64_t tile;     // of them a workgroup's, a multiple of kBlock
  int64_t tiles;
  uint32_t* counts; // [tiles][experts], or null with one tile
  int64_t* offsets;
  int32_t* places;
  int32_t bits;     // of an expert's number
};

// The expert of an assignment, or -1.
__device__ __forceinline__ int expert_of(const PlanArgs& a, int64_t i) {
  const int64_t e = a.index64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

// f(assignment, its expert) for from .. end, `step` lanes side by side; every lane takes part
// to the end (expert -1 past it).
template <typename F>
__device__ __forceinline__ void for_experts(const PlanArgs& a, int64_t from, int64_t end, int lane, int step, F f) {
  for (int64_t i0 = from; i0 < end; i0 += kAtATime * step) {
    int e[kAtATime];
#pragma unroll
    for (int i = 0; i < kAtATime; ++i) {
      const int64_t at = i0 + i * step + lane;
      e[i] = at < end ? expert_of(a, at) : -1;
    }
#pragma unroll
    for (int i = 0; i < kAtATime; ++i)
      if (i0 + i * step < end) f(i0 + i * step + lane, e[i]);
  }
}

__global__ __launch_bounds__(kBlock) void plan_count(PlanArgs a) {
  __shared__ uint32_t count[kMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += kBlock) count[e] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * a.tile, end = std::min(from + a.tile, a.n);
  for_experts(a, from, end, threadIdx.x, kBlock, [&](int64_t, int e) {
    if (e >= 0) atomicAdd(&count[e], 1u);
  });
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kBlock)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.experts + e] = count[e];
}

// A wave takes a quarter of the tile: counts it, finds where each expert's assignments of the
// quarter start, and goes through it 64 at a time, equal ones in their order.
__global__ __launch_bounds__(kBlock) void plan_place(PlanArgs a) {
  __shared__ uint32_t next[kWavesPerBlock][kMaxExperts];
  __shared__ uint32_t scratch[kWavesPerBlock];
  __shared__ uint2 slices[kBlock];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  for (int w = 0; w < kWavesPerBlock; ++w)
    for (int e = threadIdx.x; e < a.experts; e += kBlock) next[w][e] = 0;
  __syncthreads();
  const int64_t quarter = a.tile / kWavesPerBlock;
  const int64_t tile_end = std::min((blockIdx.x + int64_t{1}) * a.tile, a.n);
  const int64_t from = blockIdx.x * a.tile + wave * quarter, end = std::min(from + quarter, tile_end);
  for_experts(a, from, end, lane, kWave, [&](int64_t, int e) {
    if (e >= 0) atomicAdd(&next[wave][e], 1u);
  });
  __syncthreads();
  // Starts: the experts before, the tiles before, the quarters before.  Where there are fewer
  // experts than threads, several threads go through one's tiles.
  const int width = a.experts < kBlock ? 1 << a.bits : kBlock;  // experts at a time
  const int column = threadIdx.x & (width - 1), slice = threadIdx.x / width;
  uint32_t before_all = 0;
  for (int e0 = 0; e0 < a.experts; e0 += width) {
    const int e = e0 + column;
    const bool is = slice == 0 && e < a.experts;
    uint32_t before = 0, total = 0;
    if (a.counts) {
      if (e < a.experts)
#pragma unroll 8
        for (int64_t t = slice; t < a.tiles; t += kBlock / width) {
          const uint32_t c = a.counts[t * a.experts + e];
          total += c;
          before += t < blockIdx.x ? c : 0u;
        }
      slices[threadIdx.x] = make_uint2(total, before);
      __syncthreads();
      if (is)
        for (int i = 1; i < kBlock / width; ++i) {
          total += slices[i * width + column].x;
          before += slices[i * width + column].y;
        }
      __syncthreads();
    } else if (is) {
      for (int w = 0; w < kWavesPerBlock; ++w) total += next[w][e];
    }
    uint32_t sum;
    const uint32_t start = before_all + block_exclusive_sum(is ? total : 0u, scratch, &sum);
    before_all += sum;
    if (is) {
      uint32_t at = start + before;
      for (int w = 0; w < kWavesPerBlock; ++w) {
        const uint32_t c = next[w][e];
        next[w][e] = at;
        at += c;
      }
      if (blockIdx.x == 0) a.offsets[e] = start;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.experts] = before_all;
  __syncthreads();
  for_experts(a, from, end, lane, kWave, [&](int64_t i, int e) {
    const uint64_t real = __ballot(e >= 0);
    const uint64_t peers = match_low_bits(real, static_cast<uint32_t>(e), a.bits);
    const uint32_t rank = popc_below(peers);
    int place = -1;
    if (e >= 0) {
      place = static_cast<int>(next[wave][e] + rank);
      if (rank + 1 == __popcll(peers)) next[wave][e] = place + 1;  // the last of them
    }
    __builtin_amdgcn_wave_barrier();
    if (i < end) a.places[i] = place;
  });
}

struct MoveArgs {
  const void* x;         // dispatch: [rows, cols]; combine: the experts' rows
  const void* residual;  // or null
  const void* grad;
  const float* weights;  // [rows][k], or null: ones
  const int32_t* places;
  const int64_t* total;  // how many places are taken
  void* out;
  float* dweights;       // or null
  int64_t x_stride, r_stride, g_stride, out_stride;
  int64_t rows, cols;
  int32_t k, shift;  // 2^shift lanes have a row
};

// f(WHOLE: whether the thread's chunk at column c ends within the row, known to the compiler)
template <int ST, typename F>
__device__ __forceinline__ void with_end(int64_t c, int64_t cols, F f) {
  if (c + 16 / StorageTraits<ST>::bytes <= cols) f(std::true_type{});
  else f(std::false_type{});
}

// A chunk at column c of the row at element `at`.  Loads have no branches, so that several are
// on their way together: past a row's end the last value is read again, and zeros come of it.
template <int ST>
struct Chunk {
  static constexpr int E = 16 / StorageTraits<ST>::bytes;
  using T = typename Stored<ST>::type;
  StoredVec<ST, E> v = {};
  template <bool WHOLE>
  __device__ __forceinline__ void load(const void* base, int64_t at, int64_t c, int64_t cols) {
    if constexpr (WHOLE) {
      v = load_vec<ST, E>(base, at + c);
    } else {
      T one[E];
#pragma unroll
      for (int i = 0; i < E; ++i) one[i] = static_cast<const T*>(base)[at + (c + i < cols ? c + i : cols - 1)];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = c + i < cols ? one[i] : static_cast<T>(0.0f);
    }
  }
  template <bool WHOLE>
  __device__ __forceinline__ void store(void* base, int64_t at, int64_t c, int64_t cols) const {
    if constexpr (WHOLE) {
      store_vec<ST, E>(base, at + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (c + i < cols) static_cast<T*>(base)[at + c + i] = v[i];
    }
  }
};

// f(j0, how many: up to 4, known to the compiler) for a row's k assignments, four at a time.
template <typename F>
__device__ __forceinline__ void by_fours(int k, F f) {
  int j0 = 0;
  for (; j0 + 4 <= k; j0 += 4) f(j0, std::integral_constant<int, 4>{});
  if (k - j0 == 3) f(j0, std::integral_constant<int, 3>{});
  else if (k - j0 == 2) f(j0, std::integral_constant<int, 2>{});
  else if (k - j0 == 1) f(j0, std::integral_constant<int, 1>{});
}

// The places of C assignments from i on, -1 for none: a wrong one is none.
template <int C>
__device__ __forceinline__ void places_of(const MoveArgs& a, int64_t i, int32_t (&p)[C]) {
#pragma unroll
  for (int j = 0; j < C; ++j) p[j] = a.places[i + j];
#pragma unroll
  for (int j = 0; j < C; ++j) p[j] = p[j] >= 0 && p[j] < a.rows * a.k ? p[j] : -1;
}

// f(n, c) for the chunks of all rows: 2^shift lanes have a row.
template <int E, typename F>
__device__ __forceinline__ void over_chunks(const MoveArgs& a, F f) {
  const int64_t step = (static_cast<int64_t>(gridDim.x) * kBlock) >> a.shift;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) >> a.shift;
  const int lane = static_cast<int>(threadIdx.x) & ((1 << a.shift) - 1);
  for (int64_t n = first; n < a.rows; n += step)
    for (int64_t c = lane * E; c < a.cols; c += E << a.shift) f(n, c);
}

// A thread reads a chunk of a row once and writes it to the row's places (read again for each
// place the rows would be most of the traffic).
template <int ST>
__global__ __launch_bounds__(kBlock) void dispatch_rows(MoveArgs a) {
  const int64_t total = *a.total;
  over_chunks<Chunk<ST>::E>(a, [&](int64_t n, int64_t c) {
    with_end<ST>(c, a.cols, [&](auto whole_) {
      constexpr bool whole = whole_;
      Chunk<ST> v;
      v.template load<whole>(a.x, n * a.x_stride, c, a.cols);
      by_fours(a.k, [&](int j0, auto some_) {
        constexpr int some = some_;
        int32_t p[some];
        places_of(a, n * a.k + j0, p);
#pragma unroll
        for (int j = 0; j < some; ++j)
          if (p[j] >= 0) v.template store<whole>(a.out, p[j] * a.out_stride, c, a.cols);
      });
      // the places that nobody has
      for (int64_t i = n * a.k > total ? n * a.k : total; i < (n + 1) * a.k; ++i)
        Chunk<ST>().template store<whole>(a.out, i * a.out_stride, c, a.cols);
    });
  });
}

// A thread has a chunk of a row: four of the experts' rows at a time, on their way together; one
// that is not there is read at place 0 and left out.
template <int ST>
__global__ __launch_bounds__(kBlock) void combine_rows(MoveArgs a) {
  constexpr int E = Chunk<ST>::E;
  over_chunks<E>(a, [&](int64_t n, int64_t c) {
    with_end<ST>(c, a.cols, [&](auto whole_) {
      constexpr bool whole = whole_;
      float sum[E] = {};
      if (a.residual) {
        Chunk<ST> r;
        r.template load<whole>(a.residual, n * a.r_stride, c, a.cols);
#pragma unroll
        for (int i = 0; i < E; ++i) sum[i] = static_cast<float>(r.v[i]);
      }
      by_fours(a.k, [&](int j0, auto some_) {
        constexpr int some = some_;
        int32_t p[some];
        float w[some];
        Chunk<ST> v[some];
#pragma unroll
        for (int j = 0; j < some; ++j) w[j] = 1.0f;
        if (a.weights) {
#pragma unroll
          for (int j = 0; j < some; ++j) w[j] = a.weights[n * a.k + j0 + j];
        }
        places_of(a, n * a.k + j0, p);
#pragma unroll
        for (int j = 0; j < some; ++j)
          v[j].template load<whole>(a.x, (p[j] < 0 ? 0 : p[j]) * a.x_stride, c, a.cols);
#pragma unroll
        for (int j = 0; j < some; ++j)
#pragma unroll
          for (int i = 0; i < E; ++i) sum[i] += p[j] < 0 ? 0.0f : w[j] * static_cast<float>(v[j].v[i]);
      });
      Chunk<ST> out;
#pragma unroll
      for (int i = 0; i < E; ++i) out.v[i] = static_cast<typename Stored<ST>::type>(sum[i]);
      out.template store<whole>(a.out, n * a.out_stride, c, a.cols);
    });
  });
}

// A wave has a row: its gradient, weighted, to the row's places, and the products with the
// experts' rows there.
template <int ST>
__global__ __launch_bounds__(kBlock) void combine_gradients(MoveArgs a) {
  constexpr int E = Chunk<ST>::E;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t total = *a.total;
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wave; n < a.rows;
       n += static_cast<int64_t>(gridDim.x) * kWavesPerBlock) {
    by_fours(a.k, [&](int j0, auto some_) {
      constexpr int some = some_;
      const int64_t i0 = n * a.k + j0;
      int32_t p[some];
      float w[some], dot[some] = {};
      places_of(a, i0, p);
#pragma unroll
      for (int j = 0; j < some; ++j) w[j] = a.weights[i0 + j];
      for (int64_t c = lane * E; c < a.cols; c += 64 * E)
        with_end<ST>(c, a.cols, [&](auto whole_) {
          constexpr bool whole = whole_;
          Chunk<ST> g, y[some], out;
          g.template load<whole>(a.grad, n * a.g_stride, c, a.cols);
          if (a.dweights) {
#pragma unroll
            for (int j = 0; j < some; ++j)
              y[j].template load<whole>(a.x, (p[j] < 0 ? 0 : p[j]) * a.x_stride, c, a.cols);
          }
#pragma unroll
          for (int j = 0; j < some; ++j)
            if (p[j] >= 0) {
#pragma unroll
              for (int e = 0; e < E; ++e) {
                out.v[e] = static_cast<typename Stored<ST>::type>(w[j] * static_cast<float>(g.v[e]));
                dot[j] += static_cast<float>(g.v[e]) * static_cast<float>(y[j].v[e]);
              }
              out.template store<whole>(a.out, p[j] * a.out_stride, c, a.cols);
            }
        });
      if (a.dweights) {
#pragma unroll
        for (int d = 32; d; d >>= 1)
#pragma unroll
          for (int j = 0; j < some; ++j) dot[j] += __shfl_xor(dot[j], d);
#pragma unroll
        for (int j = 0; j < some; ++j)
          if (lane == j) a.dweights[i0 + j] = dot[j];
      }
    });
    // the places that nobody has
    for (int64_t i = n * a.k > total ? n * a.k : total; i < (n + 1) * a.k; ++i)
      for (int64_t c = lane * E; c < a.cols; c += 64 * E)
        with_end<ST>(c, a.cols, [&](auto whole_) {
          Chunk<ST>().template store<whole_>(a.out, i * a.out_stride, c, a.cols);
        });
  }
}

constexpr int64_t kMaxCols = int64_t{1} << 20;

int64_t tile_of(int64_t n) {
  const int64_t each = (n + kMostTiles - 1) / kMostTiles;
  return std::max(kTile, (each + kBlock - 1) / kBlock * kBlock);
}

size_t plan_bytes(int64_t n, int64_t experts) {
  const int64_t tiles = (n + tile_of(n) - 1) / tile_of(n);
  return tiles > 1 ? static_cast<size_t>(tiles) * experts * sizeof(uint32_t) : 0;
}

tbe_status check_plan(int64_t rows, int64_t k, int64_t experts) {
  if (rows < 0 || k < 1 || experts < 1) return TBE_ERR_INVALID_ARGUMENT;
  if (k > 64 || rows > ((int64_t{1} << 31) - 1) / k || experts > kMaxExperts) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

tbe_status check_move(int64_t rows, int64_t k, int64_t cols, int32_t dtype) {
  if (rows < 0 || k < 1 || cols < 1 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  if (k > 64 || rows > ((int64_t{1} << 31) - 1) / k || cols > kMaxCols) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

MoveArgs move_args(const int32_t* places, int64_t rows, int64_t k, int64_t cols, int32_t dtype) {
  MoveArgs a{};
  a.places = places;
  a.rows = rows;
  a.k = static_cast<int32_t>(k);
  a.cols = cols;
  const int64_t e = 16 / dtype_bytes(dtype);
  while (a.shift < 6 && e << a.shift < cols) ++a.shift;
  return a;
}

dim3 grid_of(int64_t threads) {
  return dim3(static_cast<unsigned>(std::min<int64_t>((threads + kBlock - 1) / kBlock, int64_t{1} << 22)));
}

}  // namespace

extern "C" {

tbe_status tbe_dispatch_plan_size(int64_t rows, int64_t k, int64_t experts, size_t* workspace_bytes) {
  if (!workspace_bytes) return TBE_ERR_INVALID_ARGUMENT;
  const tbe_status st = check_plan(rows, k, experts);
  if (st == TBE_OK) *workspace_bytes = plan_bytes(rows * k, experts);
  return st;
}

tbe_status tbe_dispatch_plan(const void* ids, int32_t index_dtype, int64_t rows, int64_t k, int64_t experts,
                             int64_t* offsets, int32_t* places, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const tbe_status st = check_plan(rows, k, experts);
  if (st != TBE_OK) return st;
  if (index_dtype != TBE_I32 && index_dtype != TBE_I64) return TBE_ERR_INVALID_ARGUMENT;
  if (!offsets || !aligned_to(offsets, 8) || (rows > 0 && (!ids || !places)) || !aligned_to(places, 4) ||
      !aligned_to(ids, index_dtype == TBE_I64 ? 8 : 4))
    return TBE_ERR_INVALID_ARGUMENT;
  PlanArgs a{};
  a.ids = ids;
  a.index64 = index_dtype == TBE_I64;
  a.experts = static_cast<int32_t>(experts);
  a.n = rows * k;
  a.tile = tile_of(a.n);
  a.tiles = std::max<int64_t>(1, (a.n + a.tile - 1) / a.tile);
  a.offsets = offsets;
  a.places = places;
  while ((int64_t{1} << a.bits) < experts) ++a.bits;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.tiles > 1) {
    if (!workspace || !aligned_to(workspace, 256)) return TBE_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < plan_bytes(a.n, experts)) return TBE_ERR_WORKSPACE_TOO_SMALL;
    a.counts = static_cast<uint32_t*>(workspace);
    hipLaunchKernelGGL(plan_count, dim3(static_cast<unsigned>(a.tiles)), dim3(kBlock), 0, s, a);
    if (hipGetLastError() != hipSuccess) return TBE_ERR_HIP;
  }
  hipLaunchKernelGGL(plan_place, dim3(static_cast<unsigned>(a.tiles)), dim3(kBlock), 0, s, a);
  return hipGetLastError() == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

tbe_status tbe_dispatch(const void* x, int64_t x_stride, const int32_t* places, const int64_t* total,
                        void* out, int64_t out_stride, int64_t rows, int64_t k, int64_t cols, int32_t dtype,
                        void* stream) {
  const tbe_status st = check_move(rows, k, cols, dtype);
  if (st != TBE_OK || rows == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!x || !places || !total || !out || !aligned_to(x, e) || !aligned_to(out, e) || !aligned_to(places, 4) ||
      !aligned_to(total, 8))
    return TBE_ERR_INVALID_ARGUMENT;
  if ((rows > 1 && x_stride < 0) || (rows * k > 1 && out_stride < cols)) return TBE_ERR_INVALID_ARGUMENT;
  MoveArgs a = move_args(places, rows, k, cols, dtype);
  a.x = x;
  a.x_stride = x_stride;
  a.total = total;
  a.out = out;
  a.out_stride = out_stride;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid = grid_of(rows << a.shift);
  if (dtype == TBE_F32) hipLaunchKernelGGL(dispatch_rows<kF32>, grid, dim3(kBlock), 0, s, a);
  else if (dtype == TBE_F16) hipLaunchKernelGGL(dispatch_rows<kF16>, grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL(dispatch_rows<kBF16>, grid, dim3(kBlock), 0, s, a);
  return hipGetLastError() == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

tbe_status tbe_combine(const void* y, int64_t y_stride, const int32_t* places, const float* weights,
                       const void* residual, int64_t residual_stride, void* out, int64_t out_stride,
                       int64_t rows, int64_t k, int64_t cols, int32_t dtype, void* stream) {
  const tbe_status st = check_move(rows, k, cols, dtype);
  if (st != TBE_OK || rows == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!y || !places || !out || !aligned_to(y, e) || !aligned_to(out, e) || !aligned_to(residual, e) ||
      !aligned_to(places, 4) || !aligned_to(weights, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  if ((rows * k > 1 && y_stride < 0) || (rows > 1 && (out_stride < cols || (residual && residual_stride < 0))))
    return TBE_ERR_INVALID_ARGUMENT;
  MoveArgs a = move_args(places, rows, k, cols, dtype);
  a.x = y;
  a.x_stride = y_stride;
  a.weights = weights;
  a.residual = residual;
  a.r_stride = residual_stride;
  a.out = out;
  a.out_stride = out_stride;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid = grid_of(rows << a.shift);
  if (dtype == TBE_F32) hipLaunchKernelGGL(combine_rows<kF32>, grid, dim3(kBlock), 0, s, a);
  else if (dtype == TBE_F16) hipLaunchKernelGGL(combine_rows<kF16>, grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL(combine_rows<kBF16>, grid, dim3(kBlock), 0, s, a);
  return hipGetLastError() == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

tbe_status tbe_combine_backward(const void* y, int64_t y_stride, const int32_t* places, const int64_t* total,
                                const float* weights, const void* grad, int64_t grad_stride, void* dy,
                                int64_t dy_stride, float* dweights, int64_t rows, int64_t k, int64_t cols,
                                int32_t dtype, void* stream) {
  const tbe_status st = check_move(rows, k, cols, dtype);
  if (st != TBE_OK || rows == 0) return st;
  const size_t e = dtype_bytes(dtype);
  if (!places || !total || !weights || !grad || !dy || (dweights && !y) || !aligned_to(y, e) ||
      !aligned_to(grad, e) || !aligned_to(dy, e) || !aligned_to(places, 4) || !aligned_to(total, 8) ||
      !aligned_to(weights, 4) || !aligned_to(dweights, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  if ((rows * k > 1 && (y_stride < 0 || dy_stride < cols)) || (rows > 1 && grad_stride < 0))
    return TBE_ERR_INVALID_ARGUMENT;
  MoveArgs a = move_args(places, rows, k, cols, dtype);
  a.x = y;
  a.x_stride = y_stride;
  a.total = total;
  a.weights = weights;
  a.grad = grad;
  a.g_stride = grad_stride;
  a.out = dy;
  a.out_stride = dy_stride;
  a.dweights = dweights;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid = grid_of(rows * kWave);
  if (dtype == TBE_F32) hipLaunchKernelGGL(combine_gradients<kF32>, grid, dim3(kBlock), 0, s, a);
  else if (dtype == TBE_F16) hipLaunchKernelGGL(combine_gradients<kF16>, grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL(combine_gradients<kBF16>, grid, dim3(kBlock), 0, s, a);
  return hipGetLastError() == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

}  // extern "C"
