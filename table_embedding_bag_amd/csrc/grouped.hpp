// grouped.hpp -- kernels of the grouped linear layer (grouped.hip has the
// interface; grouped_f32/f16/bf16.hip each compile them for one type).
//
// The three products, each output tile a loop over the summed index:
//   kForward  y[n, m]     = sum_k x[n, k] W[g, m, k]  (+ bias[g, m])
//   kGradX    dx[n, k]    = sum_m dy[n, m] W[g, m, k]
//   kGradW    dW[g, m, k] = sum_n dy[n, m] x[n, k]    (n over the group's rows)
// Operand A is W, W, x, operand B x, dy, dy; both are k-major in kForward, B is in
// kGradX.  products.hpp has the loop over the summed index.
#pragma once

#include "grouped_plan.hpp"
#include "layers.hpp"
#include "tiles.hpp"
#ifdef TBE_GROUPED_KERNELS
#include "products.hpp"
#endif

namespace tbe {

struct GroupedArgs {
  int64_t rows, groups, K, M;  // K = in_features, M = out_features
  const void* x;
  const void* weight;  // [groups, M, K]
  const void* bias;    // [groups, M] or null
  const void* offsets;
  void* y;
  const void* grad;    // [rows, M]
  void* dx;
  void* dw;
  void* db;
  int64_t x_stride, y_stride, grad_stride, dx_stride;
  int32_t index64;
  int32_t layout;      // kOddRows, kWordRows or kChunkRows, of every operand
  // The weights' gradient: groups of more than chunk rows are summed in chunks
  // (0: never), whose sums go to parts [slots][M * K] and bias_parts [slots][M].
  int64_t chunk, slots;
  float* parts;
  float* bias_parts;
};

// The products of one call; defined for each type in its own file.
hipError_t launch_grouped_f32(const GroupedArgs& a, bool backward, hipStream_t s);
hipError_t launch_grouped_f16(const GroupedArgs& a, bool backward, hipStream_t s);
hipError_t launch_grouped_bf16(const GroupedArgs& a, bool backward, hipStream_t s);

#ifdef TBE_GROUPED_KERNELS

namespace {

enum Product { kForward, kGradX, kGradW };

__device__ __forceinline__ int64_t group_offset(const GroupedArgs& a, int64_t g) {
  const int64_t o = a.index64 ? static_cast<const int64_t*>(a.offsets)[g]
                              : static_cast<const int32_t*>(a.offsets)[g];
  return o < 0 ? 0 : (o > a.rows ? a.rows : o);
}

// Which tile of the groups' ragged tilings a workgroup takes.
struct Tile {
  int64_t group, first, end;  // rows of the group
  int64_t ta, tb;             // tile numbers along A's and B's free index
};

// Row tiles of TB rows, `na` tiles along the other index; false where the
// workgroup has none.  Every wave works it out for itself: 64 groups at a time,
// and with no more than that from one read of the offsets.
template <int TB>
__device__ bool find_row_tile(const GroupedArgs& a, uint32_t id, uint32_t blocks, int64_t na, Tile* t) {
  const int lane = lane_id();
  uint32_t lo = 0, rows = 0, tiles = 0, incl = 0;  // of the lane's group
  const auto take = [&](int64_t g0) {
    lo = rows = 0;
    if (g0 + lane < a.groups) {
      const int64_t first = group_offset(a, g0 + lane), n = group_offset(a, g0 + lane + 1) - first;
      lo = static_cast<uint32_t>(first);
      rows = n > 0 ? static_cast<uint32_t>(n) : 0u;
    }
    tiles = (rows + TB - 1) / TB;
    incl = wave_inclusive_sum(tiles);
  };
  int64_t total = 0;
  for (int64_t g0 = 0; g0 < a.groups; g0 += 64) {
    take(g0);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  int64_t q;
  if (!tile_number(id, blocks, total * na, &q)) return false;
  for (int64_t g0 = 0; g0 < a.groups; g0 += 64) {
    if (a.groups > 64) take(g0);
    const uint64_t past = __ballot(static_cast<int64_t>(incl) * na > q);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int64_t before = __builtin_amdgcn_readlane(incl - tiles, l);
      t->group = g0 + l;
      t->first = __builtin_amdgcn_readlane(lo, l);
      t->end = t->first + __builtin_amdgcn_readlane(rows, l);
      band_order(q - before * na, na, __builtin_amdgcn_readlane(tiles, l), &t->ta, &t->tb);
      return true;
    }
    q -= static_cast<int64_t>(__builtin_amdgcn_readlane(incl, 63)) * na;
  }
  return false;
}


// Row chunk `unit` of the groups' chunks of a.chunk rows (an empty group has one):
// its group and rows, and its slot among the chunks of the groups that have
// several, or -1; false where there are fewer.
struct Unit {
  int64_t group, first, end, slot;
};
__device__ bool find_chunk(const GroupedArgs& a, int64_t unit, Unit* u) {
  const int lane = lane_id();
  int64_t slots = 0;
  for (int64_t g0 = 0; g0 < a.groups; g0 += 64) {
    int64_t lo = 0, n = 0;
    const bool real = g0 + lane < a.groups;
    if (real) {
      lo = group_offset(a, g0 + lane);
      n = group_offset(a, g0 + lane + 1) - lo;
      n = n > 0 ? n : 0;
    }
    uint32_t chunks = static_cast<uint32_t>((n + a.chunk - 1) / a.chunk);
    if (real && chunks == 0) chunks = 1;
    const uint32_t many = chunks > 1 ? chunks : 0;
    const uint32_t incl = wave_inclusive_sum(chunks), slot = wave_inclusive_sum(many);
    const uint64_t past = __ballot(static_cast<int64_t>(incl) > unit);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int64_t c = unit - __builtin_amdgcn_readlane(incl - chunks, l);
      const int64_t rows = __builtin_amdgcn_readlane(static_cast<uint32_t>(n), l);
      u->group = g0 + l;
      u->first = __builtin_amdgcn_readlane(static_cast<uint32_t>(lo), l) + c * a.chunk;
      u->end = u->first + (rows - c * a.chunk < a.chunk ? rows - c * a.chunk : a.chunk);
      u->slot = __builtin_amdgcn_readlane(many, l)
                    ? slots + __builtin_amdgcn_readlane(slot - many, l) + c
                    : -1;
      return true;
    }
    unit -= __builtin_amdgcn_readlane(incl, 63);
    slots += __builtin_amdgcn_readlane(slot, 63);
  }
  return false;
}

// The group with the r-th most rows (of up to 64; more are taken as they come).
__device__ int64_t ranked_group(const GroupedArgs& a, int64_t r) {
  if (a.groups > 64) return r;
  const int lane = lane_id();
  int32_t n = -1;
  if (lane < a.groups) n = static_cast<int32_t>(group_offset(a, lane + 1) - group_offset(a, lane));
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const int32_t other = __builtin_amdgcn_readlane(n, g);
    rank += other > n || (other == n && g < lane);
  }
  const uint64_t is = __ballot(lane < a.groups && rank == r);
  return is ? __builtin_ctzll(is) : r;
}

// A long sum in two floats: what each addition rounds off is exact in fp32 and added up
// beside it, so that the sum is off by some half steps of itself whatever its length.
// (One float's additions round one way once the sum is large: 32768 rows of 0.1 came out
// 1.5e-4 off.)
struct LongSum {
  float sum = 0.0f, low = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float s = sum + v, from = s - sum;
    low += (sum - (s - from)) + (v - from);
    sum = s;
  }
  // An infinite sum leaves NaN in low.
  __device__ __forceinline__ float value() const {
    return __builtin_isfinite(low) ? sum + low : sum;
  }
};
// The sum of a few values, two by two.
template <int N>
__device__ __forceinline__ float sum_of(const float (&v)[N]) {
  static_assert(N == 4 || N == 8);
  const float four = (v[0] + v[1]) + (v[2] + v[3]);
  if constexpr (N == 4) return four;
  else return four + ((v[4] + v[5]) + (v[6] + v[7]));
}

// The tile that workgroup `id` of a product's `blocks` takes.
template <int ST, Product P, typename S, int LAYOUT>
__device__ __forceinline__ void product(const GroupedArgs& a, uint32_t id, uint32_t blocks,
                                        unsigned char* lds) {
  constexpr bool kAKmaj = P == kForward, kBKmaj = P != kGradW;
  constexpr int kAhead = kHeldSlices<S, LAYOUT>;
  using OpA = Operand<ST, kAKmaj, S::TA, S::NW, LAYOUT, S::RB, kAhead>;
  using OpB = Operand<ST, kBKmaj, S::TB, S::NW, LAYOUT, S::RB, kAhead>;
  constexpr int bytes = StorageTraits<ST>::bytes;

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t cols = P == kForward ? a.M : a.K;      // of the output: A's free index
  const int64_t na = (cols + S::TA - 1) / S::TA;
  Tile t;
  int64_t slot = -1;
  if constexpr (P == kGradW) {
    // A group's (or chunk's) tiles spread over all XCDs, each taking a contiguous
    // part of them; groups with the most rows come first, so that short ones fill
    // the gaps at the end.
    const int64_t nb = (a.M + S::TB - 1) / S::TB, tiles = na * nb, unit = id / tiles;
    const int64_t q = xcd_contiguous_block(static_cast<int>(id - unit * tiles),
                                           static_cast<int>(tiles));
    if (a.chunk) {
      Unit u;
      if (!find_chunk(a, unit, &u)) return;
      t.group = u.group, t.first = u.first, t.end = u.end, slot = u.slot;
      if (slot >= a.slots) return;  // groups that overlap: bad offsets
    } else {
      if (unit >= a.groups) return;  // where workgroups are rounded up to the XCDs
      t.group = ranked_group(a, unit);
      t.first = group_offset(a, t.group);
      t.end = group_offset(a, t.group + 1);
      if (t.end < t.first) t.end = t.first;
    }
    band_order(q, na, nb, &t.ta, &t.tb);
  } else {
    if (!find_row_tile<S::TB>(a, id, blocks, na, &t)) return;
  }
  const int64_t a0 = t.ta * S::TA, b0 = t.tb * S::TB;
  const int64_t out_rows = P == kGradW ? a.M - b0 : t.end - t.first - b0;
  const int64_t depth = P == kForward ? a.K : P == kGradX ? a.M : t.end - t.first;
  if (out_rows <= 0) return;
  const char* w = static_cast<const char*>(a.weight) + t.group * a.M * a.K * bytes;
  const char* x = static_cast<const char*>(a.x) + t.first * a.x_stride * bytes;
  const char* dy = static_cast<const char*>(a.grad) + t.first * a.grad_stride * bytes;

  OpA oa;
  OpB ob;
  if constexpr (P == kForward) {
    oa.init(w + a0 * a.K * bytes, a.K, cols - a0, depth, wave, lane);
    ob.init(x + b0 * a.x_stride * bytes, a.x_stride, out_rows, depth, wave, lane);
  } else if constexpr (P == kGradX) {
    oa.init(w + a0 * bytes, a.K, cols - a0, depth, wave, lane);
    ob.init(dy + b0 * a.grad_stride * bytes, a.grad_stride, out_rows, depth, wave, lane);
  } else {
    oa.init(x + a0 * bytes, a.x_stride, cols - a0, depth, wave, lane);
    ob.init(dy + b0 * bytes, a.grad_stride, out_rows, depth, wave, lane);
  }

  const int wa = (wave % S::NA) * S::WA * 32, wb = (wave / S::NA) * S::WB * 32;
  f32x16 acc[S::WA][S::WB];
#pragma unroll
  for (int i = 0; i < S::WA; ++i)
#pragma unroll
    for (int j = 0; j < S::WB; ++j) acc[i][j] = f32x16{};

  // The bias's gradient: the sums of operand B's columns (dy) over the rows, by the
  // waves that have them first, each lane half of the rows.
  const bool sums = P == kGradW && a.db && t.ta == 0 && wave % S::NA == 0;
  LongSum column_sum[S::WB];
  auto add_columns = [&](const u32x4 (&fragments)[S::WB]) {
#pragma unroll
    for (int j = 0; j < S::WB; ++j) {
      const auto v = __builtin_bit_cast(StoredVec<ST, 16 / bytes>, fragments[j]);
      float f[16 / bytes];
#pragma unroll
      for (int e = 0; e < 16 / bytes; ++e) f[e] = static_cast<float>(v[e]);
      column_sum[j].add(sum_of(f));
    }
  };
  accumulate<ST, S, LAYOUT>(oa, ob, depth, lds, wa, wb, wave, lane, acc,
                            [&](const u32x4 (&fragments)[S::WB]) {
                              if constexpr (P == kGradW)
                                if (sums) add_columns(fragments);
                            });

#pragma unroll
  for (int i = 0; i < S::WA; ++i) {
    const int64_t c0 = a0 + wa + 32 * i;   // output columns c0 .. c0 + 31
    if (c0 >= cols) continue;
    if constexpr (P == kForward) {
      if (a.bias) {  // one value for each of the lane's columns, the same for all rows
        f32x16 b;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t c = c0 + 8 * q + 4 * (lane >> 5), at = t.group * a.M + c;
          StoredVec<ST, 4> four = {};
          if (c + 4 <= cols) {
            four = load_vec<ST, 4>(a.bias, at);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c + e < cols) four[e] = static_cast<const typename Stored<ST>::type*>(a.bias)[at + e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) b[4 * q + e] = static_cast<float>(four[e]);
        }
#pragma unroll
        for (int j = 0; j < S::WB; ++j) acc[i][j] += b;
      }
    }
#pragma unroll
    for (int j = 0; j < S::WB; ++j) {
      const int64_t r = b0 + wb + 32 * j + (lane & 31);
      const bool row = r - b0 < out_rows;
      if (P == kGradW && slot >= 0) {
        store_fragment<kF32>(a.parts + (slot * a.M + r) * a.K + c0, acc[i][j], cols - c0, row, lane);
        continue;
      }
      char* p;
      if constexpr (P == kForward)
        p = static_cast<char*>(a.y) + ((t.first + r) * a.y_stride + c0) * bytes;
      else if constexpr (P == kGradX)
        p = static_cast<char*>(a.dx) + ((t.first + r) * a.dx_stride + c0) * bytes;
      else
        p = static_cast<char*>(a.dw) + ((t.group * a.M + r) * a.K + c0) * bytes;
      store_fragment<ST>(p, acc[i][j], cols - c0, row, lane);
    }
  }
  if constexpr (P == kGradW) {
    if (sums) {
#pragma unroll
      for (int j = 0; j < S::WB; ++j) {
        const float half = column_sum[j].value(), v = half + __shfl_xor(half, 32);
        const int64_t m = b0 + wb + 32 * j + lane;
        if (lane < 32 && m < a.M) {
          if (slot >= 0) a.bias_parts[slot * a.M + m] = v;
          else store_one<ST>(a.db, t.group * a.M + m, v);
        }
      }
    }
  }
}

template <int ST, Product P, typename S, int LAYOUT>
__global__ __launch_bounds__(S::threads) void grouped_product(GroupedArgs a) {
  __shared__ __align__(1024) unsigned char lds[kLdsBytes<S, LAYOUT>];
  product<ST, P, S, LAYOUT>(a, blockIdx.x, gridDim.x, lds);
}

// Both gradients' products where their tiles have one shape: the second's fill the
// CUs that the first's last round leaves idle.  `first` workgroups, a multiple of
// the XCDs, have the weights'.
template <int ST, typename S, int LAYOUT>
__global__ __launch_bounds__(S::threads) void grouped_gradients(GroupedArgs a, uint32_t first) {
  __shared__ __align__(1024) unsigned char lds[kLdsBytes<S, LAYOUT>];
  if (blockIdx.x < first) product<ST, kGradW, S, LAYOUT>(a, blockIdx.x, first, lds);
  else product<ST, kGradX, S, LAYOUT>(a, blockIdx.x - first, gridDim.x - first, lds);
}

// The chunks' sums of a group, first chunk first, to its gradients.
template <int ST>
__global__ __launch_bounds__(kBlock) void grouped_join(GroupedArgs a, int64_t blocks) {
  const int64_t g = blockIdx.x / blocks, block = blockIdx.x - g * blocks;
  int64_t slot = 0, mine = 0;  // of this group's first chunk; its chunks
  const int lane = lane_id();
  for (int64_t g0 = 0; g0 <= g; g0 += 64) {
    uint32_t many = 0;
    if (g0 + lane <= g) {
      const int64_t n = group_offset(a, g0 + lane + 1) - group_offset(a, g0 + lane);
      many = n > a.chunk ? static_cast<uint32_t>((n + a.chunk - 1) / a.chunk) : 0;
    }
    const uint32_t sum = wave_inclusive_sum(many);
    slot += __builtin_amdgcn_readlane(sum, 63);
    if (g - g0 < 64) mine = __builtin_amdgcn_readlane(many, static_cast<int>(g - g0));
  }
  slot -= mine;
  // written by its only chunk; or bad offsets
  if (mine == 0 || slot + mine > a.slots) return;
  const int64_t all = a.M * a.K;
  const int64_t e0 = (block * kBlock + threadIdx.x) * 4;
  if (e0 < all) {
    f32x4 sum = {};
    const int n = all - e0 < 4 ? static_cast<int>(all - e0) : 4;
    const float* p = a.parts + slot * all + e0;
    if (n == 4) {
#pragma unroll 8
      for (int64_t c = 0; c < mine; ++c) sum += load_vec<kF32, 4>(p, c * all);
      StoredVec<ST, 4> out;
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = static_cast<typename Stored<ST>::type>(sum[j]);
      store_vec<ST, 4>(a.dw, g * all + e0, out);
    } else {
      for (int64_t c = 0; c < mine; ++c)
        for (int j = 0; j < n; ++j) sum[j] += p[c * all + j];
      for (int j = 0; j < n; ++j) store_one<ST>(a.dw, g * all + e0 + j, sum[j]);
    }
  }
  if (a.db) {
    const int64_t m = block * kBlock + threadIdx.x;
    if (m < a.M) {
      LongSum sum;
#pragma unroll 8
      for (int64_t c = 0; c < mine; ++c) sum.add(a.bias_parts[(slot + c) * a.M + m]);
      store_one<ST>(a.db, g * a.M + m, sum.value());
    }
  }
}

// The bias's gradient where the weights' is not wanted: a workgroup sums 64 columns
// of one group, 16 rows at a time.
template <int ST>
__global__ __launch_bounds__(1024) void grouped_bias_grad(GroupedArgs a) {
  __shared__ float part[16][64];
  const int64_t g = blockIdx.y;
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t end = group_offset(a, g + 1);
  LongSum sum;
  if (c < a.M) {
    int64_t n = group_offset(a, g) + w;
    for (; n + 48 < end; n += 64) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = load_one<ST>(a.grad, (n + 16 * i) * a.grad_stride + c);
      sum.add(sum_of(f));
    }
    for (; n < end; n += 16) sum.add(load_one<ST>(a.grad, n * a.grad_stride + c));
  }
  part[w][lane] = sum.value();
  __syncthreads();
  if (w == 0 && c < a.M) {
    LongSum all;
    for (int i = 0; i < 16; ++i) all.add(part[i][lane]);
    store_one<ST>(a.db, g * a.M + c, all.value());
  }
}

// Workgroups of a product.
template <Product P, typename S>
int64_t workgroups(const GroupedArgs& a) {
  const int64_t na = ceil_div(P == kForward ? a.M : a.K, S::TA);
  // a group's last row tile (or chunk) may be partial: at most one more for each group
  const int64_t units = P != kGradW ? a.rows / S::TB + std::min(a.groups, a.rows)
                        : a.chunk   ? a.rows / a.chunk + a.groups
                                    : a.groups;
  return na * units * (P == kGradW ? ceil_div(a.M, S::TB) : 1);
}

// f(the layout, known to the compiler).  (16384 rows in 8 equal groups, bf16, forward:
// odd rows 1021 -> 1021 66 us, 4095 -> 4095 628; rows of words 1022 57, 4094 526 (as odd
// ones 605); chunks 1024 45, 4096 467.)
template <int ST, typename F>
void with_layout(const GroupedArgs& a, F f) {
  if (a.layout == kChunkRows) return f(std::integral_constant<int, kChunkRows>{});
  if constexpr (StorageTraits<ST>::bytes == 2)
    if (a.layout == kOddRows) return f(std::integral_constant<int, kOddRows>{});
  f(std::integral_constant<int, kWordRows>{});
}

template <int ST, Product P, typename S>
hipError_t launch_product(const GroupedArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(workgroups<P, S>(a)));
  with_layout<ST>(a, [&](auto layout) {
    hipLaunchKernelGGL((grouped_product<ST, P, S, layout>), grid, dim3(S::threads), 0, s, a);
  });
  return hipGetLastError();
}

template <int ST, typename S>
hipError_t launch_gradients(const GroupedArgs& a, hipStream_t s) {
  const int64_t first = (workgroups<kGradW, S>(a) + 7) / 8 * 8;
  const dim3 grid(static_cast<unsigned>(first + workgroups<kGradX, S>(a)));
  with_layout<ST>(a, [&](auto layout) {
    hipLaunchKernelGGL((grouped_gradients<ST, S, layout>), grid, dim3(S::threads), 0, s, a,
                       static_cast<uint32_t>(first));
  });
  return hipGetLastError();
}

// Tiles of 256 x 256 feed the matrix cores with the fewest bytes: at 32768 x 4096 ->
// 4096 bf16 they run at 1.1 PFLOP/s of random values and 1.5 of zeros, so it is the
// power that bounds them (four waves of 128 x 128 a tile, slices of half the length,
// four slices by LDS, or 256 x 128 with two workgroups a CU: 1.03 to 1.5 ms instead of
// 1.0).
using Large = Shape<256, 256, 2, 4, 2, 128>;
using Medium = Shape<128, 128, 2, 2, 2, 128>;
using Square = Shape<64, 64, 2, 2, 4, 128>;
using Narrow = Shape<128, 32, 4, 1, 4, 128>;

template <int ST, Product P>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t s) {
  const int tile = row_tile(a.rows, a.groups, P == kForward ? a.M : a.K, ST);
  if constexpr (ST != kF32)
    if (tile == 256) return launch_product<ST, P, Large>(a, s);
  return tile == 128   ? launch_product<ST, P, Medium>(a, s)
         : tile == 64  ? launch_product<ST, P, Square>(a, s)
                       : launch_product<ST, P, Narrow>(a, s);
}

template <int ST>
hipError_t launch_backward(const GroupedArgs& a, hipStream_t s) {
  const bool dx = a.dx && a.rows > 0;
  hipError_t e = hipSuccess;
  if (a.dw) {
    const BackwardPlan plan = plan_backward(a.rows, a.groups, a.K, a.M, dx, ST);
    const bool both = plan.both;
    if (dx && !both) e = launch_rows<ST, kGradX>(a, s);
    if (e != hipSuccess) return e;
    const auto go = [&](auto shape) {
      using S = decltype(shape);
      return both ? launch_gradients<ST, S>(a, s) : launch_product<ST, kGradW, S>(a, s);
    };
    if constexpr (ST == kF32)
      e = plan.w.tile == 128 ? go(Medium{}) : go(Square{});
    else
      e = plan.w.tile == 256 ? go(Large{}) : plan.w.tile == 128 ? go(Medium{}) : go(Square{});
    if (e != hipSuccess || plan.w.slots == 0) return e;
    const int64_t blocks = ceil_div(std::max(ceil_div(a.M * a.K, 4), a.M), kBlock);
    hipLaunchKernelGGL((grouped_join<ST>), dim3(static_cast<unsigned>(blocks * a.groups)),
                       dim3(kBlock), 0, s, a, blocks);
    return hipGetLastError();
  }
  if (dx) e = launch_rows<ST, kGradX>(a, s);
  if (e == hipSuccess && a.db) {
    hipLaunchKernelGGL((grouped_bias_grad<ST>),
                       dim3(static_cast<unsigned>(ceil_div(a.M, 64)), static_cast<unsigned>(a.groups)),
                       dim3(1024), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

template <int ST>
hipError_t launch_grouped(const GroupedArgs& a, bool backward, hipStream_t s) {
  return backward ? launch_backward<ST>(a, s) : launch_rows<ST, kForward>(a, s);
}

}  // namespace

#endif  // TBE_GROUPED_KERNELS

}  // namespace tbe
