// grouped.hpp -- kernels of the grouped linear layer (grouped.hip has the
// interface; grouped_f32/f16/bf16.hip each compile them for one type).
//
// The three products, each output tile a loop over the summed index:
//   kForward  y[n, m]     = sum_k x[n, k] W[g, m, k]  (+ bias[g, m])
//   kGradX    dx[n, k]    = sum_m dy[n, m] W[g, m, k]
//   kGradW    dW[g, m, k] = sum_n dy[n, m] x[n, k]    (n over the group's rows)
// Operand A is the one whose free index runs along the output's rows in memory
// (W, W, x), operand B the other (x, dy, dy): the matrix instruction leaves
// four neighbours of its row index in a lane, so they make wide stores.  An
// operand is "k-major" where the summed index is the one adjacent in memory
// (both in kForward, B in kGradX) and "free-major" otherwise.
//
// A workgroup stages slices of 128 bytes of the summed index (64 16-bit or 32
// fp32 values) of both operands in LDS, in 16-byte chunks:
//   k-major     row r of the tile at 128 r, chunk c at slot c ^ (r / 2 & 7), so that
//               16 lanes that read one chunk of 16 rows cover the 256 bytes of the
//               banks once (c ^ (r & 7) made half of the reads' cycles conflicts);
//   free-major  row k of the slice at k * (tile width), 16-bit chunks c at slot
//               c ^ 4 (k & 3): the transposing LDS read takes 4 rows x 16 columns
//               for each 16 lanes, and this spreads the rows over the banks.
// Aligned operands go from memory to LDS directly (buffer loads that write LDS,
// their descriptor's bounds giving zeros past the rows' and the group's ends);
// others through registers, element by element at the ends.
#pragma once

#include "layers.hpp"

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
  int32_t direct;      // every operand's rows are whole, aligned 16-byte chunks
};

// The products of one call; defined for each type in its own file.
hipError_t launch_grouped_f32(const GroupedArgs& a, bool backward, hipStream_t s);
hipError_t launch_grouped_f16(const GroupedArgs& a, bool backward, hipStream_t s);
hipError_t launch_grouped_bf16(const GroupedArgs& a, bool backward, hipStream_t s);

#ifdef TBE_GROUPED_KERNELS

namespace {

enum Product { kForward, kGradX, kGradW };

using f32x16 = float __attribute__((ext_vector_type(16)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using i16x4 = short __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

#define TBE_LDS(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int kRowBytes = 128;                 // of the summed index in a slice
constexpr uint32_t kOutside = 0x80000000u;     // past every descriptor's end

// Tile shape: TA x TB outputs, NA x NB waves, NS slices of LDS.
template <int TA_, int TB_, int NA_, int NB_, int NS_>
struct Shape {
  static constexpr int TA = TA_, TB = TB_, NA = NA_, NB = NB_, NS = NS_;
  static constexpr int NW = NA * NB, threads = 64 * NW;
  static constexpr int WA = TA / NA / 32, WB = TB / NB / 32;  // 32 x 32 outputs a wave
  static constexpr int stage = (TA + TB) * kRowBytes;
};

__device__ __forceinline__ int64_t group_offset(const GroupedArgs& a, int64_t g) {
  const int64_t o = a.index64 ? static_cast<const int64_t*>(a.offsets)[g]
                              : static_cast<const int32_t*>(a.offsets)[g];
  return o < 0 ? 0 : (o > a.rows ? a.rows : o);
}

// Which tile of the groups' ragged tilings a workgroup takes.  Workgroups go
// round robin to the XCDs; each XCD takes a contiguous range of tiles, and
// within a group the tiles run in bands of 8 row tiles, so that what an XCD
// works on at one time shares operand tiles in its L2.
struct Tile {
  int64_t group, first, end;  // rows of the group
  int64_t ta, tb;             // tile numbers along A's and B's free index
};

__device__ __forceinline__ void band_order(int64_t q, int64_t na, int64_t nb, Tile* t) {
  constexpr int64_t kBand = 8;
  const int64_t band = q / (kBand * na), r = q - band * kBand * na;
  const int64_t height = nb - band * kBand < kBand ? nb - band * kBand : kBand;
  t->ta = r / height;
  t->tb = band * kBand + r % height;
}

// Row tiles of TB rows, `na` tiles along the other index; false where the
// workgroup has none.  Every wave works it out for itself: 64 groups at a time.
template <int TB>
__device__ bool find_row_tile(const GroupedArgs& a, int64_t na, Tile* t) {
  const int lane = lane_id();
  int64_t total = 0;
  for (int64_t g0 = 0; g0 < a.groups; g0 += 64) {
    int64_t n = 0;
    if (g0 + lane < a.groups) {
      n = group_offset(a, g0 + lane + 1) - group_offset(a, g0 + lane);
      n = n > 0 ? (n + TB - 1) / TB : 0;
    }
    total += __builtin_amdgcn_readlane(wave_inclusive_sum(static_cast<uint32_t>(n)), 63);
  }
  total *= na;
  if (static_cast<int64_t>(blockIdx.x) >= total) return false;
  int64_t q = xcd_contiguous_block(static_cast<int>(blockIdx.x), static_cast<int>(total));
  for (int64_t g0 = 0; g0 < a.groups; g0 += 64) {
    int64_t lo = 0, n = 0;
    if (g0 + lane < a.groups) {
      lo = group_offset(a, g0 + lane);
      n = group_offset(a, g0 + lane + 1) - lo;
      n = n > 0 ? n : 0;
    }
    const uint32_t tiles = static_cast<uint32_t>((n + TB - 1) / TB);
    const uint32_t incl = wave_inclusive_sum(tiles);
    const uint64_t past = __ballot(static_cast<int64_t>(incl) * na > q);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int64_t before = __builtin_amdgcn_readlane(incl - tiles, l);
      t->group = g0 + l;
      t->first = static_cast<int64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(lo), l));
      t->end = t->first + __builtin_amdgcn_readlane(static_cast<uint32_t>(n), l);
      band_order(q - before * na, na, __builtin_amdgcn_readlane(tiles, l), t);
      return true;
    }
    q -= static_cast<int64_t>(__builtin_amdgcn_readlane(incl, 63)) * na;
  }
  return false;
}

// 16 bytes a lane from a buffer to LDS at `lds` + 16 lane; zeros for offsets past
// the buffer's end.  In assembly (it writes no register) because the compiler,
// which cannot tell the slices apart, waits for all such loads before it reads
// LDS with the transposing instruction; wait_loads() waits for them here.  (m0
// is never kept by the compiler, which sets it before each use of its own.)
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t offset, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
      ::"s"(lds), "v"(offset), "s"(rsrc)
      : "memory");
}

// One operand of a tile: where its chunks come from and which exist.
//   KMAJ: `free` rows of the tile at base + r * stride, the summed index along them.
//   else: rows of the summed index at base + k * stride, `free` columns along them.
template <int ST, bool KMAJ, int R, int NW, bool DIRECT>
struct Operand {
  static constexpr int bytes = StorageTraits<ST>::bytes;
  static constexpr int EL = 16 / bytes;            // values in a chunk
  static constexpr int BK = kRowBytes / bytes;     // summed values in a slice
  static constexpr int CPR = KMAJ ? 8 : R * bytes / 16;  // chunks in a row
  static constexpr int NL = R * 8 / (64 * NW);     // chunks a thread
  static constexpr int kFragmentReads = KMAJ ? 1 : bytes == 2 ? 2 : 4;
  static_assert(NL >= 1, "every thread has a chunk");

  const char* base;
  int64_t stride;            // bytes
  int32_t free, depth;       // bounds of the free index from the tile's start, of the summed one
  uint32_t off[DIRECT ? NL : 1];
  uint32_t column[DIRECT ? NL : 1];
  u32x4 held[DIRECT ? 1 : NL];

  // Row and (global) chunk that thread's i-th LDS chunk holds.
  static __device__ __forceinline__ void place(int i, int wave, int lane, int* row, int* chunk) {
    const int q = (i * NW + wave) * 64 + lane;
    *row = q / CPR;
    const int slot = q % CPR;
    if constexpr (KMAJ) *chunk = slot ^ (*row >> 1 & 7);
    else if constexpr (bytes == 2) *chunk = slot ^ ((4 * (*row & 3)) & (CPR - 1));
    else *chunk = slot;
  }

  __device__ __forceinline__ void init(const void* p, int64_t stride_, int64_t free_, int64_t depth_,
                                       int wave, int lane) {
    base = static_cast<const char*>(p);
    stride = stride_ * bytes;
    free = static_cast<int32_t>(free_ < R ? free_ : R);
    depth = static_cast<int32_t>(depth_);
    if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        int row, chunk;
        place(i, wave, lane, &row, &chunk);
        const bool inside = (KMAJ ? row : chunk * EL) < free;
        off[i] = inside ? static_cast<uint32_t>(row * stride) + chunk * 16 : kOutside;
        column[i] = KMAJ ? chunk * EL : row;   // along the summed index
      }
    }
  }

  // Start the loads of the slice at k0: into LDS at `to`, or into registers.
  __device__ __forceinline__ void issue(int32_t k0, unsigned char* to, int wave, int lane) {
    const int32_t left = depth - k0;  // at most 0: a slice past the end, all zeros
    if constexpr (DIRECT) {
      const char* p = base + (KMAJ ? static_cast<int64_t>(k0) * bytes : k0 * stride);
      int64_t extent;
      if constexpr (KMAJ) extent = (free - 1) * stride + static_cast<int64_t>(left) * bytes;
      else extent = ((left < BK ? left : BK) - 1) * stride + static_cast<int64_t>(free) * bytes;
      const uint32_t records = left > 0 ? static_cast<uint32_t>(extent) : 0u;
      const uint64_t at = reinterpret_cast<uint64_t>(p);
      const u32x4 rsrc = {static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32) & 0xFFFFu, records,
                          0x00020000u};
      const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(TBE_LDS(void, to)));
#pragma unroll
      for (int i = 0; i < NL; ++i)
        load_to_lds(rsrc, static_cast<int32_t>(column[i]) < left ? off[i] : kOutside,
                    lds + (i * NW + wave) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        int row, chunk;
        place(i, wave, lane, &row, &chunk);
        const int32_t r = KMAJ ? row : chunk * EL;        // free index
        const int32_t k = KMAJ ? chunk * EL : row;        // summed index
        const int64_t e = KMAJ ? k0 + k : r;              // first element along the memory row
        const char* p = base + (KMAJ ? r * stride : static_cast<int64_t>(k0 + k) * stride);
        const int32_t room = KMAJ ? left - k : free - r;  // elements of the chunk that exist
        const bool any = KMAJ ? r < free : k < left;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (any && room >= EL) {
          v = __builtin_bit_cast(u32x4, load_vec<ST, EL>(p, e));
        } else if (any && room > 0) {
          StoredVec<ST, EL> w = __builtin_bit_cast(StoredVec<ST, EL>, v);
#pragma unroll
          for (int j = 0; j < EL; ++j)
            if (j < room) w[j] = reinterpret_cast<const typename Stored<ST>::type*>(p)[e + j];
          v = __builtin_bit_cast(u32x4, w);
        }
        held[i] = v;
      }
    }
  }

  // Registers to LDS (operands that are not loaded there directly).
  __device__ __forceinline__ void put(unsigned char* to, int wave, int lane) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        *reinterpret_cast<u32x4*>(to + (i * NW + wave) * 1024 + lane * 16) = held[i];
    }
  }

  // The lane's fragment of the 32 free indices from `at`, 16 bytes of the summed
  // index: those of chunk 2 kk + lane / 32.  k-major: one chunk.  Free-major,
  // 16-bit: two transposing reads, four summed values each; fp32: four values.
  static __device__ __forceinline__ u32x4 fragment(const unsigned char* from, int at, int kk,
                                                   int lane) {
    if constexpr (KMAJ) {
      const int row = at + (lane & 31), chunk = (2 * kk + (lane >> 5)) ^ (lane >> 1 & 7);
      return *reinterpret_cast<const u32x4*>(from + row * kRowBytes + chunk * 16);
    } else if constexpr (bytes == 2) {
      const int k = 16 * kk + 8 * (lane >> 5) + ((lane & 15) >> 2);
      const int col = at + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      const int slot = (col >> 3) ^ ((4 * (k & 3)) & (CPR - 1));
      const unsigned char* p = from + k * (CPR * 16) + slot * 16 + (col & 7) * 2;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(TBE_LDS(i16x4, p));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(TBE_LDS(i16x4, p + 4 * CPR * 16));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int k = 4 * (2 * kk + (lane >> 5)), col = at + (lane & 31);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(from) + k * R + col;
      return u32x4{p[0], p[R], p[2 * R], p[3 * R]};
    }
  }
};

template <int ST>
__device__ __forceinline__ f32x16 multiply(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (ST == kBF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(StoredVec<kBF16, 8>, a),
                                                   __builtin_bit_cast(StoredVec<kBF16, 8>, b), c, 0,
                                                   0, 0);
  } else if constexpr (ST == kF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(StoredVec<kF16, 8>, a),
                                                  __builtin_bit_cast(StoredVec<kF16, 8>, b), c, 0, 0,
                                                  0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0,
                                               0);
    return c;
  }
}

// Store the lane's 16 values of a 32 x 32 output: row index b = lane % 32, columns
// 8 (i / 4) + 4 (lane / 32) + i % 4 of the row p, of which `cols` exist.
template <int ST>
__device__ __forceinline__ void store_fragment(void* p, const f32x16& v, int64_t cols, bool row,
                                               int lane) {
  if constexpr (ST == kF32) {
    if (!row) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t c = 8 * q + 4 * (lane >> 5);
      const f32x4 w = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      if (c + 4 <= cols) {
        store_vec<kF32, 4>(p, c, w);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < cols) store_one<kF32>(p, c + j, w[j]);
      }
    }
  } else {
    // Lanes l and l + 32 hold the two halves of 8 neighbours each: exchange, so
    // that a lane has all 8 of one of two groups.
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t g[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const StoredVec<ST, 2> two = {
              static_cast<typename Stored<ST>::type>(v[8 * q + 4 * h + 2 * j]),
              static_cast<typename Stored<ST>::type>(v[8 * q + 4 * h + 2 * j + 1])};
          g[h][j] = __builtin_bit_cast(uint32_t, two);
        }
      u32x4 out;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const auto s = __builtin_amdgcn_permlane32_swap(g[0][j], g[1][j], false, false);
        out[j] = s[0];
        out[2 + j] = s[1];
      }
      const int64_t c = 16 * q + 8 * (lane >> 5);
      const StoredVec<ST, 8> w = __builtin_bit_cast(StoredVec<ST, 8>, out);
      if (!row) continue;
      if (c + 8 <= cols) {
        store_vec<ST, 8>(p, c, w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < cols) static_cast<typename Stored<ST>::type*>(p)[c + j] = w[j];
      }
    }
  }
}

// The order of a quarter's instructions: reads and products in turn.
// Left to itself the compiler moves the reads behind the products, next to their
// use, and every quarter starts with a wait for LDS.
template <int READS, int PRODUCTS>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < (READS > PRODUCTS ? READS : PRODUCTS); ++i) {
    constexpr int kRead = 0x100, kProduct = 0x8;
    if (i < READS) __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
    if (i < PRODUCTS) __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int ST, Product P, typename S, bool DIRECT>
__global__ __launch_bounds__(S::threads) void grouped_product(GroupedArgs a) {
  constexpr bool kAKmaj = P == kForward, kBKmaj = P != kGradW;
  using OpA = Operand<ST, kAKmaj, S::TA, S::NW, DIRECT>;
  using OpB = Operand<ST, kBKmaj, S::TB, S::NW, DIRECT>;
  constexpr int BK = OpA::BK;
  constexpr int bytes = StorageTraits<ST>::bytes;
  __shared__ __align__(1024) unsigned char lds[S::NS * S::stage];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t cols = P == kForward ? a.M : a.K;      // of the output: A's free index
  const int64_t na = (cols + S::TA - 1) / S::TA;
  Tile t;
  if constexpr (P == kGradW) {
    const int64_t nb = (a.M + S::TB - 1) / S::TB;
    const int64_t q = xcd_contiguous_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    t.group = q / (na * nb);
    t.first = group_offset(a, t.group);
    t.end = group_offset(a, t.group + 1);
    if (t.end < t.first) t.end = t.first;
    band_order(q - t.group * na * nb, na, nb, &t);
  } else {
    if (!find_row_tile<S::TB>(a, na, &t)) return;
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

  auto read = [&](const unsigned char* from, int kk, u32x4 (&fa)[S::WA], u32x4 (&fb)[S::WB]) {
#pragma unroll
    for (int j = 0; j < S::WB; ++j)
      fb[j] = OpB::fragment(from + S::TA * kRowBytes, wb + 32 * j, kk, lane);
#pragma unroll
    for (int i = 0; i < S::WA; ++i) fa[i] = OpA::fragment(from, wa + 32 * i, kk, lane);
  };
  auto products = [&](const u32x4 (&fa)[S::WA], const u32x4 (&fb)[S::WB]) {
#pragma unroll
    for (int i = 0; i < S::WA; ++i)
#pragma unroll
      for (int j = 0; j < S::WB; ++j) acc[i][j] = multiply<ST>(fa[i], fb[j], acc[i][j]);
  };

  const int32_t slices = static_cast<int32_t>((depth + BK - 1) / BK);
  if constexpr (DIRECT) {
    // All NS buffers are in flight; slices past the end load nothing, but count.
    // Each quarter's fragments are read while the one before is multiplied, those
    // of a slice's first quarter at the end of the slice before: the wait for the
    // slice's loads and the barrier come before a last quarter, whose fragments
    // are in registers, and its products cover what follows.
    constexpr int kLoads = OpA::NL + OpB::NL;
    constexpr int kReads = S::WA * OpA::kFragmentReads + S::WB * OpB::kFragmentReads;
    constexpr int kProducts = S::WA * S::WB * (bytes == 4 ? 4 : 1);
#pragma unroll
    for (int s = 0; s < S::NS; ++s) {
      oa.issue(s * BK, lds + s * S::stage, wave, lane);
      ob.issue(s * BK, lds + s * S::stage + S::TA * kRowBytes, wave, lane);
    }
    u32x4 fa[2][S::WA], fb[2][S::WB];
    unsigned char* at = lds;
    wait_loads<(S::NS - 1) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(at, 0, fa[0], fb[0]);
    for (int32_t s = 0; s < slices; ++s) {
#pragma unroll
      for (int kk = 0; kk < 3; ++kk) {
        read(at, kk + 1, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
        products(fa[kk & 1], fb[kk & 1]);
        interleave<kReads, kProducts>();
      }
      unsigned char* next = at + S::stage == lds + S::NS * S::stage ? lds : at + S::stage;
      wait_loads<(S::NS - 2) * kLoads>();  // this wave's loads of the next slice are in LDS
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // and its reads of this one done
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      oa.issue((s + S::NS) * BK, at, wave, lane);
      ob.issue((s + S::NS) * BK, at + S::TA * kRowBytes, wave, lane);
      read(next, 0, fa[0], fb[0]);
      products(fa[1], fb[1]);
      interleave<kReads, kProducts>();
      at = next;
    }
    wait_loads<0>();
  } else {
    oa.issue(0, lds, wave, lane);
    ob.issue(0, lds, wave, lane);
    oa.put(lds, wave, lane);
    ob.put(lds + S::TA * kRowBytes, wave, lane);
    __syncthreads();
    for (int32_t s = 0; s < slices; ++s) {
      oa.issue((s + 1) * BK, lds, wave, lane);
      ob.issue((s + 1) * BK, lds, wave, lane);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        u32x4 fa[S::WA], fb[S::WB];
        read(lds + (s & 1) * S::stage, kk, fa, fb);
        products(fa, fb);
      }
      unsigned char* next = lds + ((s + 1) & 1) * S::stage;
      oa.put(next, wave, lane);
      ob.put(next + S::TA * kRowBytes, wave, lane);
      __syncthreads();
    }
  }

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
}

// dbias: a workgroup sums 64 columns of one group, four rows at a time.
template <int ST>
__global__ __launch_bounds__(kBlock) void grouped_bias_grad(GroupedArgs a) {
  __shared__ float part[4][64];
  const int64_t g = blockIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float sum = 0.0f;
  if (c < a.M)
    for (int64_t n = group_offset(a, g) + w; n < group_offset(a, g + 1); n += 4)
      sum += load_one<ST>(a.grad, n * a.grad_stride + c);
  part[w][threadIdx.x & 63] = sum;
  __syncthreads();
  if (w == 0 && c < a.M)
    store_one<ST>(a.db, g * a.M + c,
                  (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                      (part[2][threadIdx.x] + part[3][threadIdx.x]));
}

inline int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

template <int ST, Product P, typename S>
hipError_t launch_product(const GroupedArgs& a, hipStream_t s) {
  const int64_t na = ceil_div(P == kForward ? a.M : a.K, S::TA);
  // a group's last row tile may be partial: at most one more for each group
  const int64_t nb = P == kGradW ? a.groups * ceil_div(a.M, S::TB)
                                 : a.rows / S::TB + std::min(a.groups, a.rows);
  const dim3 grid(static_cast<unsigned>(na * nb));
  if (a.direct)
    hipLaunchKernelGGL((grouped_product<ST, P, S, true>), grid, dim3(S::threads), 0, s, a);
  else
    hipLaunchKernelGGL((grouped_product<ST, P, S, false>), grid, dim3(S::threads), 0, s, a);
  return hipGetLastError();
}

using Large = Shape<256, 256, 2, 4, 2>;
using Medium = Shape<128, 128, 2, 2, 2>;
using Small = Shape<128, 32, 4, 1, 4>;

template <int ST, Product P>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t s) {
  const int64_t mean = a.rows / a.groups, cols = P == kForward ? a.M : a.K;
  if (mean <= 32) return launch_product<ST, P, Small>(a, s);
  if (mean >= 256 && ceil_div(a.rows, 256) * ceil_div(cols, 256) >= 256)
    return launch_product<ST, P, Large>(a, s);
  return launch_product<ST, P, Medium>(a, s);
}

template <int ST>
hipError_t launch_grouped(const GroupedArgs& a, bool backward, hipStream_t s) {
  if (!backward) return launch_rows<ST, kForward>(a, s);
  hipError_t e = hipSuccess;
  if (a.dx && a.rows > 0) e = launch_rows<ST, kGradX>(a, s);
  if (e == hipSuccess && a.dw) {
    if (a.groups * ceil_div(a.M, 256) * ceil_div(a.K, 256) >= 256)
      e = launch_product<ST, kGradW, Large>(a, s);
    else
      e = launch_product<ST, kGradW, Medium>(a, s);
  }
  if (e == hipSuccess && a.db) {
    hipLaunchKernelGGL((grouped_bias_grad<ST>),
                       dim3(static_cast<unsigned>(ceil_div(a.M, 64)), static_cast<unsigned>(a.groups)),
                       dim3(kBlock), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

#endif  // TBE_GROUPED_KERNELS

}  // namespace tbe
