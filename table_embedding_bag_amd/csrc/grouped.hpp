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
// A workgroup stages slices of RB = 128 or 64 bytes of the summed index of both
// operands in LDS, in 16-byte chunks:
//   k-major     row r of the tile at RB r, chunk c at slot c ^ (r / 2 & 7) (128) or
//               c ^ (r / 4 & 3) (64), so that 16 lanes that read one chunk of 16 rows
//               cover the 256 bytes of the banks once (c ^ (r & 7) made half of the
//               reads' cycles conflicts);
//   free-major  row k of the slice at k * (tile width), 16-bit chunks c at slot
//               c ^ 4 (k & 3): the transposing LDS read takes 4 rows x 16 columns
//               for each 16 lanes, and this spreads the rows over the banks.
// Slices come by one of two ways.  Through registers, a slice or two ahead of LDS:
// the registers are buffers beside LDS's two, so a load has a whole slice's
// products to arrive.  Or, where tiles are small and memory is what counts, from
// memory to LDS directly, several slices ahead (aligned operands only).
// All loads are buffer loads, whose descriptor's bounds give zeros past the rows'
// and the group's ends.  Where rows are not whole aligned chunks, what follows a
// row's end is masked in the last slice; where they start between words, a chunk
// is loaded as the aligned words it lies in and shifted into place.
#pragma once

#include <type_traits>

#include "grouped_plan.hpp"
#include "layers.hpp"
#include "tiles.hpp"

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

using f32x16 = float __attribute__((ext_vector_type(16)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using i16x4 = short __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

#define TBE_LDS(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr uint32_t kOutside = 0x80000000u;      // past every descriptor's end
constexpr uint32_t kBufferFlags = 0x00020000u;  // of a descriptor: 32-bit data, no swizzle

// Tile shape: TA x TB outputs, NA x NB waves, NS slices of LDS with RB bytes of
// the summed index each.
template <int TA_, int TB_, int NA_, int NB_, int NS_, int RB_>
struct Shape {
  static constexpr int TA = TA_, TB = TB_, NA = NA_, NB = NB_, NS = NS_, RB = RB_;
  static constexpr int NW = NA * NB, threads = 64 * NW;
  static constexpr int WA = TA / NA / 32, WB = TB / NB / 32;  // 32 x 32 outputs a wave
  static constexpr int stage = (TA + TB) * RB;
};

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

// 16 bytes a lane from a buffer to LDS at `lds` + 16 lane; zeros for offsets past
// the buffer's end.  In assembly (it writes no register) because the compiler,
// which cannot tell the slices apart, waits for all such loads before it reads
// LDS with the transposing instruction; wait_loads() waits for them here.
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t offset, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
      ::"s"(lds), "v"(offset), "s"(rsrc)
      : "memory", "m0");
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

// One operand of a tile: where its chunks come from and which exist.
//   KMAJ: `free` rows of the tile at base + r * stride, the summed index along them.
//   else: rows of the summed index at base + k * stride, `free` columns along them.
//   AHEAD slices are held in registers where they come that way.
template <int ST, bool KMAJ, int R, int NW, int LAYOUT, int RB, int AHEAD>
struct Operand {
  static constexpr bool DIRECT = LAYOUT == kChunkRows;
  static constexpr int bytes = StorageTraits<ST>::bytes;
  static constexpr int EL = 16 / bytes;            // values in a chunk
  static constexpr int BK = RB / bytes;     // summed values in a slice
  static constexpr int CPR = KMAJ ? RB / 16 : R * bytes / 16;  // chunks in a row
  static constexpr int NL = R * RB / 16 / (64 * NW);     // chunks a thread
  static constexpr bool SHIFT = LAYOUT == kOddRows;     // rows may start between words
  static_assert(!SHIFT || bytes == 2);
  static constexpr int kFragmentReads = KMAJ ? 1 : bytes == 2 ? 2 : 4;
  static_assert(NL >= 1, "every thread has a chunk");

  const char* base;
  int64_t stride;            // bytes
  int32_t free, depth;       // bounds of the free index from the tile's start, of the summed one
  uint32_t off[NL];
  uint32_t column[NL];
  u32x4 held[AHEAD][NL];
  uint32_t more[AHEAD][SHIFT ? NL : 1];  // the word after
  uint32_t skew;                  // bytes from the aligned word before base to base
  uint32_t shift[AHEAD] = {};     // bit i: the chunk held starts between words
  const char* from;  // the slice aimed at
  uint32_t records;
  int32_t left;

  // What a k-major row's chunk numbers are xored with: rows that lie 256 bytes (all
  // banks) apart differ in it.
  static __device__ __forceinline__ int swizzle(int row) {
    return RB == 128 ? row >> 1 & 7 : row >> 2 & 3;
  }
  // Row and (global) chunk that thread's i-th LDS chunk holds.
  static __device__ __forceinline__ void place(int i, int wave, int lane, int* row, int* chunk) {
    const int q = (i * NW + wave) * 64 + lane;
    *row = q / CPR;
    const int slot = q % CPR;
    if constexpr (KMAJ) *chunk = slot ^ swizzle(*row);
    else if constexpr (bytes == 2) *chunk = slot ^ ((4 * (*row & 3)) & (CPR - 1));
    else *chunk = slot;
  }

  __device__ __forceinline__ void init(const void* p, int64_t stride_, int64_t free_, int64_t depth_,
                                       int wave, int lane) {
    skew = SHIFT ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 2u : 0u;
    base = static_cast<const char*>(p) - skew;
    stride = stride_ * bytes;
    free = static_cast<int32_t>(free_ < R ? free_ : R);
    depth = static_cast<int32_t>(depth_);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      int row, chunk;
      place(i, wave, lane, &row, &chunk);
      const bool inside = (KMAJ ? row : chunk * EL) < free;
      off[i] = inside ? static_cast<uint32_t>(row * stride) + chunk * 16 + skew : kOutside;
      column[i] = KMAJ ? chunk * EL : row;   // along the summed index
    }
  }

  // The slice at k0 for the loads that follow (past the end: all zeros), ...
  __device__ __forceinline__ void aim(int32_t k0) {
    left = depth - k0;
    from = base + (KMAJ ? static_cast<int64_t>(k0) * bytes : k0 * stride);
    int64_t extent;
    if constexpr (KMAJ) extent = (free - 1) * stride + static_cast<int64_t>(left) * bytes;
    else extent = ((left < BK ? left : BK) - 1) * stride + static_cast<int64_t>(free) * bytes;
    // up to the end of the word that holds the last value
    if constexpr (!DIRECT && bytes == 2) extent = (extent + skew + 3) & ~int64_t{3};
    records = left > 0 ? static_cast<uint32_t>(extent) : 0u;
  }
  // ... and, directly, the load of the thread's i-th chunk of it into the slice at `to`.
  __device__ __forceinline__ void load(int i, unsigned char* to, int wave) const {
    const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(TBE_LDS(void, to)));
    const uint64_t at = reinterpret_cast<uint64_t>(from);
    const u32x4 rsrc = {static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32) & 0xFFFFu, records,
                        kBufferFlags};
    load_to_lds(rsrc, static_cast<int32_t>(column[i]) < left ? off[i] : kOutside,
                lds + (i * NW + wave) * 1024);
  }

  // Through registers: the load of the i-th chunk of the slice aimed at into the
  // slice held at h, ...
  __device__ __forceinline__ void fetch(int i, int h) {
    const auto rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), 0,
                                                        static_cast<int>(records), kBufferFlags);
    uint32_t o = static_cast<int32_t>(column[i]) < left ? off[i] : kOutside;
    if constexpr (SHIFT) {
      more[h][i] = __builtin_amdgcn_raw_buffer_load_b32(rows, (o & ~3u) + 16, 0, 0);
      shift[h] = (shift[h] & ~(1u << i)) | (o >> 1 & 1u) << i;
      o &= ~3u;
    }
    held[h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, o, 0, 0));
  }
  // ... and its write into the slice at `to`, when the slice AHEAD after it is aimed at.
  __device__ __forceinline__ void put(int i, int h, unsigned char* to, int wave, int lane) const {
    u32x4 v = held[h][i];
    if constexpr (SHIFT) {
      const uint32_t by = (shift[h] >> i & 1u) * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = __builtin_amdgcn_alignbit(j < 3 ? held[h][i][j < 3 ? j + 1 : 0] : more[h][i],
                                         held[h][i][j], by);
    }
    if constexpr (!DIRECT && KMAJ) {
      const int32_t held_left = left + AHEAD * BK;
      if (held_left < BK) {  // the last: nothing past the summed index's end
        const int32_t room = (held_left - static_cast<int32_t>(column[i])) * bytes * 8;  // bits
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int32_t bits = room - 32 * j;
          v[j] &= bits >= 32 ? ~0u : bits <= 0 ? 0u : (1u << bits) - 1u;
        }
      }
    }
    *reinterpret_cast<u32x4*>(to + (i * NW + wave) * 1024 + lane * 16) = v;
  }

  // The lane's fragment of the 32 free indices from `at`, 16 bytes of the summed
  // index: those of chunk 2 kk + lane / 32.  k-major: one chunk.  Free-major,
  // 16-bit: two transposing reads, four summed values each; fp32: four values.
  static __device__ __forceinline__ u32x4 fragment(const unsigned char* from, int at, int kk,
                                                   int lane) {
    if constexpr (KMAJ) {
      const int row = at + (lane & 31), chunk = (2 * kk + (lane >> 5)) ^ swizzle(lane & 31);
      return *reinterpret_cast<const u32x4*>(from + row * RB + chunk * 16);
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

// The order of some instructions: reads and products in turn.  Left to itself the
// compiler moves the reads behind the products, next to their use, and every
// step starts with a wait for LDS.
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

// for (i = FROM; i < TO; ++i) with i known to the compiler.
template <int FROM, int TO, typename F>
__device__ __forceinline__ void repeat(F f) {
  if constexpr (FROM < TO) {
    f(std::integral_constant<int, FROM>{});
    repeat<FROM + 1, TO>(f);
  }
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// LDS's buffers: for slices that come by registers two.
template <typename S, int LAYOUT>
constexpr int kLdsBytes = (LAYOUT == kChunkRows && S::NS > 2 ? S::NS : 2) * S::stage;

// The tile that workgroup `id` of a product's `blocks` takes.
template <int ST, Product P, typename S, int LAYOUT>
__device__ __forceinline__ void product(const GroupedArgs& a, uint32_t id, uint32_t blocks,
                                        unsigned char* lds) {
  constexpr bool kAKmaj = P == kForward, kBKmaj = P != kGradW;
  // Slices past LDS's two in registers: one where a slice's products take long enough
  // for a load to arrive, two where tiles are small (three take longer to start: 8191 x
  // 250 -> 130 fp32, both directions, 53 us instead of 51).
  constexpr bool kThroughLds = LAYOUT == kChunkRows && S::NS > 2;
  constexpr int kAhead = !kThroughLds && S::NS > 2 ? 2 : 1;
  using OpA = Operand<ST, kAKmaj, S::TA, S::NW, LAYOUT, S::RB, kAhead>;
  using OpB = Operand<ST, kBKmaj, S::TB, S::NW, LAYOUT, S::RB, kAhead>;
  constexpr int BK = OpA::BK, KK = S::RB / 32;  // of a slice: values, steps of 32 bytes
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

  // Fragment f of a step: first B's, then A's.
  auto read = [&](const unsigned char* from, int kk, int f, u32x4 (&fa)[S::WA], u32x4 (&fb)[S::WB]) {
    if (f < S::WB)
      fb[f < S::WB ? f : 0] = OpB::fragment(from + S::TA * S::RB, wb + 32 * f, kk, lane);
    else
      fa[f < S::WB ? 0 : f - S::WB] = OpA::fragment(from, wa + 32 * (f - S::WB), kk, lane);
  };
  constexpr int kFragments = S::WA + S::WB, kTiles = S::WA * S::WB;

  const int32_t slices = static_cast<int32_t>((depth + BK - 1) / BK);
  constexpr int kLoads = OpA::NL + OpB::NL;
  u32x4 fa[2][S::WA], fb[2][S::WB];
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
  // Part p of n of a step: reads of the next step's fragments and products of this
  // one's, taking turns.
  auto part = [&](auto p_, auto parts, auto kk_, const unsigned char* next_step) {
    constexpr int p = p_, n = parts, kk = kk_;
    constexpr int f0 = p * kFragments / n, f1 = (p + 1) * kFragments / n;
    constexpr int t0 = p * kTiles / n, t1 = (p + 1) * kTiles / n;
    constexpr int kFragmentB = f1 < S::WB ? f1 - f0 : f0 < S::WB ? S::WB - f0 : 0;
#pragma unroll
    for (int f = f0; f < f1; ++f) read(next_step, (kk + 1) % KK, f, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
#pragma unroll
    for (int t = t0; t < t1; ++t)
      acc[t / S::WB][t % S::WB] =
          multiply<ST>(fa[kk & 1][t / S::WB], fb[kk & 1][t % S::WB], acc[t / S::WB][t % S::WB]);
    interleave<kFragmentB * OpB::kFragmentReads + (f1 - f0 - kFragmentB) * OpA::kFragmentReads,
               (t1 - t0) * (bytes == 4 ? 4 : 1)>();
    if constexpr (P == kGradW && p == n - 1)
      if (sums) add_columns(fb[kk & 1]);
  };
  if constexpr (kThroughLds) {
    // Of the NS buffers one is read, NS - 2 are in flight and one, read before, is
    // being filled; slices past the end load nothing, but count.  A step's loads,
    // the reads of the next step's fragments and its products take turns: loads all
    // at once block the wave, in front of its products, until the memory pipeline
    // has taken them (1.1 ms of a 0.85 ms product).  A slice's first fragments are
    // read at the end of the slice before: the wait for the slice's loads and the
    // barrier come before a last step, whose fragments are in registers, and its
    // products cover what follows.
    constexpr int kBefore = (KK - 1) * kLoads / KK;  // a slice's loads before that wait
    auto load = [&](int i, unsigned char* to) {
      if (i < OpA::NL) oa.load(i < OpA::NL ? i : 0, to, wave);
      else ob.load(i < OpA::NL ? 0 : i - OpA::NL, to + S::TA * S::RB, wave);
    };
#pragma unroll
    for (int s = 0; s < S::NS - 1; ++s) {
      oa.aim(s * BK);
      ob.aim(s * BK);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load(i, lds + s * S::stage);
    }
    unsigned char *at = lds, *fill = lds + (S::NS - 1) * S::stage;
    wait_loads<(S::NS - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < kFragments; ++f) read(at, 0, f, fa[0], fb[0]);
    for (int32_t s = 0; s < slices; ++s) {
      unsigned char* next = at + S::stage == lds + S::NS * S::stage ? lds : at + S::stage;
      oa.aim((s + S::NS - 1) * BK);
      ob.aim((s + S::NS - 1) * BK);
      repeat<0, KK>([&](auto kk_) {
        constexpr int kk = kk_, kFrom = kk * kLoads / KK, kTo = (kk + 1) * kLoads / KK;
        constexpr int kParts = kTo - kFrom > 1 ? kTo - kFrom : 1;
        if constexpr (kk == KK - 1) {
          // this wave's loads of the next slice are in LDS, its reads of this one done
          wait_loads<(S::NS - 3) * kLoads + kBefore>();
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
        repeat<0, kParts>([&](auto p_) {
          if constexpr (kFrom + p_ < kTo) load(kFrom + p_, fill);
          part(p_, std::integral_constant<int, kParts>{}, kk_, kk == KK - 1 ? next : at);
        });
      });
      fill = at;
      at = next;
    }
    wait_loads<0>();
  } else {
    // While slice s is read from its buffer, the registers' slice s + 1 goes into the
    // other one, chunk by chunk, and each chunk's register takes its load of slice
    // s + 1 + kAhead at once: a load has kAhead slices' products to arrive.  All writes
    // come before the last step, which reads the next slice's first fragments.
    auto fetch = [&](int i, int h) {
      if (i < OpA::NL) oa.fetch(i < OpA::NL ? i : 0, h);
      else ob.fetch(i < OpA::NL ? 0 : i - OpA::NL, h);
    };
    auto put = [&](int i, int h, unsigned char* to) {
      if (i < OpA::NL) oa.put(i < OpA::NL ? i : 0, h, to, wave, lane);
      else ob.put(i < OpA::NL ? 0 : i - OpA::NL, h, to + S::TA * S::RB, wave, lane);
    };
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      oa.aim(h * BK);
      ob.aim(h * BK);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) fetch(i, h);
    }
    oa.aim(kAhead * BK);
    ob.aim(kAhead * BK);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      put(i, 0, lds);
      fetch(i, 0);
    }
    __syncthreads();
#pragma unroll
    for (int f = 0; f < kFragments; ++f) read(lds, 0, f, fa[0], fb[0]);
    auto slice = [&](int32_t s, auto h_) {
      constexpr int h = h_;
      const unsigned char* at = lds + (s & 1) * S::stage;
      unsigned char* next = lds + ((s + 1) & 1) * S::stage;
      oa.aim((s + 1 + kAhead) * BK);
      ob.aim((s + 1 + kAhead) * BK);
      repeat<0, KK>([&](auto kk_) {
        constexpr int kk = kk_;
        constexpr int kFrom = kk == KK - 1 ? kLoads : kk * kLoads / (KK - 1);
        constexpr int kTo = kk == KK - 1 ? kLoads : (kk + 1) * kLoads / (KK - 1);
        constexpr int kParts = kTo - kFrom > 1 ? kTo - kFrom : 1;
        if constexpr (kk == KK - 1) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads and writes
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
        repeat<0, kParts>([&](auto p_) {
          if constexpr (kFrom + p_ < kTo) {
            put(kFrom + p_, h, next);
            fetch(kFrom + p_, h);
          }
          part(p_, std::integral_constant<int, kParts>{}, kk_, kk == KK - 1 ? next : at);
        });
      });
    };
    for (int32_t s = 0; s < slices; s += kAhead)
      repeat<0, kAhead>([&](auto r_) {
        constexpr int r = r_;
        if (r == 0 || s + r < slices) slice(s + r, std::integral_constant<int, (r + 1) % kAhead>{});
      });
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
