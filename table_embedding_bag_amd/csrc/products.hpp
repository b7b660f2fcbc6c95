// products.hpp -- the tile products on the matrix cores that the grouped linear layer
// (grouped.hpp) and the softmax loss (softmax_loss.hpp) are made of.
//
// A tile's product is a loop over the summed index of two operands, each "k-major",
// where the summed index is the one adjacent in memory, or "free-major".  The matrix
// instruction leaves four neighbours of operand A's free index in a lane, so A is the
// operand whose free index runs along the output's rows in memory: wide stores.
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

namespace tbe {
namespace {

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
// Whether slices go from memory to LDS directly.
template <typename S, int LAYOUT>
constexpr bool kByLds = LAYOUT == kChunkRows && S::NS > 2;
// Slices past LDS's two in registers: one where a slice's products take long enough
// for a load to arrive, two where tiles are small (three take longer to start: 8191 x
// 250 -> 130 fp32, both directions, 53 us instead of 51).
template <typename S, int LAYOUT>
constexpr int kHeldSlices = !kByLds<S, LAYOUT> && S::NS > 2 ? 2 : 1;

// acc += the products of a tile's operands over the summed index, `depth` values of it.
// wa and wb: where the wave's outputs start along A's and B's free index.  step(fb) is
// called with every step's fragments of operand B.
template <int ST, typename S, int LAYOUT, typename OpA, typename OpB, typename F>
__device__ __forceinline__ void accumulate(OpA& oa, OpB& ob, int64_t depth, unsigned char* lds,
                                           int wa, int wb, int wave, int lane,
                                           f32x16 (&acc)[S::WA][S::WB], F step) {
  constexpr bool kThroughLds = kByLds<S, LAYOUT>;
  constexpr int kAhead = kHeldSlices<S, LAYOUT>;
  constexpr int BK = OpA::BK, KK = S::RB / 32;  // of a slice: values, steps of 32 bytes
  constexpr int bytes = StorageTraits<ST>::bytes;

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
    if constexpr (p == n - 1) step(fb[kk & 1]);
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
}

}  // namespace
}  // namespace tbe
