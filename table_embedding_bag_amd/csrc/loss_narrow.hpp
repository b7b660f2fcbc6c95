// loss_narrow.hpp -- the softmax loss over tables of narrow rows: 2-byte values, at most
// 128 of them in whole 16-byte chunks.
//
// A wave keeps 64 rows of one side (Q) in registers as matrix operands for the whole
// kernel; the other side's rows (T) stream through LDS, a ring of tiles filled directly
// from memory, all of the row at once.  The logits of 32 x 64 rows come out of the matrix
// cores with a row of Q in each lane and 16 rows of T in its registers.  That is what
// the forward pass sums over; and, once exponentiated and rounded, it is in place as an
// operand of the next product, whose summed index is T's row:
//   forward   Q = x, T = table:  each lane sums its row's powers
//   dx        Q = x, T = table:  dx[q] += sum_t d[q, t] table[t]
//   dtable    Q = table, T = x:  dtable[q] += sum_t d[t, q] x[t]
// so the logits' gradients never leave the registers; each pass computes the logits again.
#pragma once

#include "loss_kernels.hpp"

namespace tbe {
namespace {

constexpr int kRing = 4;  // tiles of the ring: one is read, two are in flight, one is filled

// QW of the four waves have rows of Q of their own, the others share them and take other
// rows of the tile; BL blocks of 32 rows of the tile are a wave's.
template <int SL_, int QW_, int BL_>
struct NarrowShape {
  static constexpr int SL = SL_, QW = QW_, BL = BL_;  // SL: slices of 64 values in a row
  static constexpr int TW = 4 / QW, TR = 32 * TW * BL, QR = 64 * QW;
  static constexpr int KS = 4 * SL;           // steps of 16 values
  static constexpr int NL = SL * TR / 32;     // 16-byte loads a thread for a tile
  static constexpr int stage = SL * TR * 128;
};

// A tile in LDS: slices of 64 values, rows of 128 bytes, chunk c of row r at slot
// c ^ swizzle(r): 16 lanes that read one chunk of 16 rows cover the 256 bytes of the banks
// once, and so do 32 lanes that read 32 columns of 4 rows for the transposing read.
__device__ __forceinline__ int narrow_swizzle(int row) { return (row >> 1 & 1) << 2 | (row >> 2 & 3); }

// INFO: with what is known of the tile's rows (64 bases, targets, gradients), in a ring of
// its own.
constexpr int kInfoBytes = 4 * kInfoBlock;
template <typename S, bool INFO>
struct NarrowStream {
  static constexpr int loads = S::NL + INFO;  // of a tile
  const char* base;
  const char* info;
  int64_t stride, rows;  // bytes; rows of T
  uint32_t last;         // bytes of a row that exist
  uint32_t off[S::NL];
  uint32_t lds, info_lds, info_off;
  int wave;

  __device__ __forceinline__ void with_info(const void* p, unsigned char* info_ring, int lane) {
    info = static_cast<const char*>(p);
    info_lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(TBE_LDS(void, info_ring)));
    info_off = lane * 16;
  }
  __device__ __forceinline__ void init(const void* p, int64_t stride_, int64_t rows_, int64_t K,
                                       unsigned char* ring, int wave_, int lane) {
    base = static_cast<const char*>(p);
    stride = stride_ * 2;
    rows = rows_;
    last = static_cast<uint32_t>(K) * 2;
    wave = wave_;
    lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(TBE_LDS(void, ring)));
#pragma unroll
    for (int i = 0; i < S::NL; ++i) {
      const int q = (i * 4 + wave) * 64 + lane;
      const int slice = q / (S::TR * 8), r = q / 8 % S::TR;
      const int c = slice * 8 + ((q & 7) ^ narrow_swizzle(r));
      off[i] = c * 16u < last ? static_cast<uint32_t>(r * stride) + c * 16 : kOutside;
    }
  }
  // Tile t into the ring's buffer; zeros past T's rows.
  __device__ __forceinline__ void load(int64_t t, int buffer) const {
    const int64_t left = rows - t * S::TR;
    const uint64_t at = reinterpret_cast<uint64_t>(base + t * S::TR * stride);
    const uint32_t records =
        left > 0 ? static_cast<uint32_t>(((left < S::TR ? left : S::TR) - 1) * stride) + last : 0u;
    const u32x4 rsrc = {static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32) & 0xFFFFu, records,
                        kBufferFlags};
#pragma unroll
    for (int i = 0; i < S::NL; ++i)
      load_to_lds(rsrc, off[i], lds + buffer * S::stage + (i * 4 + wave) * 1024);
    if constexpr (INFO) {  // every wave loads the same
      const uint64_t from = reinterpret_cast<uint64_t>(info + t * kInfoBytes);
      const u32x4 rows_info = {static_cast<uint32_t>(from), static_cast<uint32_t>(from >> 32) & 0xFFFFu,
                               left > 0 ? static_cast<uint32_t>(kInfoBytes) : 0u, kBufferFlags};
      load_to_lds(rows_info, info_off, info_lds + buffer * kInfoBytes);
    }
  }
};

// The wave's 64 rows of Q: lane l of block b has row 32 b + l % 32, chunks 2 k + l / 32.
template <int ST, typename S>
__device__ __forceinline__ void load_rows(const void* p, int64_t stride, int64_t first, int64_t rows,
                                          int64_t K, int lane, u32x4 (&q)[2][S::KS]) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t row = first + 32 * b + (lane & 31);
#pragma unroll
    for (int k = 0; k < S::KS; ++k) {
      const int c = 16 * k + 8 * (lane >> 5);
      StoredVec<ST, 8> v = {};
      if (row < rows) {
        if (c + 8 <= K) {
          v = load_vec<ST, 8>(p, row * stride + c);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < K) v[i] = static_cast<const typename Stored<ST>::type*>(p)[row * stride + c + i];
        }
      }
      q[b][k] = __builtin_bit_cast(u32x4, v);
    }
  }
}

// The logits of 32 rows of the tile (from row `block` on) and the wave's 64 of Q.
template <int ST, typename S>
__device__ __forceinline__ void narrow_logits(const unsigned char* tile, int block, int lane,
                                              const u32x4 (&q)[2][S::KS], f32x16 (&z)[2]) {
  const int row = block + (lane & 31), s = narrow_swizzle(lane & 31);
  z[0] = f32x16{};
  z[1] = f32x16{};
#pragma unroll
  for (int k = 0; k < S::KS; ++k) {
    const int chunk = (2 * (k & 3) + (lane >> 5)) ^ s;
    const u32x4 t = *reinterpret_cast<const u32x4*>(tile + ((k >> 2) * S::TR + row) * 128 + chunk * 16);
    z[0] = multiply<ST>(t, q[0][k], z[0]);
    z[1] = multiply<ST>(t, q[1][k], z[1]);
  }
}

// acc[b][c] += the products of the tile's 32 rows' columns 32 c .. 32 c + 31 and d: the
// summed index runs over rows in the order in which the logits came out, 4 (lane / 32) + i
// and 8 more for the two halves of a step.
template <int ST, typename S>
__device__ __forceinline__ void narrow_product(const unsigned char* tile, int block, int lane,
                                               const u32x4 (&d)[2][2], f32x16 (&acc)[2][2 * S::SL]) {
  const int j = (lane & 15) >> 2, h = lane >> 5;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int c = 0; c < 2 * S::SL; ++c) {
      i16x4 half[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = block + 16 * t + 8 * e + 4 * h + j;
        const int chunk = (4 * (c & 1) + 2 * (lane >> 4 & 1) + (lane >> 1 & 1)) ^ ((j >> 1) << 2 | e << 1 | h);
        const unsigned char* p = tile + ((c >> 1) * S::TR + row) * 128 + chunk * 16 + (lane & 1) * 8;
        half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(TBE_LDS(i16x4, p));
      }
      const u32x4 a =
          __builtin_bit_cast(u32x4, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
      acc[0][c] = multiply<ST>(a, d[0][t], acc[0][c]);
      acc[1][c] = multiply<ST>(a, d[1][t], acc[1][c]);
    }
}

// What follows is done where the branch is taken alone: the compiler would rather do it
// always and choose afterwards (the forward pass took every power twice).
__device__ __forceinline__ void rarely() { asm volatile(""); }

// Which of the lane's 16 values of a block is row `at` of its 32, or -1.
__device__ __forceinline__ int32_t element_of(int64_t at, bool real, int lane) {
  if (!real || at < 0 || at >= 32 || (at >> 2 & 1) != lane >> 5) return -1;
  const int32_t r = static_cast<int32_t>(at);
  return (r >> 3) * 4 + (r & 3);
}
__device__ __forceinline__ void subtract_at(f32x16& z, int32_t element, float v) {
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] -= element == e ? v : 0.0f;
}

// f(the ring's buffer, the tile's number) for the tiles first .. last, each when it is there.
template <typename Stream, typename F>
__device__ __forceinline__ void stream_tiles(const Stream& stream, int64_t first, int64_t last, F f) {
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) stream.load(first + i, i);
  int at = 0;
  for (int64_t t = first; t < last; ++t) {
    wait_loads<(kRing - 2) * Stream::loads>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of the tile before
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    stream.load(t + kRing - 1, (at + kRing - 1) % kRing);  // past the end: zeros
    f(at, t);
    at = (at + 1) % kRing;
  }
  wait_loads<0>();
}

// Forward.  A row's reference m is that of the first block (or of the last one whose
// powers grew past 2^80 of it): no maximum is looked for otherwise, as fp32 holds sums of
// 2^20 such powers, and what lies far below the reference does not count.
template <int ST, typename S>
__global__ __launch_bounds__(kBlock, 2) void loss_narrow_forward(LossArgs a) {
  __shared__ __align__(1024) unsigned char ring[kRing * S::stage];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nb = (a.rows + S::QR - 1) / S::QR;
  int64_t segment, tb;
  band_order(xcd_contiguous_block(blockIdx.x, gridDim.x), a.forward.segments, nb, &segment, &tb);
  const int64_t n0 = tb * S::QR + wave % S::QW * 64;
  const int64_t first = segment * a.forward.run;
  const int64_t last = first + a.forward.run < a.forward.tiles ? first + a.forward.run : a.forward.tiles;
  NarrowStream<S, false> stream;
  stream.init(a.table, a.table_stride, a.vocab, a.K, ring, wave, lane);
  u32x4 q[2][S::KS];
  load_rows<ST, S>(a.x, a.x_stride, n0, a.rows, a.K, lane, q);
  float m[2] = {kNegInf, kNegInf}, sum[2] = {0.0f, 0.0f};
  int64_t target[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t n = n0 + 32 * b + (lane & 31);
    target[b] = n < a.rows ? target_of(a, n) : -1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads are counted from here
  stream_tiles(stream, first, last, [&](int buffer, int64_t t) {
    const unsigned char* tile = ring + buffer * S::stage;
#pragma unroll
    for (int block = 0; block < S::BL; ++block) {
      const int at = 32 * (wave / S::QW * S::BL + block);
      const int64_t v0 = t * S::TR + at, left = a.vocab - v0;
      if (left <= 0) continue;
      f32x16 z[2];
      narrow_logits<ST, S>(tile, at, lane, q, z);
      if (left < 32) {  // the last: nothing past the table's end
        rarely();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (place_of(0, e, lane) >= left) z[0][e] = z[1][e] = kNegInf;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int32_t hit = element_of(target[b] - v0, target[b] >= 0, lane);
        if (__any(hit >= 0)) {
          rarely();
          float logit = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) logit = hit == e ? z[b][e] : logit;
          if (hit >= 0) a.target_logit[n0 + 32 * b + (lane & 31)] = logit;
        }
        const auto powers = [&](float from) {
          float part[4] = {};
#pragma unroll
          for (int e = 0; e < 16; ++e)
            part[e & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(z[b][e], a.exponent, -from));
          return (part[0] + part[1]) + (part[2] + part[3]);
        };
        const bool unset = m[b] == kNegInf;
        float part = powers(unset ? 0.0f : m[b]);
        const bool again = unset || !(part <= 0x1p80f);  // each lane for itself
        if (__any(again)) {
          rarely();
          float top = z[b][0];
#pragma unroll
          for (int e = 1; e < 16; ++e) top = fmaxf(top, z[b][e]);
          const float next = fmaxf(m[b], top * a.exponent), from = next == kNegInf ? 0.0f : next;
          const float other = powers(from);
          if (again) {
            part = other;
            sum[b] *= __builtin_amdgcn_exp2f(m[b] - from);
            m[b] = next;
          }
        }
        sum[b] += part;
      }
    }
  });
  // the two halves of a wave, then the waves that share their rows
  __syncthreads();
  float2* joined = reinterpret_cast<float2*>(ring);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float2 other = make_float2(__shfl_xor(m[b], 32), __shfl_xor(sum[b], 32));
    const float2 both = join_sums(make_float2(m[b], sum[b]), other);
    if (lane < 32) joined[(wave / S::QW) * S::QR + wave % S::QW * 64 + 32 * b + lane] = both;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < S::QR; r += kBlock) {
    if (tb * S::QR + r >= a.rows) break;
    float2 v = joined[r];
#pragma unroll
    for (int w = 1; w < S::TW; ++w) v = join_sums(v, joined[w * S::QR + r]);
    a.parts[segment * a.rows + tb * S::QR + r] = v;
  }
}

// One gradient, of the table (DTABLE) or of x: of 256 rows of Q, summed over a part of T's
// tiles.  Sums go to the part, or rounded to the output where there is one.
template <int ST, typename S, bool DTABLE>
__global__ __launch_bounds__(kBlock, 2) void loss_narrow_gradient(LossArgs a, int64_t splits, int64_t run,
                                                                  float* parts, void* out) {
  static_assert(S::QW == 4 && S::BL == 2 && S::TR == 64);
  __shared__ __align__(1024) unsigned char ring[kRing * S::stage];
  __shared__ __align__(1024) unsigned char info_ring[DTABLE ? kRing * kInfoBytes : 16];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t rows_q = DTABLE ? a.vocab : a.rows, rows_t = DTABLE ? a.rows : a.vocab;
  const int64_t nb = (rows_q + S::QR - 1) / S::QR;
  int64_t split, tb;
  band_order(xcd_contiguous_block(blockIdx.x, gridDim.x), splits, nb, &split, &tb);
  const int64_t q0 = tb * S::QR + wave * 64;
  const int64_t tiles = (rows_t + S::TR - 1) / S::TR, first = split * run;
  const int64_t last = first + run < tiles ? first + run : tiles;
  NarrowStream<S, DTABLE> stream;
  u32x4 q[2][S::KS];
  if constexpr (DTABLE) {
    stream.init(a.x_rows, a.x_width, rows_t, a.x_width, ring, wave, lane);
    stream.with_info(a.row_info, info_ring, lane);
    load_rows<ST, S>(a.table, a.table_stride, q0, rows_q, a.K, lane, q);
  } else {
    stream.init(a.table, a.table_stride, rows_t, a.K, ring, wave, lane);
    load_rows<ST, S>(a.x_rows, a.x_width, q0, rows_q, a.K, lane, q);
  }
  float base[2], grad[2];  // of x's rows in the lanes
  int32_t target[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t n = q0 + 32 * b + (lane & 31);
    base[b] = __builtin_inff();
    grad[b] = 0.0f;
    target[b] = -1;
    if (!DTABLE && n < a.rows) {
      const uint32_t* info = a.row_info + n / 64 * kInfoBlock + n % 64;
      base[b] = __uint_as_float(info[0]);
      target[b] = static_cast<int32_t>(info[64]);
      grad[b] = fabsf(__uint_as_float(info[128]));
    }
  }
  f32x16 acc[2][2 * S::SL];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int c = 0; c < 2 * S::SL; ++c) acc[b][c] = f32x16{};
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads are counted from here
  stream_tiles(stream, first, last, [&](int buffer, int64_t t) {
    const unsigned char* tile = ring + buffer * S::stage;
    const float* bases = reinterpret_cast<const float*>(info_ring + buffer * kInfoBytes);
    const int32_t* words = reinterpret_cast<const int32_t*>(bases + 64);
    const float* grads = bases + 128;
#pragma unroll
    for (int block = 0; block < S::BL; ++block) {
      const int64_t t0 = t * S::TR + 32 * block;
      f32x16 z[2];
      narrow_logits<ST, S>(tile, 32 * block, lane, q, z);
      if constexpr (DTABLE) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const f32x4 four = *reinterpret_cast<const f32x4*>(bases + 32 * block + 8 * p + 4 * (lane >> 5));
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z[b][4 * p + e] =
                  __builtin_amdgcn_exp2f(__builtin_fmaf(z[b][4 * p + e], a.exponent, -four[e]));
        }
        // where the wave has a row's target, or a row's gradient is negative
        const int32_t word = words[32 * block + (lane & 31)];
        const int64_t hit = (word & ~kNegative) - q0;
        if (__any(word >= 0 && ((hit >= 0 && hit < 64) || (word & kNegative)))) {
          rarely();
          const int32_t v = static_cast<int32_t>(q0) + (lane & 31);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int at = 32 * block + 8 * p + 4 * (lane >> 5);
            const u32x4 w4 = *reinterpret_cast<const u32x4*>(words + at);
            const f32x4 g4 = *reinterpret_cast<const f32x4*>(grads + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int32_t w = static_cast<int32_t>(w4[e]), t = w & ~kNegative;  // none: below 0
              if (w >= 0 && w != t) z[0][4 * p + e] = -z[0][4 * p + e], z[1][4 * p + e] = -z[1][4 * p + e];
              z[0][4 * p + e] -= t == v ? g4[e] : 0.0f;
              z[1][4 * p + e] -= t == v + 32 ? g4[e] : 0.0f;
            }
          }
        }
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            z[b][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[b][e], a.exponent, -base[b]));
          const int32_t hit = element_of((target[b] & ~kNegative) - t0, target[b] >= 0, lane);
          if (__any(hit >= 0)) {
            rarely();
            subtract_at(z[b], hit, grad[b]);
          }
        }
      }
      u32x4 d[2][2];  // rounded to the rows' type: operands of the product
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          StoredVec<ST, 8> v;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = static_cast<typename Stored<ST>::type>(z[b][8 * s + e]);
          d[b][s] = __builtin_bit_cast(u32x4, v);
        }
      narrow_product<ST, S>(tile, 32 * block, lane, d, acc);
    }
  });
  const float undo = out ? a.factor[1] : 1.0f;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t r = q0 + 32 * b + (lane & 31);
    const float by = target[b] >= 0 && (target[b] & kNegative) ? -undo : undo;
#pragma unroll
    for (int c = 0; c < 2 * S::SL; ++c) {
      const int64_t cols = a.K - 32 * c;
      if (cols <= 0) continue;
      acc[b][c] *= by;
      if (out)
        store_fragment<ST>(static_cast<char*>(out) + (r * a.K + 32 * c) * 2, acc[b][c], cols, r < rows_q, lane);
      else
        store_fragment<kF32>(parts + (split * rows_q + r) * a.K + 32 * c, acc[b][c], cols, r < rows_q, lane);
    }
  }
}

}  // namespace
}  // namespace tbe
