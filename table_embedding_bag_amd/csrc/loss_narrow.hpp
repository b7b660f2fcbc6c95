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
//
// 2048 rows, 100000 outputs of 128, bf16: forward 66 us (0.79 PFLOP/s; powers of two take as long
// as the product), dtable 148 us (two products, 0.71: 391 workgroups take two rounds of the 256
// places, the second half empty), dx 115 us (0.91).  64 rows: forward 12 us (2.1 TB/s of the table).
#pragma once

#include "loss_kernels.hpp"

namespace tbe {
namespace {

// Tiles of the rings: the forward pass reads one while two are in flight and one is filled;
// the gradients read two.
constexpr int kRing = 4, kGradientRing = 5;

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

// Steps of 16 values of the logits of 32 rows of a tile (from row `block` on) and the wave's
// 64 of Q.
template <int ST, typename S>
__device__ __forceinline__ u32x4 tile_chunk(const unsigned char* tile, int block, int k, int lane) {
  const int row = block + (lane & 31);
  const int chunk = (2 * (k & 3) + (lane >> 5)) ^ narrow_swizzle(lane & 31);
  return *reinterpret_cast<const u32x4*>(tile + ((k >> 2) * S::TR + row) * 128 + chunk * 16);
}

// Columns 32 c .. 32 c + 31 of half t (16) of the tile's 32 rows from `block` on, an operand
// whose summed index runs over rows in the order in which the logits come out:
// 4 (lane / 32) + i, and 8 more for the second four.
template <typename S>
__device__ __forceinline__ u32x4 tile_columns(const unsigned char* tile, int block, int t, int c, int lane) {
  const int j = (lane & 15) >> 2, h = lane >> 5;
  i16x4 half[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = block + 16 * t + 8 * e + 4 * h + j;
    const int chunk = (4 * (c & 1) + 2 * (lane >> 4 & 1) + (lane >> 1 & 1)) ^ ((j >> 1) << 2 | e << 1 | h);
    const unsigned char* p = tile + ((c >> 1) * S::TR + row) * 128 + chunk * 16 + (lane & 1) * 8;
    half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(TBE_LDS(i16x4, p));
  }
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// A step is written as matrix instructions one by one, with a few vector instructions and
// reads of LDS behind each, in its shadow: what is between two of these stays there.  Left to
// itself the compiler puts all of one kind after all of another, and a matrix instruction
// right behind another holds up what follows.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }
constexpr int kReadAhead = 6;  // matrix instructions between a read and its use

// v is computed here: the compiler would move that to where v is used, behind the next
// branch and out of the matrix instructions' shadow.
template <typename T>
__device__ __forceinline__ void settled(T& v) { asm volatile("" : "+v"(v)); }

// f(t, its buffer, the buffer of the tile before) for the tiles first .. last of a ring of
// R, each when it is there; the LAG tiles before t are still being read.
template <int R, int LAG, typename Stream, typename F>
__device__ __forceinline__ void stream_tiles(const Stream& stream, int64_t first, int64_t last, F f) {
  constexpr int kAhead = R - LAG - 2;  // in flight while t is read
#pragma unroll
  for (int i = 0; i <= kAhead; ++i) stream.load(first + i, i);
  int at = 0, before = 0;
  for (int64_t t = first; t < last; ++t) {
    wait_loads<kAhead * Stream::loads>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of the buffer to fill
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    stream.load(t + kAhead + 1, at + kAhead + 1 < R ? at + kAhead + 1 : at + kAhead + 1 - R);
    f(t, at, before);
    before = at;
    at = at + 1 < R ? at + 1 : 0;
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
  float from[2] = {0.0f, 0.0f}, sum[2] = {0.0f, 0.0f};  // what powers are relative to, their sum
  bool unset[2] = {true, true};                          // no reference yet
  int32_t target[2];  // tables have at most 2^30 rows
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t n = n0 + 32 * b + (lane & 31);
    target[b] = n < a.rows ? static_cast<int32_t>(target_of(a, n)) : -1;
  }
  // A step takes the logits of a block of the tile while it sums the powers of the block
  // before: matrix and vector instructions in turn.
  f32x16 z[2] = {f32x16{}, f32x16{}};
  float part[2][4];
  const auto add_power = [&](int b, int e) {
    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(z[b][e], a.exponent, -from[b]));
    part[b][e & 3] = e < 4 ? p : part[b][e & 3] + p;
  };
  const auto block_sum = [&](int b) { return (part[b][0] + part[b][1]) + (part[b][2] + part[b][3]); };
  // What is done of a block once its powers are summed; v0: its first row.
  const auto settle = [&](int64_t v0) {
    const int32_t first_v = static_cast<int32_t>(v0);
    const auto near = [&](int b) { return static_cast<uint32_t>(target[b] - first_v) < 32u; };  // none: no
    if (__any(near(0) || near(1))) {
      rarely();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int32_t hit = element_of(target[b] - first_v, near(b), lane);
        float logit = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) logit = hit == e ? z[b][e] : logit;
        if (hit >= 0) a.target_logit[n0 + 32 * b + (lane & 31)] = logit;
      }
    }
    float now[2] = {block_sum(0), block_sum(1)};
    const auto again = [&](int b) { return unset[b] || !(now[b] <= 0x1p80f); };  // each lane for itself
    if (__any(again(0) || again(1))) {
      rarely();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float top = z[b][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, z[b][e]);
        const float next = fmaxf(unset[b] ? kNegInf : from[b], top * a.exponent);
        const bool still = next == kNegInf, change = again(b);
        const float keep = from[b];
        if (change) from[b] = still ? 0.0f : next;
#pragma unroll
        for (int e = 0; e < 16; ++e) add_power(b, e);
        if (change) {
          now[b] = block_sum(b);
          sum[b] = unset[b] ? sum[b] : sum[b] * __builtin_amdgcn_exp2f(keep - from[b]);
          unset[b] = still;
        }
      }
    }
    sum[0] += now[0];
    sum[1] += now[1];
  };
  const auto mask_end = [&](int64_t v0) {  // nothing past the table's end
    if (a.vocab - v0 < 32) {
      rarely();
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (place_of(0, e, lane) >= a.vocab - v0) z[0][e] = z[1][e] = kNegInf;
    }
  };
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads are counted from here
  int64_t v_before = -1;  // of the block whose powers are due
  stream_tiles<kRing, 0>(stream, first, last, [&](int64_t t, int buffer, int) {
    const unsigned char* tile = ring + buffer * S::stage;
#pragma unroll
    for (int block = 0; block < S::BL; ++block) {
      const int at = 32 * (wave / S::QW * S::BL + block);
      f32x16 next[2] = {f32x16{}, f32x16{}};
      u32x4 chunk[S::KS];
#pragma unroll
      for (int k = 0; k < 3; ++k) chunk[k] = tile_chunk<ST, S>(tile, at, k, lane);
      repeat<0, 2 * S::KS>([&](auto op_) {
        constexpr int op = op_, k = op / 2, kEach = 16 / S::KS;  // powers behind each
        in_order();
        next[op % 2] = multiply<ST>(chunk[k], q[op % 2][k], next[op % 2]);
        if constexpr (op % 2 == 0 && k + 3 < S::KS) chunk[k + 3] = tile_chunk<ST, S>(tile, at, k + 3, lane);
        repeat<op * kEach, (op + 1) * kEach>([&](auto i_) {
          constexpr int b = i_ / 16, e = i_ % 16;
          add_power(b, e);
          settled(part[b][e & 3]);
        });
      });
      in_order();
      if (v_before >= 0) settle(v_before);
      z[0] = next[0];
      z[1] = next[1];
      v_before = t * S::TR + at;
      mask_end(v_before);
    }
  });
  if (v_before >= 0) {
#pragma unroll
    for (int e = 0; e < 16; ++e) add_power(0, e), add_power(1, e);
    settle(v_before);
  }
  float m[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) m[b] = unset[b] ? kNegInf : from[b];
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
__global__ __launch_bounds__(kBlock, 1) void loss_narrow_gradient(LossArgs a, int64_t splits, int64_t run,
                                                                  float* parts, void* out) {
  static_assert(S::QW == 4 && S::BL == 2 && S::TR == 64);
  __shared__ __align__(1024) unsigned char ring[kGradientRing * S::stage];
  __shared__ __align__(1024) unsigned char info_ring[DTABLE ? kGradientRing * kInfoBytes : 16];
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
      const RowInfo info = row_info(a, n);
      base[b] = info.base;
      target[b] = info.target;
      grad[b] = fabsf(info.grad);
    }
  }
  f32x16 acc[2][2 * S::SL], z[2];
  u32x4 d[2][2];  // of a block, rounded to the rows' type: operands of the product
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int c = 0; c < 2 * S::SL; ++c) acc[b][c] = f32x16{};
#pragma unroll
    for (int e = 0; e < 16; ++e) z[b][e] = kNegInf;  // powers of 0 before the first block
    d[b][0] = d[b][1] = u32x4{};
  }
  f32x4 bases[4];  // DTABLE: of the rows of z, lane / 32's share
#pragma unroll
  for (int p = 0; p < 4; ++p) bases[p] = f32x4{};
  const auto read_bases = [&](const unsigned char* info, int at, int p) {
    if constexpr (DTABLE) bases[p] = *reinterpret_cast<const f32x4*>(info + (at + 8 * p + 4 * (lane >> 5)) * 4);
  };
  // The i-th power of z.
  const auto power = [&](auto i_) {
    constexpr int i = i_, b = i / 16, e = i % 16;
    float p = __builtin_amdgcn_exp2f(
        __builtin_fmaf(z[b][e], a.exponent, DTABLE ? -bases[e / 4][e % 4] : -base[b]));
    settled(p);
    z[b][e] = p;
  };
  // The gradients of the logits from their powers; t0: the block's first row of T (real:
  // there is such a block).
  const auto settle = [&](const unsigned char* info, int at, int64_t t0, bool real) {
    if constexpr (DTABLE) {
      // where the wave has a row's target, or a row's gradient is negative
      const int32_t* words = reinterpret_cast<const int32_t*>(info + 256) + at;
      const float* grads = reinterpret_cast<const float*>(info + 512) + at;
      const int32_t word = words[lane & 31];
      const int32_t hit = (word & ~kNegative) - static_cast<int32_t>(q0);
      if (real && __any(word >= 0 && ((hit >= 0 && hit < 64) || (word & kNegative)))) {
        rarely();
        const int32_t v = static_cast<int32_t>(q0) + (lane & 31);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const u32x4 w4 = *reinterpret_cast<const u32x4*>(words + 8 * p + 4 * (lane >> 5));
          const f32x4 g4 = *reinterpret_cast<const f32x4*>(grads + 8 * p + 4 * (lane >> 5));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t w = static_cast<int32_t>(w4[e]), target_v = w & ~kNegative;  // none: below 0
            if (w >= 0 && w != target_v)
              z[0][4 * p + e] = -z[0][4 * p + e], z[1][4 * p + e] = -z[1][4 * p + e];
            z[0][4 * p + e] -= target_v == v ? g4[e] : 0.0f;
            z[1][4 * p + e] -= target_v == v + 32 ? g4[e] : 0.0f;
          }
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int32_t at = (target[b] & ~kNegative) - static_cast<int32_t>(t0);
        const bool near = target[b] >= 0 && static_cast<uint32_t>(at) < 32u;
        if (real && __any(near)) {
          rarely();
          subtract_at(z[b], element_of(at, near, lane), grad[b]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        StoredVec<ST, 8> v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = static_cast<typename Stored<ST>::type>(z[b][8 * s + e]);
        d[b][s] = __builtin_bit_cast(u32x4, v);
      }
  };
  // The i-th of the product's 4 SL parts, and the tile's columns for it.
  const auto columns_of = [&](const unsigned char* tile, int at, int i) {
    return tile_columns<S>(tile, at, i / (2 * S::SL), i % (2 * S::SL), lane);
  };
  const auto product = [&](const u32x4& columns, int i) {
    const int t = i / (2 * S::SL), c = i % (2 * S::SL);
    acc[0][c] = multiply<ST>(columns, d[0][t], acc[0][c]);
    acc[1][c] = multiply<ST>(columns, d[1][t], acc[1][c]);
  };
  u32x4 ahead[4];  // of the next step's first parts, read a step before
#pragma unroll
  for (int i = 0; i < 4; ++i) ahead[i] = u32x4{};
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads are counted from here
  // A step has three blocks in hand, one after the other in T: the logits of one, the powers
  // of the one before, the product of the one before that (in the tile before): matrix and
  // vector instructions in turn.
  const unsigned char *tile_before = ring, *info_before = info_ring;
  stream_tiles<kGradientRing, 1>(stream, first, last, [&](int64_t t, int buffer, int before) {
    const unsigned char* tile = ring + buffer * S::stage;
    const unsigned char* info = info_ring + (DTABLE ? buffer * kInfoBytes : 0);
    tile_before = ring + before * S::stage;
    info_before = info_ring + (DTABLE ? before * kInfoBytes : 0);
#pragma unroll
    for (int block = 0; block < 2; ++block) {
      f32x16 next[2] = {f32x16{}, f32x16{}};
      // The matrix instructions: the product's first four parts, whose columns are there, then
      // the logits with the other parts between them.  Reads come kReadAhead before their use,
      // those for the next step's start at the end.
      constexpr int kOps = 4 * S::KS, kRest = 4 * S::SL - 4;
      u32x4 chunk[S::KS], rest[kRest ? kRest : 1];
      const unsigned char* due = block == 0 ? info_before : info;
      repeat<0, kOps>([&](auto op_) {
        constexpr int op = op_;
        in_order();
        // Behind the first 8 come groups of 6: logits 2 k, logits 2 k + 1, part 4 + k; or, of
        // short rows, of 2.
        constexpr int kGroup = kRest ? 6 : 4, at = op - 8;
        constexpr int pair = at >= 0 ? at / kGroup : 0, in = at >= 0 ? at % kGroup : 0;
        if constexpr (op < 8) {
          constexpr int i = op / 2, c = i % (2 * S::SL), s = i / (2 * S::SL);
          acc[op % 2][c] = multiply<ST>(ahead[i], d[op % 2][s], acc[op % 2][c]);
        } else if constexpr (in < 4) {
          constexpr int k = 2 * pair + in / 2;
          next[in % 2] = multiply<ST>(chunk[k], q[in % 2][k], next[in % 2]);
        } else {
          constexpr int i = 4 + pair, c = i % (2 * S::SL), s = i / (2 * S::SL);
          acc[in % 2][c] = multiply<ST>(rest[pair], d[in % 2][s], acc[in % 2][c]);
        }
        constexpr int ahead_at = op + kReadAhead - 8;
        constexpr int pair_r = ahead_at >= 0 ? ahead_at / kGroup : 0, in_r = ahead_at >= 0 ? ahead_at % kGroup : 1;
        if constexpr (op + kReadAhead < kOps) {
          if constexpr (in_r == 0 || in_r == 2) {
            constexpr int k = 2 * pair_r + in_r / 2;
            chunk[k] = tile_chunk<ST, S>(tile, 32 * block, k, lane);
          }
          if constexpr (in_r == 4) rest[pair_r] = columns_of(tile_before, 32 * block, 4 + pair_r);
        }
        if constexpr (kOps - op <= 4) {
          constexpr int i = 4 - (kOps - op);
          ahead[i] = block == 0 ? columns_of(tile_before, 32, i) : columns_of(tile, 0, i);
        }
        constexpr int kEach = 32 / kOps;  // powers
        repeat<op * kEach, (op + 1) * kEach>(power);
      });
      in_order();
#pragma unroll
      for (int p = 0; p < 4; ++p) read_bases(info, 32 * block, p);  // of `next`
      settle(due, block == 0 ? 32 : 0, t * S::TR - (block == 0 ? 32 : 0),
             block == 1 || t > first);
      if constexpr (!DTABLE) {  // rows past the table's end: no powers
        if (rows_t - t * S::TR - 32 * block < 32) {
          rarely();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (place_of(0, e, lane) >= rows_t - t * S::TR - 32 * block) next[0][e] = next[1][e] = kNegInf;
        }
      }
      z[0] = next[0];
      z[1] = next[1];
    }
  });
  // the last tile's products, its second block's powers
  {
    const int buffer = static_cast<int>((last - 1 - first) % kGradientRing);
    tile_before = ring + buffer * S::stage;
    info_before = info_ring + (DTABLE ? buffer * kInfoBytes : 0);
#pragma unroll
    for (int i = 0; i < 4 * S::SL; ++i) product(columns_of(tile_before, 0, i), i);
    repeat<0, 32>(power);
    settle(info_before, 32, (last - 1) * S::TR + 32, true);
#pragma unroll
    for (int i = 0; i < 4 * S::SL; ++i) product(columns_of(tile_before, 32, i), i);
  }
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
