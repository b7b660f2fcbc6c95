// scan.hip -- the gated linear recurrence over jagged sequences, per channel
//   h_t = a_t h_{t-1} + b_t x_t,   h_{-1} = initial,
// with a = sigmoid(g), b = 1 - a = sigmoid(-g) or a = g, b = 1, its backward
// pass
//   lam_t = dh_t + a_{t+1} lam_{t+1}   (grad_final after the last token)
//   dx_t = b_t lam_t
//   dg_t = lam_t (h_{t-1} - x_t) a_t b_t   or   lam_t h_{t-1}
//   dinitial = a_0 lam_0
// and the step that takes one token for each sequence.  States are fp32;
// h, dx and dg are rounded once, to the rows' type.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "layers.hpp"

using namespace tbe;

namespace {

struct Gates {
  float a, b;
};

// sigmoid(g) and sigmoid(-g) from one exponential of -|g|: neither overflows
// nor loses the smaller one to cancellation.  exp(-|g|) = 2^t (1 + r ln 2) with
// t + r = -|g| log2 e, r what the product's rounding left out; the reciprocal
// gets one Newton step.  Both are good to some 2^-23 relative; expf and two
// divisions cost three times as much and made the backward pass wait for them.
template <bool SIGMOID>
__device__ __forceinline__ Gates gates(float g) {
  if constexpr (!SIGMOID) return {g, 1.0f};
  constexpr double kLog2e = 1.4426950408889634074;
  constexpr float kHigh = static_cast<float>(kLog2e);
  constexpr float kLow = static_cast<float>(kLog2e - static_cast<double>(kHigh));
  const float m = fabsf(g) > 128.0f ? -128.0f : -fabsf(g);  // infinities stay out of r, NaN passes
  const float t = m * kHigh;
  const float r = fmaf(m, kLow, fmaf(m, kHigh, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  const float z = fmaf(p, r * 0.69314718f, p);
  const float d = 1.0f + z;
  float hi = __builtin_amdgcn_rcpf(d);
  hi = fmaf(fmaf(-d, hi, 1.0f), hi, hi);
  const float lo = z * hi;
  return g >= 0.0f ? Gates{hi, lo} : Gates{lo, hi};
}

// --- one token for each sequence ---------------------------------------------

template <int ST, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void step_kernel(const void* x, int64_t x_stride,
                                                      const void* gate, int64_t gate_stride,
                                                      const float* state, int64_t state_stride,
                                                      void* h, float* next, uint32_t items,
                                                      uint32_t vecs, int32_t dim) {
  const uint32_t i = blockIdx.x * kBlock + threadIdx.x;
  if (i >= items) return;
  const uint32_t s = i / vecs;
  const int32_t c = static_cast<int32_t>(i - s * vecs) * 4;
  const int64_t out = static_cast<int64_t>(s) * dim + c;
  if (c + 4 <= dim) {
    const auto xv = load_vec<ST, 4>(x, s * x_stride + c);
    const auto gv = load_vec<ST, 4>(gate, s * gate_stride + c);
    StoredVec<kF32, 4> v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (state) v = load_vec<kF32, 4>(state, s * state_stride + c);
    StoredVec<ST, 4> hv;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Gates t = gates<SIGMOID>(static_cast<float>(gv[k]));
      v[k] = t.a * v[k] + t.b * static_cast<float>(xv[k]);
      hv[k] = static_cast<typename Stored<ST>::type>(v[k]);
    }
    store_vec<kF32, 4>(next, out, v);
    store_vec<ST, 4>(h, out, hv);
    return;
  }
  for (int k = 0; c + k < dim; ++k) {
    const Gates t = gates<SIGMOID>(load_one<ST>(gate, s * gate_stride + c + k));
    const float v0 = state ? state[s * state_stride + c + k] : 0.0f;
    const float v = t.a * v0 + t.b * load_one<ST>(x, s * x_stride + c + k);
    next[out + k] = v;
    store_one<ST>(h, out + k, v);
  }
}

// --- whole sequences -----------------------------------------------------------

struct ScanArgs {
  int64_t tokens, seqs, dim;
  const void* x;
  const void* gate;
  const void* offsets;
  int32_t index64;
  const float* initial;  // null: zeros
  int64_t x_stride, gate_stride, initial_stride;
  // forward
  void* h;
  float* final;
  float* carry;  // null: not kept
  // backward
  const float* carried;
  const void* grad_h;         // null: zeros
  const float* grad_final;    // null: zeros
  int64_t grad_h_stride, grad_final_stride;
  void* dx;
  void* dgate;
  int64_t dx_stride, dgate_stride;
  float* dinitial;            // null: not asked for
};

// Offsets are clamped to the tokens, so that bad ones read and write nothing out of range.
__device__ __forceinline__ int64_t offset_at(const ScanArgs& a, int64_t s) {
  const int64_t o = a.index64 ? static_cast<const int64_t*>(a.offsets)[s]
                              : static_cast<const int32_t*>(a.offsets)[s];
  return o < 0 ? 0 : (o > a.tokens ? a.tokens : o);
}

// The token axis is cut into tiles whatever the sequences: W waves of T tokens
// each (a span), and 64 V channels, V neighbours a lane.  Within its span a wave
// reduces the recurrence to "state out = A state in + B" per channel, the waves'
// pairs join in LDS, and the tiles' in the workspace: a tile publishes its own
// (A, B), or, where a sequence starts inside, the state it ends with, which
// depends on no earlier tile; it then looks back for the nearest tile whose end
// state is known and folds the pairs between, first tile first, into its own
// start state and the end state it publishes.  Every state is the same sequence
// of operations whichever tile was found, so results do not depend on timing.
// The waves then run their tokens from their start states.  One pass: inputs are
// read once and stay in registers in between.
//
// What passes between tiles is written and read with 8- and 4-byte device-scope
// atomics; a value is there once it differs from all ones (a NaN that canonical()
// never lets through).  Tiles are numbered by a ticket taken at a workgroup's
// start, so every tile waited for is running or done.
constexpr int kCarry = 8;                  // tokens between the states that are carried
constexpr uint64_t kNoPair = ~uint64_t{0};
constexpr uint32_t kNoState = ~uint32_t{0};
constexpr uint32_t kSpinLimit = 1u << 22;  // polls before a wait gives up (states turn NaN)

struct ScanWork {
  uint32_t* ticket;
  int32_t* lo;       // [tiles + 1]: first offset at or past the tile's first token
  uint64_t* pairs;   // [tiles, dim]
  uint32_t* states;  // [tiles, dim]
  int64_t tiles;
  int32_t channel_blocks;
};

__device__ __forceinline__ float canonical(float v) {
  return v != v ? __uint_as_float(0x7FC00000u) : v;
}
__device__ __forceinline__ uint64_t ld_pair(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t ld_state(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_pair(uint64_t* p, float A, float B) {
  const uint64_t v = static_cast<uint64_t>(__float_as_uint(canonical(B))) << 32 |
                     __float_as_uint(canonical(A));
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_state(uint32_t* p, float v) {
  __hip_atomic_store(p, __float_as_uint(canonical(v)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Before the tiles: nothing published, the tiles' first offsets found, and the
// empty sequences' outputs, which belong to no token (copied from `from`).
__global__ __launch_bounds__(kBlock) void scan_prepare(ScanArgs a, ScanWork w, int32_t tile_tokens,
                                                       const float* from, int64_t from_stride,
                                                       float* to) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t all = static_cast<int64_t>(gridDim.x) * kBlock;
  if (id == 0) *w.ticket = 0u;
  const int64_t words = w.tiles * a.dim;
  for (int64_t i = id; i < words; i += all) {
    w.pairs[i] = kNoPair;
    w.states[i] = kNoState;
  }
  if (w.tiles > 0)
    for (int64_t k = id; k <= w.tiles; k += all) {
      const int64_t token = k * tile_tokens;
      int64_t lo = 0, hi = a.seqs + 1;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (offset_at(a, mid) < token) lo = mid + 1;
        else hi = mid;
      }
      w.lo[k] = static_cast<int32_t>(lo);
    }
  if (!to) return;
  const int lane = lane_id();
  for (int64_t s0 = id - lane; s0 < a.seqs; s0 += all) {
    const int64_t s = s0 + lane;
    uint64_t empty = __ballot(s < a.seqs && offset_at(a, s) >= offset_at(a, s + 1));
    for (; empty; empty &= empty - 1) {
      const int64_t e = s0 + __builtin_ctzll(empty);
      for (int64_t c = lane; c < a.dim; c += 64)
        to[e * a.dim + c] = from ? from[e * from_stride + c] : 0.0f;
    }
  }
}

// What the waves of a tile share.
template <int V, int W, int T>
struct TileShared {
  static constexpr int kWindow = 2 * W;  // tiles looked back on at a time
  uint32_t ticket;
  int32_t lists[2][W * T];               // sequence that starts at / ends with a token, or -1
  uint32_t resets[W];                    // the wave's span holds a reset
  float A[W][64 * V], B[W][64 * V];
  float pair_a[kWindow][64 * V], pair_b[kWindow][64 * V];
  uint32_t state[kWindow][64 * V];
};

// Which sequences start in and end with the tile's tokens.
template <int V, int W, int T>
__device__ __forceinline__ void list_sequences(const ScanArgs& a, const ScanWork& w, int64_t tile,
                                               TileShared<V, W, T>& sh) {
  constexpr int kTokens = W * T;
  const int64_t t0 = tile * kTokens;
  const int64_t lo = w.lo[tile], hi = w.lo[tile + 1];
  for (int64_t i = lo + threadIdx.x; i <= hi && i <= a.seqs; i += 64 * W) {
    const int64_t o = offset_at(a, i);
    const int64_t at = o - t0;
    if (i < a.seqs && at >= 0 && at < kTokens && offset_at(a, i + 1) > o)
      sh.lists[0][at] = static_cast<int32_t>(i);
    if (i > 0 && at >= 1 && at <= kTokens && offset_at(a, i - 1) < o)
      sh.lists[1][at - 1] = static_cast<int32_t>(i - 1);
  }
}

// A tile's start state per channel (the state after its predecessor in scan
// order), the tile's own pair, and the end state published.  STEP: +1 where
// tile k follows tile k - 1, -1 where it follows tile k + 1.
template <int V, int W, int T, int STEP>
__device__ __forceinline__ void join_tiles(const ScanArgs& a, const ScanWork& w, int64_t tile,
                                           int64_t c0, bool mine, TileShared<V, W, T>& sh,
                                           float (&start)[V]) {
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  // the tile's pair: wave by wave in scan order
  float A[V], B[V];
  bool reset = false;
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
  for (int q = 0; q < W; ++q) {
    const int i = STEP > 0 ? q : W - 1 - q;
    const bool r = sh.resets[i];
    reset |= r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float wa = sh.A[i][lane * V + v], wb = sh.B[i][lane * V + v];
      B[v] = r ? wb : fmaf(wa, B[v], wb);
      A[v] *= wa;
    }
  }
  const bool first = STEP > 0 ? tile == 0 : tile == w.tiles - 1;
  const int64_t here = tile * a.dim + c0;
  if (wave == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (mine) {
        if (reset || first) st_state(w.states + here + v, B[v]);
        else st_pair(w.pairs + here + v, A[v], B[v]);
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) start[v] = 0.0f;
  // no state comes in where the tile's first token (in scan order) starts afresh
  if (first || sh.lists[STEP > 0 ? 0 : 1][STEP > 0 ? 0 : W * T - 1] >= 0) return;
  constexpr int kWindow = TileShared<V, W, T>::kWindow;
  uint32_t spins = 0;
  for (int round = 0;; ++round) {
    // The first look is at the nearest tile alone (with short sequences it knows
    // its end state by itself), the later ones at the whole window.
    const int n = round == 0 ? 1 : kWindow;
    __syncthreads();
    for (int e = wave; e < n; e += W) {
      const int64_t k = tile - static_cast<int64_t>(STEP) * (e + 1);
      const bool real = k >= 0 && k < w.tiles;
      uint64_t pair[V];
      uint32_t state[V];
      bool there;
      do {
        there = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          pair[v] = 0;
          state[v] = 0;
          if (real && mine) {
            state[v] = ld_state(w.states + k * a.dim + c0 + v);
            pair[v] = ld_pair(w.pairs + k * a.dim + c0 + v);
            there = there && (state[v] != kNoState || pair[v] != kNoPair);
          }
        }
        if (__all(there)) break;
        if (++spins > kSpinLimit) break;
        __builtin_amdgcn_s_sleep(1);
      } while (true);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sh.pair_a[e][lane * V + v] = __uint_as_float(static_cast<uint32_t>(pair[v]));
        sh.pair_b[e][lane * V + v] = __uint_as_float(static_cast<uint32_t>(pair[v] >> 32));
        sh.state[e][lane * V + v] = state[v];
      }
    }
    __syncthreads();
    // from the nearest tile whose end state is there, through the pairs of those
    // after it (a tile without a state has its pair)
    bool have[V];
#pragma unroll
    for (int v = 0; v < V; ++v) have[v] = false;
    for (int e = n - 1; e >= 0; --e)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t s = sh.state[e][lane * V + v];
        const float on = fmaf(sh.pair_a[e][lane * V + v], start[v], sh.pair_b[e][lane * V + v]);
        start[v] = s != kNoState ? __uint_as_float(s) : on;
        have[v] = have[v] || s != kNoState;
      }
    bool all = true;
#pragma unroll
    for (int v = 0; v < V; ++v) all = all && have[v];
    if (__all(all)) break;
    if (round > static_cast<int>(kSpinLimit >> 4)) {
#pragma unroll
      for (int v = 0; v < V; ++v) start[v] = __uint_as_float(0x7FC00000u);
      break;
    }
  }
  if (wave == 0 && !reset) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (mine) st_state(w.states + here + v, fmaf(A[v], start[v], B[v]));
  }
}

// The state a wave starts from: the tile's, taken through the waves before it.
template <int V, int W, int T, int STEP>
__device__ __forceinline__ void wave_start(const TileShared<V, W, T>& sh, int wave, int lane,
                                           float (&state)[V]) {
#pragma unroll
  for (int q = 0; q < W; ++q) {
    const int i = STEP > 0 ? q : W - 1 - q;
    if (STEP > 0 ? i < wave : i > wave) {
      const bool r = sh.resets[i];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float wb = sh.B[i][lane * V + v];
        state[v] = r ? wb : fmaf(sh.A[i][lane * V + v], state[v], wb);
      }
    }
  }
}

// A buffer descriptor: loads past `bytes` give 0, stores there are dropped.  The
// spans' loads and stores go through these, so that no branch parts them and all
// of a wave's loads are in flight together.
__device__ __forceinline__ auto buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0,
                                           static_cast<int>(bytes > 0 ? bytes : 0), 0x00020000);
}
using Buffer = decltype(buffer(nullptr, 0));
constexpr uint32_t kOutside = 0x80000000u;  // past every descriptor's end

// One lane's V channels: 2, 4 or 8 bytes.
template <int BYTES>
struct Word;
template <>
struct Word<2> {
  using type = uint16_t;
  static __device__ __forceinline__ type load(Buffer b, uint32_t o) {
    return __builtin_amdgcn_raw_buffer_load_b16(b, o, 0, 0);
  }
  static __device__ __forceinline__ void store(type v, Buffer b, uint32_t o) {
    __builtin_amdgcn_raw_buffer_store_b16(v, b, o, 0, 0);
  }
};
template <>
struct Word<4> {
  using type = uint32_t;
  static __device__ __forceinline__ type load(Buffer b, uint32_t o) {
    return __builtin_amdgcn_raw_buffer_load_b32(b, o, 0, 0);
  }
  static __device__ __forceinline__ void store(type v, Buffer b, uint32_t o) {
    __builtin_amdgcn_raw_buffer_store_b32(v, b, o, 0, 0);
  }
};
template <>
struct Word<8> {
  using type = uint32_t __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ type load(Buffer b, uint32_t o) {
    return __builtin_amdgcn_raw_buffer_load_b64(b, o, 0, 0);
  }
  static __device__ __forceinline__ void store(type v, Buffer b, uint32_t o) {
    __builtin_amdgcn_raw_buffer_store_b64(v, b, o, 0, 0);
  }
};
template <int ST, int V>
using RowWord = Word<StorageTraits<ST>::bytes * V>;

// The span's rows from column `c` (the workgroup's first) of `base`; a lane's V
// channels are at byte `lane_off` (kOutside: none).
template <int ST>
__device__ __forceinline__ Buffer span_buffer(const void* base, int64_t stride, int64_t t0,
                                              int tokens, int64_t c, int64_t dim) {
  constexpr int b = StorageTraits<ST>::bytes;
  return buffer(static_cast<const char*>(base) + (t0 * stride + c) * b,
                tokens > 0 && base ? ((tokens - 1) * stride + dim - c) * b : 0);
}
template <int ST, int V, int T>
__device__ __forceinline__ void load_span(Buffer rows, int64_t stride, uint32_t lane_off,
                                          StoredVec<ST, V> (&out)[T]) {
  const uint32_t step = static_cast<uint32_t>(stride) * StorageTraits<ST>::bytes;
#pragma unroll
  for (int i = 0; i < T; ++i)
    out[i] = __builtin_bit_cast(StoredVec<ST, V>, RowWord<ST, V>::load(rows, lane_off + i * step));
}
// The rows of `base` of the sequences whose bits are set in mask (list: lane i
// holds the sequence of token i), 0 for the others.
template <int V, int T>
__device__ __forceinline__ void load_marked(const float* base, int64_t stride, uint32_t mask,
                                            int32_t list, int64_t c, int64_t dim, uint32_t lane_off,
                                            float (&out)[T][V]) {
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) out[i][v] = 0.0f;
  if (!base || !mask) return;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int64_t s = __builtin_amdgcn_readlane(list, i);
    const Buffer row = buffer(base + (s < 0 ? 0 : s * stride) + c, s < 0 ? 0 : (dim - c) * 4);
    const auto r = __builtin_bit_cast(StoredVec<kF32, V>, RowWord<kF32, V>::load(row, lane_off));
#pragma unroll
    for (int v = 0; v < V; ++v) out[i][v] = r[v];
  }
}
template <int ST, int V>
__device__ __forceinline__ void store_row(Buffer rows, uint32_t off, const float (&f)[V]) {
  StoredVec<ST, V> o;
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = static_cast<typename Stored<ST>::type>(f[v]);
  RowWord<ST, V>::store(__builtin_bit_cast(typename RowWord<ST, V>::type, o), rows, off);
}

// Tile and channels of a workgroup, in the order of the tickets, and the lists cleared.
template <int V, int W, int T>
__device__ __forceinline__ uint32_t take_ticket(const ScanWork& w, TileShared<V, W, T>& sh) {
  if (threadIdx.x == 0) sh.ticket = atomicAdd(w.ticket, 1u);
  for (int i = threadIdx.x; i < 2 * W * T; i += 64 * W) (&sh.lists[0][0])[i] = -1;
  __syncthreads();
  return sh.ticket;
}

template <int ST, int V, bool SIGMOID, int W, int T>
__global__ __launch_bounds__(64 * W, 4) void scan_tiles(ScanArgs a, ScanWork w) {
  __shared__ TileShared<V, W, T> sh;
  const uint32_t ticket = take_ticket(w, sh);
  const int64_t tile = ticket / w.channel_blocks;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = static_cast<int64_t>(ticket % w.channel_blocks) * (64 * V), c0 = c + lane * V;
  const bool mine = c0 < a.dim;  // V divides dim
  constexpr int bytes = StorageTraits<ST>::bytes;
  const uint32_t at = mine ? lane * V * bytes : kOutside, at32 = mine ? lane * V * 4 : kOutside;
  const int64_t t0 = tile * (W * T) + wave * T;
  const int tokens = static_cast<int>(a.tokens - t0 < 0 ? 0 : a.tokens - t0 < T ? a.tokens - t0
                                                                                     : T);
  StoredVec<ST, V> x[T], g[T];
  load_span<ST, V, T>(span_buffer<ST>(a.gate, a.gate_stride, t0, tokens, c, a.dim), a.gate_stride, at, g);
  load_span<ST, V, T>(span_buffer<ST>(a.x, a.x_stride, t0, tokens, c, a.dim), a.x_stride, at, x);
  list_sequences<V, W, T>(a, w, tile, sh);
  __syncthreads();
  const int32_t starts = lane < T ? sh.lists[0][wave * T + lane] : -1;
  const int32_t ends = lane < T ? sh.lists[1][wave * T + lane] : -1;
  const uint32_t first = static_cast<uint32_t>(__ballot(starts >= 0));
  const uint32_t last = static_cast<uint32_t>(__ballot(ends >= 0));
  float init[T][V];
  load_marked<V, T>(a.initial, a.initial_stride, first, starts, c, a.dim, at32, init);

  // state_i = first ? u_i : k_i state_{i-1} + u_i, the state before a first token being in its u
  float k[T][V], u[T][V], A[V], B[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const bool f = first >> i & 1u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gates t = gates<SIGMOID>(static_cast<float>(g[i][v]));
      const bool in = i < tokens;
      k[i][v] = in ? t.a : 1.0f;
      const float in_x = t.b * static_cast<float>(x[i][v]);
      u[i][v] = f ? fmaf(t.a, init[i][v], in_x) : in ? in_x : 0.0f;
      B[v] = f ? u[i][v] : fmaf(k[i][v], B[v], u[i][v]);
      A[v] *= k[i][v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[wave][lane * V + v] = A[v];
    sh.B[wave][lane * V + v] = B[v];
  }
  if (lane == 0) sh.resets[wave] = first;
  __syncthreads();
  float state[V];
  join_tiles<V, W, T, 1>(a, w, tile, c0, mine, sh, state);
  wave_start<V, W, T, 1>(sh, wave, lane, state);
  const Buffer carry = span_buffer<kF32>(a.carry, a.dim, t0 / kCarry, (tokens + kCarry - 1) / kCarry, c,
                                         a.dim);
  const Buffer h = span_buffer<ST>(a.h, a.dim, t0, tokens, c, a.dim);
  const uint32_t step = static_cast<uint32_t>(a.dim) * bytes;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const bool f = first >> i & 1u;
    if (i % kCarry == 0 && a.carry)
      store_row<kF32, V>(carry, at32 + i / kCarry * static_cast<uint32_t>(a.dim) * 4, state);
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = f ? u[i][v] : fmaf(k[i][v], state[v], u[i][v]);
    store_row<ST, V>(h, at + i * step, state);
    if (last >> i & 1u) {
      const int64_t s = __builtin_amdgcn_readlane(ends, i);
      store_row<kF32, V>(span_buffer<kF32>(a.final, a.dim, s, 1, c, a.dim), at32, state);
    }
  }
}

template <int ST, int V, bool SIGMOID, int W, int T>
__global__ __launch_bounds__(64 * W, 4) void scan_tiles_back(ScanArgs a, ScanWork w) {
  __shared__ TileShared<V, W, T> sh;
  const uint32_t ticket = take_ticket(w, sh);
  const int64_t tile = w.tiles - 1 - ticket / w.channel_blocks;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = static_cast<int64_t>(ticket % w.channel_blocks) * (64 * V), c0 = c + lane * V;
  const bool mine = c0 < a.dim;  // V divides dim
  constexpr int bytes = StorageTraits<ST>::bytes;
  const uint32_t at = mine ? lane * V * bytes : kOutside, at32 = mine ? lane * V * 4 : kOutside;
  const int64_t t0 = tile * (W * T) + wave * T;
  const int tokens = static_cast<int>(a.tokens - t0 < 0 ? 0 : a.tokens - t0 < T ? a.tokens - t0
                                                                                     : T);
  StoredVec<ST, V> x[T], g[T], dh[T];
  load_span<ST, V, T>(span_buffer<ST>(a.gate, a.gate_stride, t0, tokens, c, a.dim), a.gate_stride, at, g);
  load_span<ST, V, T>(span_buffer<ST>(a.x, a.x_stride, t0, tokens, c, a.dim), a.x_stride, at, x);
  load_span<ST, V, T>(span_buffer<ST>(a.grad_h, a.grad_h_stride, t0, tokens, c, a.dim), a.grad_h_stride,
                   at, dh);
  float state[V];
  {
    const auto r = __builtin_bit_cast(
        StoredVec<kF32, V>,
        RowWord<kF32, V>::load(span_buffer<kF32>(a.carried, a.dim, t0 / kCarry, tokens > 0, c, a.dim),
                               at32));
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = r[v];
  }
  list_sequences<V, W, T>(a, w, tile, sh);
  __syncthreads();
  const int32_t starts = lane < T ? sh.lists[0][wave * T + lane] : -1;
  const int32_t ends = lane < T ? sh.lists[1][wave * T + lane] : -1;
  const uint32_t first = static_cast<uint32_t>(__ballot(starts >= 0));
  const uint32_t last = static_cast<uint32_t>(__ballot(ends >= 0));
  // before[i]: the state before token i; lam_i = up_i + (last ? 0 : mu_{i+1}), mu_i = a_i lam_i,
  // the gradient of a final state being in its up
  float before[T][V], up[T][V], A[V], B[V];
  load_marked<V, T>(a.initial, a.initial_stride, first, starts, c, a.dim, at32, before);
  load_marked<V, T>(a.grad_final, a.grad_final_stride, last, ends, c, a.dim, at32, up);
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const bool f = first >> i & 1u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gates t = gates<SIGMOID>(static_cast<float>(g[i][v]));
      before[i][v] = f ? before[i][v] : state[v];
      const float u = t.b * static_cast<float>(x[i][v]);
      // as the forward pass rounds it
      state[v] = f ? fmaf(t.a, before[i][v], u) : fmaf(t.a, state[v], u);
      up[i][v] += static_cast<float>(dh[i][v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
  for (int i = T - 1; i >= 0; --i) {
    const bool l = last >> i & 1u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float k = i < tokens ? gates<SIGMOID>(static_cast<float>(g[i][v])).a : 1.0f;
      B[v] = k * (l ? up[i][v] : up[i][v] + B[v]);
      A[v] *= k;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[wave][lane * V + v] = A[v];
    sh.B[wave][lane * V + v] = B[v];
  }
  if (lane == 0) sh.resets[wave] = last;
  __syncthreads();
  float mu[V];
  join_tiles<V, W, T, -1>(a, w, tile, c0, mine, sh, mu);
  wave_start<V, W, T, -1>(sh, wave, lane, mu);
  const Buffer dxs = span_buffer<ST>(a.dx, a.dx_stride, t0, tokens, c, a.dim);
  const Buffer dgs = span_buffer<ST>(a.dgate, a.dgate_stride, t0, tokens, c, a.dim);
  const uint32_t dx_step = static_cast<uint32_t>(a.dx_stride) * bytes;
  const uint32_t dg_step = static_cast<uint32_t>(a.dgate_stride) * bytes;
#pragma unroll
  for (int i = T - 1; i >= 0; --i) {
    const bool l = last >> i & 1u;
    float dx[V], dg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gates t = gates<SIGMOID>(static_cast<float>(g[i][v]));
      const float lam = l ? up[i][v] : up[i][v] + mu[v];
      dx[v] = t.b * lam;
      dg[v] = SIGMOID ? lam * (before[i][v] - static_cast<float>(x[i][v])) * (t.a * t.b)
                      : lam * before[i][v];
      mu[v] = i < tokens ? t.a * lam : mu[v];
    }
    store_row<ST, V>(dxs, at + i * dx_step, dx);
    store_row<ST, V>(dgs, at + i * dg_step, dg);
    if (a.dinitial && (first >> i & 1u)) {
      const int64_t s = __builtin_amdgcn_readlane(starts, i);
      store_row<kF32, V>(span_buffer<kF32>(a.dinitial, a.dim, s, 1, c, a.dim), at32, mu);
    }
  }
}

// Waves in a tile and tokens in a wave's span.  The backward pass holds twice as
// much for each token: its spans are as short as the carry's rows.
constexpr int kForwardWaves = 8, kForwardSpan = 16;
constexpr int kBackWaves = 8, kBacT = kCarry;
constexpr int kForwardTokens = kForwardWaves * kForwardSpan, kBackTokens = kBackWaves * kBacT;

template <int ST, int V, bool SIGMOID>
hipError_t launch_tiles(const ScanArgs& a, const ScanWork& w, bool back, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(w.tiles * w.channel_blocks));
  if (back)
    hipLaunchKernelGGL((scan_tiles_back<ST, V, SIGMOID, kBackWaves, kBacT>), grid,
                       dim3(64 * kBackWaves), 0, s, a, w);
  else
    hipLaunchKernelGGL((scan_tiles<ST, V, SIGMOID, kForwardWaves, kForwardSpan>), grid,
                       dim3(64 * kForwardWaves), 0, s, a, w);
  return hipGetLastError();
}

template <int ST, int V>
hipError_t launch_tiles(const ScanArgs& a, const ScanWork& w, int32_t kind, bool back,
                        hipStream_t s) {
  return kind == TBE_GATE_SIGMOID ? launch_tiles<ST, V, true>(a, w, back, s)
                                  : launch_tiles<ST, V, false>(a, w, back, s);
}

// Channels a lane: two neighbours of 16-bit rows, where every row starts at an
// even element and a wave's 128 channels are not mostly past the end.
int lane_channels(const tbe_scan_input* in, const ScanArgs& a) {
  if (in->dtype == TBE_F32 || a.dim <= 64 || a.dim % 2) return 1;
  const auto even = [](const void* p, int64_t stride) { return aligned_to(p, 4) && stride % 2 == 0; };
  return even(a.x, a.x_stride) && even(a.gate, a.gate_stride) && even(a.h, 0) &&
                 even(a.grad_h, a.grad_h_stride) && even(a.dx, a.dx_stride) &&
                 even(a.dgate, a.dgate_stride)
             ? 2
             : 1;
}

int64_t tiles_of(int64_t tokens, bool back) {
  const int64_t n = back ? kBackTokens : kForwardTokens;
  return (tokens + n - 1) / n;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace: ticket, first offsets, pairs, states.
size_t workspace_bytes_of(int64_t tokens, int64_t dim) {
  const size_t tiles = static_cast<size_t>(tiles_of(tokens, kBackTokens < kForwardTokens));
  return 256 + up256((tiles + 1) * 4) + up256(tiles * dim * 8) + up256(tiles * dim * 4);
}

hipError_t launch_scan(ScanArgs a, const tbe_scan_input* in, bool back, void* workspace,
                       hipStream_t s) {
  if (a.tokens <= 1)  // a single row's stride says nothing
    a.x_stride = a.gate_stride = a.grad_h_stride = a.dx_stride = a.dgate_stride = a.dim;
  ScanWork w{};
  w.tiles = tiles_of(a.tokens, back);
  const int v = lane_channels(in, a);
  w.channel_blocks = static_cast<int32_t>((a.dim + 64 * v - 1) / (64 * v));
  char* p = static_cast<char*>(workspace);
  w.ticket = reinterpret_cast<uint32_t*>(p);
  p += 256;
  w.lo = reinterpret_cast<int32_t*>(p);
  p += up256(static_cast<size_t>(w.tiles + 1) * 4);
  w.pairs = reinterpret_cast<uint64_t*>(p);
  p += up256(static_cast<size_t>(w.tiles) * a.dim * 8);
  w.states = reinterpret_cast<uint32_t*>(p);
  const int64_t work = std::max(w.tiles * a.dim, a.seqs);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((work + kBlock - 1) / kBlock, 1024));
  hipLaunchKernelGGL(scan_prepare, dim3(static_cast<unsigned>(blocks)), dim3(kBlock), 0, s, a, w,
                     back ? kBackTokens : kForwardTokens,
                     back ? a.grad_final : a.initial,
                     back ? a.grad_final_stride : a.initial_stride, back ? a.dinitial : a.final);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || w.tiles == 0) return e;
  if (in->dtype == TBE_F32) return launch_tiles<kF32, 1>(a, w, in->gate_kind, back, s);
  if (in->dtype == TBE_F16)
    return v == 2 ? launch_tiles<kF16, 2>(a, w, in->gate_kind, back, s)
                  : launch_tiles<kF16, 1>(a, w, in->gate_kind, back, s);
  return v == 2 ? launch_tiles<kBF16, 2>(a, w, in->gate_kind, back, s)
                : launch_tiles<kBF16, 1>(a, w, in->gate_kind, back, s);
}

// A span's rows lie within a buffer descriptor's reach.
constexpr int64_t kMaxRow = int64_t{1} << 24;

// Sizes a call can take: 31-bit tokens and sequences, 2^32 threads in a launch.
tbe_status check_sizes(int64_t tokens, int64_t seqs, int64_t dim, int32_t dtype) {
  constexpr int64_t kMax = 0x7FFFFFFF;
  if (tokens < 0 || seqs < 0 || dim < 1 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  if (seqs == 0 && tokens > 0) return TBE_ERR_INVALID_ARGUMENT;
  if (tokens >= kMax || seqs >= kMax || dim > kMaxRow) return TBE_ERR_UNSUPPORTED;
  // 512 threads for 64 tokens of 64 channels
  if ((tokens + 63) / 64 * ((dim + 63) / 64) >= (int64_t{1} << 23)) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

size_t carry_bytes_of(int64_t tokens, int64_t dim) {
  return static_cast<size_t>((tokens + kCarry - 1) / kCarry) * static_cast<size_t>(dim) * sizeof(float);
}

tbe_status check_input(const tbe_scan_input* in) {
  if (!in) return TBE_ERR_INVALID_ARGUMENT;
  const tbe_status st = check_sizes(in->tokens, in->seqs, in->dim, in->dtype);
  if (st != TBE_OK) return st;
  if (in->gate_kind != TBE_GATE_SIGMOID && in->gate_kind != TBE_GATE_DECAY)
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->index_dtype != TBE_I32 && in->index_dtype != TBE_I64) return TBE_ERR_INVALID_ARGUMENT;
  const size_t e = dtype_bytes(in->dtype);
  if (in->seqs > 0 && !in->offsets) return TBE_ERR_INVALID_ARGUMENT;
  if (!aligned_to(in->offsets, in->index_dtype == TBE_I64 ? 8 : 4)) return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 0 && (!in->x || !in->gate || !aligned_to(in->x, e) || !aligned_to(in->gate, e)))
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 1 && (in->x_stride > kMaxRow || in->gate_stride > kMaxRow))
    return TBE_ERR_UNSUPPORTED;
  if (in->x_stride < 0 || in->gate_stride < 0 || in->initial_stride < 0 ||
      !aligned_to(in->initial, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  return TBE_OK;
}

tbe_status check_workspace(const tbe_scan_input* in, const void* workspace, size_t bytes) {
  if (!workspace || !aligned_to(workspace, 256)) return TBE_ERR_INVALID_ARGUMENT;
  return bytes < workspace_bytes_of(in->tokens, in->dim) ? TBE_ERR_WORKSPACE_TOO_SMALL : TBE_OK;
}

ScanArgs scan_args(const tbe_scan_input* in) {
  ScanArgs a{};
  a.tokens = in->tokens;
  a.seqs = in->seqs;
  a.dim = in->dim;
  a.x = in->x;
  a.gate = in->gate;
  a.offsets = in->offsets;
  a.index64 = in->index_dtype == TBE_I64;
  a.initial = in->initial;
  a.x_stride = in->x_stride;
  a.gate_stride = in->gate_stride;
  a.initial_stride = in->initial_stride;
  return a;
}

}  // namespace

extern "C" {

tbe_status tbe_scan_step(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride,
                         const float* state, int64_t state_stride, void* h, float* next_state,
                         int64_t seqs, int64_t dim, int32_t dtype, int32_t gate_kind,
                         void* stream) {
  const tbe_status st = check_sizes(0, seqs, dim, dtype);
  if (st != TBE_OK) return st;
  if (gate_kind != TBE_GATE_SIGMOID && gate_kind != TBE_GATE_DECAY) return TBE_ERR_INVALID_ARGUMENT;
  if (seqs == 0) return TBE_OK;
  const size_t e = dtype_bytes(dtype);
  if (!x || !gate || !h || !next_state || !aligned_to(x, e) || !aligned_to(gate, e) ||
      !aligned_to(h, e) || !aligned_to(state, 4) || !aligned_to(next_state, 4) || x_stride < 0 ||
      gate_stride < 0 || state_stride < 0)
    return TBE_ERR_INVALID_ARGUMENT;
  const int64_t vecs = (dim + 3) / 4;
  if (seqs * vecs > 0xFFFFFF00ll) return TBE_ERR_UNSUPPORTED;  // 2^32 threads in a launch
  const uint32_t items = static_cast<uint32_t>(seqs * vecs);
  const dim3 grid((items + kBlock - 1) / kBlock);
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, s, x, x_stride, gate, gate_stride, state,
                       state_stride, h, next_state, items, static_cast<uint32_t>(vecs),
                       static_cast<int32_t>(dim));
  };
  const bool sig = gate_kind == TBE_GATE_SIGMOID;
  if (dtype == TBE_F32) sig ? go(step_kernel<kF32, true>) : go(step_kernel<kF32, false>);
  else if (dtype == TBE_F16) sig ? go(step_kernel<kF16, true>) : go(step_kernel<kF16, false>);
  else sig ? go(step_kernel<kBF16, true>) : go(step_kernel<kBF16, false>);
  return hipGetLastError() == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

tbe_status tbe_scan_sizes(int64_t tokens, int64_t seqs, int64_t dim, int32_t dtype,
                          size_t* carry_bytes, size_t* workspace_bytes) {
  if (!carry_bytes || !workspace_bytes) return TBE_ERR_INVALID_ARGUMENT;
  const tbe_status st = check_sizes(tokens, seqs, dim, dtype);
  if (st != TBE_OK) return st;
  *carry_bytes = carry_bytes_of(tokens, dim);
  *workspace_bytes = seqs > 0 ? workspace_bytes_of(tokens, dim) : 0;
  return TBE_OK;
}

tbe_status tbe_scan_forward(const tbe_scan_input* in, void* h, float* final, float* carry,
                            void* workspace, size_t workspace_bytes, void* stream) {
  tbe_status st = check_input(in);
  if (st != TBE_OK) return st;
  if (in->seqs == 0) return TBE_OK;
  st = check_workspace(in, workspace, workspace_bytes);
  if (st != TBE_OK) return st;
  if (!final || !aligned_to(final, 4) || !aligned_to(carry, 16) ||
      (in->tokens > 0 && (!h || !aligned_to(h, dtype_bytes(in->dtype)))))
    return TBE_ERR_INVALID_ARGUMENT;
  ScanArgs a = scan_args(in);
  a.h = h;
  a.final = final;
  a.carry = carry;
  return launch_scan(a, in, false, workspace, static_cast<hipStream_t>(stream)) == hipSuccess
             ? TBE_OK
             : TBE_ERR_HIP;
}

tbe_status tbe_scan_backward(const tbe_scan_input* in, const float* carry, const void* grad_h,
                             int64_t grad_h_stride, const float* grad_final,
                             int64_t grad_final_stride, void* dx, int64_t dx_stride, void* dgate,
                             int64_t dgate_stride, float* dinitial, void* workspace,
                             size_t workspace_bytes, void* stream) {
  tbe_status st = check_input(in);
  if (st != TBE_OK) return st;
  if (in->seqs == 0) return TBE_OK;
  st = check_workspace(in, workspace, workspace_bytes);
  if (st != TBE_OK) return st;
  const size_t e = dtype_bytes(in->dtype);
  if (grad_h_stride < 0 || grad_final_stride < 0 || !aligned_to(grad_h, e) ||
      !aligned_to(grad_final, 4) || !aligned_to(dinitial, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 0 && (!carry || !aligned_to(carry, 16) || !dx || !dgate || !aligned_to(dx, e) ||
                         !aligned_to(dgate, e)))
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 1 && (dx_stride < in->dim || dgate_stride < in->dim))
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 1 && (grad_h_stride > kMaxRow || dx_stride > kMaxRow || dgate_stride > kMaxRow))
    return TBE_ERR_UNSUPPORTED;
  ScanArgs a = scan_args(in);
  a.carried = carry;
  a.grad_h = grad_h;
  a.grad_h_stride = grad_h_stride;
  a.grad_final = grad_final;
  a.grad_final_stride = grad_final_stride;
  a.dx = dx;
  a.dx_stride = dx_stride;
  a.dgate = dgate;
  a.dgate_stride = dgate_stride;
  a.dinitial = dinitial;
  return launch_scan(a, in, true, workspace, static_cast<hipStream_t>(stream)) == hipSuccess
             ? TBE_OK
             : TBE_ERR_HIP;
}

}  // extern "C"
