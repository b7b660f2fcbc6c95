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
//
// Every input is read and every output written once, 16 bytes a token and channel
// of 16-bit rows for both directions, and memory would bound that: 4 sequences of
// 16384 x 1024 bf16 move 1.0 GB, 194 us at a copy's 5.2 TB/s.  They take 273 us (3.7
// TB/s), 8192 of about 20 x 256 175 us (4.1).  A tile waits 6 of its 11 us for the
// states before it (reads and writes between XCDs, about a microsecond each way),
// and of the rest about half is arithmetic: some 30 vector instructions a token and
// channel forwards, 50 backwards.  With short sequences the wait is 3 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layers.hpp"

using namespace tbe;

namespace {

struct Gates {
  float a, b;
};

// sigmoid(g) and sigmoid(-g) from one exponential of -|g|: neither overflows
// nor loses the smaller one to cancellation.  exp(-|g|) = 2^t (1 + r) with
// t + r / ln 2 = -|g| log2 e, r what t leaves out.  bf16 gates have 8 bits, so t
// is exact with a log2 e of 16; others take the product's rounding back with two
// fused operations.  The reciprocal is the hardware's, good to a step of 2^-23,
// as is the exponential.
template <int ST, bool SIGMOID>
__device__ __forceinline__ Gates gates(float g) {
  if constexpr (!SIGMOID) return {g, 1.0f};
  constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;
  // infinities stay out of r, NaN passes
  const float m = __builtin_elementwise_maximum(-fabsf(g), -128.0f);
  float t, r;
  if constexpr (ST == kBF16) {
    constexpr float kHigh = 47274.0f / 32768.0f;
    t = m * kHigh;
    r = m * static_cast<float>((kLog2e - static_cast<double>(kHigh)) * kLn2);
  } else {
    constexpr float kHigh = static_cast<float>(kLog2e);
    constexpr float kLow = static_cast<float>(kLog2e - static_cast<double>(kHigh));
    t = m * kHigh;
    r = fmaf(m, kLow, fmaf(m, kHigh, -t)) * static_cast<float>(kLn2);
  }
  const float p = __builtin_amdgcn_exp2f(t);
  const float z = fmaf(p, r, p);
  const float hi = __builtin_amdgcn_rcpf(1.0f + z), lo = z * hi;
  return g >= 0.0f ? Gates{hi, lo} : Gates{lo, hi};
}

// --- one token for each sequence ---------------------------------------------

// Four channels a thread, everything read and written once: 2048 x 128 fp32 take
// 3.1 us, most of it the launch; 10 us a call with what the host does for it.
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
      const Gates t = gates<ST, SIGMOID>(static_cast<float>(gv[k]));
      v[k] = t.a * v[k] + t.b * static_cast<float>(xv[k]);
      hv[k] = static_cast<typename Stored<ST>::type>(v[k]);
    }
    store_vec<kF32, 4>(next, out, v);
    store_vec<ST, 4>(h, out, hv);
    return;
  }
  for (int k = 0; c + k < dim; ++k) {
    const Gates t = gates<ST, SIGMOID>(load_one<ST>(gate, s * gate_stride + c + k));
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

// A scan in one pass over tiles that look back at what earlier ones published (Merrill,
// Garland, "Single-pass parallel prefix scan with decoupled look-back", 2016), in groups.
//
// The token axis is cut into tiles whatever the sequences: W waves of T tokens
// each (a span), and 64 V channels, V neighbours a lane.  Within its span a wave
// reduces the recurrence to "state out = A state in + B" per channel, the waves'
// pairs join in LDS, and the tiles' in the workspace.  A tile publishes its own
// (A, B) or, where a sequence starts inside, the state it ends with, which
// depends on no earlier tile.  Eight tiles make a group; its last tile
// publishes the group's pair or state the same way, and, once it knows the state
// the group starts from, the group's end state.  A tile's start state is that of
// its group (the nearest earlier group whose end state is there, taken through
// the pairs of the groups between) taken through the tiles before it in the
// group, or from the nearest of them that knows its state: within a group nothing
// waits for a chain, and the chain has one link for 8 tiles.  Every state is the
// same sequence of operations whatever was found when, so results do not depend
// on timing.  The waves then run their tokens from their start states.  One pass:
// inputs are read once and stay in registers in between.
//
// What passes between tiles is written and read with 8- and 4-byte device-scope
// atomics; a value is there once it differs from all ones (a NaN that canonical()
// never lets through).  Workgroups start in the order of their numbers, so the
// tiles waited for are running; nothing rests on that: a wait ends after
// max_polls, and the tile then walks its sequence's earlier tokens itself.  (A
// ticket taken at each workgroup's start, which would fix the order, costs 14 ns
// a workgroup on its one counter.)
constexpr int kCarry = 8;                  // tokens between the states that are carried
constexpr uint64_t kNoPair = ~uint64_t{0};
constexpr uint32_t kNoState = ~uint32_t{0};
constexpr uint32_t kMaxPolls = 1u << 16;   // each about a microsecond

constexpr int kGroup = 8;                  // tiles

// What a row of `dim` channels publishes: a pair, a state, or both.
struct Published {
  uint64_t* pairs;
  uint32_t* states;
};
struct ScanWork {
  int2* marks;       // [tokens]: the sequences that start and end with a token, or -1
  Published tile;    // [tiles, dim]: a pair or a state
  Published group;   // [groups, dim]: a pair, then a state
  int64_t tiles, rows;  // rows: of all published ones, tiles first
  uint32_t channel_blocks;
  uint32_t max_polls;
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

// The first offset at or past `token`: 64 probes at a time.
__device__ __forceinline__ int64_t find_offset(const ScanArgs& a, int64_t token) {
  const int lane = lane_id();
  int64_t lo = 0, hi = a.seqs + 1;
  while (hi > lo) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step - 1;
    const int below = __popcll(__ballot(at < hi && offset_at(a, at) < token));
    lo += below * step;
    if (step == 1) break;
    hi = lo + step - 1 < hi ? lo + step - 1 : hi;
  }
  return lo;
}

// Before the tiles: nothing published, each token's sequences marked (a wave
// takes 64 tokens), and the empty sequences' outputs, which belong to no token,
// copied from `from`.
__global__ __launch_bounds__(kBlock) void scan_prepare(ScanArgs a, ScanWork w, const float* from,
                                                       int64_t from_stride, float* to) {
  __shared__ int2 marks[kWavesPerBlock][64];
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t all = static_cast<int64_t>(gridDim.x) * kBlock;
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  for (int64_t t0 = id - lane; t0 < a.tokens; t0 += all) {
    marks[wave][lane] = make_int2(-1, -1);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int64_t end = t0 + 64;
    bool more = true;
    for (int64_t i0 = find_offset(a, t0); more && i0 <= a.seqs; i0 += 64) {
      const int64_t i = i0 + lane < a.seqs ? i0 + lane : a.seqs;
      const int64_t o = offset_at(a, i), next = offset_at(a, i < a.seqs ? i + 1 : i),
                    before = offset_at(a, i > 0 ? i - 1 : i);
      const bool in = i0 + lane <= a.seqs;
      if (in && o >= t0 && o < end && next > o) marks[wave][o - t0].x = static_cast<int32_t>(i);
      if (in && o > t0 && o <= end && before < o)
        marks[wave][o - 1 - t0].y = static_cast<int32_t>(i - 1);
      more = __all(o <= end);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (t0 + lane < a.tokens) w.marks[t0 + lane] = marks[wave][lane];
  }
  const int64_t words = w.rows * a.dim;
  for (int64_t i = id; i < words; i += all) {
    w.tile.pairs[i] = kNoPair;
    w.tile.states[i] = kNoState;
  }
  if (!to) return;
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

// The sequence that holds the token before `token` (a thread by itself).
__device__ int64_t sequence_before(const ScanArgs& a, int64_t token) {
  int64_t lo = 0, hi = a.seqs + 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (offset_at(a, mid) < token) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

// Waves in a tile: 4, or 8 where sequences span tiles.  Fewer wait less for each
// other (8192 sequences of about 20 x 256 bf16: 63 and 104 us with 4, 76 and 144
// with 8; 2048 of 1-32 x 100 fp32: 13 and 18, 14 and 22), more make the chain of
// tiles shorter (4 of 16384 x 1024 bf16: 111 and 165 us with 8, 126 and 235 with 4;
// 256 of 256 x 512: 49 and 81, 53 and 93; 256 of 128 x 512: both 28 and 46).
constexpr int kFewWaves = 4, kManyWaves = 8;

// What the waves of a tile share.
template <int V, int W, int T>
struct TileShared {
  uint32_t resets[W];                    // tokens of the wave's span that start afresh
  float A[W][64 * V], B[W][64 * V];
  uint64_t pair[kGroup][64 * V];         // of the tiles before this one in its group
  uint32_t state[kGroup][64 * V];
  uint64_t group_pair[W][64 * V];        // of the W groups before this one
  uint32_t group_state[W][64 * V];
  uint32_t kind[kGroup], group_kind[W];
};

// An entry as a wave reads it.
enum Kind : uint32_t { kAbsent, kPair, kState };
template <int V>
struct Entry {
  uint64_t pair[V];
  uint32_t state[V];
  // What is there of row r for all the wave's channels.
  __device__ __forceinline__ Kind read(const Published& p, int64_t at, bool mine) {
    bool paired = true, known = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      pair[v] = 0;
      state[v] = 0;
      if (mine) {
        state[v] = ld_state(p.states + at + v);
        pair[v] = ld_pair(p.pairs + at + v);
      }
      known = known && state[v] != kNoState;
      paired = paired && pair[v] != kNoPair;
    }
    return __all(known) ? kState : __all(paired) ? kPair : kAbsent;
  }
};
// GROWS: gates may be above 1, and their products infinite.
// The product of gates' products: 0 where either is, also beside an infinite one.  (A
// gate that is itself infinite or NaN shows in B.)
template <bool GROWS>
__device__ __forceinline__ float times(float A, float a) {
  return GROWS && (A == 0.0f || a == 0.0f) ? 0.0f : A * a;
}
// The state after tokens of which (A, B) is the pair.  B is the state they make of 0,
// token after token, so 0 needs no product: 0 times an infinite A would be NaN.
template <bool GROWS>
__device__ __forceinline__ float after(float A, float state, float B) {
  return GROWS && state == 0.0f ? B : fmaf(A, state, B);
}
template <bool GROWS>
__device__ __forceinline__ float after(uint64_t pair, float state) {
  return after<GROWS>(__uint_as_float(static_cast<uint32_t>(pair)), state,
                      __uint_as_float(static_cast<uint32_t>(pair >> 32)));
}
__device__ __forceinline__ float pair_a(uint64_t p) {
  return __uint_as_float(static_cast<uint32_t>(p));
}

// A tile's start state per channel (the state after its predecessor in scan
// order), and the tile's and its group's entries published.  STEP: +1 where tile
// k follows tile k - 1, -1 where it follows tile k + 1; tiles and groups are
// numbered in scan order here.  walk(start) works the start state out from the
// inputs, for waits that give up.
template <int V, int W, int T, int STEP, bool GROWS, typename Walk>
__device__ __forceinline__ void join_tiles(const ScanArgs& a, const ScanWork& w, int64_t tile,
                                           int64_t c0, bool mine, TileShared<V, W, T>& sh,
                                           float (&start)[V], Walk walk) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t k = STEP > 0 ? tile : w.tiles - 1 - tile, group = k / kGroup;
  const int in_group = static_cast<int>(k % kGroup);
  const bool first = k == 0, last = in_group == kGroup - 1;
  // the tile's pair, which the first wave publishes: wave by wave in scan order
  float A[V], B[V];
  bool reset = first;
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll 2
  for (int q = 0; q < (wave == 0 ? W : 0); ++q) {
    const int i = STEP > 0 ? q : W - 1 - q;
    const bool r = sh.resets[i] != 0u;
    reset |= r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float wa = sh.A[i][lane * V + v], wb = sh.B[i][lane * V + v];
      B[v] = r ? wb : after<GROWS>(wa, B[v], wb);
      A[v] = times<GROWS>(A[v], wa);
    }
  }
  const int64_t at = k * a.dim + c0, group_at = group * a.dim + c0;
  const auto publish = [&](const Published& p, int64_t to, bool known) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (mine) {
        if (known) st_state(p.states + to + v, B[v]);
        else st_pair(p.pairs + to + v, A[v], B[v]);
      }
  };
  if (wave == 0) {
    publish(w.tile, at, reset);
    if (last && reset) publish(w.group, group_at, true);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) start[v] = 0.0f;
  // No state comes in where the tile's first token (in scan order) starts afresh.
  if (first || (STEP > 0 ? sh.resets[0] & 1u : sh.resets[W - 1] >> (T - 1) & 1u)) return;

  // The tiles before this one in the group, nearest first, up to the nearest that
  // knows its state.  Where sequences are short (few waves), the nearest alone is
  // looked at first, and mostly does; where they are long, all at once (4 of 16384 x
  // 1024 bf16: 112 and 198 us instead of 114 and 206).
  uint32_t polls = 0;
  int depth = 0;        // tiles taken
  bool known = false, given_up = false;
  while (depth < in_group && !known && !given_up) {
    const int n = depth == 0 && W == kFewWaves ? 1 : in_group;
    for (int e = depth + wave; e < n; e += W) {
      Entry<V> x;
      Kind kind;
      for (;; ++polls) {
        kind = x.read(w.tile, (k - 1 - e) * a.dim + c0, mine);
        if (kind != kAbsent || polls >= w.max_polls) break;
        __builtin_amdgcn_s_sleep(1);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sh.pair[e][lane * V + v] = x.pair[v];
        sh.state[e][lane * V + v] = x.state[v];
      }
      if (lane == 0) sh.kind[e] = kind;
    }
    __syncthreads();
    const uint32_t kind = lane >= depth && lane < n ? sh.kind[lane] : kPair;
    const uint64_t states = __ballot(kind == kState), absent = __ballot(kind == kAbsent);
    const int to = states ? __builtin_ctzll(states) + 1 : n;
    given_up = absent != 0 && __builtin_ctzll(absent) < to;
    known = states != 0;
    depth = to;
  }

  // The state the group starts from, unless a tile of the group knows its own.
  float ga[V], gb[V];  // the group's pair
#pragma unroll
  for (int v = 0; v < V; ++v) ga[v] = 1.0f, gb[v] = 0.0f;
  const bool chained = !known && !given_up && group > 0;
  if (chained) {
    if (wave == 0 && last && !reset) {  // first tile first
#pragma unroll 4
      for (int e = kGroup - 2; e >= 0; --e)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint64_t p = sh.pair[e][lane * V + v];
          gb[v] = after<GROWS>(p, gb[v]);
          ga[v] = times<GROWS>(ga[v], pair_a(p));
        }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gb[v] = after<GROWS>(A[v], gb[v], B[v]);
        ga[v] = times<GROWS>(ga[v], A[v]);
        if (mine) st_pair(w.group.pairs + group_at + v, ga[v], gb[v]);
      }
    }
    // Wave e watches the e-th group before; each wave goes on by itself as soon as
    // the nearest state is there with the pairs of the groups after it.
    volatile uint32_t* kinds = sh.group_kind;
    const bool real = group - 1 - wave >= 0;
    uint32_t seen = kAbsent;
    int found = -1;
    for (;; ++polls) {
      if (seen != kState) {
        Entry<V> x;
        const uint32_t now = real ? x.read(w.group, (group - 1 - wave) * a.dim + c0, mine) : kPair;
        if (now > seen) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (now == kPair) sh.group_pair[wave][lane * V + v] = x.pair[v];
            else sh.group_state[wave][lane * V + v] = x.state[v];
          }
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
          if (lane == 0) kinds[wave] = now;
          seen = now;
        }
      }
      uint32_t kind[W];
#pragma unroll
      for (int e = 0; e < W; ++e) kind[e] = kinds[e];
      found = -1;
#pragma unroll
      for (int e = W - 1; e >= 0; --e) found = kind[e] == kState ? e : kind[e] == kPair ? found : -1;
      found = __builtin_amdgcn_readfirstlane(found);
      if (found >= 0 || polls >= w.max_polls) break;
      __builtin_amdgcn_s_sleep(1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    given_up = found < 0;
    if (!given_up) {
#pragma unroll
      for (int v = 0; v < V; ++v) start[v] = __uint_as_float(sh.group_state[found][lane * V + v]);
      for (int e = found - 1; e >= 0; --e)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint64_t p = sh.group_pair[e][lane * V + v];
          start[v] = after<GROWS>(p, start[v]);
        }
#pragma unroll
      for (int v = 0; v < V; ++v) gb[v] = after<GROWS>(ga[v], start[v], gb[v]);  // the group's end
    }
  }
  if (given_up) {
    walk(start);
  } else {
    if (known) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        start[v] = __uint_as_float(sh.state[depth - 1][lane * V + v]);
    }
#pragma unroll 4
    for (int e = known ? depth - 2 : depth - 1; e >= 0; --e)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint64_t p = sh.pair[e][lane * V + v];
        start[v] = after<GROWS>(p, start[v]);
      }
  }
  if (wave == 0 && last && !reset) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (mine)
        st_state(w.group.states + group_at + v,
                 chained && !given_up ? gb[v] : after<GROWS>(A[v], start[v], B[v]));
  }
}

// The state a wave starts from: the tile's, taken through the waves before it.
template <int V, int W, int T, int STEP, bool GROWS>
__device__ __forceinline__ void wave_start(const TileShared<V, W, T>& sh, int wave, int lane,
                                           float (&state)[V]) {
#pragma unroll 2
  for (int q = 0; q < W; ++q) {
    const int i = STEP > 0 ? q : W - 1 - q;
    if (STEP > 0 ? i < wave : i > wave) {
      const bool r = sh.resets[i];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float wb = sh.B[i][lane * V + v];
        state[v] = r ? wb : after<GROWS>(sh.A[i][lane * V + v], state[v], wb);
      }
    }
  }
}

// Has v in its register from here on.  Without it the compiler puts the last
// operations on a span's values off until they are used, holds more than their
// results in the meantime, and spills.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

// Whether the products of all the wave's channels are finite.
template <int V>
__device__ __forceinline__ bool finite(const float (&A)[V]) {
  bool f = true;
#pragma unroll
  for (int v = 0; v < V; ++v) f = f && __builtin_isfinite(A[v]);
  return __all(f);
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

// The span's rows from column `c` (the workgroup's first) of `base`, a descriptor
// for each, made in scalar registers: one for them all needs each row's offset in
// a vector register of its own.  A lane's V channels are at byte `lane_off`
// (kOutside: none).
struct Span {
  const char* base;
  uint32_t step, bytes;  // between rows, of a row
  int tokens;
  __device__ __forceinline__ Buffer row(int i) const {
    return buffer(base + static_cast<uint64_t>(step) * i, i < tokens ? bytes : 0u);
  }
};
template <int ST>
__device__ __forceinline__ Span span(const void* base, int64_t stride, int64_t t0, int tokens,
                                     int64_t c, int64_t dim) {
  constexpr int b = StorageTraits<ST>::bytes;
  return {static_cast<const char*>(base) + (t0 * stride + c) * b, static_cast<uint32_t>(stride * b),
          static_cast<uint32_t>((dim - c) * b), base ? tokens : 0};
}
template <int ST, int V, int T>
__device__ __forceinline__ void load_span(const Span& rows, uint32_t lane_off,
                                          StoredVec<ST, V> (&out)[T]) {
#pragma unroll
  for (int i = 0; i < T; ++i)
    out[i] = __builtin_bit_cast(StoredVec<ST, V>, RowWord<ST, V>::load(rows.row(i), lane_off));
}
// The rows of `base` of the sequences whose bits are set in mask (list: lane at +
// i holds the sequence of token i), 0 for the others.
template <int V, int T>
__device__ __forceinline__ void load_marked(const float* base, int64_t stride, uint32_t mask,
                                            int32_t list, int at, int64_t c, int64_t dim,
                                            uint32_t lane_off,
                                            float (&out)[T][V]) {
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) out[i][v] = 0.0f;
  if (!base || !mask) return;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int64_t s = __builtin_amdgcn_readlane(list, at + i);
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

// Which tile (in scan order) and channels a workgroup takes.  Workgroups go round
// robin to the XCDs: an XCD takes all the channels of each eighth tile.
struct Place {
  int64_t tile;
  uint32_t channels;
};
__device__ __forceinline__ Place place_of(const ScanWork& w) {
  const uint32_t eight = blockIdx.x / 8, row = eight / w.channel_blocks;
  return {static_cast<int64_t>(row) * 8 + blockIdx.x % 8, eight - row * w.channel_blocks};
}

// Tokens in a wave's span, and whether the backward pass works its gates out again
// after the join instead of keeping them.  It holds twice as much for each token as
// the forward pass; without the gates, rows of 2 bytes need half of that.  Where
// sequences are long and the wait for the join is more than half of a tile's time,
// spans of 16 halve the number of waits (4 of 16384 x 1024 bf16: 198 -> 170 us);
// the forward pass with spans of 32 and gates worked out again went from 112 to 136.
constexpr int kForwardSpan = 16;
constexpr int back_span(int waves) { return waves == kManyWaves ? 16 : 8; }
template <int ST>
constexpr bool gates_again(int waves) {
  return waves == kManyWaves && StorageTraits<ST>::bytes == 2;
}

// A row's values anew: what was computed from them before is not kept for later.
template <int ST, int V>
__device__ __forceinline__ void renew(StoredVec<ST, V>& row) {
  using W = typename RowWord<ST, V>::type;
  W w = __builtin_bit_cast(W, row);
  if constexpr (sizeof(W) == 2) {
    uint32_t wide = w;
    asm volatile("" : "+v"(wide));
    w = static_cast<W>(wide);
  } else {
    asm volatile("" : "+v"(w));
  }
  row = __builtin_bit_cast(StoredVec<ST, V>, w);
}

template <int ST, int V, bool SIGMOID, int W, int T>
__global__ __launch_bounds__(64 * W, 4) void scan_tiles(ScanArgs a, ScanWork w) {
  __shared__ TileShared<V, W, T> sh;
  const Place place = place_of(w);
  if (place.tile >= w.tiles) return;
  const int64_t tile = place.tile;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = static_cast<int64_t>(place.channels) * (64 * V), c0 = c + lane * V;
  const bool mine = c0 < a.dim;  // V divides dim
  constexpr int bytes = StorageTraits<ST>::bytes;
  const uint32_t at = mine ? lane * V * bytes : kOutside, at32 = mine ? lane * V * 4 : kOutside;
  const int64_t t0 = tile * (W * T) + wave * T;
  const int tokens = static_cast<int>(a.tokens - t0 < 0 ? 0 : a.tokens - t0 < T ? a.tokens - t0
                                                                                     : T);
  // First of all: their answer does not wait for the rows' then.
  const int2 marks = lane < tokens ? w.marks[t0 + lane] : make_int2(-1, -1);
  StoredVec<ST, V> x[T], g[T];
  load_span<ST, V, T>(span<ST>(a.gate, a.gate_stride, t0, tokens, c, a.dim), at, g);
  load_span<ST, V, T>(span<ST>(a.x, a.x_stride, t0, tokens, c, a.dim), at, x);
  if (threadIdx.x < W) sh.group_kind[threadIdx.x] = kAbsent;
  const int32_t starts = marks.x, ends = marks.y;
  const uint32_t first = static_cast<uint32_t>(__ballot(starts >= 0));
  const uint32_t last = static_cast<uint32_t>(__ballot(ends >= 0));
  // state_i = first ? u_i : k_i state_{i-1} + u_i, the state before a first token being in its u
  float k[T][V], u[T][V], A[V], B[V];
  // A span in the middle of a sequence, T tokens long, has nothing to choose.
  const bool plain = first == 0u && tokens == T;
  auto reduce = [&](auto plain_) {
    constexpr bool kPlain = plain_;
    float init[4][V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool f = !kPlain && (first >> i & 1u), in = kPlain || i < tokens;
      if (!kPlain && i % 4 == 0)  // initial states of four tokens at a time: few spans have more starts
        load_marked<V, 4>(a.initial, a.initial_stride, first >> i & 15u, starts, i, c, a.dim, at32, init);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gates t = gates<ST, SIGMOID>(static_cast<float>(g[i][v]));
        const float in_x = t.b * static_cast<float>(x[i][v]);
        k[i][v] = in ? t.a : 1.0f;
        u[i][v] = f ? fmaf(t.a, init[i % 4][v], in_x) : in ? in_x : 0.0f;
        settle(k[i][v]), settle(u[i][v]);
        B[v] = f ? u[i][v] : fmaf(k[i][v], B[v], u[i][v]);
        A[v] *= k[i][v];
      }
    }
  };
  if (plain) reduce(std::true_type{});
  else reduce(std::false_type{});
  if constexpr (!SIGMOID) {
    if (!finite(A)) {  // gates above 1 that pass fp32's range, maybe with one of 0 behind
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] = 1.0f;
#pragma unroll
        for (int i = 0; i < T; ++i) A[v] = times<true>(A[v], k[i][v]);
      }
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
  join_tiles<V, W, T, 1, !SIGMOID>(a, w, tile, c0, mine, sh, state, [&](float (&v)[V]) {
    // the sequence that the tile's first token goes on
    const int64_t end = tile * (W * T), s = sequence_before(a, end);
    if (s < 0 || s >= a.seqs) return;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (!mine) continue;
      v[q] = a.initial ? a.initial[s * a.initial_stride + c0 + q] : 0.0f;
      for (int64_t t = offset_at(a, s); t < end; ++t) {
        const Gates n = gates<ST, SIGMOID>(load_one<ST>(a.gate, t * a.gate_stride + c0 + q));
        v[q] = fmaf(n.a, v[q], n.b * load_one<ST>(a.x, t * a.x_stride + c0 + q));
      }
    }
  });
  wave_start<V, W, T, 1, !SIGMOID>(sh, wave, lane, state);
  const Span carry = span<kF32>(a.carry, a.dim, t0 / kCarry, (tokens + kCarry - 1) / kCarry, c,
                                         a.dim);
  const Span h = span<ST>(a.h, a.dim, t0, tokens, c, a.dim);
  auto run = [&](auto plain_) {
    constexpr bool kPlain = plain_;
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool f = !kPlain && (first >> i & 1u);
      if (i % kCarry == 0 && a.carry) store_row<kF32, V>(carry.row(i / kCarry), at32, state);
#pragma unroll
      for (int v = 0; v < V; ++v) state[v] = f ? u[i][v] : fmaf(k[i][v], state[v], u[i][v]);
      store_row<ST, V>(h.row(i), at, state);
      if (!kPlain && (last >> i & 1u)) {
        const int64_t s = __builtin_amdgcn_readlane(ends, i);
        store_row<kF32, V>(span<kF32>(a.final, a.dim, s, 1, c, a.dim).row(0), at32, state);
      }
    }
  };
  if (plain && last == 0u) run(std::true_type{});
  else run(std::false_type{});
}

template <int ST, int V, bool SIGMOID, int W, int T>
__global__ __launch_bounds__(64 * W, 4) void scan_tiles_back(ScanArgs a, ScanWork w) {
  __shared__ TileShared<V, W, T> sh;
  const Place place = place_of(w);
  if (place.tile >= w.tiles) return;
  const int64_t tile = w.tiles - 1 - place.tile;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = static_cast<int64_t>(place.channels) * (64 * V), c0 = c + lane * V;
  const bool mine = c0 < a.dim;  // V divides dim
  constexpr int bytes = StorageTraits<ST>::bytes;
  const uint32_t at = mine ? lane * V * bytes : kOutside, at32 = mine ? lane * V * 4 : kOutside;
  const int64_t t0 = tile * (W * T) + wave * T;
  const int tokens = static_cast<int>(a.tokens - t0 < 0 ? 0 : a.tokens - t0 < T ? a.tokens - t0
                                                                                     : T);
  // First of all: their answer does not wait for the rows' then.
  const int2 marks = lane < tokens ? w.marks[t0 + lane] : make_int2(-1, -1);
  StoredVec<ST, V> x[T], g[T], dh[T];
  load_span<ST, V, T>(span<ST>(a.gate, a.gate_stride, t0, tokens, c, a.dim), at, g);
  load_span<ST, V, T>(span<ST>(a.x, a.x_stride, t0, tokens, c, a.dim), at, x);
  load_span<ST, V, T>(span<ST>(a.grad_h, a.grad_h_stride, t0, tokens, c, a.dim), at, dh);
  float state[V];
  {
    const auto r = __builtin_bit_cast(
        StoredVec<kF32, V>,
        RowWord<kF32, V>::load(span<kF32>(a.carried, a.dim, t0 / kCarry, tokens > 0, c, a.dim).row(0), at32));
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = r[v];
  }
  if (threadIdx.x < W) sh.group_kind[threadIdx.x] = kAbsent;
  const int32_t starts = marks.x, ends = marks.y;
  const uint32_t first = static_cast<uint32_t>(__ballot(starts >= 0));
  const uint32_t last = static_cast<uint32_t>(__ballot(ends >= 0));
  // lam_i = up_i + (last ? 0 : mu_{i+1}), mu_i = a_i lam_i, the gradient of a final
  // state being in its up; dgate_i = q_i lam_i with q_i of the state before token i
  // The span's pair is summed in the order of its tokens: mu_0 = sum_i (a_0 .. a_i) up_i
  // up to the first last token.
  constexpr bool kAgain = gates_again<ST>(W);
  constexpr int kMarked = kAgain ? 4 : T;  // tokens whose marked rows are loaded together
  float ka[kAgain ? 1 : T][V], kb[kAgain ? 1 : T][V], up[kAgain ? 1 : T][V], q[T][V], A[V], B[V];
  float final_up[kMarked][V];
  // A span in the middle of a sequence, T tokens long, has nothing to choose.
  const bool plain = (first | last) == 0u && tokens == T;
  auto load_final = [&](int i) {
    load_marked<V, kMarked>(a.grad_final, a.grad_final_stride, last >> i & ((1u << kMarked) - 1u), ends,
                            i, c, a.dim, at32, final_up);
  };
  auto reduce = [&](auto plain_) {
    constexpr bool kPlain = plain_;
    float init[kMarked][V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool f = !kPlain && (first >> i & 1u), in = kPlain || i < tokens;
      const bool passed = !kPlain && (last & ((1u << i) - 1u)) != 0u;
      if (!kPlain && i % kMarked == 0) {
        load_marked<V, kMarked>(a.initial, a.initial_stride, first >> i & ((1u << kMarked) - 1u),
                                starts, i, c, a.dim, at32, init);
        load_final(i);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gates t = gates<ST, SIGMOID>(static_cast<float>(g[i][v]));
        const float before = f ? init[i % kMarked][v] : state[v], xi = static_cast<float>(x[i][v]);
        float at_ = in ? t.a : 1.0f, bt = t.b, ut = static_cast<float>(dh[i][v]);
        if (!kPlain) ut += final_up[i % kMarked][v];
        state[v] = fmaf(t.a, before, t.b * xi);  // as the forward pass rounds it
        q[i][v] = SIGMOID ? (before - xi) * (t.a * t.b) : before;
        settle(at_), settle(bt), settle(q[i][v]), settle(ut);
        if constexpr (!kAgain) ka[i][v] = at_, kb[i][v] = bt, up[i][v] = ut;
        A[v] *= at_;
        B[v] = passed ? B[v] : fmaf(A[v], ut, B[v]);
      }
    }
  };
  if (plain) reduce(std::true_type{});
  else reduce(std::false_type{});
  // Gates above 1, whose products pass fp32's range, make terms of that sum infinite or
  // NaN.  Then both once more, mu_0 token after token, from memory: rare, and registers
  // are full.
  if constexpr (!SIGMOID) {
    if (!finite(A)) {
      bool again[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        again[v] = mine && !__builtin_isfinite(A[v]);
        if (again[v]) A[v] = 1.0f, B[v] = 0.0f;
      }
#pragma unroll 1
      for (int i = tokens - 1; i >= 0; --i) {
        const bool l = last >> i & 1u;
        const int64_t t = t0 + i, s = __builtin_amdgcn_readlane(ends, i);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (!again[v]) continue;
          float ut = a.grad_h ? load_one<ST>(a.grad_h, t * a.grad_h_stride + c0 + v) : 0.0f;
          if (l && a.grad_final) ut += a.grad_final[s * a.grad_final_stride + c0 + v];
          const float at_ = load_one<ST>(a.gate, t * a.gate_stride + c0 + v);
          A[v] = times<true>(A[v], at_);
          B[v] = at_ * (l ? ut : ut + B[v]);
        }
      }
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
  join_tiles<V, W, T, -1, !SIGMOID>(a, w, tile, c0, mine, sh, mu, [&](float (&v)[V]) {
    // the sequence that the token after the tile goes on
    const int64_t begin = (tile + 1) * (W * T);
    const int64_t s = sequence_before(a, begin);
    if (s < 0 || s >= a.seqs) return;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (!mine) continue;
      v[q] = a.grad_final ? a.grad_final[s * a.grad_final_stride + c0 + q] : 0.0f;
      for (int64_t t = offset_at(a, s + 1) - 1; t >= begin; --t) {
        const float up = a.grad_h ? load_one<ST>(a.grad_h, t * a.grad_h_stride + c0 + q) : 0.0f;
        v[q] = gates<ST, SIGMOID>(load_one<ST>(a.gate, t * a.gate_stride + c0 + q)).a * (up + v[q]);
      }
    }
  });
  wave_start<V, W, T, -1, !SIGMOID>(sh, wave, lane, mu);
  const Span dxs = span<ST>(a.dx, a.dx_stride, t0, tokens, c, a.dim);
  const Span dgs = span<ST>(a.dgate, a.dgate_stride, t0, tokens, c, a.dim);
  if constexpr (kAgain) {
#pragma unroll
    for (int i = 0; i < T; ++i) renew<ST, V>(g[i]), renew<ST, V>(dh[i]);
  }
  auto run = [&](auto plain_) {
    constexpr bool kPlain = plain_;
#pragma unroll
    for (int i = T - 1; i >= 0; --i) {
      const bool l = !kPlain && (last >> i & 1u), in = kPlain || i < tokens;
      if (!kPlain && kAgain && i % kMarked == kMarked - 1) load_final(i - kMarked + 1);
      float dx[V], dg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float at_, bt, ut;
        if constexpr (kAgain) {
          const Gates t = gates<ST, SIGMOID>(static_cast<float>(g[i][v]));
          at_ = in ? t.a : 1.0f, bt = t.b, ut = static_cast<float>(dh[i][v]);
          if (!kPlain) ut += final_up[i % kMarked][v];
        } else {
          at_ = ka[i][v], bt = kb[i][v], ut = up[i][v];
        }
        const float lam = l ? ut : ut + mu[v];
        dx[v] = bt * lam;
        dg[v] = lam * q[i][v];
        mu[v] = at_ * lam;
      }
      store_row<ST, V>(dxs.row(i), at, dx);
      store_row<ST, V>(dgs.row(i), at, dg);
      if (!kPlain && a.dinitial && (first >> i & 1u)) {
        const int64_t s = __builtin_amdgcn_readlane(starts, i);
        store_row<kF32, V>(span<kF32>(a.dinitial, a.dim, s, 1, c, a.dim).row(0), at32, mu);
      }
    }
  };
  if (plain) run(std::true_type{});
  else run(std::false_type{});
}

int waves_of(int64_t tokens, int64_t seqs) { return tokens < seqs * 256 ? kFewWaves : kManyWaves; }

template <int ST, int V, bool SIGMOID, int W>
hipError_t launch_tiles(const ScanArgs& a, const ScanWork& w, bool back, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((w.tiles + 7) / 8 * 8 * w.channel_blocks));
  if (back)
    hipLaunchKernelGGL((scan_tiles_back<ST, V, SIGMOID, W, back_span(W)>), grid, dim3(64 * W), 0, s, a,
                       w);
  else
    hipLaunchKernelGGL((scan_tiles<ST, V, SIGMOID, W, kForwardSpan>), grid, dim3(64 * W), 0, s, a, w);
  return hipGetLastError();
}
template <int ST, int V, bool SIGMOID>
hipError_t launch_tiles(const ScanArgs& a, const ScanWork& w, bool back, hipStream_t s) {
  return waves_of(a.tokens, a.seqs) == kFewWaves
             ? launch_tiles<ST, V, SIGMOID, kFewWaves>(a, w, back, s)
             : launch_tiles<ST, V, SIGMOID, kManyWaves>(a, w, back, s);
}

template <int ST, int V>
hipError_t launch_tiles(const ScanArgs& a, const ScanWork& w, int32_t kind, bool back,
                        hipStream_t s) {
  return kind == TBE_GATE_SIGMOID ? launch_tiles<ST, V, true>(a, w, back, s)
                                  : launch_tiles<ST, V, false>(a, w, back, s);
}

// Channels a lane: two neighbours of 16-bit rows, where every row starts at an
// even element and a wave's 128 channels are not mostly past the end (8192
// sequences of about 20 x 256 bf16 in packed rows, both directions: 173 us, 175 with
// one; 4 of 16384 x 1024: 262 and 263).
int lane_channels(const tbe_scan_input* in, const ScanArgs& a) {
  if (in->dtype == TBE_F32 || a.dim <= 64 || a.dim % 2) return 1;
  const auto even = [](const void* p, int64_t stride) { return aligned_to(p, 4) && stride % 2 == 0; };
  return even(a.x, a.x_stride) && even(a.gate, a.gate_stride) && even(a.h, 0) &&
                 even(a.grad_h, a.grad_h_stride) && even(a.dx, a.dx_stride) &&
                 even(a.dgate, a.dgate_stride)
             ? 2
             : 1;
}

int64_t tiles_of(int64_t tokens, int64_t seqs, bool back) {
  const int w = waves_of(tokens, seqs);
  const int64_t n = w * (back ? back_span(w) : kForwardSpan);
  return (tokens + n - 1) / n;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int64_t groups_of(int64_t tiles) { return (tiles + kGroup - 1) / kGroup; }

// The workspace: marks, pairs and states of tiles and groups.
size_t workspace_bytes_of(int64_t tokens, int64_t seqs, int64_t dim) {
  static_assert(back_span(kFewWaves) <= kForwardSpan && back_span(kManyWaves) <= kForwardSpan,
                "the forward pass has no more tiles");
  const int64_t tiles = tiles_of(tokens, seqs, true);
  const size_t words = static_cast<size_t>((tiles + groups_of(tiles)) * dim);
  return up256(static_cast<size_t>(tokens) * 8) + up256(words * 8) + up256(words * 4);
}

hipError_t launch_scan(ScanArgs a, const tbe_scan_input* in, bool back, void* workspace,
                       hipStream_t s) {
  if (a.tokens <= 1)  // a single row's stride says nothing
    a.x_stride = a.gate_stride = a.grad_h_stride = a.dx_stride = a.dgate_stride = a.dim;
  ScanWork w{};
  w.tiles = tiles_of(a.tokens, a.seqs, back);
  const int v = lane_channels(in, a);
  w.channel_blocks = static_cast<uint32_t>((a.dim + 64 * v - 1) / (64 * v));
  w.rows = w.tiles + groups_of(w.tiles);
  char* p = static_cast<char*>(workspace);
  w.marks = reinterpret_cast<int2*>(p);
  p += up256(static_cast<size_t>(a.tokens) * 8);
  w.tile.pairs = reinterpret_cast<uint64_t*>(p);
  p += up256(static_cast<size_t>(w.rows) * a.dim * 8);
  w.tile.states = reinterpret_cast<uint32_t*>(p);
  w.group.pairs = w.tile.pairs + w.tiles * a.dim;
  w.group.states = w.tile.states + w.tiles * a.dim;
  w.max_polls = in->max_polls == 0  ? kMaxPolls
                : in->max_polls < 0 ? 0u
                                    : static_cast<uint32_t>(in->max_polls);
  const int64_t work = std::max(std::max(w.rows * a.dim, a.tokens), a.seqs);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((work + kBlock - 1) / kBlock, 1024));
  hipLaunchKernelGGL(scan_prepare, dim3(static_cast<unsigned>(blocks)), dim3(kBlock), 0, s, a, w,
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

// A row lies within a buffer descriptor's reach.
constexpr int64_t kMaxRow = int64_t{1} << 23;

// Sizes a call can take: 31-bit tokens and sequences, 2^32 threads in a launch.
tbe_status check_sizes(int64_t tokens, int64_t seqs, int64_t dim, int32_t dtype) {
  constexpr int64_t kMax = 0x7FFFFFFF;
  if (tokens < 0 || seqs < 0 || dim < 1 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  if (seqs == 0 && tokens > 0) return TBE_ERR_INVALID_ARGUMENT;
  if (tokens >= kMax || seqs >= kMax || dim > kMaxRow) return TBE_ERR_UNSUPPORTED;
  // 256 threads for 32 tokens of 64 channels at most, tiles rounded up to 8
  if ((tokens + 511) / 512 * 8 * ((dim + 63) / 64) >= (int64_t{1} << 23))
    return TBE_ERR_UNSUPPORTED;
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
  const size_t need = workspace_bytes_of(in->tokens, in->seqs, in->dim);
  if (need == 0) return TBE_OK;  // no tokens
  if (!workspace || !aligned_to(workspace, 256)) return TBE_ERR_INVALID_ARGUMENT;
  return bytes < need ? TBE_ERR_WORKSPACE_TOO_SMALL : TBE_OK;
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
  *workspace_bytes = seqs > 0 ? workspace_bytes_of(tokens, seqs, dim) : 0;
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
