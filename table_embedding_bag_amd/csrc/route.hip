// route.hip -- the choice of k experts for each row, and its gradient.
//
// Scores are softmax or sigmoid of a row's logits; experts are chosen by score + bias,
// where there are groups first the groups, by their best or their best two; the weights
// are the chosen experts' scores (without the bias), over their sum where renormalised.
//
// The choice is that of exact arithmetic, equal scores going to the lower index.  Without a bias
// scores lie in the order of the logits, so the logits are compared.  A lane sorts its experts'
// keys once, as whole numbers that end in the expert's number, and the row takes the best
// of its lanes' heads k times.  Logits of 16 bits leave room for the whole number, so
// equal ones need nothing more; otherwise keys lose their last 4 bits to it, and
// where two that follow each other lie closer than that and fp32 scores may be off, the
// wave chooses again in 64 bits.
//
// The second look bounds it, where there is one (32768 x 256 bf16, 8 of them in 4 of 8 groups by
// sigmoid + bias: 17 MB, 4 us at a copy's rate): 22 us where no row is in doubt (15 by the logits
// themselves), 43 with biases that differ, where 0.8% of the rows are and a few late waves work on
// alone, and 76 with biases of 0, where equal logits put a third of the rows in doubt.  By the
// logits themselves instructions do: 1000 a wave, vector units busy in 58%.  Backward 11 us for
// 18 MB: the chosen experts' values go through LDS (conflicts in two thirds of its cycles) between
// two barriers.  A row has 16 lanes where that leaves a lane 16 experts at most, so that four rows
// share a wave's steps.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "layers.hpp"
#include "route_keys.hpp"

using namespace tbe;

namespace {

struct RouteArgs {
  const void* logits;
  const float* bias;  // or null
  int32_t* ids;       // [rows][k]
  float* weights;
  const int32_t* ids_in;
  const float* grad;  // [rows][k]
  void* dlogits;
  int64_t stride, out_stride, rows;
  int32_t experts, k;
  int32_t groups, per, top_groups;  // per: experts of a group
  uint32_t inverse;                 // ceil(2^32 / per) (0 for per = 1)
  int32_t sigmoid, top2, renormalize;
  int32_t by_score;                 // chosen by score, not by logit
  float scale;
};

constexpr int kMaxExperts = 1024, kMaxGroups = 16, kMaxChosen = 16;
constexpr float kNegInf = -__builtin_inff();

template <typename T>
constexpr T kDead = static_cast<T>(__builtin_nan(""));  // an expert that cannot be chosen

// The result of op over the L lanes of a row, in each of them.
template <int CTRL>
__device__ __forceinline__ uint32_t move_lanes(uint32_t v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL, typename T>
__device__ __forceinline__ T swap(T v) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, move_lanes<CTRL>(__builtin_bit_cast(uint32_t, v)));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = move_lanes<CTRL>(static_cast<uint32_t>(u));
    const uint64_t hi = move_lanes<CTRL>(static_cast<uint32_t>(u >> 32));
    return __builtin_bit_cast(T, hi << 32 | lo);
  }
}
template <int L, typename T, typename F>
__device__ __forceinline__ T over_row(T v, F op) {
  // Neighbours, pairs, quads and halves of 16 lanes change places, so that both sides of
  // every step add the same two values: all lanes get the same sum to the last bit.
  v = op(v, swap<0xB1>(v));
  v = op(v, swap<0x4E>(v));
  v = op(v, swap<0x141>(v));
  v = op(v, swap<0x140>(v));
  if constexpr (L == 64) {
    v = op(v, __shfl_xor(v, 16));
    v = op(v, __shfl_xor(v, 32));
  }
  return v;
}
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct Min {
  __device__ int operator()(int a, int b) const { return a < b ? a : b; }
};
struct Sum {
  template <typename T>
  __device__ T operator()(T a, T b) const { return a + b; }
};

// Experts of one load: of 16 bytes, or all V of a lane.
template <int ST, int V>
constexpr int kWidth = V < 16 / StorageTraits<ST>::bytes ? V : 16 / StorageTraits<ST>::bytes;
// A lane's experts: V consecutive ones, the row's L lanes in order; ...
template <int L, int V>
struct Layout {
  static __device__ __forceinline__ int expert(int j, int lane) { return lane * V + j; }
};
// ... or, where the whole row is written, loads side by side.
template <int ST, int L, int V>
struct Striped {
  static constexpr int W = kWidth<ST, V>;
  static __device__ __forceinline__ int expert(int j, int lane) { return (j / W) * (L * W) + lane * W + j % W; }
};

// A wave's LDS operations so far are done.
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ float usable(float v) {  // NaN counts as -infinity
  return v >= kNegInf ? fminf(v, 3.402823466e38f) : kNegInf;
}

template <int ST, typename Lay, int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int lane, float (&l)[V]) {
  constexpr int W = kWidth<ST, V>;
#pragma unroll
  for (int j = 0; j < V; j += W) {
    const int e = Lay::expert(j, lane);
    if (e + W <= a.experts) {
      const StoredVec<ST, W> v = load_vec<ST, W>(a.logits, row * a.stride + e);
#pragma unroll
      for (int i = 0; i < W; ++i) l[j + i] = usable(static_cast<float>(v[i]));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        l[j + i] = e + i < a.experts ? usable(load_one<ST>(a.logits, row * a.stride + e + i)) : kNegInf;
    }
  }
}

// The best n of a row's keys (dead ones are NaN), the lowest index among equals: lane t < n
// of the row gets the t-th's index.
template <int L, int V, typename T, typename F>
__device__ __forceinline__ int choose(T (&key)[V], int n, int lane, F index) {
  int mine = 0;
  for (int t = 0; t < n; ++t) {
    T top = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) top = Max()(top, key[j]);
    top = over_row<L>(top, Max());
    int at = 1 << 30;
#pragma unroll
    for (int j = 0; j < V; ++j) at = key[j] == top && index(j) < at ? index(j) : at;
    at = over_row<L>(at, Min());
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = index(j) == at ? kDead<T> : key[j];
    if (lane == t) mine = at;
  }
  return mine;
}

// The lane's experts' biases, 0 past the last.
template <int L, int V>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int lane, float (&bias)[V]) {
  constexpr int W = kWidth<kF32, V>;
#pragma unroll
  for (int j = 0; j < V; j += W) {
    const int e = Layout<L, V>::expert(j, lane);
    if (e + W <= a.experts) {
      const StoredVec<kF32, W> v = load_vec<kF32, W>(a.bias, e);
#pragma unroll
      for (int i = 0; i < W; ++i) bias[j + i] = usable(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) bias[j + i] = e + i < a.experts ? usable(a.bias[e + i]) : 0.0f;
    }
  }
}

// The scores the experts are chosen by, and the largest there can be without the bias.
template <int L, int V>
__device__ __forceinline__ float make_keys(const RouteArgs& a, const float (&l)[V], int lane, float (&key)[V]) {
  float most = 1.0f;
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[j]));
  } else {
    float top = l[0], sum = 0.0f;
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, l[j]);
    top = over_row<L>(top, Max());
    if (top == kNegInf) top = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      key[j] = __expf(l[j] - top);
      sum += key[j];
    }
    sum = over_row<L>(sum, Sum());
    most = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] *= most;
  }
  if (a.bias) {
    float bias[V];
    load_bias<L, V>(a, lane, bias);
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] += bias[j];
  }
  return most;
}

// The score of group `lane` (below a.groups) from the row's keys in LDS.
template <typename T>
__device__ __forceinline__ T score_group(const RouteArgs& a, const T* key, int lane) {
  T one = key[lane * a.per], two = static_cast<T>(-__builtin_inf());
#pragma unroll 4
  for (int i = 1; i < a.per; ++i) {
    const T x = key[lane * a.per + i];
    two = Max()(two, x < one ? x : one);
    one = Max()(one, x);
  }
  return a.top2 ? one + two : one;
}

template <int L, int V>
__device__ __forceinline__ void find_groups(const RouteArgs& a, int lane, int (&group)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = Layout<L, V>::expert(j, lane);
    group[j] = a.inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(e), a.inverse)) : e;
    if (e >= a.experts) group[j] = -1;
  }
}

__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t x = a, y = b;
  a = x > y ? x : y;
  b = x > y ? y : x;
}

// The best first (Batcher's merge exchange).
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&s)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) exchange(s[i + j], s[i + j + k]);
}

// Whether groups are whole lanes, a power of two of them.
template <int V>
__device__ __forceinline__ bool groups_of_lanes(const RouteArgs& a) {
  return a.per % V == 0 && (a.per / V & (a.per / V - 1)) == 0;
}
// The best two of 2^shift neighbouring lanes' best two.
template <int L, typename T>
__device__ __forceinline__ void best_two(T& one, T& two, int shift) {
  const auto join = [&](T o1, T o2) {
    const T least = one < o1 ? one : o1;
    two = Max()(least, Max()(two, o2));
    one = Max()(one, o1);
  };
  if (shift > 0) join(swap<0xB1>(one), swap<0xB1>(two));
  if (shift > 1) join(swap<0x4E>(one), swap<0x4E>(two));
  if (shift > 2) join(swap<0x141>(one), swap<0x141>(two));
  if (shift > 3) join(swap<0x140>(one), swap<0x140>(two));
  if (L == 64 && shift > 4) join(__shfl_xor(one, 16), __shfl_xor(two, 16));
  if (L == 64 && shift > 5) join(__shfl_xor(one, 32), __shfl_xor(two, 32));
}

// The choice of a row in 64 bits; lane t < k gets the t-th expert.  key: the row's experts in
// LDS.  Few rows come here, and those wait for what is not in the instruction cache: loops
// with short bodies (unrolled whole it took 100 us), whose reads are in flight together.
template <int L, int V>
__device__ int choose_exactly(const RouteArgs& a, const float (&l)[V], int lane, double* key) {
  // a logit and its bias lie where the key will
  float2* const pair = reinterpret_cast<float2*>(key);
  float bias[V] = {};
  if (a.bias) load_bias<L, V>(a, lane, bias);
#pragma unroll
  for (int j = 0; j < V; ++j) pair[Layout<L, V>::expert(j, lane)] = make_float2(l[j], bias[j]);
  lds_done();
  constexpr int kEach = V < 4 ? V : 4;  // experts at a time
  const auto over_experts = [&](auto f) {  // lane's are lane, lane + L, ...
#pragma unroll 1
    for (int j = 0; j < V; j += kEach)
#pragma unroll
      for (int i = 0; i < kEach; ++i) f((j + i) * L + lane, (j + i) * L + lane < a.experts);
  };
  if (a.by_score) {
    double top = 0.0, sum = 1.0;
    if (!a.sigmoid) {
      float most = kNegInf;
      over_experts([&](int e, bool is) { most = fmaxf(most, is ? pair[e].x : kNegInf); });
      most = over_row<L>(most, Max());
      top = most == kNegInf ? 0.0 : static_cast<double>(most);
      sum = 0.0;
      over_experts([&](int e, bool is) { sum += is ? exp(static_cast<double>(pair[e].x) - top) : 0.0; });
      sum = over_row<L>(sum, Sum());
      if (sum == 0.0) sum = 1.0;
    }
    over_experts([&](int e, bool) {
      const float2 p = pair[e];
      const double v = p.x, x = exp(a.sigmoid ? -v : v - top);
      key[e] = (a.sigmoid ? 1.0 / (1.0 + x) : x / sum) + static_cast<double>(p.y);
    });
  } else {
    over_experts([&](int e, bool) { key[e] = pair[e].x; });
  }
  lds_done();
  if (a.groups > 1) {
    double best[1] = {kDead<double>};
    if (lane < a.groups) best[0] = score_group<double>(a, key, lane);
    const int mine = choose<L, 1, double>(best, a.top_groups, lane, [&](int) { return lane; });
    const int bits = over_row<L>(lane < a.top_groups ? 1 << (mine & 31) : 0, [](int x, int y) { return x | y; });
    over_experts([&](int e, bool) {
      if (!(bits >> (a.inverse ? __umulhi(static_cast<uint32_t>(e), a.inverse) : e) & 1)) key[e] = kDead<double>;
    });
    lds_done();
  }
  int mine = 0;
#pragma unroll 1
  for (int t = 0; t < a.k; ++t) {
    double best = kDead<double>;
    int at = 1 << 30;
    over_experts([&](int e, bool is) {
      const double x = is ? key[e] : kDead<double>;
      if (x > best || (x == x && best != best)) best = x, at = e;
    });
    const double top = over_row<L>(best, Max());
    at = over_row<L>(best == top ? at : 1 << 30, Min());
    if (lane == t) mine = at;
    if (at < a.experts && at % L == lane) key[at] = kDead<double>;
    lds_done();
  }
  return mine < a.experts ? mine : 0;
}

// Keys as whole numbers in the same order, their last `bits` bits an expert's number
// counted down; 0 for an expert that cannot be chosen.
__device__ __forceinline__ uint32_t in_order(float f) { return key_of_float(__float_as_uint(f + 0.0f)); }  // no -0
__device__ __forceinline__ float value_of(uint32_t key, uint32_t bits) {
  return __uint_as_float(float_of_key(key, bits));
}
struct MaxKey {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// Whether two keys that follow each other, off by 2^-19 of their size (which is at most
// `size` for both together) where they end in a number, may lie less than room apart.
__device__ __forceinline__ bool too_close(float before, float after, float size, float room) {
  if (after == kNegInf) return before == kNegInf;
  return !(before - after - 3.814697265625e-6f * size > room);
}

// The row's choice by fp32 keys; lane t < k gets the t-th expert.  close: two that follow each
// other, the first one that was not chosen among them, may have changed places, as their
// difference is off by up to room.  NUMBER: keys end in the whole number, and are exact.
// shared: the row's LDS.
template <int L, int V, bool NUMBER>
__device__ __forceinline__ int choose_experts(const RouteArgs& a, const float (&key)[V], int lane, float room,
                                              float* shared, bool* close) {
  constexpr uint32_t kBits = NUMBER ? kMaxExperts - 1 : 15;
  uint32_t s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = Layout<L, V>::expert(j, lane);
    s[j] = e < a.experts ? (in_order(key[j]) & ~kBits) | (kBits - (NUMBER ? e : j)) : 0u;
  }
  const int first_lane = L == 64 ? 0 : lane_id() & 48;
  // The lane whose head is the row's best, the lowest of several.  There always is one: open
  // groups and experts of theirs are as many as are taken, at least, and -infinity counts too.
  const auto best_lane = [&](bool is) {
    const uint64_t all = __ballot(is) >> first_lane;
    return __builtin_ctzll(L == 64 ? all | 1ull << 63 : (all & 0xFFFFu) | 0x8000u);  // always one of them
  };
  bool doubt = false;
  if (a.groups > 1) {
    const bool whole = groups_of_lanes<V>(a);
    const int shift = whole ? __builtin_ctz(a.per / V) : 0;
    float score, size = -1.0f;  // of the lane's group, or of group `lane`
    if (whole) sort_down<V>(s);
    if (whole) {
      float one = value_of(s[0], kBits), two = V > 1 ? value_of(s[V > 1 ? 1 : 0], kBits) : -__builtin_inff();
      best_two<L>(one, two, shift);
      score = a.top2 ? one + two : one;
      // (-infinity is off by nothing)
      const auto size_of = [](float v) { return v > kNegInf ? fabsf(v) : 0.0f; };
      size = over_row<L>(lane >> shift < a.groups ? size_of(one) + (a.top2 ? size_of(two) : 0.0f) : 0.0f, Max());
      // one lane for each group
      if (lane >> shift >= a.groups || lane & ((1 << shift) - 1)) score = kDead<float>;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) shared[Layout<L, V>::expert(j, lane)] = key[j];
      lds_done();
      score = lane < a.groups ? score_group<float>(a, shared, lane) : kDead<float>;
    }
    int bits = 0;
    float before = 0.0f;
    for (int t = 0;; ++t) {
      const float top = over_row<L>(score, Max());
      // sums of two are twice as far off
      if (t > 0 && !NUMBER)
        doubt = doubt || too_close(before, top, size < 0.0f ? fabsf(before) + fabsf(top) : 2.0f * size, 2.0f * room);
      if (t == a.top_groups) break;
      const int at = best_lane(score == top);
      if (lane == at) score = kDead<float>;
      bits |= 1 << (at >> shift);
      before = top;
    }
    if (whole) {
      const int mine = lane >> shift;
      if (mine >= a.groups || !(bits >> mine & 1))
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0u;
    } else {
      int group[V];
      find_groups<L, V>(a, lane, group);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (group[j] < 0 || !(bits >> group[j] & 1)) s[j] = 0u;
      sort_down<V>(s);
    }
  } else {
    sort_down<V>(s);
  }
  int mine = 0;
  uint32_t before = 0;
  for (int t = 0;; ++t) {
    if (NUMBER && t == a.k) break;
    const uint32_t top = over_row<L>(s[0], MaxKey());
    if (!NUMBER && t > 0 && top != 0u) {
      const float x = value_of(before, kBits), y = value_of(top, kBits);
      doubt = doubt || too_close(x, y, fabsf(x) + fabsf(y), room);
    }
    if (t == a.k) break;
    bool out = s[0] == top;
    int id;
    if constexpr (NUMBER) {
      id = kBits - (top & kBits);
    } else {
      const int at = best_lane(out);
      id = at * V + 15 - (top & 15u);
      out = lane == at;
    }
    if (lane == t) mine = id;
#pragma unroll
    for (int j = 1; j < V; ++j) s[j - 1] = out ? s[j] : s[j - 1];
    s[V - 1] = out ? 0u : s[V - 1];
    before = top;
  }
  *close = doubt;
  return mine;
}

// Scores' exponentials relative to the row's chosen (or all) experts, and what they add up to:
// the weights of the chosen before `scale`.
struct Weights {
  float share;  // over the chosen experts' sum
  float score;  // itself
};
// l: of lane t < k the chosen expert's logit, else -infinity; all: largest logit and the sum
// of exponentials relative to it over all experts (softmax that is not renormalised).
template <int L>
__device__ __forceinline__ Weights weigh(const RouteArgs& a, float l, float all_top, float all_sum) {
  const float top = over_row<L>(l, Max());
  float e;
  // sigmoid's numerator and denominator, both times the same power: large negative logits
  // keep their ratio
  if (a.sigmoid) e = l == kNegInf ? 0.0f : expf(fminf(l, 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(l)));
  else e = l == kNegInf ? 0.0f : expf(l - top);
  Weights w{0.0f, 0.0f};
  const float sum = over_row<L>(e, Sum());
  if (sum > 0.0f) w.share = e / sum;
  if (a.sigmoid) w.score = l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l) / (1.0f + expf(l));
  else if (all_sum > 0.0f) w.score = expf(l - all_top) / all_sum;
  return w;
}

// The largest of a row's logits, and the sum of exponentials relative to it.
template <int L, int V>
__device__ __forceinline__ float2 sum_all(const float (&l)[V]) {
  float top = l[0], sum = 0.0f;
#pragma unroll
  for (int j = 1; j < V; ++j) top = fmaxf(top, l[j]);
  top = over_row<L>(top, Max());
  if (top == kNegInf) return make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < V; ++j) sum += expf(l[j] - top);
  return make_float2(top, over_row<L>(sum, Sum()));
}

template <int L>
constexpr int kRowsOfBlock = kBlock / L;

template <int ST, int L, int V, bool BY_SCORE>
__global__ __launch_bounds__(kBlock) void route_forward(RouteArgs a) {
  const int lane = threadIdx.x % L, r = threadIdx.x / L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsOfBlock<L> + r;
  const int64_t from = row < a.rows ? row : a.rows - 1;  // all lanes take part to the end
  __shared__ double exact[kRowsOfBlock<L>][L * V];
  float* const shared = reinterpret_cast<float*>(exact[r]);
  float l[V];
  load_logits<ST, Layout<L, V>, V>(a, from, lane, l);
  int mine;
  bool close = false;
  if constexpr (BY_SCORE) {
    // What fp32 scores may be off by: sums of 1024 terms in a tree and exponentials, 2^-19
    // of the largest score; a sigmoid 2^-22; twice that for a difference, and room.
    float key[V];
    const float most = make_keys<L, V>(a, l, lane, key);
    mine = choose_experts<L, V, false>(a, key, lane, a.sigmoid ? 0x1p-19f : most * 0x1p-16f, shared, &close);
  } else {
    mine = choose_experts<L, V, ST != kF32>(a, l, lane, 0.0f, shared, &close);
  }
  if (__any(close)) {
    const int other = choose_exactly<L, V>(a, l, lane, exact[r]);
    if (close) mine = other;
  }
  float2 all = make_float2(0.0f, 0.0f);
  if (!a.sigmoid && !a.renormalize) all = sum_all<L, V>(l);
  const float chosen = lane < a.k ? usable(load_one<ST>(a.logits, from * a.stride + mine)) : kNegInf;
  const Weights w = weigh<L>(a, chosen, all.x, all.y);
  if (lane < a.k && row < a.rows) {
    a.ids[row * a.k + lane] = mine;
    a.weights[row * a.k + lane] = a.scale * (a.renormalize ? w.share : w.score);
  }
}

// The gradient of the weights: of the chosen experts' logits, through the sum of all where
// softmax's scores are not renormalised.
template <int ST, int L, int V>
__global__ __launch_bounds__(kBlock) void route_backward(RouteArgs a) {
  using Lay = Striped<ST, L, V>;
  constexpr int W = Lay::W;
  __shared__ float shared[kRowsOfBlock<L>][L * V];
  const int lane = threadIdx.x % L, r = threadIdx.x / L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsOfBlock<L> + r;
  const int64_t from = row < a.rows ? row : a.rows - 1;
  const bool through = !a.sigmoid && !a.renormalize;
  float l[V];
  float2 all = make_float2(0.0f, 0.0f);
  if (through) {
    load_logits<ST, Lay, V>(a, from, lane, l);
    all = sum_all<L, V>(l);
  }
  int id = -1;
  float g = 0.0f;
  if (lane < a.k) {
    id = a.ids_in[from * a.k + lane];
    g = a.grad[from * a.k + lane] * a.scale;
    if (id < 0 || id >= a.experts) id = -1, g = 0.0f;
  }
  const float chosen = id >= 0 ? usable(load_one<ST>(a.logits, from * a.stride + id)) : kNegInf;
  const Weights w = weigh<L>(a, chosen, all.x, all.y);
  float d, sum = 0.0f;
  if (a.renormalize) {
    // an expert without weight passes nothing back, whatever its gradient holds
    const float mean = over_row<L>(w.share > 0.0f ? w.share * g : 0.0f, Sum());
    d = w.share > 0.0f ? w.share * (g - mean) : 0.0f;
    if (a.sigmoid) d *= 1.0f / (1.0f + expf(chosen));
  } else {
    d = w.score > 0.0f ? w.score * g : 0.0f;
    if (a.sigmoid) d *= 1.0f / (1.0f + expf(chosen));
    else sum = over_row<L>(d, Sum());
  }
#pragma unroll
  for (int j = 0; j < V; ++j) shared[r][Lay::expert(j, lane)] = 0.0f;
  __syncthreads();
  // an expert that was given twice gets both: by the first of its lanes
  float total = 0.0f;
  bool first = id >= 0;
  for (int t = 0; t < a.k; ++t) {
    const int other = __shfl(id, t, L);
    const float v = __shfl(d, t, L);
    if (other == id) {
      total += v;
      first = first && t >= lane;
    }
  }
  if (first) shared[r][id] = total;
  __syncthreads();
  if (row >= a.rows) return;
#pragma unroll
  for (int j = 0; j < V; j += W) {
    const int e = Lay::expert(j, lane);
    float out[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      out[i] = shared[r][e + i];
      if (through && all.y > 0.0f) out[i] -= expf(l[j + i] - all.x) / all.y * sum;
    }
    if (e + W <= a.experts) {
      StoredVec<ST, W> v;
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = static_cast<typename Stored<ST>::type>(out[i]);
      store_vec<ST, W>(a.dlogits, row * a.out_stride + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (e + i < a.experts) store_one<ST>(a.dlogits, row * a.out_stride + e + i, out[i]);
    }
  }
}

template <int ST, int L, int V>
hipError_t launch_shape(const RouteArgs& a, bool backward, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.rows + kRowsOfBlock<L> - 1) / kRowsOfBlock<L>));
  if (backward) hipLaunchKernelGGL((route_backward<ST, L, V>), grid, dim3(kBlock), 0, s, a);
  else if (a.by_score) hipLaunchKernelGGL((route_forward<ST, L, V, true>), grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL((route_forward<ST, L, V, false>), grid, dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

// 16 lanes a row, four rows a wave, up to 256 experts, else a wave.
template <int ST>
hipError_t launch_route(const RouteArgs& a, bool backward, hipStream_t s) {
  return a.experts <= 16    ? launch_shape<ST, 16, 1>(a, backward, s)
         : a.experts <= 32  ? launch_shape<ST, 16, 2>(a, backward, s)
         : a.experts <= 64  ? launch_shape<ST, 16, 4>(a, backward, s)
         : a.experts <= 128 ? launch_shape<ST, 16, 8>(a, backward, s)
         : a.experts <= 256 ? launch_shape<ST, 16, 16>(a, backward, s)
                            : launch_shape<ST, 64, 16>(a, backward, s);
}

hipError_t launch(const RouteArgs& a, int32_t dtype, bool backward, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == TBE_F32   ? launch_route<kF32>(a, backward, s)
         : dtype == TBE_F16 ? launch_route<kF16>(a, backward, s)
                            : launch_route<kBF16>(a, backward, s);
}

tbe_status check(RouteArgs* a, const void* logits, int64_t stride, int64_t rows, int64_t experts, int64_t k,
                 int32_t dtype, int32_t scores, double scale) {
  if (rows < 0 || experts < 1 || k < 1 || k > experts || !known_dtype(dtype) ||
      (scores != TBE_SCORES_SOFTMAX && scores != TBE_SCORES_SIGMOID) || !std::isfinite(scale) ||
      !std::isfinite(static_cast<float>(scale)))
    return TBE_ERR_INVALID_ARGUMENT;
  if (experts > kMaxExperts || k > kMaxChosen || rows > (int64_t{1} << 25)) return TBE_ERR_UNSUPPORTED;
  if (rows > 0 && (!logits || !aligned_to(logits, dtype_bytes(dtype)))) return TBE_ERR_INVALID_ARGUMENT;
  if (rows > 1 && stride < 0) return TBE_ERR_INVALID_ARGUMENT;
  a->logits = logits;
  a->stride = stride;
  a->rows = rows;
  a->experts = static_cast<int32_t>(experts);
  a->k = static_cast<int32_t>(k);
  a->sigmoid = scores == TBE_SCORES_SIGMOID;
  a->scale = static_cast<float>(scale);
  return TBE_OK;
}

}  // namespace

extern "C" {

tbe_status tbe_route(const void* logits, int64_t logits_stride, const float* bias, int32_t* ids,
                     float* weights, int64_t rows, int64_t experts, int64_t k, int64_t groups,
                     int64_t top_groups, int32_t dtype, int32_t scores, int32_t group_score,
                     int32_t renormalize, double scale, void* stream) {
  RouteArgs a{};
  const tbe_status st = check(&a, logits, logits_stride, rows, experts, k, dtype, scores, scale);
  if (st != TBE_OK) return st;
  if (groups < 1 || groups > experts || experts % groups || top_groups < 1 || top_groups > groups ||
      k > experts / groups * top_groups ||
      (group_score != TBE_GROUP_BEST && group_score != TBE_GROUP_BEST_TWO) || !aligned_to(bias, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  if (groups > kMaxGroups) return TBE_ERR_UNSUPPORTED;
  if (rows == 0) return TBE_OK;
  if (!ids || !weights || !aligned_to(ids, 4) || !aligned_to(weights, 4)) return TBE_ERR_INVALID_ARGUMENT;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  if (groups > top_groups) {  // else every group is in
    a.groups = static_cast<int32_t>(groups);
    a.top_groups = static_cast<int32_t>(top_groups);
    a.per = static_cast<int32_t>(experts / groups);
    a.inverse = a.per == 1 ? 0u : static_cast<uint32_t>((uint64_t{1} << 32) / a.per + 1);
    a.top2 = group_score == TBE_GROUP_BEST_TWO && a.per > 1;
  }
  a.by_score = bias || a.top2;
  a.renormalize = renormalize != 0;
  return launch(a, dtype, false, stream) == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

tbe_status tbe_route_backward(const void* logits, int64_t logits_stride, const int32_t* ids,
                              const float* grad, void* dlogits, int64_t dlogits_stride, int64_t rows,
                              int64_t experts, int64_t k, int32_t dtype, int32_t scores,
                              int32_t renormalize, double scale, void* stream) {
  RouteArgs a{};
  const tbe_status st = check(&a, logits, logits_stride, rows, experts, k, dtype, scores, scale);
  if (st != TBE_OK || rows == 0) return st;
  if (!ids || !grad || !dlogits || !aligned_to(ids, 4) || !aligned_to(grad, 4) ||
      !aligned_to(dlogits, dtype_bytes(dtype)) || (rows > 1 && dlogits_stride < experts))
    return TBE_ERR_INVALID_ARGUMENT;
  a.ids_in = ids;
  a.grad = grad;
  a.dlogits = dlogits;
  a.out_stride = dlogits_stride;
  a.renormalize = renormalize != 0;
  return launch(a, dtype, true, stream) == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

}  // extern "C"
