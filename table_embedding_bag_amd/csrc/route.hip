// route.hip -- the choice of k experts for each row, and its gradient.
//
// Scores are softmax or sigmoid of a row's logits; experts are chosen by score + bias,
// where there are groups first the groups, by their best or their best two; the weights
// are the chosen experts' scores (without the bias), over their sum where renormalised.
//
// The choice is that of exact arithmetic, equal scores going to the lower index.  Without a bias
// scores lie in the order of the logits, so the logits are compared.  Otherwise scores are
// compared in fp32, and where two that follow each other lie closer than fp32 may be off,
// the wave does the same again in 64 bits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "layers.hpp"

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
template <typename T>
__device__ __forceinline__ T Abs(T v) {
  return v < 0 ? -v : v;
}
struct Min {
  __device__ int operator()(int a, int b) const { return a < b ? a : b; }
};
struct Sum {
  template <typename T>
  __device__ T operator()(T a, T b) const { return a + b; }
};

// A lane's experts: V of them in vectors of W, the row's L lanes side by side.
template <int L, int V>
struct Layout {
  static constexpr int W = V < 4 ? V : 4;
  static __device__ __forceinline__ int expert(int j, int lane) {
    return (j / W) * (L * W) + lane * W + j % W;
  }
};

__device__ __forceinline__ float usable(float v) {  // NaN counts as -infinity
  return v >= kNegInf ? fminf(v, 3.402823466e38f) : kNegInf;
}

template <int ST, int L, int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int lane, float (&l)[V]) {
  using Lay = Layout<L, V>;
  constexpr int W = Lay::W;
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
// of the row gets the t-th's index.  gap: the least difference of two that follow each other,
// the first one that was not chosen among them, less 2^-22 of their sizes.
template <int L, int V, typename T, typename F>
__device__ __forceinline__ int choose(T (&key)[V], int n, int lane, F index, T* gap) {
  int mine = 0;
  T before = 0, least = static_cast<T>(__builtin_inf());
  for (int t = 0;; ++t) {
    if (t == n && !gap) break;
    T top = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) top = Max()(top, key[j]);
    top = over_row<L>(top, Max());
    if (gap && t > 0) {
      const T room = before - top - static_cast<T>(2.384185791015625e-7) * (Abs(before) + Abs(top));
      least = room < least ? room : least;  // NaN (none left): no
    }
    if (t == n) break;
    int at = 1 << 30;
#pragma unroll
    for (int j = 0; j < V; ++j) at = key[j] == top && index(j) < at ? index(j) : at;
    at = over_row<L>(at, Min());
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = index(j) == at ? kDead<T> : key[j];
    if (lane == t) mine = at;
    before = top;
  }
  if (gap) *gap = least;
  return mine;
}

// The keys the experts are chosen by, in T.
template <int L, int V, typename T>
__device__ __forceinline__ T make_keys(const RouteArgs& a, const float (&l)[V], int lane, T (&key)[V]) {
  using Lay = Layout<L, V>;
  T most = 1;  // largest score
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (sizeof(T) == 8) key[j] = 1.0 / (1.0 + exp(-static_cast<double>(l[j])));
      else key[j] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[j]));
    }
  } else {
    float top = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, l[j]);
    top = over_row<L>(top, Max());
    if (top == kNegInf) top = 0.0f;
    T sum = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (sizeof(T) == 8) key[j] = exp(static_cast<double>(l[j]) - static_cast<double>(top));
      else key[j] = __expf(l[j] - top);
      sum += key[j];
    }
    sum = over_row<L>(sum, Sum());
    most = sum > 0 ? 1 / sum : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] *= most;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = Lay::expert(j, lane);
    if (e >= a.experts) key[j] = kDead<T>;
    else if (a.bias) key[j] += static_cast<T>(a.bias[e]);
  }
  return most;
}

// The row's choice by its keys; lane t < k gets the t-th expert.
template <int L, int V, typename T>
__device__ __forceinline__ int choose_experts(const RouteArgs& a, T (&key)[V], int lane, T* shared, T* gap) {
  using Lay = Layout<L, V>;
  T gap_groups = static_cast<T>(__builtin_inf());
  if (a.groups > 1) {
    // Expert e of group q lies at e + q of the row's keys in LDS, so that lanes that go
    // through a group each read different banks.
    int group[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = Lay::expert(j, lane);
      group[j] = a.inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(e), a.inverse)) : e;
      if (e < a.experts) shared[e + group[j]] = key[j];
    }
    __syncthreads();
    T best[1] = {kDead<T>};
    if (lane < a.groups) {
      const T* from = shared + lane * (a.per + 1);
      T one = from[0], two = static_cast<T>(-__builtin_inf());
      for (int i = 1; i < a.per; ++i) {
        const T x = from[i];
        two = Max()(two, x < one ? x : one);
        one = Max()(one, x);
      }
      best[0] = a.top2 ? one + two : one;
    }
    const int mine = choose<L, 1, T>(best, a.top_groups, lane, [&](int) { return lane; },
                                     gap ? &gap_groups : nullptr);
    const int bits = over_row<L>(lane < a.top_groups ? 1 << mine : 0, [](int x, int y) { return x | y; });
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (!(bits >> group[j] & 1)) key[j] = kDead<T>;
    __syncthreads();
  }
  const int mine = choose<L, V, T>(key, a.k, lane, [&](int j) { return Lay::expert(j, lane); }, gap);
  if (gap && gap_groups < *gap) *gap = gap_groups;
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
// Keys of a row in LDS: one more for each group.
template <int L, int V>
constexpr int kSharedKeys = L * V + kMaxGroups;

template <int ST, int L, int V>
__global__ __launch_bounds__(kBlock) void route_forward(RouteArgs a) {
  __shared__ double shared[kRowsOfBlock<L>][kSharedKeys<L, V>];
  const int lane = threadIdx.x % L, r = threadIdx.x / L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsOfBlock<L> + r;
  const int64_t from = row < a.rows ? row : a.rows - 1;  // all lanes take part to the end
  float l[V], key[V];
  load_logits<ST, L, V>(a, from, lane, l);
  float* const fast = reinterpret_cast<float*>(shared[r]);
  int mine;
  if (a.bias || a.top2) {
    float gap;
    const float most = make_keys<L, V, float>(a, l, lane, key);
    mine = choose_experts<L, V, float>(a, key, lane, fast, &gap);
    // What fp32 may be off by: sums of 1024 terms in a tree and exponentials, 2^-19 of the
    // largest score; a sigmoid 2^-22; twice that for a difference, again for sums of two.
    const float room = a.sigmoid ? 1.9073486328125e-6f : most * 1.52587890625e-5f;
    const bool close = !(gap > room);
    if (__syncthreads_or(close)) {
      double exact[V];
      make_keys<L, V, double>(a, l, lane, exact);
      const int other = choose_experts<L, V, double>(a, exact, lane, shared[r], nullptr);
      if (close) mine = other;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = Layout<L, V>::expert(j, lane) < a.experts ? l[j] : kDead<float>;
    mine = choose_experts<L, V, float>(a, key, lane, fast, nullptr);
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
  using Lay = Layout<L, V>;
  __shared__ float shared[kRowsOfBlock<L>][L * V];
  const int lane = threadIdx.x % L, r = threadIdx.x / L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsOfBlock<L> + r;
  const int64_t from = row < a.rows ? row : a.rows - 1;
  const bool through = !a.sigmoid && !a.renormalize;
  float l[V];
  float2 all = make_float2(0.0f, 0.0f);
  if (through) {
    load_logits<ST, L, V>(a, from, lane, l);
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
  for (int j = 0; j < V; j += Lay::W) {
    const int e = Lay::expert(j, lane);
    float out[Lay::W];
#pragma unroll
    for (int i = 0; i < Lay::W; ++i) {
      out[i] = shared[r][e + i];
      if (through && all.y > 0.0f) out[i] -= expf(l[j + i] - all.x) / all.y * sum;
    }
    if (e + Lay::W <= a.experts) {
      StoredVec<ST, Lay::W> v;
#pragma unroll
      for (int i = 0; i < Lay::W; ++i) v[i] = static_cast<typename Stored<ST>::type>(out[i]);
      store_vec<ST, Lay::W>(a.dlogits, row * a.out_stride + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < Lay::W; ++i)
        if (e + i < a.experts) store_one<ST>(a.dlogits, row * a.out_stride + e + i, out[i]);
    }
  }
}

template <int ST, int L, int V>
hipError_t launch_shape(const RouteArgs& a, bool backward, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.rows + kRowsOfBlock<L> - 1) / kRowsOfBlock<L>));
  if (backward) hipLaunchKernelGGL((route_backward<ST, L, V>), grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL((route_forward<ST, L, V>), grid, dim3(kBlock), 0, s, a);
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
