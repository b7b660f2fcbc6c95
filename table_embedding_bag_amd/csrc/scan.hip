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

#include "layers.hpp"

using namespace tbe;

namespace {

struct Gates {
  float a, b;
};

// sigmoid(g) and sigmoid(-g) from one exponential of -|g|: neither overflows
// nor loses the smaller one to cancellation.
template <bool SIGMOID>
__device__ __forceinline__ Gates gates(float g) {
  if constexpr (!SIGMOID) return {g, 1.0f};
  const float z = expf(-fabsf(g));
  const float hi = 1.0f / (1.0f + z), lo = z / (1.0f + z);
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

template <typename IT>
__device__ __forceinline__ int64_t offset_at(const ScanArgs& a, int64_t s) {
  const int64_t o = static_cast<const IT*>(a.offsets)[s];
  return o < 0 ? 0 : (o > a.tokens ? a.tokens : o);
}

// A thread walks one channel of one sequence.
template <int ST, bool SIGMOID, typename IT>
__global__ __launch_bounds__(kBlock) void scan_walk(ScanArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t s = i / a.dim, c = i - s * a.dim;
  if (s >= a.seqs) return;
  const int64_t lo = offset_at<IT>(a, s), hi = offset_at<IT>(a, s + 1);
  float v = a.initial ? a.initial[s * a.initial_stride + c] : 0.0f;
  for (int64_t t = lo; t < hi; ++t) {
    if (a.carry) a.carry[t * a.dim + c] = v;
    const Gates k = gates<SIGMOID>(load_one<ST>(a.gate, t * a.gate_stride + c));
    v = k.a * v + k.b * load_one<ST>(a.x, t * a.x_stride + c);
    store_one<ST>(a.h, t * a.dim + c, v);
  }
  a.final[s * a.dim + c] = v;
}

template <int ST, bool SIGMOID, typename IT>
__global__ __launch_bounds__(kBlock) void scan_walk_back(ScanArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t s = i / a.dim, c = i - s * a.dim;
  if (s >= a.seqs) return;
  const int64_t lo = offset_at<IT>(a, s), hi = offset_at<IT>(a, s + 1);
  float mu = a.grad_final ? a.grad_final[s * a.grad_final_stride + c] : 0.0f;
  for (int64_t t = hi - 1; t >= lo; --t) {
    const Gates k = gates<SIGMOID>(load_one<ST>(a.gate, t * a.gate_stride + c));
    const float before = a.carried[t * a.dim + c];
    const float lam = (a.grad_h ? load_one<ST>(a.grad_h, t * a.grad_h_stride + c) : 0.0f) + mu;
    store_one<ST>(a.dx, t * a.dx_stride + c, k.b * lam);
    float dg = lam * before;
    if constexpr (SIGMOID)
      dg = lam * (before - load_one<ST>(a.x, t * a.x_stride + c)) * (k.a * k.b);
    store_one<ST>(a.dgate, t * a.dgate_stride + c, dg);
    mu = k.a * lam;
  }
  if (a.dinitial) a.dinitial[s * a.dim + c] = mu;
}

template <int ST, bool SIGMOID, typename IT>
hipError_t launch_scan(const ScanArgs& a, bool back, hipStream_t s) {
  const int64_t blocks = (a.seqs * a.dim + kBlock - 1) / kBlock;
  if (back)
    hipLaunchKernelGGL((scan_walk_back<ST, SIGMOID, IT>), dim3(static_cast<unsigned>(blocks)),
                       dim3(kBlock), 0, s, a);
  else
    hipLaunchKernelGGL((scan_walk<ST, SIGMOID, IT>), dim3(static_cast<unsigned>(blocks)),
                       dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int ST>
hipError_t launch_scan(const ScanArgs& a, int32_t kind, int32_t index, bool back, hipStream_t s) {
  if (kind == TBE_GATE_SIGMOID)
    return index == TBE_I64 ? launch_scan<ST, true, int64_t>(a, back, s)
                            : launch_scan<ST, true, int32_t>(a, back, s);
  return index == TBE_I64 ? launch_scan<ST, false, int64_t>(a, back, s)
                          : launch_scan<ST, false, int32_t>(a, back, s);
}

hipError_t launch_scan(const ScanArgs& a, const tbe_scan_input* in, bool back, hipStream_t s) {
  return in->dtype == TBE_F32   ? launch_scan<kF32>(a, in->gate_kind, in->index_dtype, back, s)
         : in->dtype == TBE_F16 ? launch_scan<kF16>(a, in->gate_kind, in->index_dtype, back, s)
                                : launch_scan<kBF16>(a, in->gate_kind, in->index_dtype, back, s);
}

constexpr int64_t kMaxElements = int64_t{1} << 38;

// Sizes a call can take: 31-bit tokens, sequences and channels.
tbe_status check_sizes(int64_t tokens, int64_t seqs, int64_t dim, int32_t dtype) {
  if (tokens < 0 || seqs < 0 || dim < 1 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  if (seqs == 0 && tokens > 0) return TBE_ERR_INVALID_ARGUMENT;
  if (tokens >= 0x7FFFFFFF || seqs >= 0x7FFFFFFF || dim >= 0x7FFFFFFF) return TBE_ERR_UNSUPPORTED;
  if (tokens > kMaxElements / dim || seqs > kMaxElements / dim) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

size_t carry_bytes_of(int64_t tokens, int64_t dim) {
  return static_cast<size_t>(tokens) * static_cast<size_t>(dim) * sizeof(float);
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
  if (in->x_stride < 0 || in->gate_stride < 0 || in->initial_stride < 0 ||
      !aligned_to(in->initial, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  return TBE_OK;
}

ScanArgs scan_args(const tbe_scan_input* in) {
  ScanArgs a{};
  a.tokens = in->tokens;
  a.seqs = in->seqs;
  a.dim = in->dim;
  a.x = in->x;
  a.gate = in->gate;
  a.offsets = in->offsets;
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
  *workspace_bytes = 0;
  return TBE_OK;
}

tbe_status tbe_scan_forward(const tbe_scan_input* in, void* h, float* final, float* carry,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const tbe_status st = check_input(in);
  if (st != TBE_OK) return st;
  if (in->seqs == 0) return TBE_OK;
  if (!final || !aligned_to(final, 4) || !aligned_to(carry, 16) ||
      (in->tokens > 0 && (!h || !aligned_to(h, dtype_bytes(in->dtype)))))
    return TBE_ERR_INVALID_ARGUMENT;
  ScanArgs a = scan_args(in);
  a.h = h;
  a.final = final;
  a.carry = carry;
  return launch_scan(a, in, false, static_cast<hipStream_t>(stream)) == hipSuccess ? TBE_OK
                                                                                   : TBE_ERR_HIP;
}

tbe_status tbe_scan_backward(const tbe_scan_input* in, const float* carry, const void* grad_h,
                             int64_t grad_h_stride, const float* grad_final,
                             int64_t grad_final_stride, void* dx, int64_t dx_stride, void* dgate,
                             int64_t dgate_stride, float* dinitial, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const tbe_status st = check_input(in);
  if (st != TBE_OK) return st;
  if (in->seqs == 0) return TBE_OK;
  const size_t e = dtype_bytes(in->dtype);
  if (grad_h_stride < 0 || grad_final_stride < 0 || !aligned_to(grad_h, e) ||
      !aligned_to(grad_final, 4) || !aligned_to(dinitial, 4))
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 0 && (!carry || !aligned_to(carry, 16) || !dx || !dgate || !aligned_to(dx, e) ||
                         !aligned_to(dgate, e)))
    return TBE_ERR_INVALID_ARGUMENT;
  if (in->tokens > 1 && (dx_stride < in->dim || dgate_stride < in->dim))
    return TBE_ERR_INVALID_ARGUMENT;
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
  return launch_scan(a, in, true, static_cast<hipStream_t>(stream)) == hipSuccess ? TBE_OK
                                                                                  : TBE_ERR_HIP;
}

}  // extern "C"
