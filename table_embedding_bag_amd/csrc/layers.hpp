// layers.hpp -- helpers shared by the kernels of the row layers (dropout.hip,
// scan.hip, grouped.hip).  Internal; the public interface is tbe.h.
#pragma once

#include "common.hpp"
#include "tbe.h"

namespace tbe {

template <int ST>
struct Stored {
  using type = float;
};
template <>
struct Stored<kF16> {
  using type = _Float16;
};
template <>
struct Stored<kBF16> {
  using type = __bf16;
};

template <int ST, int E>
using StoredVec = typename Stored<ST>::type __attribute__((ext_vector_type(E)));

// E consecutive stored elements, the address aligned to one element only: one
// wide load (global memory takes any alignment).
template <int ST, int E>
__device__ __forceinline__ StoredVec<ST, E> load_vec(const void* base, int64_t e) {
  StoredVec<ST, E> v;
  __builtin_memcpy(&v, static_cast<const char*>(base) + e * StorageTraits<ST>::bytes,
                   E * StorageTraits<ST>::bytes);
  return v;
}
template <int ST, int E>
__device__ __forceinline__ void store_vec(void* base, int64_t e, const StoredVec<ST, E>& v) {
  __builtin_memcpy(static_cast<char*>(base) + e * StorageTraits<ST>::bytes, &v,
                   E * StorageTraits<ST>::bytes);
}

template <int ST>
__device__ __forceinline__ float load_one(const void* base, int64_t e) {
  return static_cast<float>(static_cast<const typename Stored<ST>::type*>(base)[e]);
}
// Rounds to nearest, ties to even: the one rounding of a result held in fp32.
template <int ST>
__device__ __forceinline__ void store_one(void* base, int64_t e, float v) {
  static_cast<typename Stored<ST>::type*>(base)[e] = static_cast<typename Stored<ST>::type>(v);
}

inline bool known_dtype(int32_t dtype) { return dtype >= TBE_F32 && dtype <= TBE_BF16; }
inline int dtype_bytes(int32_t dtype) { return dtype == TBE_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace tbe
