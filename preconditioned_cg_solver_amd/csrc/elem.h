// Storage types of the operators along sequences, of the norms and of the AdamW step,
// and the type each is computed in: fp64 for fp64, fp32 for everything else.
#pragma once

#include <hip/hip_runtime.h>

#include "sla.h"

namespace sla {

using bf16_t = __bf16;
using f16_t = _Float16;

template <typename T>
struct Compute {
  using type = float;
};
template <>
struct Compute<double> {
  using type = double;
};

inline size_t dtype_bytes(int32_t dt) { return dt == SLA_F64 ? 8 : dt == SLA_F32 ? 4 : 2; }

// N consecutive elements moved by one load or store when aligned to N of them.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// A word as wide as a pack.
template <size_t BYTES>
struct WordOf {
  typedef unsigned type __attribute__((ext_vector_type(BYTES / 4)));
};
template <>
struct WordOf<4> {
  using type = unsigned;
};
template <>
struct WordOf<2> {
  using type = unsigned short;
};

// Reads and writes of packs, past the caches if STREAM.  (Not a choice at run time: the
// compiler would make one access of both.)
template <bool STREAM, int N, typename T>
__device__ __forceinline__ Pack<T, N> get_pack(const T* from) {
  using W = typename WordOf<sizeof(Pack<T, N>)>::type;
  if constexpr (STREAM)
    return __builtin_bit_cast(Pack<T, N>, __builtin_nontemporal_load((const W*)from));
  return *(const Pack<T, N>*)from;
}
template <bool STREAM, int N, typename T>
__device__ __forceinline__ void put_pack(T* to, const Pack<T, N>& v) {
  using W = typename WordOf<sizeof(Pack<T, N>)>::type;
  if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(W, v), (W*)to);
  else *(Pack<T, N>*)to = v;
}

}  // namespace sla
