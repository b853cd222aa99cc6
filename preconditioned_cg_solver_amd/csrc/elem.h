// Storage types of the recurrences and of the AdamW step, and the type each
// is computed in: fp64 for fp64, fp32 for everything else.
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

}  // namespace sla
