// Sums of parts that workgroups left in a workspace, in a fixed order.
#pragma once

#include "seq.h"

namespace sla {
namespace {

constexpr int kSumWaves = 16;

// Up to three arrays of `rows` rows of n elements each.
template <typename C>
struct RowSums {
  const C* part[3];
  C* out[3];
  int64_t n[3], stride[3], groups[3];  // elements, from row to row, workgroups
  int64_t rows;
};

// A workgroup sums 64 elements, its waves taking a part of the rows each: few
// elements and many rows still have enough loads on their way (1024 rows x 2048: 4
// waves 32 us, 16 waves 7).
template <typename C>
__global__ __launch_bounds__(kSumWaves * 64) void sum_rows(RowSums<C> p) {
  __shared__ C red[kSumWaves][64];
  int64_t g = blockIdx.x;
  int k = 0;
  while (k < 2 && g >= p.groups[k]) g -= p.groups[k++];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t at = g * 64 + lane, step = p.stride[k];
  const int64_t each = (p.rows + kSumWaves - 1) / kSumWaves;
  const int64_t r0 = wave * each, r1 = min(r0 + each, p.rows);
  C s = C(0);
  if (at < p.n[k]) {
    const C* const from = p.part[k] + at;
#pragma unroll 8
    for (int64_t r = r0; r < r1; ++r) s += from[r * step];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave || at >= p.n[k]) return;
#pragma unroll
  for (int o = 1; o < kSumWaves; ++o) s += red[o][lane];
  p.out[k][at] = s;
}

// Arrays without an `out` are left alone.
template <typename C>
sla_status sum_of_rows(RowSums<C> r, hipStream_t s) {
  int64_t groups = 0;
  for (int k = 0; k < 3; ++k) {
    if (!r.out[k]) r.n[k] = 0;
    groups += r.groups[k] = (r.n[k] + 63) / 64;
  }
  if (!groups) return SLA_OK;
  sum_rows<C><<<(unsigned)groups, kSumWaves * 64, 0, s>>>(r);
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}

}  // namespace
}  // namespace sla
