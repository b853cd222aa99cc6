// Parts shared by the operators along sequences: the activations and their slopes, and
// sums over lanes.
#pragma once

#include <hip/hip_runtime.h>

#include "elem.h"
#include "internal.h"
#include "offsets.h"

namespace sla {

// Orders a wave's LDS accesses before and after it: its lanes exchange data
// without a barrier, for LDS serves a wave's accesses in their order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Waits for loads of values here, and not where they are used: in a loop that would
// be a wait for whatever was loaded last, the next tile.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void settle(double& v) { asm volatile("" : "+v"(v)); }
template <int N, typename C>
__device__ __forceinline__ void settle(C (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) settle(v[j]);
}

// A barrier that waits for a wave's LDS accesses but not, as __syncthreads does, for
// its stores to memory.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 2^v; in fp32 results under 2^-126 are 0.
__device__ __forceinline__ float pow2(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ double pow2(double v) { return exp2(v); }

// 1 / (1 + e^-v).
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}
__device__ __forceinline__ double sigmoid(double v) { return 1.0 / (1.0 + exp(-v)); }

// v sigmoid(v) from s = sigmoid(v): -infinity gives -0, where the plain product is NaN
// (s is NaN if v is, which the maximum would hide).
__device__ __forceinline__ float silu_of(float v, float s) { return fmaxf(v, -3e38f) * s; }
__device__ __forceinline__ double silu_of(double v, double s) { return fmax(v, -1e308) * s; }
template <typename C>
__device__ __forceinline__ C silu(C v) {
  return silu_of(v, sigmoid(v));
}
// Its slope, s (1 + v (1 - s)): s (1 - s) is 0 long before v reaches the bounds.
__device__ __forceinline__ float silu_slope(float v, float s) {
  return s + __builtin_amdgcn_fmed3f(v, -1e4f, 1e4f) * (s * (1.0f - s));
}
__device__ __forceinline__ double silu_slope(double v, double s) {
  return s + fmin(fmax(v, -1e5), 1e5) * (s * (1.0 - s));
}

// log(1 + e^v), and the slope sigmoid(v).  With w = 1 + e as rounded, log(w) + (e - (w -
// 1)) / w has the accuracy of log(1 + e) for every e; above 30 (fp64: 40) the sum is v
// to the last place.
__device__ __forceinline__ float softplus(float v, float& slope) {
  const float e = __builtin_amdgcn_exp2f(1.44269504f * v), w = 1.0f + e;
  const float r = __builtin_amdgcn_rcpf(w);
  const float l = 0.693147181f * __builtin_amdgcn_logf(w) + (e - (w - 1.0f)) * r;
  const bool big = v > 30.0f;
  slope = big ? 1.0f : e * r;
  return big ? v : l;
}
__device__ __forceinline__ double softplus(double v, double& slope) {
  const double e = exp(v);
  const bool big = v > 40.0;
  slope = big ? 1.0 : e / (1.0 + e);
  return big ? v : log1p(e);
}

// Lane exchanges of either width: with the halves (the 16-lane rows) of a wave
// swapped between two values, their sum holds in each half (row) one of the two
// sums over a lane and its partner.
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_rows(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_halves(double& a, double& b) {
  const auto lo = __builtin_amdgcn_permlane32_swap(__double2loint(a), __double2loint(b), false,
                                                   false);
  const auto hi = __builtin_amdgcn_permlane32_swap(__double2hiint(a), __double2hiint(b), false,
                                                   false);
  a = __hiloint2double((int)hi[0], (int)lo[0]);
  b = __hiloint2double((int)hi[1], (int)lo[1]);
}
__device__ __forceinline__ void swap_rows(double& a, double& b) {
  const auto lo = __builtin_amdgcn_permlane16_swap(__double2loint(a), __double2loint(b), false,
                                                   false);
  const auto hi = __builtin_amdgcn_permlane16_swap(__double2hiint(a), __double2hiint(b), false,
                                                   false);
  a = __hiloint2double((int)hi[0], (int)lo[0]);
  b = __hiloint2double((int)hi[1], (int)lo[1]);
}
// Both sums over pairs of lanes, 32 apart: of a in the lower half, of b in the upper.
template <typename C>
__device__ __forceinline__ C fold_halves(C a, C b) {
  swap_halves(a, b);
  return a + b;
}
// Both sums over pairs of lanes, 16 apart: of a in the even rows, of b in the odd.
template <typename C>
__device__ __forceinline__ C fold_rows(C a, C b) {
  swap_rows(a, b);
  return a + b;
}
// The value of another lane of the 16-lane row (a DPP pattern).
template <int CTRL>
__device__ __forceinline__ float from_lane(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ double from_lane(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf, 0xf, false);
  return __hiloint2double(hi, lo);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;             // within a quad
constexpr int kRor4 = 0x124, kRor8 = 0x128;  // rotations of a row

}  // namespace sla
