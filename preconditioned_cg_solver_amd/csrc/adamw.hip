// AdamW over many tensors in one launch, with states in 32 or in 8 bits.
//
// Work is cut into blocks of 256 elements, one wave64 each (four consecutive
// elements per lane); in 8 bits a block is also what shares a base.  A
// device table, written when the handle is created, lists the tensors and
// the blocks; only the gradients' addresses, which change from step to step,
// travel with the launch as kernel arguments.  Nothing is reduced over more than
// a block and there are no atomics: a step's bits do not depend on its order.
//
// What bounds it: an element's 28 bytes with fp32 states (120M of them 536 to
// 582 us between cards, 5.8 to 6.3 TB/s) and its 14 bytes with 8-bit ones and a
// bf16 gradient (60M: 131 to 140 us, 6.0 to 6.4 TB/s), where an elementwise sum
// of large arrays reaches 6.2; with bf16 parameters and 8-bit states (10 bytes)
// the rounding's arithmetic, some 80 instructions an element (9M: 26 to 27 us,
// 3.5 TB/s); below a million elements the launch (60000 in 24 tensors: 3.3 us).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "device_util.h"
#include "elem.h"
#include "internal.h"

namespace sla {
namespace {

constexpr int kBlock = 256;          // elements per block
constexpr int kPerLane = kBlock / 64;
constexpr int kChunkBlocks = kWaves;  // blocks per workgroup
// Gradient addresses per launch: with the other arguments they stay within
// the 4 KB that a launch can carry.
constexpr int kGrads = 448;
// Bytes of a step above which it goes past the caches (the last-level cache
// has 256 MB).  Through and past them, with the reading back of 8-bit states:
// 120M fp32 elements 572 and 544 us, 60M with 8-bit states 214 and 202 us,
// 9M bf16 with 8-bit states (90 MB) 35.3 and 36.2 us.
constexpr int64_t kCacheBytes = 256 << 20;
constexpr int kTopM = 126, kTopV = 254;      // highest finite codes
constexpr int kBadM = 127, kBadV = 255;      // not finite

// Parameter and gradient types, a launch each.
enum Kind { K_F32 = 0, K_F32_BF16 = 1, K_BF16 = 2, K_F64 = 3, K_KINDS = 4 };

struct Tensor {
  void* p;
  void* copy;
  int64_t numel;
  int64_t block0;  // first block in the states
};
// kChunkBlocks consecutive blocks of one tensor.
struct Chunk {
  int32_t tensor;  // in the order of its kind
  int32_t first;   // block of the tensor, in units of kChunkBlocks
};

struct State {
  float *m32, *v32;          // 32 bits
  uint8_t *m8, *v8;          // 8 bits
  uint16_t *mbase, *vbase;
};

struct Step {
  const Tensor* tensors;  // of the kind
  const Chunk* chunks;    // of this launch
  State st;
  float b1, b1c, b2, b2c;      // beta and 1 - beta
  float decay, rate, root, eps;  // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  double decay64;
  uint32_t key;
  int32_t tensor0;        // of grads[0]
  const float* scale;
};
struct Grads {
  const void* g[kGrads];
};
static_assert(sizeof(Step) + sizeof(Grads) <= 4096, "kernel arguments");

__host__ __device__ inline uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x9E3779B1u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}
// 32 random bits of elements e, e + 1, ... e + kPerLane - 1 (places in the
// padded order; e is a multiple of kPerLane).
__device__ __forceinline__ void noise(uint32_t key, uint64_t e, uint32_t (&r)[kPerLane]) {
  const uint32_t hi = (uint32_t)(e >> 32), k = hi ? key ^ mix(hi) : key;
#pragma unroll
  for (uint32_t j = 0; j < kPerLane; ++j)
    r[j] = mix((uint32_t)e * 0x9E3779B1u + (j * 0x9E3779B1u + k));
}

// Largest over the 64 lanes, in every lane: within 16-lane rows by DPP moves,
// across rows and halves by the lane swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_max<0x141>(v);  // row_half_mirror
  v = dpp_max<0x140>(v);  // row_mirror
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)r[0], (uint32_t)r[1]);
  const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)h[0], (uint32_t)h[1]);
}

// The 8-bit form (see sla.h): patterns of finite magnitudes are below this.
constexpr uint32_t kInf = 0x7f800000u;
constexpr uint32_t kMost = (kInf >> 20) - 1;  // the largest finite level

// FINITE: no code of the wave's stands for a value that is not (the step's
// arithmetic bounds its 8-bit form, and these tests are a fifth of it).
template <bool FINITE>
__device__ __forceinline__ float decode(uint32_t code, uint32_t base, uint32_t bad, float worst) {
  const float v = code == 0 ? 0.0f : __uint_as_float((code + base) << 20);
  return !FINITE && code == bad ? worst : v;
}
template <bool FINITE>
__device__ __forceinline__ float decode_v(uint32_t c, uint32_t base) {
  return decode<FINITE>(c, base, kBadV, INFINITY);
}
template <bool FINITE>
__device__ __forceinline__ float decode_m(uint32_t c, uint32_t base) {
  const uint32_t sign = (c & 128) << 24;
  return __uint_as_float(__float_as_uint(decode<FINITE>(c & 127, base, kBadM, NAN)) | sign);
}
// Whether one of the four codes in m or v is kBadM or kBadV: a zero byte in
// the complement, which subtracting one from each byte shows in its top bit.
__device__ __forceinline__ bool bad_codes(uint32_t m, uint32_t v) {
  const uint32_t a = (~m & 0x7f7f7f7fu) - 0x01010101u, b = (~v - 0x01010101u) & v;
  return ((a | b) & 0x80808080u) != 0;
}

// Largest pattern of a wave's block; FINITE: of those that are.
template <bool FINITE>
__device__ __forceinline__ uint32_t top_of(const uint32_t (&bits)[kPerLane]) {
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) mx = max(mx, !FINITE || bits[j] < kInf ? bits[j] : 0);
  return __builtin_amdgcn_readfirstlane(wave_max(mx));
}
// The base under which every value up to `mx`, rounded up by less than `up`,
// has a code of at most `top`.
__device__ __forceinline__ uint32_t base_of(uint32_t mx, int top, uint32_t up) {
  const uint32_t k = min((mx + up) >> 20, kMost);
  return k > (uint32_t)top ? k - (uint32_t)top : 0;
}
// add < 2^20, so that a zero's code is 0.
template <bool FINITE>
__device__ __forceinline__ uint32_t encode(uint32_t bits, uint32_t add, uint32_t base, int least,
                                           int top, int bad) {
  const int c = (int)((bits + add) >> 20) - (int)base;
  return !FINITE && bits >= kInf ? bad : (uint32_t)min(max(c, least), top);
}
template <bool FINITE>
__device__ __forceinline__ uint32_t encode_v(uint32_t bits, uint32_t add, uint32_t base) {
  return encode<FINITE>(bits, add, base, (int)min(bits, 1u), kTopV, kBadV);
}
template <bool FINITE>
__device__ __forceinline__ uint32_t encode_m(uint32_t bits, uint32_t add, uint32_t base) {
  return encode<FINITE>(bits, add, base, 0, kTopM, kBadM);
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int KIND>
struct Types {
  using P = float;
  using G = float;
};
template <>
struct Types<K_F32_BF16> {
  using P = float;
  using G = bf16_t;
};
template <>
struct Types<K_BF16> {
  using P = bf16_t;
  using G = bf16_t;
};
template <>
struct Types<K_F64> {
  using P = double;
  using G = double;
};

// rate m / (root sqrt(v) + eps), by the hardware's root and reciprocal (each
// within a unit in the last place; the full-precision sequences would make
// the 8-bit step wait for its arithmetic).  They take no subnormal numbers:
// v counts as 2^-126 at least, unless it is NaN (the maximum that keeps those).
__device__ __forceinline__ float update(const Step& q, float m, float v) {
  const float s = __builtin_amdgcn_sqrtf(__builtin_elementwise_maximum(v, 0x1p-126f));
  return m * __builtin_amdgcn_rcpf(s * q.root + q.eps) * q.rate;
}

// A bf16 parameter's new value, rounded up with the probability of its
// remainder (16 random bits).  A NaN that arithmetic gave is quiet and stays
// one without its low bits.
__device__ __forceinline__ bf16_t round_bf16(float x, uint32_t r16) {
  const uint32_t u = __float_as_uint(x) + (__builtin_isfinite(x) ? r16 : 0);
  return __builtin_bit_cast(bf16_t, (uint16_t)(u >> 16));
}

// m' and v', in the order of operations that sla.h's formulas give and with
// every product rounded by itself, so that the 8-bit codes do not depend on
// what the compiler would contract.
__device__ __forceinline__ void moments(const Step& q, float g, float& m, float& v) {
#pragma clang fp contract(off)
  m = m * q.b1 + g * q.b1c;
  v = v * q.b2 + (g * g) * q.b2c;
}

// A pointer from the table, known to be to global memory.
template <typename T>
__device__ __forceinline__ T* global(const void* p) {
  return (T*)(__attribute__((address_space(1))) T*)(uintptr_t)p;
}

// Four elements of a lane, at any address that is a multiple of their size.
// NT: past the caches, for a step that moves more than they hold.
template <typename T>
using Quad4 = unsigned __attribute__((ext_vector_type(sizeof(T)), aligned(sizeof(T))));
template <bool NT, typename T>
__device__ __forceinline__ void load4(const T* from, T (&to)[kPerLane]) {
  const Quad4<T> w = ld_stream<NT>((const Quad4<T>*)from);
  __builtin_memcpy(to, &w, sizeof to);
}
template <bool NT, typename T>
__device__ __forceinline__ void store4(T* to, const T (&from)[kPerLane]) {
  Quad4<T> w;
  __builtin_memcpy(&w, from, sizeof w);
  if constexpr (NT) __builtin_nontemporal_store(w, (Quad4<T>*)to);
  else *(Quad4<T>*)to = w;
}

// A lane's part of a block: as read, and after the step.
template <int KIND, int BITS>
struct Quad {
  using P = typename Types<KIND>::P;
  using G = typename Types<KIND>::G;
  using S = std::conditional_t<BITS == 32, float, uint8_t>;
  P p[kPerLane];
  G g[kPerLane];
  Pack<S, kPerLane> m, v;
  uint32_t bm, bv;
};

// PART: the block ends with the tensor, after `left` elements of this lane.
template <int KIND, int BITS, bool NT, bool PART>
__device__ __forceinline__ void read_quad(const Step& q, const Tensor& t,
                                          const typename Types<KIND>::G* gr, int64_t blk,
                                          Quad<KIND, BITS>& d) {
  using Q = Quad<KIND, BITS>;
  const int64_t i = blk * kBlock + kPerLane * (threadIdx.x & 63);
  const int64_t at = t.block0 * kBlock + i;  // in the states
  const auto* p = global<const typename Q::P>(t.p);
  if constexpr (PART) {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      d.p[j] = i + j < t.numel ? p[i + j] : (typename Q::P)0.0f;
      d.g[j] = i + j < t.numel ? gr[i + j] : (typename Q::G)0.0f;
    }
  } else {
    load4<NT>(p + i, d.p);
    load4<NT>(gr + i, d.g);
  }
  if constexpr (BITS == 32) {
    load4<NT>(q.st.m32 + at, d.m.v);
    load4<NT>(q.st.v32 + at, d.v.v);
  } else {
    load4<NT>(q.st.m8 + at, d.m.v);
    load4<NT>(q.st.v8 + at, d.v.v);
    d.bm = q.st.mbase[t.block0 + blk];
    d.bv = q.st.vbase[t.block0 + blk];
  }
}

template <int KIND, int BITS, bool NT, bool PART>
__device__ __forceinline__ void step_quad(const Step& q, const Tensor& t, float scale,
                                          int64_t blk, Quad<KIND, BITS>& d) {
  using Q = Quad<KIND, BITS>;
  const int lane = threadIdx.x & 63;
  const int64_t i = blk * kBlock + kPerLane * lane, at = t.block0 * kBlock + i;
  float m[kPerLane], v[kPerLane];
  uint32_t rnd[kPerLane] = {}, mb[kPerLane], vb[kPerLane];
  bf16_t low[kPerLane];
  if (BITS == 8 || KIND == K_BF16) noise(q.key, (uint64_t)at, rnd);
  if constexpr (BITS == 32) {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) m[j] = d.m.v[j], v[j] = d.v.v[j];
  } else {
    auto decode4 = [&](auto finite) {
      constexpr bool kFinite = decltype(finite)::value;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        m[j] = decode_m<kFinite>(d.m.v[j], d.bm), v[j] = decode_v<kFinite>(d.v.v[j], d.bv);
    };
    if (__any(bad_codes(__builtin_bit_cast(uint32_t, d.m), __builtin_bit_cast(uint32_t, d.v))))
      decode4(std::false_type{});
    else decode4(std::true_type{});
  }
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const bool in = !PART || i + j < t.numel;
    using W = std::conditional_t<KIND == K_F64, double, float>;
    const float g = (float)((W)d.g[j] * (W)scale);
    moments(q, g, m[j], v[j]);
    if (!in) m[j] = v[j] = 0.0f;
    const float up = update(q, m[j], v[j]);
    if constexpr (KIND == K_F64) {
      d.p[j] = d.p[j] * q.decay64 - (double)up;
    } else if constexpr (KIND == K_BF16) {
      d.p[j] = round_bf16((float)d.p[j] * q.decay - up, mix(rnd[j] + 0x6A09E667u) & 0xffff);
    } else {
      d.p[j] = d.p[j] * q.decay - up;
      low[j] = (bf16_t)d.p[j];
    }
    mb[j] = magnitude(m[j]);
    vb[j] = magnitude(v[j]);
  }
  auto* p = global<typename Q::P>(t.p);
  bf16_t* copy = t.copy ? global<bf16_t>(t.copy) : nullptr;
  if constexpr (PART) {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      if (i + j < t.numel) {
        p[i + j] = d.p[j];
        if ((KIND == K_F32 || KIND == K_F32_BF16) && copy) copy[i + j] = low[j];
      }
    }
  } else {
    store4<NT>(p + i, d.p);
    if ((KIND == K_F32 || KIND == K_F32_BF16) && copy) store4<false>(copy + i, low);
  }
  if constexpr (BITS == 32) {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) d.m.v[j] = m[j], d.v.v[j] = v[j];
    store4<NT>(q.st.m32 + at, d.m.v);
    store4<NT>(q.st.v32 + at, d.v.v);
  } else {
    uint32_t bm = top_of<false>(mb), bv = top_of<false>(vb);
    auto encode4 = [&](auto finite) {
      constexpr bool kFinite = decltype(finite)::value;
      bm = base_of(bm, kTopM, 0xfffff);
      bv = base_of(bv, kTopV, 0xfffff);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        const uint32_t cm = encode_m<kFinite>(mb[j], ((rnd[j] & 0xffff) << 4) + 8, bm);
        d.m.v[j] = (uint8_t)(cm | (m[j] < 0.0f ? 128u : 0u));
        d.v.v[j] = (uint8_t)encode_v<kFinite>(vb[j], ((rnd[j] >> 16) << 4) + 8, bv);
      }
    };
    if (max(bm, bv) < kInf) {
      encode4(std::true_type{});
    } else {
      // (keeps the compiler from doing this for every block beforehand)
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) asm volatile("" : "+v"(mb[j]), "+v"(vb[j]));
      bm = top_of<true>(mb), bv = top_of<true>(vb);
      encode4(std::false_type{});
    }
    store4<NT>(q.st.m8 + at, d.m.v);
    store4<NT>(q.st.v8 + at, d.v.v);
    if (lane == 0) {
      q.st.mbase[t.block0 + blk] = (uint16_t)bm;
      q.st.vbase[t.block0 + blk] = (uint16_t)bv;
    }
  }
}

// One step of every parameter of a launch, a block per wave.  (Two or four
// blocks, all read before the first is stepped: 120M fp32 elements 572 us with one,
// 581 with two, 580 with four; 9M bf16 with 8-bit states 33.7, 35.4 and 37.6 us.)
template <int KIND, int BITS, bool NT>
__global__ __launch_bounds__(kWG) void adamw_step(Step q, Grads grads) {
  const float scale = q.scale ? *q.scale : 1.0f;
  if (!(fabsf(scale) < INFINITY)) return;
  const Chunk ch = q.chunks[blockIdx.x];
  const int tensor = __builtin_amdgcn_readfirstlane(ch.tensor);
  const void* grad = grads.g[tensor - q.tensor0];
  if (!grad) return;
  const auto* gr = global<const typename Types<KIND>::G>(grad);
  const Tensor t = q.tensors[tensor];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blk = (int64_t)__builtin_amdgcn_readfirstlane(ch.first) * kChunkBlocks + wave;
  Quad<KIND, BITS> d;
  if ((blk + 1) * kBlock <= t.numel) {
    read_quad<KIND, BITS, NT, false>(q, t, gr, blk, d);
    step_quad<KIND, BITS, NT, false>(q, t, scale, blk, d);
  } else if (blk * kBlock < t.numel) {
    read_quad<KIND, BITS, NT, true>(q, t, gr, blk, d);
    step_quad<KIND, BITS, NT, true>(q, t, scale, blk, d);
  }
}

// The values of 8-bit states: four significant bits, which bf16 holds.
// Bound by its 6 bytes an element: 60M in 63 us, 5.7 TB/s.
__global__ __launch_bounds__(kWG) void adamw_read8(State st, int64_t blk0, int64_t blocks,
                                                   bf16_t* m, bf16_t* v) {
  const int64_t blk = blk0 + (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int64_t at = blk * kBlock + kPerLane * (threadIdx.x & 63);
  const auto cm = *(const Pack<uint8_t, 4>*)(st.m8 + at);
  const auto cv = *(const Pack<uint8_t, 4>*)(st.v8 + at);
  const uint32_t bm = st.mbase[blk], bv = st.vbase[blk];
  Pack<bf16_t, 4> om, ov;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    om.v[j] = (bf16_t)decode_m<false>(cm.v[j], bm);
    ov.v[j] = (bf16_t)decode_v<false>(cv.v[j], bv);
  }
  *(Pack<bf16_t, 4>*)(m + at) = om;
  *(Pack<bf16_t, 4>*)(v + at) = ov;
}

// States from values, to the nearest level (10 bytes an element: 60M in
// 115 us on a first call).
__global__ __launch_bounds__(kWG) void adamw_write8(State st, int64_t blk0, int64_t blocks,
                                                    const float* m, const float* v) {
  const int64_t blk = blk0 + (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int lane = threadIdx.x & 63;
  const int64_t at = blk * kBlock + kPerLane * lane;
  const auto pm = *(const Pack<float, 4>*)(m + at);
  const auto pv = *(const Pack<float, 4>*)(v + at);
  uint32_t mb[kPerLane], vb[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) mb[j] = magnitude(pm.v[j]), vb[j] = magnitude(pv.v[j]);
  const uint32_t bm = base_of(top_of<true>(mb), kTopM, 0x80000);
  const uint32_t bv = base_of(top_of<true>(vb), kTopV, 0x80000);
  Pack<uint8_t, 4> cm, cv;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    cm.v[j] = (uint8_t)(encode_m<false>(mb[j], 0x80000, bm) | (pm.v[j] < 0.0f ? 128u : 0u));
    cv.v[j] = (uint8_t)encode_v<false>(vb[j], 0x80000, bv);
  }
  *(Pack<uint8_t, 4>*)(st.m8 + at) = cm;
  *(Pack<uint8_t, 4>*)(st.v8 + at) = cv;
  if (lane == 0) st.mbase[blk] = (uint16_t)bm, st.vbase[blk] = (uint16_t)bv;
}

// Plain copies between the 32-bit states and the caller's arrays: a lane copies
// as much of a block as it steps.
__global__ __launch_bounds__(kWG) void copy4(const float* a, float* b, int64_t blk0,
                                             int64_t blocks) {
  const int64_t i = blk0 * 64 + (int64_t)blockIdx.x * kWG + threadIdx.x;
  if (i < blocks * 64) ((Pack<float, 4>*)b)[i] = ((const Pack<float, 4>*)a)[i];
}

sla_status refuse(const char* msg) {
  set_error(msg);
  return SLA_ERR_INVALID_ARG;
}

int kind_of(const sla_adamw_tensor& t) {
  if (t.dtype == SLA_F32 && t.grad_dtype == SLA_F32) return K_F32;
  if (t.dtype == SLA_F32 && t.grad_dtype == SLA_BF16) return K_F32_BF16;
  if (t.dtype == SLA_BF16 && t.grad_dtype == SLA_BF16) return K_BF16;
  if (t.dtype == SLA_F64 && t.grad_dtype == SLA_F64) return K_F64;
  return -1;
}

bool aligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

struct Sizes {
  int64_t blocks = 0, chunks = 0;
  size_t state = 0, table = 0;
};

sla_status check_tensors(const sla_adamw_tensor* ts, int32_t n, int32_t bits, Sizes* z) {
  if (n < 0 || (n > 0 && !ts)) return refuse("bad tensor list");
  if (bits != 8 && bits != 32) {
    set_error("states have 8 or 32 bits");
    return SLA_ERR_UNSUPPORTED;
  }
  for (int32_t i = 0; i < n; ++i) {
    const sla_adamw_tensor& t = ts[i];
    for (const sla_dtype d : {t.dtype, t.grad_dtype})
      if (d != SLA_F64 && d != SLA_F32 && d != SLA_BF16 && d != SLA_F16)
        return refuse("unknown dtype");
    if (kind_of(t) < 0) {
      set_error("unsupported parameter and gradient dtypes");
      return SLA_ERR_UNSUPPORTED;
    }
    if (t.d_copy && t.dtype != SLA_F32) {
      set_error("only an fp32 parameter can keep a bf16 copy");
      return SLA_ERR_UNSUPPORTED;
    }
    if (t.numel < 0 || t.numel >= ((int64_t)1 << 40)) return refuse("bad tensor size");
    if (t.numel > 0 && !t.d_param) return refuse("a parameter is NULL");
    if (!aligned(t.d_param, dtype_bytes(t.dtype)) || !aligned(t.d_copy, 2))
      return refuse("a parameter is not aligned to its elements");
    const int64_t blocks = (t.numel + kBlock - 1) / kBlock;
    z->blocks += blocks;
    z->chunks += (blocks + kChunkBlocks - 1) / kChunkBlocks;
  }
  if (z->chunks >= (1 << 28)) {
    set_error("too many elements for one handle");
    return SLA_ERR_UNSUPPORTED;
  }
  const size_t padded = (size_t)z->blocks * kBlock;
  z->state = bits == 32 ? 8 * padded : 2 * padded + 4 * (size_t)z->blocks;
  z->table = align_up((size_t)n * sizeof(Tensor)) + (size_t)z->chunks * sizeof(Chunk);
  return SLA_OK;
}

// A launch has less than 2^32 threads.
constexpr int64_t kMostGroups = (((int64_t)1 << 32) - 1) / kWG;
// Calls launch(first block, grid) for all blocks, one a wave.
template <typename F>
sla_status in_launches(int64_t blocks, F&& launch) {
  for (int64_t at = 0; at < blocks; at += kMostGroups * kWaves) {
    const int64_t groups = (blocks - at + kWaves - 1) / kWaves;
    launch(at, dim3((unsigned)std::min(groups, kMostGroups)));
    SLA_HIP(hipGetLastError());
  }
  return SLA_OK;
}

// One launch of a kind: a range of its tensors (kGrads at most) and of its
// chunks (kMostGroups at most).
struct Launch {
  int kind;
  int32_t tensor0, tensors;
  int64_t chunk0, chunks;
};

// Memory that a step writes for a tensor.
struct Span {
  uintptr_t begin, end;
  int32_t tensor;
};
// Whether two of the spans that `used` takes overlap; they are sorted by begin.
template <typename F>
bool overlap(const std::vector<Span>& spans, F&& used) {
  uintptr_t end = 0;
  for (const Span& s : spans) {
    if (!used(s.tensor)) continue;
    if (s.begin < end) return true;
    end = std::max(end, s.end);
  }
  return false;
}
// The spans that overlap another one, sorted.
std::vector<Span> shared_spans(const sla_adamw_tensor* ts, int32_t n) {
  std::vector<Span> all, some;
  for (int32_t i = 0; i < n; ++i) {
    if (ts[i].numel == 0) continue;
    const uintptr_t p = (uintptr_t)ts[i].d_param, c = (uintptr_t)ts[i].d_copy;
    all.push_back({p, p + ts[i].numel * dtype_bytes(ts[i].dtype), i});
    if (c) all.push_back({c, c + ts[i].numel * dtype_bytes(SLA_BF16), i});
  }
  std::sort(all.begin(), all.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t end = 0;  // of those before
  for (size_t k = 0; k < all.size(); ++k) {
    if (all[k].begin < end || (k + 1 < all.size() && all[k + 1].begin < all[k].end))
      some.push_back(all[k]);
    end = std::max(end, all[k].end);
  }
  return some;
}

}  // namespace
}  // namespace sla

struct sla_adamw {
  int32_t n = 0, bits = 32;
  int64_t blocks = 0;
  bool streams = false;                    // a step moves more than the caches hold
  const sla::Tensor* d_tensors = nullptr;  // sorted by kind
  const sla::Chunk* d_chunks = nullptr;
  sla::State st = {};
  int32_t kind0[sla::K_KINDS] = {};        // first tensor of each kind
  std::vector<int32_t> order;              // caller's index of each
  std::vector<size_t> align;               // of its gradient
  std::vector<sla::Launch> launches;
  std::vector<sla::Span> shared;           // of tensors that share memory
};

namespace sla {
namespace {

sla_status build(sla_adamw* o, const sla_adamw_tensor* ts, void* d_state, void* d_table,
                 const Sizes& z, hipStream_t s) {
  const size_t tbytes = align_up((size_t)o->n * sizeof(Tensor));
  std::vector<char> table(z.table);
  Tensor* ht = (Tensor*)table.data();
  Chunk* hc = (Chunk*)(table.data() + tbytes);
  std::vector<int64_t> block0((size_t)o->n);
  int64_t blocks = 0, bytes = 0;
  for (int32_t i = 0; i < o->n; ++i) {
    block0[i] = blocks;
    blocks += (ts[i].numel + kBlock - 1) / kBlock;
    bytes += ts[i].numel * (int64_t)(2 * dtype_bytes(ts[i].dtype) + dtype_bytes(ts[i].grad_dtype) +
                                     (o->bits == 32 ? 16 : 4));
  }
  o->blocks = blocks;
  o->shared = shared_spans(ts, o->n);
  o->streams = bytes > kCacheBytes;
  int64_t nc = 0;
  for (int kind = 0; kind < K_KINDS; ++kind) {
    o->kind0[kind] = (int32_t)o->order.size();
    for (int32_t i = 0; i < o->n; ++i) {
      if (kind_of(ts[i]) != kind || ts[i].numel == 0) continue;
      const int32_t pos = (int32_t)o->order.size(), local = pos - o->kind0[kind];
      if (local % kGrads == 0) o->launches.push_back({kind, local, 0, nc, 0});
      o->order.push_back(i);
      o->align.push_back(dtype_bytes(ts[i].grad_dtype));
      ht[pos] = {ts[i].d_param, ts[i].d_copy, ts[i].numel, block0[i]};
      const int64_t nb = (ts[i].numel + kBlock - 1) / kBlock;
      for (int64_t b = 0; b < nb; b += kChunkBlocks) {
        if (o->launches.back().chunks == kMostGroups)
          o->launches.push_back({kind, local, 0, nc, 0});
        Launch& l = o->launches.back();
        hc[nc++] = {local, (int32_t)(b / kChunkBlocks)};
        l.tensors = local - l.tensor0 + 1;
        ++l.chunks;
      }
    }
  }
  o->d_tensors = (const Tensor*)d_table;
  o->d_chunks = (const Chunk*)((char*)d_table + tbytes);
  const size_t padded = (size_t)blocks * kBlock;
  if (o->bits == 32) {
    o->st.m32 = (float*)d_state;
    o->st.v32 = o->st.m32 + padded;
  } else {
    o->st.m8 = (uint8_t*)d_state;
    o->st.v8 = o->st.m8 + padded;
    o->st.mbase = (uint16_t*)(o->st.v8 + padded);
    o->st.vbase = o->st.mbase + blocks;
  }
  if (z.table) SLA_HIP(hipMemcpyAsync(d_table, table.data(), z.table, hipMemcpyHostToDevice, s));
  SLA_HIP(hipStreamSynchronize(s));
  return SLA_OK;
}

template <int BITS, bool NT>
void launch(const Launch& l, const Step& q, const Grads& g, hipStream_t s) {
  const dim3 grid((unsigned)l.chunks);
  switch (l.kind) {
    case K_F32: adamw_step<K_F32, BITS, NT><<<grid, kWG, 0, s>>>(q, g); break;
    case K_F32_BF16: adamw_step<K_F32_BF16, BITS, NT><<<grid, kWG, 0, s>>>(q, g); break;
    case K_BF16: adamw_step<K_BF16, BITS, NT><<<grid, kWG, 0, s>>>(q, g); break;
    default: adamw_step<K_F64, BITS, NT><<<grid, kWG, 0, s>>>(q, g); break;
  }
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

sla_status sla_adamw_sizes(const sla_adamw_tensor* h_tensors, int32_t n_tensors,
                           int32_t state_bits, size_t* state_bytes, size_t* table_bytes,
                           int64_t* padded) {
  Sizes z;
  const sla_status st = check_tensors(h_tensors, n_tensors, state_bits, &z);
  if (st != SLA_OK) return st;
  if (!state_bytes || !table_bytes || !padded) return refuse("NULL result");
  *state_bytes = z.state;
  *table_bytes = z.table;
  *padded = z.blocks * kBlock;
  return SLA_OK;
}

sla_status sla_adamw_create(sla_adamw_t* out, const sla_adamw_tensor* h_tensors,
                            int32_t n_tensors, int32_t state_bits, void* d_state,
                            size_t state_bytes, void* d_table, size_t table_bytes,
                            void* stream) {
  if (!out) return refuse("out is NULL");
  *out = nullptr;
  Sizes z;
  sla_status st = check_tensors(h_tensors, n_tensors, state_bits, &z);
  if (st != SLA_OK) return st;
  if ((z.state && !d_state) || state_bytes < z.state) return refuse("state buffer too small");
  if ((z.table && !d_table) || table_bytes < z.table) return refuse("table buffer too small");
  if (!aligned(d_state, 256) || !aligned(d_table, 256))
    return refuse("the state and table buffers must be 256-byte aligned");
  TraceRange tr("sla_adamw_create");
  sla_adamw* o = new (std::nothrow) sla_adamw();
  if (!o) {
    set_error("host allocation failed");
    return SLA_ERR_OOM;
  }
  o->n = n_tensors;
  o->bits = state_bits;
  try {
    st = build(o, h_tensors, d_state, d_table, z, (hipStream_t)stream);
  } catch (const std::bad_alloc&) {
    st = SLA_ERR_OOM;
  }
  if (st != SLA_OK) {
    if (st == SLA_ERR_OOM) set_error("host allocation failed");
    delete o;
    return st;
  }
  *out = o;
  return SLA_OK;
}

sla_status sla_adamw_destroy(sla_adamw_t opt) {
  delete opt;
  return SLA_OK;
}

sla_status sla_adamw_step(sla_adamw_t opt, const void* const* h_grads,
                          const sla_adamw_hyper* h, const float* d_grad_scale, void* stream) {
  if (!opt || !h || (opt->n > 0 && !h_grads)) return refuse("NULL argument");
  auto nonneg = [](double v) { return std::isfinite(v) && v >= 0.0; };
  if (!nonneg(h->lr) || !nonneg(h->weight_decay) || !nonneg(h->eps))
    return refuse("lr, weight_decay and eps must be finite and not negative");
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
    return refuse("the betas must be in [0, 1)");
  if (h->step < 1) return refuse("step must be at least 1");
  if (!aligned(d_grad_scale, 4)) return refuse("grad_scale is misaligned");
  for (size_t k = 0; k < opt->order.size(); ++k)
    if (!aligned(h_grads[opt->order[k]], opt->align[k]))
      return refuse("a gradient is not aligned to its elements");
  if (overlap(opt->shared, [&](int32_t i) { return h_grads[i] != nullptr; }))
    return refuse("tensors that share memory have gradients in the same step");
  TraceRange tr("sla_adamw_step");
  Step q{};
  q.st = opt->st;
  q.b1 = (float)h->beta1;
  q.b1c = (float)(1.0 - h->beta1);
  q.b2 = (float)h->beta2;
  q.b2c = (float)(1.0 - h->beta2);
  q.decay64 = 1.0 - h->lr * h->weight_decay;
  q.decay = (float)q.decay64;
  q.rate = (float)(h->lr / (1.0 - std::pow(h->beta1, (double)h->step)));
  q.root = (float)(1.0 / std::sqrt(1.0 - std::pow(h->beta2, (double)h->step)));
  q.eps = (float)h->eps;
  q.key = mix((uint32_t)h->seed ^ mix((uint32_t)(h->seed >> 32) ^ mix((uint32_t)h->step)));
  q.scale = d_grad_scale;
  for (const Launch& l : opt->launches) {
    Grads g;
    const int32_t at = opt->kind0[l.kind] + l.tensor0;
    for (int32_t k = 0; k < l.tensors; ++k) g.g[k] = h_grads[opt->order[at + k]];
    q.tensors = opt->d_tensors + opt->kind0[l.kind];
    q.chunks = opt->d_chunks + l.chunk0;
    q.tensor0 = l.tensor0;
    const hipStream_t s = (hipStream_t)stream;
    const auto f = opt->bits == 32 ? opt->streams ? launch<32, true> : launch<32, false>
                                   : opt->streams ? launch<8, true> : launch<8, false>;
    f(l, q, g, s);
    SLA_HIP(hipGetLastError());
  }
  return SLA_OK;
}

sla_status sla_adamw_get_state(sla_adamw_t opt, void* d_m, void* d_v, void* stream) {
  if (!opt) return refuse("handle is NULL");
  if (opt->blocks == 0) return SLA_OK;
  if (!d_m || !d_v || d_m == d_v) return refuse("m and v must be distinct non-NULL arrays");
  if (!aligned(d_m, 16) || !aligned(d_v, 16)) return refuse("m and v must be 16-byte aligned");
  hipStream_t s = (hipStream_t)stream;
  return in_launches(opt->blocks, [&](int64_t blk0, dim3 grid) {
    if (opt->bits == 32) {
      copy4<<<grid, kWG, 0, s>>>(opt->st.m32, (float*)d_m, blk0, opt->blocks);
      copy4<<<grid, kWG, 0, s>>>(opt->st.v32, (float*)d_v, blk0, opt->blocks);
    } else {
      adamw_read8<<<grid, kWG, 0, s>>>(opt->st, blk0, opt->blocks, (bf16_t*)d_m, (bf16_t*)d_v);
    }
  });
}

sla_status sla_adamw_set_state(sla_adamw_t opt, const float* d_m, const float* d_v,
                               void* stream) {
  if (!opt) return refuse("handle is NULL");
  if (opt->blocks == 0) return SLA_OK;
  if (!d_m || !d_v) return refuse("m and v must be non-NULL arrays");
  if (!aligned(d_m, 16) || !aligned(d_v, 16)) return refuse("m and v must be 16-byte aligned");
  hipStream_t s = (hipStream_t)stream;
  return in_launches(opt->blocks, [&](int64_t blk0, dim3 grid) {
    if (opt->bits == 32) {
      copy4<<<grid, kWG, 0, s>>>(d_m, opt->st.m32, blk0, opt->blocks);
      copy4<<<grid, kWG, 0, s>>>(d_v, opt->st.v32, blk0, opt->blocks);
    } else {
      adamw_write8<<<grid, kWG, 0, s>>>(opt->st, blk0, opt->blocks, d_m, d_v);
    }
  });
}

}  // extern "C"
