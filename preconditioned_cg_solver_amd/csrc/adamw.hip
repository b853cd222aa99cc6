// AdamW over many tensors in one launch, with states in 32 or in 8 bits.
//
// Work is cut into blocks of 256 elements, one wave64 each (four consecutive
// elements per lane); in 8 bits a block is also what shares a base.  A
// device table, written when the handle is created, lists the tensors and
// the blocks; only the gradients' addresses, which change from step to step,
// travel with the launch as kernel arguments.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "elem.h"
#include "internal.h"

namespace sla {
namespace {

constexpr int kBlock = 256;          // elements per block
constexpr int kPerLane = kBlock / 64;
constexpr int kChunkBlocks = 16;     // blocks per workgroup
// Gradient addresses per launch: with the other arguments they stay within
// the 4 KB that a launch can carry.
constexpr int kGrads = 448;
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
// 32 random bits of element e (place in the padded order).
__device__ __forceinline__ uint32_t noise(uint32_t key, uint64_t e) {
  const uint32_t hi = (uint32_t)(e >> 32);
  return mix((uint32_t)e * 0x9E3779B1u + (key ^ mix(hi) * (hi != 0)));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

// The 8-bit form (see sla.h): patterns of finite magnitudes are below this.
constexpr uint32_t kInf = 0x7f800000u;
constexpr uint32_t kMost = (kInf >> 20) - 1;  // the largest finite level

__device__ __forceinline__ float decode(uint32_t code, uint32_t base, uint32_t bad, float worst) {
  const float v = __uint_as_float((code + base) << 20);
  return code == 0 ? 0.0f : code == bad ? worst : v;
}
__device__ __forceinline__ float decode_v(uint32_t c, uint32_t base) {
  return decode(c, base, kBadV, INFINITY);
}
__device__ __forceinline__ float decode_m(uint32_t c, uint32_t base) {
  return copysignf(decode(c & 127, base, kBadM, NAN), (c & 128) ? -1.0f : 1.0f);
}

// Largest finite pattern of a wave's block, and the base under which every
// value rounded up by less than `up` has a code of at most `top`.
__device__ __forceinline__ uint32_t base_of(const uint32_t (&bits)[kPerLane], int top,
                                            uint32_t up) {
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) mx = max(mx, bits[j] < kInf ? bits[j] : 0);
  mx = wave_max(mx);
  const uint32_t k = min((mx + up) >> 20, kMost);
  return k > (uint32_t)top ? k - (uint32_t)top : 0;
}
__device__ __forceinline__ uint32_t encode_v(uint32_t bits, uint32_t add, uint32_t base) {
  const int c = (int)((bits + add) >> 20) - (int)base;
  return bits == 0 ? 0 : bits >= kInf ? kBadV : (uint32_t)min(max(c, 1), kTopV);
}
__device__ __forceinline__ uint32_t encode_m(uint32_t bits, uint32_t add, uint32_t base) {
  const int c = (int)((bits + add) >> 20) - (int)base;
  return bits == 0 ? 0 : bits >= kInf ? kBadM : (uint32_t)min(max(c, 0), kTopM);
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

// A bf16 parameter's new value, rounded up with the probability of its
// remainder (16 random bits).
__device__ __forceinline__ bf16_t round_bf16(float x, uint32_t r16) {
  uint32_t u = __float_as_uint(x);
  if ((u & kInf) != kInf) u += r16;
  else if (u & 0x7fffff) u |= 0x400000;  // a NaN stays one without its low bits
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

template <int KIND, int BITS>
__global__ __launch_bounds__(kWG) void adamw_step(Step q, Grads grads) {
  using P = typename Types<KIND>::P;
  using G = typename Types<KIND>::G;
  const float scale = q.scale ? *q.scale : 1.0f;
  if (!(fabsf(scale) < INFINITY)) return;
  const Chunk ch = q.chunks[blockIdx.x];
  const G* gr = (const G*)grads.g[ch.tensor - q.tensor0];
  if (!gr) return;
  const Tensor t = q.tensors[ch.tensor];
  P* p = (P*)t.p;
  bf16_t* copy = (bf16_t*)t.copy;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int b = wave; b < kChunkBlocks; b += kWaves) {
    const int64_t blk = (int64_t)ch.first * kChunkBlocks + b;
    const int64_t e0 = blk * kBlock;
    if (e0 >= t.numel) break;
    const int64_t at = (t.block0 + blk) * kBlock + kPerLane * lane;  // in the states
    float m[kPerLane], v[kPerLane];
    if constexpr (BITS == 32) {
      const auto pm = *(const Pack<float, 4>*)(q.st.m32 + at);
      const auto pv = *(const Pack<float, 4>*)(q.st.v32 + at);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) m[j] = pm.v[j], v[j] = pv.v[j];
    } else {
      const auto pm = *(const Pack<uint8_t, 4>*)(q.st.m8 + at);
      const auto pv = *(const Pack<uint8_t, 4>*)(q.st.v8 + at);
      const uint32_t bm = q.st.mbase[t.block0 + blk], bv = q.st.vbase[t.block0 + blk];
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) m[j] = decode_m(pm.v[j], bm), v[j] = decode_v(pv.v[j], bv);
    }
    uint32_t rnd[kPerLane] = {};
    uint32_t mb[kPerLane], vb[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int64_t i = e0 + kPerLane * lane + j;
      const bool in = i < t.numel;
      if (BITS == 8 || KIND == K_BF16) rnd[j] = noise(q.key, (uint64_t)(at + j));
      float g = 0.0f;
      if (in) {
        if constexpr (KIND == K_F64) g = (float)(q.scale ? gr[i] * (double)scale : gr[i]);
        else g = q.scale ? (float)gr[i] * scale : (float)gr[i];
      }
      moments(q, g, m[j], v[j]);
      if (!in) m[j] = v[j] = 0.0f;
      if (in) {
        const float up = m[j] / (sqrtf(v[j]) * q.root + q.eps) * q.rate;
        if constexpr (KIND == K_F64) {
          p[i] = p[i] * q.decay64 - (double)up;
        } else if constexpr (KIND == K_BF16) {
          p[i] = round_bf16((float)p[i] * q.decay - up, mix(rnd[j] + 0x6A09E667u) & 0xffff);
        } else {
          const float np = p[i] * q.decay - up;
          p[i] = np;
          if (copy) copy[i] = (bf16_t)np;
        }
      }
      mb[j] = magnitude(m[j]);
      vb[j] = magnitude(v[j]);
    }
    if constexpr (BITS == 32) {
      Pack<float, 4> pm, pv;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) pm.v[j] = m[j], pv.v[j] = v[j];
      *(Pack<float, 4>*)(q.st.m32 + at) = pm;
      *(Pack<float, 4>*)(q.st.v32 + at) = pv;
    } else {
      const uint32_t bm = base_of(mb, kTopM, 0xfffff), bv = base_of(vb, kTopV, 0xfffff);
      Pack<uint8_t, 4> pm, pv;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        const uint32_t cm = encode_m(mb[j], ((rnd[j] & 0xffff) << 4) + 8, bm);
        pm.v[j] = (uint8_t)(cm | (m[j] < 0.0f ? 128u : 0u));
        pv.v[j] = (uint8_t)encode_v(vb[j], ((rnd[j] >> 16) << 4) + 8, bv);
      }
      *(Pack<uint8_t, 4>*)(q.st.m8 + at) = pm;
      *(Pack<uint8_t, 4>*)(q.st.v8 + at) = pv;
      if (lane == 0) {
        q.st.mbase[t.block0 + blk] = (uint16_t)bm;
        q.st.vbase[t.block0 + blk] = (uint16_t)bv;
      }
    }
  }
}

// The values of 8-bit states: four significant bits, which bf16 holds.
__global__ __launch_bounds__(kWG) void adamw_read8(State st, int64_t blocks, bf16_t* m,
                                                   bf16_t* v) {
  const int64_t blk = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int64_t at = blk * kBlock + kPerLane * (threadIdx.x & 63);
  const auto cm = *(const Pack<uint8_t, 4>*)(st.m8 + at);
  const auto cv = *(const Pack<uint8_t, 4>*)(st.v8 + at);
  const uint32_t bm = st.mbase[blk], bv = st.vbase[blk];
  Pack<bf16_t, 4> om, ov;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    om.v[j] = (bf16_t)decode_m(cm.v[j], bm);
    ov.v[j] = (bf16_t)decode_v(cv.v[j], bv);
  }
  *(Pack<bf16_t, 4>*)(m + at) = om;
  *(Pack<bf16_t, 4>*)(v + at) = ov;
}

// States from values, to the nearest level.
__global__ __launch_bounds__(kWG) void adamw_write8(State st, int64_t blocks, const float* m,
                                                    const float* v) {
  const int64_t blk = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int lane = threadIdx.x & 63;
  const int64_t at = blk * kBlock + kPerLane * lane;
  const auto pm = *(const Pack<float, 4>*)(m + at);
  const auto pv = *(const Pack<float, 4>*)(v + at);
  uint32_t mb[kPerLane], vb[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) mb[j] = magnitude(pm.v[j]), vb[j] = magnitude(pv.v[j]);
  const uint32_t bm = base_of(mb, kTopM, 0x80000), bv = base_of(vb, kTopV, 0x80000);
  Pack<uint8_t, 4> cm, cv;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    cm.v[j] = (uint8_t)(encode_m(mb[j], 0x80000, bm) | (pm.v[j] < 0.0f ? 128u : 0u));
    cv.v[j] = (uint8_t)encode_v(vb[j], 0x80000, bv);
  }
  *(Pack<uint8_t, 4>*)(st.m8 + at) = cm;
  *(Pack<uint8_t, 4>*)(st.v8 + at) = cv;
  if (lane == 0) st.mbase[blk] = (uint16_t)bm, st.vbase[blk] = (uint16_t)bv;
}

// Plain copies between the 32-bit states and the caller's arrays.
__global__ __launch_bounds__(kWG) void copy4(const float* a, float* b, int64_t quads) {
  const int64_t i = (int64_t)blockIdx.x * kWG + threadIdx.x;
  if (i < quads) ((Pack<float, 4>*)b)[i] = ((const Pack<float, 4>*)a)[i];
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

// One launch of a kind: a range of its tensors (kGrads at most) and of its
// chunks.
struct Launch {
  int kind;
  int32_t tensor0, tensors;
  int64_t chunk0, chunks;
};

}  // namespace
}  // namespace sla

struct sla_adamw {
  int32_t n = 0, bits = 32;
  int64_t blocks = 0;
  const sla::Tensor* d_tensors = nullptr;  // sorted by kind
  const sla::Chunk* d_chunks = nullptr;
  sla::State st = {};
  int32_t kind0[sla::K_KINDS] = {};        // first tensor of each kind
  std::vector<int32_t> order;              // caller's index of each
  std::vector<size_t> align;               // of its gradient
  std::vector<sla::Launch> launches;
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
  int64_t blocks = 0;
  for (int32_t i = 0; i < o->n; ++i) {
    block0[i] = blocks;
    blocks += (ts[i].numel + kBlock - 1) / kBlock;
  }
  o->blocks = blocks;
  int64_t nc = 0;
  for (int kind = 0; kind < K_KINDS; ++kind) {
    o->kind0[kind] = (int32_t)o->order.size();
    for (int32_t i = 0; i < o->n; ++i) {
      if (kind_of(ts[i]) != kind || ts[i].numel == 0) continue;
      const int32_t pos = (int32_t)o->order.size(), local = pos - o->kind0[kind];
      if (local % kGrads == 0) o->launches.push_back({kind, local, 0, nc, 0});
      Launch& l = o->launches.back();
      o->order.push_back(i);
      o->align.push_back(dtype_bytes(ts[i].grad_dtype));
      ht[pos] = {ts[i].d_param, ts[i].d_copy, ts[i].numel, block0[i]};
      const int64_t nb = (ts[i].numel + kBlock - 1) / kBlock;
      for (int64_t b = 0; b < nb; b += kChunkBlocks)
        hc[nc++] = {local, (int32_t)(b / kChunkBlocks)};
      l.tensors = local - l.tensor0 + 1;
      l.chunks = nc - l.chunk0;
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

template <int BITS>
void launch(const Launch& l, const Step& q, const Grads& g, hipStream_t s) {
  const dim3 grid((unsigned)l.chunks);
  switch (l.kind) {
    case K_F32: adamw_step<K_F32, BITS><<<grid, kWG, 0, s>>>(q, g); break;
    case K_F32_BF16: adamw_step<K_F32_BF16, BITS><<<grid, kWG, 0, s>>>(q, g); break;
    case K_BF16: adamw_step<K_BF16, BITS><<<grid, kWG, 0, s>>>(q, g); break;
    default: adamw_step<K_F64, BITS><<<grid, kWG, 0, s>>>(q, g); break;
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
    if (opt->bits == 32) launch<32>(l, q, g, (hipStream_t)stream);
    else launch<8>(l, q, g, (hipStream_t)stream);
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
  if (opt->bits == 32) {
    const int64_t quads = opt->blocks * (kBlock / 4);
    const dim3 grid((unsigned)((quads + kWG - 1) / kWG));
    copy4<<<grid, kWG, 0, s>>>(opt->st.m32, (float*)d_m, quads);
    copy4<<<grid, kWG, 0, s>>>(opt->st.v32, (float*)d_v, quads);
  } else {
    adamw_read8<<<dim3((unsigned)((opt->blocks + kWaves - 1) / kWaves)), kWG, 0, s>>>(
        opt->st, opt->blocks, (bf16_t*)d_m, (bf16_t*)d_v);
  }
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}

sla_status sla_adamw_set_state(sla_adamw_t opt, const float* d_m, const float* d_v,
                               void* stream) {
  if (!opt) return refuse("handle is NULL");
  if (opt->blocks == 0) return SLA_OK;
  if (!d_m || !d_v) return refuse("m and v must be non-NULL arrays");
  if (!aligned(d_m, 16) || !aligned(d_v, 16)) return refuse("m and v must be 16-byte aligned");
  hipStream_t s = (hipStream_t)stream;
  if (opt->bits == 32) {
    const int64_t quads = opt->blocks * (kBlock / 4);
    const dim3 grid((unsigned)((quads + kWG - 1) / kWG));
    copy4<<<grid, kWG, 0, s>>>(d_m, opt->st.m32, quads);
    copy4<<<grid, kWG, 0, s>>>(d_v, opt->st.v32, quads);
  } else {
    adamw_write8<<<dim3((unsigned)((opt->blocks + kWaves - 1) / kWaves)), kWG, 0, s>>>(
        opt->st, opt->blocks, d_m, d_v);
  }
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}

}  // extern "C"
