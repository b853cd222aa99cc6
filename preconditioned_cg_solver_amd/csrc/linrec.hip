// Gated linear recurrences along a sequence and their adjoint.
//
// Forward substitution of a unit lower bidiagonal system per sequence and
// channel, h_t = a_t h_{t-1} + b_t, and back substitution of its transpose
// for the gradients, lambda_t = dh_t + a_{t+1} lambda_{t+1}.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "elem.h"
#include "internal.h"

namespace sla {
namespace {

// A workgroup takes kChunk consecutive steps of 64 V channels: each of its
// kWaves waves kSub steps, a lane V channels of them.
constexpr int kSub = 32;
constexpr int kChunk = kWaves * kSub;

// The coefficient and the weight of x at one step, 1 / (1 + e^-g) and
// 1 / (1 + e^g), from e = exp(-|g|) so that neither is a difference of
// nearly equal numbers and neither overflows.  `small` is the smaller one;
// the other is 1 - small to half a unit in the last place.
__device__ __forceinline__ float small_of(float g) {
  const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(g));
  const float d = 1.0f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(fmaf(-d, r, 1.0f), r, r);
  return e * r;
}
__device__ __forceinline__ double small_of(double g) {
  const double e = exp(-fabs(g));
  return e / (1.0 + e);
}

// A step's coefficient and weight in one number: the smaller of the two,
// negative where that is the weight (g >= 0).
template <typename C>
__device__ __forceinline__ void unfold(C s, C& a, C& keep) {
  const C m = fabs(s), big = C(1) - m;
  const bool neg = signbit(s);
  a = neg ? big : m;
  keep = neg ? m : big;
}

template <int GATE, typename C>
__device__ __forceinline__ void coefficients(C g, C x, C& a, C& b) {
  if constexpr (GATE == SLA_GATE_SIGMOID) {
    C keep;
    unfold(copysign(small_of(g), -g), a, keep);
    b = keep * x;
  } else {
    a = g;
    b = x;
  }
}

template <typename T>
struct Args {
  using C = typename Compute<T>::type;
  const T* x;
  const T* gate;
  const T* grad_h;
  const C* h0;
  const C* grad_last;
  T* h;
  C* h_last;
  C* saved;      // the state after each chunk
  T* grad_x;
  T* grad_gate;
  C* grad_h0;
  const int64_t* offsets;
  int64_t x_seq, x_step, g_seq, g_step, d_seq, d_step;
  int64_t n_seq, steps, dim;
  int chunks;        // dense: of each sequence
  int blocks;        // channel blocks
  int64_t rows;      // rows of `saved`
  // joining the chunks of a sequence
  int* ticket;
  C* sums;           // [row][channel][2]: a chunk's product of a and its sum from a zero start
  C* ends;           // [row][channel]: what leaves the chunk (forward: h; backward: mu)
  const int* row_seq;  // packed: the sequence of a row
};

// A packed sequence's first row.  Rows offset / kChunk + s are distinct and
// leave each sequence at least ceil(length / kChunk) of them, without any sum
// over the lengths.
__device__ __forceinline__ int64_t first_row(const int64_t* offsets, int64_t steps, int64_t s) {
  return min(max(offsets[s], (int64_t)0), steps) / kChunk + s;
}

// A chunk: its sequence, place and length.
struct Where {
  int64_t s, row;
  int64_t x, g, d, out;  // element offsets of the sequence's first step
  int64_t len;           // of the sequence
  int64_t c, after;      // chunks before and after it
};

// Chunk `row` of a packed sequence or of the dense sequence s.  Whatever the
// offsets hold, the steps lie in [0, p.steps) and 0 <= c.
template <typename T>
__device__ __forceinline__ Where locate(const Args<T>& p, int64_t s, int64_t row) {
  Where w;
  w.s = s;
  w.row = row;
  if (p.offsets) {
    const int64_t o0 = min(max(p.offsets[s], (int64_t)0), p.steps);
    const int64_t o1 = min(max(p.offsets[s + 1], o0), p.steps);
    w.len = o1 - o0;
    w.c = p.row_seq ? max(row - (o0 / kChunk + s), (int64_t)0) : 0;
    w.x = o0 * p.x_step;
    w.g = o0 * p.g_step;
    w.d = o0 * p.d_step;
    w.out = o0 * p.dim;
  } else {
    w.len = p.steps;
    w.c = row - s * p.chunks;
    w.x = s * p.x_seq;
    w.g = s * p.g_seq;
    w.d = s * p.d_seq;
    w.out = s * p.steps * p.dim;
  }
  w.after = max((w.len + kChunk - 1) / kChunk - 1 - w.c, (int64_t)0);
  return w;
}

// Words of `sums` and `ends` that have not been written hold all ones, a NaN
// that no published number is (publish() sees to that), so a word carries its
// own flag and needs no fence.
template <typename C>
using Word = std::conditional_t<sizeof(C) == 8, unsigned long long, unsigned>;
template <typename C>
__device__ __forceinline__ bool written(C v) {
  return __builtin_bit_cast(Word<C>, v) != ~Word<C>(0);
}
template <typename C>
__device__ __forceinline__ void publish(C* to, C v) {
  Word<C> u = __builtin_bit_cast(Word<C>, v);
  if (u == ~Word<C>(0)) u = __builtin_bit_cast(Word<C>, C(NAN));
  __hip_atomic_store((Word<C>*)to, u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename C>
__device__ __forceinline__ C look(const C* at) {
  return __builtin_bit_cast(
      C, __hip_atomic_load((const Word<C>*)at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// What enters a chunk, from the chunks before it (forward: STEP = -1) or
// after it (backward: STEP = 1), `have` of them in the sequence: the nearest
// one whose end is known, carried over the sums of those between.  The sums
// are applied one by one from the far end, as each chunk's own end is
// computed, so the bits do not depend on how far the look went.  K ends are
// tried at once, in one trip to memory.
template <int K, int V, int STEP, typename C>
__device__ __forceinline__ bool try_carry(const C* ends, const C* sums, int64_t dim, int have,
                                          C (&carry)[V]) {
  C e[K][V], a[K][V], m[K][V];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (j < have) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[j][v] = look(ends + STEP * j * dim + v);
        if (j + 1 < K) {
          a[j][v] = look(sums + 2 * (STEP * j * dim + v));
          m[j][v] = look(sums + 2 * (STEP * j * dim + v) + 1);
        }
      }
    }
  }
  bool found = false, open = true;  // open: the sums so far are all known
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (j < have && open && !found) {
      bool known = true, sum = true;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        known = known && written(e[j][v]);
        if (j + 1 < K) sum = sum && written(a[j][v]) && written(m[j][v]);
      }
      if (__all(known)) {
        found = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          C h = e[j][v];
#pragma unroll
          for (int q = j - 1; q >= 0; --q) h = a[q][v] * h + m[q][v];
          carry[v] = h;
        }
      } else if (!__all(sum)) {
        open = false;
      }
    }
  }
  return found;
}

// Every chunk publishes its sums before it waits for anything, and a chunk
// waits only for chunks whose tickets were drawn before its own, by
// workgroups that therefore run already: the wait ends.
template <int V, int STEP, typename C>
__device__ __forceinline__ void wait_carry(const C* ends, const C* sums, int64_t dim, int have,
                                           C (&carry)[V]) {
  if (try_carry<2, V, STEP>(ends, sums, dim, have, carry)) return;
  while (!try_carry<8, V, STEP>(ends, sums, dim, have, carry)) __builtin_amdgcn_s_sleep(1);
}

// Marks every word as not written, zeroes the ticket and finds each row's
// sequence: the last one that begins at or before it.
template <typename C>
__global__ __launch_bounds__(kWG) void rec_begin(Word<C>* sums, int64_t n_sums, Word<C>* ends,
                                                 int64_t n_ends, int* ticket, int* row_seq,
                                                 int64_t rows, const int64_t* offsets,
                                                 int64_t n_seq, int64_t steps) {
  const int64_t i0 = (int64_t)blockIdx.x * kWG + threadIdx.x, n = (int64_t)gridDim.x * kWG;
  if (i0 == 0) *ticket = 0;
  for (int64_t i = i0; i < n_sums; i += n) sums[i] = ~Word<C>(0);
  for (int64_t i = i0; i < n_ends; i += n) ends[i] = ~Word<C>(0);
  if (!row_seq) return;
  for (int64_t r = i0; r < rows; r += n) {
    int64_t lo = 0, hi = n_seq;  // first_row(lo) <= r < first_row(hi)
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (first_row(offsets, steps, mid) <= r) lo = mid;
      else hi = mid;
    }
    row_seq[r] = (int)lo;
  }
}

// This workgroup's chunk and channel block.  CHAIN: by ticket, so that the
// chunks it waits for are under way, all sequences' first chunks first
// (packed: in the order of rows); REVERSE: from the last chunk on.
template <bool CHAIN, bool REVERSE, typename T>
__device__ __forceinline__ Where my_chunk(const Args<T>& p, int& block) {
  if constexpr (!CHAIN) {
    const int64_t s = blockIdx.x / (unsigned)p.blocks;
    block = blockIdx.x % (unsigned)p.blocks;
    return locate(p, s, p.offsets ? 0 : s * p.chunks);
  } else {
    __shared__ int drawn;
    if (threadIdx.x == 0)
      drawn = __hip_atomic_fetch_add(p.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const unsigned k = __builtin_amdgcn_readfirstlane(drawn);
    block = k % (unsigned)p.blocks;
    unsigned r = k / (unsigned)p.blocks;
    if (p.offsets) {
      const int64_t row = REVERSE ? p.rows - 1 - r : r;
      return locate(p, p.row_seq[row], row);
    }
    unsigned c = r / (unsigned)p.n_seq;
    const int64_t s = r % (unsigned)p.n_seq;
    if (REVERSE) c = p.chunks - 1 - c;
    return locate(p, s, s * p.chunks + c);
  }
}

// Rows [0, nv) of kSub, V channels each; rows from nv on are the last one
// again.  `base` is uniform, so the row addresses are scalar.
template <int V, typename T>
__device__ __forceinline__ void load_rows(const T* base, int64_t step, unsigned lane_at, int nv,
                                          Pack<T, V> (&r)[kSub]) {
  if (nv == kSub) {
#pragma unroll
    for (int i = 0; i < kSub; ++i) r[i] = *(const Pack<T, V>*)(base + i * step + lane_at);
  } else {
#pragma unroll
    for (int i = 0; i < kSub; ++i)
      r[i] = *(const Pack<T, V>*)(base + min(i, nv - 1) * step + lane_at);
  }
}

// WAVES: waves along the steps of a chunk (kWaves, or 1 where the whole
// sequence fits one wave's rows; then each wave has its own channels).
template <typename T, int GATE, int V, int WAVES, bool CHAIN>
__global__ __launch_bounds__(kWG, 2) void rec_forward(Args<T> p) {
  using C = typename Compute<T>::type;
  constexpr int kWidth = 64 * V;
  __shared__ C s_a[WAVES][kWidth], s_m[WAVES][kWidth], s_in[kWidth];
  int block;
  const Where w = my_chunk<CHAIN, false>(p, block);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = WAVES == 1 ? 0 : wave;
  const int64_t ch = ((int64_t)block * (kWaves / WAVES) + (WAVES == 1 ? wave : 0)) * kWidth +
                     lane * V;
  const bool act = ch < p.dim;
  const int64_t at = act ? ch : 0;
  const int64_t t0 = w.c * kChunk + part * kSub;
  const int nv = (int)min(max(w.len - t0, (int64_t)0), (int64_t)kSub);

  C a[kSub][V], b[kSub][V];
  if (nv > 0) {
    Pack<T, V> x[kSub], g[kSub];
    load_rows<V>(p.gate + w.g + t0 * p.g_step, p.g_step, (unsigned)at, nv, g);
    load_rows<V>(p.x + w.x + t0 * p.x_step, p.x_step, (unsigned)at, nv, x);
#pragma unroll
    for (int i = 0; i < kSub; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        coefficients<GATE, C>((C)g[i].v[v], (C)x[i].v[v], a[i][v], b[i][v]);
        if (i >= nv) a[i][v] = C(1), b[i][v] = C(0);
      }
  } else {
#pragma unroll
    for (int i = 0; i < kSub; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) a[i][v] = C(1), b[i][v] = C(0);
  }

  C h[V];
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C pa = C(1), pm = C(0);
#pragma unroll
      for (int i = 0; i < kSub; ++i) {
        pm = a[i][v] * pm + b[i][v];
        pa *= a[i][v];
      }
      s_a[wave][lane * V + v] = pa;
      s_m[wave][lane * V + v] = pm;
    }
    __syncthreads();
  }
  if (wave == 0 || WAVES == 1) {
    const int64_t row_at = w.row * p.dim + at;
    C ca[V], cm[V];
    if constexpr (CHAIN) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ca[v] = C(1), cm[v] = C(0);
#pragma unroll
        for (int q = 0; q < WAVES; ++q) {
          cm[v] = s_a[q][lane * V + v] * cm[v] + s_m[q][lane * V + v];
          ca[v] *= s_a[q][lane * V + v];
        }
        if (act) {
          publish(p.sums + 2 * (row_at + v), ca[v]);
          publish(p.sums + 2 * (row_at + v) + 1, cm[v]);
        }
      }
    }
    if (!CHAIN || w.c == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = p.h0 ? p.h0[w.s * p.dim + at + v] : C(0);
    } else {
      wait_carry<V, -1>(p.ends + row_at - p.dim, p.sums + 2 * (row_at - p.dim), p.dim,
                        (int)min(w.c, (int64_t)64), h);
    }
    if constexpr (CHAIN) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (act) publish(p.ends + row_at + v, ca[v] * h[v] + cm[v]);
    }
    if (w.len == 0 && w.c == 0 && act && p.h_last) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_last[w.s * p.dim + at + v] = h[v];
    }
    if constexpr (WAVES > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) s_in[lane * V + v] = h[v];
    }
  }
  if constexpr (WAVES > 1) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = s_in[lane * V + v];
      for (int q = 0; q < wave; ++q)
        h[v] = s_a[q][lane * V + v] * h[v] + s_m[q][lane * V + v];
    }
  }
  if (nv == 0 || !act) return;
  T* out = p.h + w.out + t0 * p.dim;
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    Pack<T, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = a[i][v] * h[v] + b[i][v];
      o.v[v] = (T)h[v];
    }
    if (i < nv) *(Pack<T, V>*)(out + i * p.dim + (unsigned)at) = o;
  }
  // rows past the end leave h as it was
  if (t0 + nv == w.len && p.h_last) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.h_last[w.s * p.dim + at + v] = h[v];
  }
}

template <typename T, int GATE, int V, int WAVES, bool CHAIN>
__global__ __launch_bounds__(kWG, 2) void rec_backward(Args<T> p) {
  using C = typename Compute<T>::type;
  constexpr int kWidth = 64 * V;
  constexpr bool kSig = GATE == SLA_GATE_SIGMOID;
  __shared__ C s_a[WAVES][kWidth], s_m[WAVES][kWidth], s_u[WAVES][kWidth], s_in[kWidth],
      s_mu[kWidth];
  int block;
  const Where w = my_chunk<CHAIN, true>(p, block);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = WAVES == 1 ? 0 : wave;
  const int64_t ch = ((int64_t)block * (kWaves / WAVES) + (WAVES == 1 ? wave : 0)) * kWidth +
                     lane * V;
  const bool act = ch < p.dim;
  const int64_t at = act ? ch : 0;
  const int64_t t0 = w.c * kChunk + part * kSub;
  const int nv = (int)min(max(w.len - t0, (int64_t)0), (int64_t)kSub);

  // f: linear the coefficient, sigmoid coefficient and weight folded into one
  // number.  z: x, later h_{t-1} - x (linear: h_{t-1}).
  C f[kSub][V], z[kSub][V];
  Pack<T, V> d[kSub];
  if (nv > 0) {
    Pack<T, V> x[kSub], g[kSub];
    load_rows<V>(p.gate + w.g + t0 * p.g_step, p.g_step, (unsigned)at, nv, g);
    load_rows<V>(p.x + w.x + t0 * p.x_step, p.x_step, (unsigned)at, nv, x);
    if (p.grad_h) load_rows<V>(p.grad_h + w.d + t0 * p.d_step, p.d_step, (unsigned)at, nv, d);
#pragma unroll
    for (int i = 0; i < kSub; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const C gv = (C)g[i].v[v];
        f[i][v] = kSig ? copysign(small_of(gv), -gv) : gv;
        z[i][v] = (C)x[i].v[v];
        if (i >= nv) f[i][v] = kSig ? C(-0.0) : C(1), z[i][v] = C(0);
        if (i >= nv || !p.grad_h) d[i].v[v] = (T)0.0f;
      }
  } else {
#pragma unroll
    for (int i = 0; i < kSub; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        f[i][v] = kSig ? C(-0.0) : C(1), z[i][v] = C(0), d[i].v[v] = (T)0.0f;
  }
  // Each pass over the steps unfolds f again: held unfolded, the two arrays
  // would not fit the registers, so the compiler is kept from reusing them.
  auto step = [&](C& fv, C& a, C& keep) {
    if constexpr (kSig) {
      asm volatile("" : "+v"(fv));
      unfold(fv, a, keep);
    } else {
      a = fv, keep = C(1);
    }
  };

  C h[V], mu[V];
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C pa = C(1), pm = C(0), pu = C(0), a, keep;
#pragma unroll
      for (int i = 0; i < kSub; ++i) {
        step(f[i][v], a, keep);
        pm = a * pm + (kSig ? keep * z[i][v] : z[i][v]);
        pa *= a;
      }
#pragma unroll
      for (int i = kSub - 1; i >= 0; --i) {
        step(f[i][v], a, keep);
        pu = a * ((C)d[i].v[v] + pu);
      }
      s_a[wave][lane * V + v] = pa;
      s_m[wave][lane * V + v] = pm;
      s_u[wave][lane * V + v] = pu;
    }
    __syncthreads();
  }
  if (wave == 0 || WAVES == 1) {
    const int64_t row_at = w.row * p.dim + at;
    C ca[V], cu[V];
    if constexpr (CHAIN) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ca[v] = C(1), cu[v] = C(0);
#pragma unroll
        for (int q = WAVES - 1; q >= 0; --q) {
          cu[v] = s_a[q][lane * V + v] * cu[v] + s_u[q][lane * V + v];
          ca[v] *= s_a[q][lane * V + v];
        }
        if (act) {
          publish(p.sums + 2 * (row_at + v), ca[v]);
          publish(p.sums + 2 * (row_at + v) + 1, cu[v]);
        }
      }
    }
    if (w.c == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = p.h0 ? p.h0[w.s * p.dim + at + v] : C(0);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = p.saved[row_at - p.dim + v];
    }
    if (!CHAIN || w.after == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) mu[v] = p.grad_last ? p.grad_last[w.s * p.dim + at + v] : C(0);
    } else {
      wait_carry<V, 1>(p.ends + row_at + p.dim, p.sums + 2 * (row_at + p.dim), p.dim,
                       (int)min(w.after, (int64_t)64), mu);
    }
    if constexpr (CHAIN) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (act) publish(p.ends + row_at + v, ca[v] * mu[v] + cu[v]);
    }
    if (w.len == 0 && w.c == 0 && act && p.grad_h0) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.grad_h0[w.s * p.dim + at + v] = mu[v];
    }
    if constexpr (WAVES > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) s_in[lane * V + v] = h[v], s_mu[lane * V + v] = mu[v];
    }
  }
  if constexpr (WAVES > 1) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = s_in[lane * V + v];
      for (int q = 0; q < wave; ++q)
        h[v] = s_a[q][lane * V + v] * h[v] + s_m[q][lane * V + v];
      mu[v] = s_mu[lane * V + v];
      for (int q = WAVES - 1; q > wave; --q)
        mu[v] = s_a[q][lane * V + v] * mu[v] + s_u[q][lane * V + v];
    }
  }
  if (nv == 0 || !act) return;
#pragma unroll
  for (int i = 0; i < kSub; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C a, keep;
      step(f[i][v], a, keep);
      const C before = h[v], x = z[i][v];
      h[v] = a * h[v] + (kSig ? keep * x : x);
      z[i][v] = kSig ? before - x : before;
    }
  T* ox = p.grad_x + w.out + t0 * p.dim;
  T* og = p.grad_gate + w.out + t0 * p.dim;
#pragma unroll
  for (int i = kSub - 1; i >= 0; --i) {
    Pack<T, V> rx, rg;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C a, keep;
      step(f[i][v], a, keep);
      const C lam = (C)d[i].v[v] + mu[v];
      mu[v] = a * lam;
      rx.v[v] = (T)(kSig ? lam * keep : lam);
      rg.v[v] = (T)(kSig ? mu[v] * z[i][v] * keep : lam * z[i][v]);
    }
    if (i < nv) {
      *(Pack<T, V>*)(ox + i * p.dim + (unsigned)at) = rx;
      *(Pack<T, V>*)(og + i * p.dim + (unsigned)at) = rg;
    }
  }
  // mu has passed the first step
  if (t0 == 0 && p.grad_h0) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.grad_h0[w.s * p.dim + at + v] = mu[v];
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

sla_status refuse(const char* msg) {
  set_error(msg);
  return SLA_ERR_INVALID_ARG;
}

// Rows of kept states (see span_of).
int64_t saved_rows(const sla_linrec_shape& q) {
  if (q.d_offsets) return q.steps / kChunk + q.n_seq;
  return q.n_seq * ((q.steps + kChunk - 1) / kChunk);
}

bool empty(const sla_linrec_shape& q) { return q.n_seq == 0 || q.dim == 0; }
bool no_steps(const sla_linrec_shape& q) { return empty(q) || q.steps == 0; }

sla_status check_shape(const sla_linrec_shape* q) {
  if (!q) return refuse("shape is NULL");
  if (q->n_seq < 0 || q->steps < 0 || q->dim < 0) return refuse("negative size");
  if (q->dtype != SLA_F64 && q->dtype != SLA_F32 && q->dtype != SLA_BF16 && q->dtype != SLA_F16)
    return refuse("unknown dtype");
  if (q->gate != SLA_GATE_LINEAR && q->gate != SLA_GATE_SIGMOID) return refuse("unknown gate");
  const int64_t seqs = q->d_offsets ? 1 : q->n_seq;
  if (q->n_seq >= INT32_MAX || q->dim >= INT32_MAX || q->steps >= ((int64_t)1 << 40) ||
      (__int128)(q->steps / kChunk + 1) * q->n_seq >= ((__int128)1 << 60) || (__int128)seqs * q->steps * q->dim >= ((__int128)1 << 60) ||
      (__int128)q->n_seq * q->dim >= ((__int128)1 << 60) ||
      (__int128)(saved_rows(*q) + q->n_seq) * ((q->dim + 63) / 64) >= INT32_MAX) {
    set_error("sizes beyond what one launch can index");
    return SLA_ERR_UNSUPPORTED;
  }
  return SLA_OK;
}

size_t state_bytes(const sla_linrec_shape& q) { return q.dtype == SLA_F64 ? 8 : 4; }

// Calls f with the storage type and the gate of the shape.
template <typename F>
sla_status with_types(const sla_linrec_shape& q, F&& f) {
  auto gate = [&](auto t) {
    return q.gate == SLA_GATE_SIGMOID
               ? f(t, std::integral_constant<int, SLA_GATE_SIGMOID>{})
               : f(t, std::integral_constant<int, SLA_GATE_LINEAR>{});
  };
  switch (q.dtype) {
    case SLA_F64: return gate(double{});
    case SLA_F32: return gate(float{});
    case SLA_BF16: return gate(bf16_t{});
    default: return gate(f16_t{});
  }
}

// Whether no sequence has more than one chunk, whatever the offsets.
bool one_chunk(const sla_linrec_shape& q) { return q.steps <= kChunk; }

// The workspace of a call that joins chunks: the ticket, the rows'
// sequences, the chunks' sums and (always, though the forward call has them
// in d_saved when that is given) their ends.
struct Work {
  size_t rows_at = 0, sums_at = 0, ends_at = 0, bytes = 0;
};
Work work_of(const sla_linrec_shape& q) {
  Work w;
  if (no_steps(q) || one_chunk(q)) return w;
  const size_t words = (size_t)saved_rows(q) * q.dim * state_bytes(q);
  w.rows_at = align_up(sizeof(int));
  w.sums_at = w.rows_at + (q.d_offsets ? align_up((size_t)saved_rows(q) * sizeof(int)) : 0);
  w.ends_at = w.sums_at + align_up(2 * words);
  w.bytes = w.ends_at + align_up(words);
  return w;
}

// Whether two neighbouring 16-bit channels can be moved as one word anywhere.
bool even(int64_t v) { return (v & 1) == 0; }
bool paired(const sla_linrec_shape& q, const void* p, int64_t seq, int64_t step) {
  return ((uintptr_t)p & 3) == 0 && (even(seq) || q.d_offsets || q.n_seq == 1) &&
         (even(step) || q.steps == 1);
}

template <typename T>
Args<T> common_args(const sla_linrec_shape& q, const void* x, int64_t xs, int64_t xt,
                    const void* g, int64_t gs, int64_t gt, const void* h0) {
  using C = typename Compute<T>::type;
  Args<T> p{};
  p.x = (const T*)x;
  p.gate = (const T*)g;
  p.h0 = (const C*)h0;
  p.offsets = q.d_offsets;
  p.x_seq = q.d_offsets ? 0 : xs;
  p.x_step = xt;
  p.g_seq = q.d_offsets ? 0 : gs;
  p.g_step = gt;
  p.n_seq = q.n_seq;
  p.steps = q.steps;
  p.dim = q.dim;
  p.chunks = (int)std::max<int64_t>(1, (q.steps + kChunk - 1) / kChunk);
  p.rows = saved_rows(q);
  return p;
}

// Sets up the chunks' joining and calls launch(integral V, integral WAVES,
// integral CHAIN, grid).
template <typename T, typename F>
sla_status run_chunks(const sla_linrec_shape& q, Args<T>& p, bool pairs, void* work, bool own_ends,
                      hipStream_t s, F&& launch) {
  using C = typename Compute<T>::type;
  const bool chain = !no_steps(q) && !one_chunk(q);
  if (chain) {
    const Work w = work_of(q);
    char* base = (char*)work;
    p.ticket = (int*)base;
    int* row_seq = q.d_offsets ? (int*)(base + w.rows_at) : nullptr;
    p.row_seq = row_seq;
    p.sums = (C*)(base + w.sums_at);
    if (own_ends) p.ends = (C*)(base + w.ends_at);
    const int64_t words = p.rows * p.dim;
    const int64_t want = (2 * words / 4 + kWG - 1) / kWG;
    rec_begin<C><<<dim3((unsigned)std::min<int64_t>(std::max<int64_t>(want, 1), 2048)), kWG, 0, s>>>(
        (Word<C>*)p.sums, 2 * words, (Word<C>*)p.ends, words, p.ticket, row_seq, p.rows,
        q.d_offsets, q.n_seq, q.steps);
    SLA_HIP(hipGetLastError());
  }
  const bool narrow = !chain && q.steps <= kSub;
  auto with_v = [&](auto v) {
    constexpr int V = decltype(v)::value;
    const int64_t per = 64 * V * (narrow ? kWaves : 1);
    p.blocks = (int)((q.dim + per - 1) / per);
    const int64_t rows = !chain ? q.n_seq : q.d_offsets ? p.rows : q.n_seq * p.chunks;
    const dim3 grid((unsigned)(rows * p.blocks));
    using I1 = std::integral_constant<int, 1>;
    using I4 = std::integral_constant<int, kWaves>;
    if (chain) launch(v, I4{}, std::true_type{}, grid);
    else if (narrow) launch(v, I1{}, std::false_type{}, grid);
    else launch(v, I4{}, std::false_type{}, grid);
  };
  if constexpr (sizeof(T) == 2) {
    if (pairs) with_v(std::integral_constant<int, 2>{});
    else with_v(std::integral_constant<int, 1>{});
  } else {
    (void)pairs;
    with_v(std::integral_constant<int, 1>{});
  }
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}

sla_status check_work(const sla_linrec_shape& q, const void* work, size_t bytes) {
  const size_t need = work_of(q).bytes;
  if (need && (!work || bytes < need)) return refuse("workspace too small");
  if ((uintptr_t)work & 255) return refuse("the workspace must be 256-byte aligned");
  return SLA_OK;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

sla_status sla_linrec_sizes(const sla_linrec_shape* shape, size_t* saved_bytes,
                            size_t* work_bytes) {
  const sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (!saved_bytes || !work_bytes) return refuse("NULL result");
  *saved_bytes = no_steps(*shape) ? 0 : (size_t)saved_rows(*shape) * shape->dim * state_bytes(*shape);
  *work_bytes = work_of(*shape).bytes;
  return SLA_OK;
}

sla_status sla_linrec_forward(const sla_linrec_shape* shape, const void* d_x,
                              int64_t x_seq_stride, int64_t x_step_stride, const void* d_gate,
                              int64_t gate_seq_stride, int64_t gate_step_stride,
                              const void* d_h0, void* d_h, void* d_h_last, void* d_saved,
                              void* d_work, size_t work_bytes, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (x_seq_stride < 0 || x_step_stride < 0 || gate_seq_stride < 0 || gate_step_stride < 0)
    return refuse("negative stride");
  if (empty(*shape)) return SLA_OK;
  if (!no_steps(*shape) && (!d_x || !d_gate || !d_h)) return refuse("x, gate or h is NULL");
  if (!no_steps(*shape) && (d_h == d_x || d_h == d_gate))
    return refuse("h must not be an input");
  const sla_linrec_shape& q = *shape;
  if ((st = check_work(q, d_work, work_bytes)) != SLA_OK) return st;
  TraceRange tr("sla_linrec_forward");
  const bool pairs = even(q.dim) && paired(q, d_x, x_seq_stride, x_step_stride) &&
                     paired(q, d_gate, gate_seq_stride, gate_step_stride) && paired(q, d_h, 0, 0);
  return with_types(q, [&](auto t, auto gate) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    constexpr int GATE = decltype(gate)::value;
    Args<T> p = common_args<T>(q, d_x, x_seq_stride, x_step_stride, d_gate, gate_seq_stride,
                               gate_step_stride, d_h0);
    p.h = (T*)d_h;
    p.h_last = (C*)d_h_last;
    p.ends = (C*)d_saved;
    return run_chunks<T>(q, p, pairs, d_work, !d_saved, (hipStream_t)stream,
                         [&](auto v, auto waves, auto chain, dim3 grid) {
                           rec_forward<T, GATE, decltype(v)::value, decltype(waves)::value,
                                       decltype(chain)::value>
                               <<<grid, kWG, 0, (hipStream_t)stream>>>(p);
                         });
  });
}

sla_status sla_linrec_backward(const sla_linrec_shape* shape, const void* d_x,
                               int64_t x_seq_stride, int64_t x_step_stride, const void* d_gate,
                               int64_t gate_seq_stride, int64_t gate_step_stride,
                               const void* d_h0, const void* d_saved, const void* d_grad_h,
                               int64_t grad_seq_stride, int64_t grad_step_stride,
                               const void* d_grad_last, void* d_grad_x, void* d_grad_gate,
                               void* d_grad_h0, void* d_work, size_t work_bytes, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (x_seq_stride < 0 || x_step_stride < 0 || gate_seq_stride < 0 || gate_step_stride < 0 ||
      grad_seq_stride < 0 || grad_step_stride < 0)
    return refuse("negative stride");
  if (empty(*shape)) return SLA_OK;
  if (!no_steps(*shape) && (!d_x || !d_gate || !d_saved || !d_grad_x || !d_grad_gate))
    return refuse("x, gate, the saved states or a gradient is NULL");
  if (!no_steps(*shape)) {
    for (const void* in : {d_x, d_gate, d_grad_h, d_saved})
      if (in && (in == d_grad_x || in == d_grad_gate))
        return refuse("a gradient must not be an input");
    if (d_grad_x == d_grad_gate) return refuse("the gradients must be distinct arrays");
  }
  const sla_linrec_shape& q = *shape;
  if ((st = check_work(q, d_work, work_bytes)) != SLA_OK) return st;
  TraceRange tr("sla_linrec_backward");
  const bool pairs = even(q.dim) && paired(q, d_x, x_seq_stride, x_step_stride) &&
                     paired(q, d_gate, gate_seq_stride, gate_step_stride) &&
                     paired(q, d_grad_h, grad_seq_stride, grad_step_stride) &&
                     paired(q, d_grad_x, 0, 0) && paired(q, d_grad_gate, 0, 0);
  return with_types(q, [&](auto t, auto gate) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    constexpr int GATE = decltype(gate)::value;
    Args<T> p = common_args<T>(q, d_x, x_seq_stride, x_step_stride, d_gate, gate_seq_stride,
                               gate_step_stride, d_h0);
    p.grad_h = (const T*)d_grad_h;
    p.d_seq = q.d_offsets ? 0 : grad_seq_stride;
    p.d_step = grad_step_stride;
    p.grad_last = (const C*)d_grad_last;
    p.saved = (C*)d_saved;
    p.grad_x = (T*)d_grad_x;
    p.grad_gate = (T*)d_grad_gate;
    p.grad_h0 = (C*)d_grad_h0;
    return run_chunks<T>(q, p, pairs, d_work, true, (hipStream_t)stream,
                         [&](auto v, auto waves, auto chain, dim3 grid) {
                           rec_backward<T, GATE, decltype(v)::value, decltype(waves)::value,
                                        decltype(chain)::value>
                               <<<grid, kWG, 0, (hipStream_t)stream>>>(p);
                         });
  });
}

}  // extern "C"
