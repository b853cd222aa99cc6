// Short causal convolutions along a sequence, per channel, and their adjoint.
//
// Bytes: x in and y out; x and dL/dy in and dL/dx out.  8 x 2048 x 2048 bf16 forward 26 us
// (5.2 TB/s, bound by them), backward 54 us (3.7 TB/s, the vector unit at work 65% of them).
// A thread has V neighbouring channels and walks a run of steps with the last
// inputs in registers, so each is read once but for the few before a run; the
// loads of a group of steps are on their way together.  Backward it also carries the
// unfinished sums of dL/dx, and works pre and its slope out again.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "rowsum.h"

namespace sla {
namespace {

constexpr int kLanes = 64;

template <typename T>
struct ConvArgs {
  using C = typename Compute<T>::type;
  const T *x, *state, *grad_y, *grad_last;
  int64_t x_seq, x_step, gy_seq, gy_step;
  const C *weight, *bias;
  T *y, *last, *grad_x, *grad_state;
  C* part;  // [workgroup row][tap, then bias][channel]
  const int64_t* offsets;
  int64_t n_seq, steps, dim;
  int64_t before;  // workgroups of earlier launches of the call
  int blocks;      // of 64 lanes' channels
  int side;        // waves of a workgroup that stand side by side in the channels
  int groups;      // workgroups side by side
  int run;         // steps of a thread
  int64_t runs;    // of a sequence (packed: of all)
  int64_t all;     // runs of the call
  bool silu;
  bool inlined;    // whoever walks a sequence's last step writes its last state
};

// The sequence that a step is in.
struct Seq {
  int64_t s, begin, end;
};
template <typename T>
__device__ __forceinline__ Seq seq_at(const ConvArgs<T>& p, int64_t dense, int64_t t) {
  if (!p.offsets) return {dense, 0, p.steps};
  const int64_t s = sequence_of(p.offsets, p.n_seq, t);
  return {s, p.offsets[s], p.offsets[s + 1]};
}

// The same for a step behind sequence q: mostly one of the next few.
template <typename T>
__device__ __forceinline__ Seq seq_after(const ConvArgs<T>& p, const Seq& q, int64_t t) {
  int64_t s = q.s;
  for (int i = 0; i < 4; ++i) {
    if (s + 1 >= p.n_seq || p.offsets[s + 1] > t) return {s, p.offsets[s], p.offsets[s + 1]};
    ++s;
  }
  return seq_at(p, 0, t);
}

// A thread's run of steps, from `from` to `to`; t0 <= t < t1 of them are of sequences (packed
// rows before the first and behind the last are of none).
struct Run {
  int64_t dense, t0, t1, at, col, from, to, hi;
  bool some;
};
template <int V, typename T>
__device__ __forceinline__ Run run_of(const ConvArgs<T>& p) {
  const int64_t k = p.before + blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t run = k / p.groups * (kWaves / p.side) + wave / p.side;
  Run r;
  r.col = ((k % p.groups * p.side + wave % p.side) * kLanes + (threadIdx.x & 63)) * V;
  r.some = run < p.all && r.col < p.dim;
  r.dense = p.offsets ? 0 : run / p.runs;
  r.from = (run - r.dense * p.runs) * p.run;
  r.to = min(r.from + p.run, p.steps);
  const int64_t lo = p.offsets ? row_at(p.offsets[0], 0, p.steps) : 0;
  r.hi = p.offsets ? row_at(p.offsets[p.n_seq], lo, p.steps) : p.steps;
  r.t0 = max(r.from, lo);
  r.t1 = min(r.to, r.hi);
  r.at = p.offsets ? 0 : r.dense * p.steps;
  return r;
}

// The input at time t of a sequence, or what its state holds there.
template <int K, int V, typename T>
__device__ __forceinline__ Pack<T, V> input_at(const ConvArgs<T>& p, const T* x, const Seq& q,
                                               int64_t t, int64_t col) {
  Pack<T, V> r{};
  if (t >= q.begin) {
    if (t >= 0) r = *(const Pack<T, V>*)(x + t * p.x_step);
  } else if (p.state) {
    r = *(const Pack<T, V>*)(p.state + (q.s * (K - 1) + state_at(t, q.begin, K)) * p.dim + col);
  }
  return r;
}

template <typename T, int K, int V, bool STREAM>
__global__ __launch_bounds__(kWG) void conv_forward(ConvArgs<T> p) {
  using C = typename Compute<T>::type;
  constexpr int U = 8;
  const Run r = run_of<V>(p);
  if (!r.some || r.t0 >= r.t1) return;
  C w[K][V], bias[V], past[K - 1][V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][v] = p.weight[(r.col + v) * K + k];
    bias[v] = p.bias ? p.bias[r.col + v] : C(0);
  }
  Seq q = seq_at(p, r.dense, r.t0);
  const T* const x = p.x + r.dense * p.x_seq + r.col;
  T* const y = p.y + r.at * p.dim + r.col;
  auto settle_past = [&] {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) settle(past[j]);
  };
#pragma unroll
  for (int k = 0; k < K; ++k) settle(w[k]);
  settle(bias);
  auto look_back = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const auto o = input_at<K, V>(p, x, q, t - (K - 1) + j, r.col);
#pragma unroll
      for (int v = 0; v < V; ++v) past[j][v] = (C)o.v[v];
    }
  };
  Pack<T, V> in[U], ahead[U];
  const T* from = x + r.t0 * p.x_step;
  auto fetch = [&](int left) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      ahead[i] = get_pack<STREAM, V>(from + min(i, left - 1) * p.x_step);
    from += U * p.x_step;
  };
  int left = (int)(r.t1 - r.t0);  // steps
  fetch(left);
  look_back(r.t0);
  settle_past();
  T* to = y + r.t0 * p.dim;
  for (int64_t t = r.t0; left > 0; t += U, left -= U) {
#pragma unroll
    for (int i = 0; i < U; ++i) in[i] = ahead[i];
    if (left > U) fetch(left - U);
    auto step = [&](const Pack<T, V>& x_in) {
      C pre[V];
      Pack<T, V> o;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const C now = (C)x_in.v[v];
        pre[v] = bias[v];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) pre[v] += w[k][v] * past[k][v];
        pre[v] += w[K - 1][v] * now;
#pragma unroll
        for (int k = 0; k + 1 < K - 1; ++k) past[k][v] = past[k + 1][v];
        past[K - 2][v] = now;
      }
      if (p.silu)
#pragma unroll
        for (int v = 0; v < V; ++v) pre[v] = silu(pre[v]);
#pragma unroll
      for (int v = 0; v < V; ++v) o.v[v] = (T)pre[v];
      *(Pack<T, V>*)to = o;
      to += p.dim;
    };
    if (left >= U && (!p.offsets || t + U <= q.end)) {
#pragma unroll
      for (int i = 0; i < U; ++i) step(in[i]);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (i >= left) break;
        if (p.offsets && t + i == q.end) {
          q = seq_after(p, q, t + i);
          look_back(t + i);
          settle_past();
        }
        step(in[i]);
      }
    }
  }
  if (p.inlined && p.last && r.t1 == p.steps) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Pack<T, V> o;
#pragma unroll
      for (int v = 0; v < V; ++v) o.v[v] = (T)past[j][v];
      *(Pack<T, V>*)(p.last + (r.dense * (K - 1) + j) * p.dim + r.col) = o;
    }
  }
}

// Zeros in the rows before the first sequence and behind the last: a call without such
// rows reads two offsets.
template <typename W>
__global__ __launch_bounds__(kWG) void clear_rows(const int64_t* offsets, int64_t n_seq,
                                                  int64_t steps, int64_t dim, W* y) {
  const int64_t lo = row_at(offsets[0], 0, steps), hi = row_at(offsets[n_seq], lo, steps);
  const int64_t all = (lo + steps - hi) * dim;
  for (int64_t i = (int64_t)blockIdx.x * kWG + threadIdx.x; i < all; i += (int64_t)gridDim.x * kWG)
    y[i < lo * dim ? i : i + (hi - lo) * dim] = W(0);
}

// The last states of all sequences; backward (BACK) the gradients of the states of
// those without steps, which are the last states'.
template <typename T, int K, int V, bool BACK>
__global__ __launch_bounds__(kWG) void conv_last(ConvArgs<T> p) {
  const int64_t per = p.dim / V, k = (p.before + blockIdx.x) * kWG + threadIdx.x;
  if (k >= p.n_seq * per) return;
  Seq q{k / per, 0, p.steps};
  const int64_t col = k % per * V;
  if (p.offsets) {
    q.begin = row_at(p.offsets[q.s], 0, p.steps);
    q.end = row_at(p.offsets[q.s + 1], q.begin, p.steps);
  }
  const T* const x = p.x + (p.offsets ? 0 : q.s * p.x_seq) + col;
  Pack<T, V> o[K - 1];
  if constexpr (BACK) {
    if (q.begin != q.end) return;
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      o[j] = p.grad_last
                 ? *(const Pack<T, V>*)(p.grad_last + (q.s * (K - 1) + j) * p.dim + col)
                 : Pack<T, V>{};
  } else {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) o[j] = input_at<K, V>(p, x, q, q.end - (K - 1) + j, col);
  }
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    *(Pack<T, V>*)((BACK ? p.grad_state : p.last) + (q.s * (K - 1) + j) * p.dim + col) = o[j];
}

template <typename T, int K, int V, bool STREAM>
__global__ __launch_bounds__(kWG) void conv_backward(ConvArgs<T> p) {
  using C = typename Compute<T>::type;
  constexpr int U = V == 1 ? 8 : 4;
  __shared__ C red[kWaves - 1][kLanes * V];
  const Run r = run_of<V>(p);
  C dw[K + 1][V];  // the bias's last
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = C(0);
  if (r.some && r.t0 < r.t1) {
    C w[K][V], bias[V], past[K - 1][V], sum[K][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][v] = p.weight[(r.col + v) * K + k], sum[k][v] = C(0);
      bias[v] = p.bias ? p.bias[r.col + v] : C(0);
    }
    Seq q = seq_at(p, r.dense, r.t0);
    const T* const x = p.x + r.dense * p.x_seq + r.col;
    const T* const gy = p.grad_y ? p.grad_y + r.dense * p.gy_seq + r.col : nullptr;
    T* const gx = p.grad_x + r.at * p.dim + r.col;
    auto settle_past = [&] {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) settle(past[j]);
    };
#pragma unroll
    for (int k = 0; k < K; ++k) settle(w[k]);
    settle(bias);
    auto look_back = [&](int64_t t) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const auto o = input_at<K, V>(p, x, q, t - (K - 1) + j, r.col);
#pragma unroll
        for (int v = 0; v < V; ++v) past[j][v] = (C)o.v[v];
      }
    };
    // The gradient at time t of sequence q, if this thread is the one to write it: its
    // run holds the step, or for the state the sequence's first.
    auto emit = [&](int64_t t, const C (&g)[V]) {
      T* to;
      if (t >= q.begin) {
        if (t < r.t0 || t >= r.t1) return;
        to = gx + t * p.dim;
      } else {
        const int64_t j = t - q.begin + K - 1;
        if (!p.grad_state || q.begin < r.t0 || q.begin >= r.t1 || j < 0) return;
        to = p.grad_state + (q.s * (K - 1) + j) * p.dim + r.col;
      }
      Pack<T, V> o;
#pragma unroll
      for (int v = 0; v < V; ++v) o.v[v] = (T)g[v];
      *(Pack<T, V>*)to = o;
    };
    // what is left at the end of a sequence
    auto finish = [&]() {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        if (p.grad_last) {
          const auto o =
              *(const Pack<T, V>*)(p.grad_last + (q.s * (K - 1) + j) * p.dim + r.col);
#pragma unroll
          for (int v = 0; v < V; ++v) sum[j][v] += (C)o.v[v];
        }
        emit(q.end - (K - 1) + j, sum[j]);
      }
    };
    const int64_t stop = min(r.t1 + K - 1, r.hi);
    Pack<T, V> in[U], up[U], in_ahead[U], up_ahead[U];
    const T *from = x + r.t0 * p.x_step, *gfrom = gy ? gy + r.t0 * p.gy_step : nullptr;
    auto fetch = [&](int left) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        in_ahead[i] = get_pack<STREAM, V>(from + min(i, left - 1) * p.x_step);
      from += U * p.x_step;
      if (!p.grad_y) return;
#pragma unroll
      for (int i = 0; i < U; ++i)
        up_ahead[i] = get_pack<STREAM, V>(gfrom + min(i, left - 1) * p.gy_step);
      gfrom += U * p.gy_step;
    };
#pragma unroll
    for (int i = 0; i < U; ++i) up_ahead[i] = Pack<T, V>{};
    int left = (int)(stop - r.t0);
    fetch(left);
    look_back(r.t0);
    settle_past();
    bool done = false;
    for (int64_t t = r.t0; left > 0 && !done; t += U, left -= U) {
#pragma unroll
      for (int i = 0; i < U; ++i) in[i] = in_ahead[i], up[i] = up_ahead[i];
      if (left > U) fetch(left - U);
      // A step; what it completes is the gradient of the input K - 1 steps before.
      auto step = [&](const Pack<T, V>& x_in, const Pack<T, V>& g_in, bool own) {
        C pre[V], g[V], now[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          now[v] = (C)x_in.v[v], g[v] = (C)g_in.v[v], pre[v] = bias[v];
#pragma unroll
          for (int k = 0; k < K - 1; ++k) pre[v] += w[k][v] * past[k][v];
          pre[v] += w[K - 1][v] * now[v];
        }
        if (p.silu)
#pragma unroll
          for (int v = 0; v < V; ++v) g[v] *= silu_slope(pre[v], sigmoid(pre[v]));
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int k = 0; k < K; ++k) sum[k][v] += w[k][v] * g[v];
        if (own)
#pragma unroll
          for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) dw[k][v] += g[v] * past[k][v];
            dw[K - 1][v] += g[v] * now[v];
            dw[K][v] += g[v];
          }
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int k = 0; k + 1 < K - 1; ++k) past[k][v] = past[k + 1][v];
          past[K - 2][v] = now[v];
        }
      };
      auto shift = [&] {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int v = 0; v < V; ++v) sum[k][v] = k + 1 < K ? sum[k + 1 < K ? k + 1 : k][v] : C(0);
      };
      if (t + U <= r.t1 && (!p.offsets || t + U <= q.end) && t - (K - 1) >= max(r.t0, q.begin)) {
        // a group in the middle of the run and of a sequence
        T* to = gx + (t - (K - 1)) * p.dim;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          step(in[i], up[i], true);
          Pack<T, V> o;
#pragma unroll
          for (int v = 0; v < V; ++v) o.v[v] = (T)sum[0][v];
          *(Pack<T, V>*)to = o;
          to += p.dim;
          shift();
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t at = t + i;
        if (done || i >= left) break;
        if (p.offsets && at == q.end) {
          finish();
          if (at >= r.t1) {
            done = true;
            break;
          }
          q = seq_after(p, q, at);
          look_back(at);
          settle_past();
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) sum[k][v] = C(0);
        }
        step(in[i], up[i], at < r.t1);
        emit(at - (K - 1), sum[0]);
        shift();
      }
    }
    if (!done && stop == q.end) finish();
  }
  if (p.offsets && r.some) {  // rows of no sequence have gradients of zero
    for (int64_t t = r.from; t < r.to; ++t)
      if (t < r.t0 || t >= r.t1) *(Pack<T, V>*)(p.grad_x + t * p.dim + r.col) = Pack<T, V>{};
  }
  // over the workgroup's runs, and one row of parts for it
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  C* const to = p.part + (p.before + blockIdx.x) / p.groups * (K + 1) * p.dim + r.col;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    if (wave >= p.side)
#pragma unroll
      for (int v = 0; v < V; ++v) red[wave - 1][v * kLanes + lane] = dw[k][v];
    __syncthreads();
    if (wave < p.side && r.col < p.dim) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        C s = dw[k][v];
        for (int o = wave + p.side; o < kWaves; o += p.side) s += red[o - 1][v * kLanes + lane];
        to[k * p.dim + v] = s;
      }
    }
    __syncthreads();
  }
}

// The parts of the weights' gradients summed: 64 channels of a tap a workgroup,
// the waves taking a part of the rows each.
template <typename C>
__global__ __launch_bounds__(kSumWaves * 64) void conv_sum(const C* part, int64_t rows,
                                                           int64_t dim, int width, C* grad_w,
                                                           C* grad_b) {
  __shared__ C red[kSumWaves][kLanes];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t col = (int64_t)blockIdx.x * kLanes + lane;
  const int k = blockIdx.y;
  const int64_t each = (rows + kSumWaves - 1) / kSumWaves;
  const int64_t r0 = wave * each, r1 = min(r0 + each, rows);
  const int64_t step = (width + 1) * dim;
  C s = C(0);
  if (col < dim) {
    const C* const from = part + k * dim + col;
#pragma unroll 8
    for (int64_t r = r0; r < r1; ++r) s += from[r * step];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave || col >= dim) return;
#pragma unroll
  for (int o = 1; o < kSumWaves; ++o) s += red[o][lane];
  if (k < width) grad_w[col * width + k] = s;
  else if (grad_b) grad_b[col] = s;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

sla_status refuse(const char* msg) {
  set_error(msg);
  return SLA_ERR_INVALID_ARG;
}

sla_status check_shape(const sla_conv_shape* q) {
  if (!q) return refuse("shape is NULL");
  if (q->n_seq < 0 || q->steps < 0 || q->dim < 0) return refuse("negative size");
  if (q->dtype != SLA_F64 && q->dtype != SLA_F32 && q->dtype != SLA_BF16 && q->dtype != SLA_F16)
    return refuse("unknown dtype");
  if (q->act != SLA_ACT_NONE && q->act != SLA_ACT_SILU) return refuse("unknown activation");
  if (q->width < 2 || q->width > 4) {
    set_error("a convolution has 2 to 4 taps");
    return SLA_ERR_UNSUPPORTED;
  }
  if (q->n_seq >= INT32_MAX || q->dim >= (1 << 26) || q->steps >= ((int64_t)1 << 40) ||
      (__int128)(q->d_offsets ? 1 : q->n_seq) * (q->steps + 64) * (q->dim + 64) >=
          ((__int128)1 << 58) ||
      (__int128)q->n_seq * q->dim >= ((__int128)1 << 58)) {
    set_error("sizes beyond what a call can index");
    return SLA_ERR_UNSUPPORTED;
  }
  return SLA_OK;
}

bool empty(const sla_conv_shape& q) { return q.n_seq == 0 || q.dim == 0; }

// Channels of a thread: what 8 bytes hold.
template <typename T>
constexpr int most_v() {
  return std::max(1, 8 / (int)sizeof(T));
}

struct Cut {
  int run;
  int64_t runs, all, rows;
  int blocks, side, groups;
};
Cut cut_of(const sla_conv_shape& q, int v, bool backward) {
  Cut c;
  c.blocks = (int)((q.dim + kLanes * v - 1) / (kLanes * v));
  const int64_t seqs = q.d_offsets ? 1 : q.n_seq;
  // Waves that fill the device a few times over, of runs that look back seldom.  8 x 2048 x
  // 2048 bf16, us, by the waves that are wanted: forward 2048 28.7, 4096 26.9, 8192 28.9;
  // backward 1024 69, 2048 54, 4096 61, 8192 75.  Longer runs make fewer parts of the weights'
  // gradients, shorter ones hide more of memory's latency: backward with runs of 64, 128
  // and 256 steps 8 x 4096 x 4096 bf16 200, 180, 165, 50003 x 768 fp32 103, 116, 112.
  const int64_t want = std::max<int64_t>(1, (backward ? 2048 : 4096) / (c.blocks * seqs));
  const int64_t run = (q.steps + want - 1) / want;
  const int64_t most = backward && v >= 4 ? 256 : 64;
  c.run = (int)std::min(std::max<int64_t>((run + 7) / 8 * 8, 8), most);
  c.runs = (q.steps + c.run - 1) / c.run;
  c.all = c.runs * seqs;
  // Waves stand side by side until they reach 512 bytes of a row (backward 1024), so that
  // lines which two waves share are written together.  Forward, with 1, 2 and 4: 8 x 2048 x
  // 2047 bf16 40, 34, 29 us, 50003 x 777 fp32 90, 83, 88; backward the latter 157, 152, 142.
  const int64_t piece = kLanes * v * (int64_t)dtype_bytes(q.dtype);
  c.side = 1;
  while (c.side < kWaves && c.side < c.blocks && c.side * piece < (backward ? 1024 : 512))
    c.side *= 2;
  c.groups = (c.blocks + c.side - 1) / c.side;
  c.rows = (c.all + kWaves / c.side - 1) / (kWaves / c.side);
  return c;
}

bool packs(const void* p, int64_t seq, int64_t step, size_t bytes, int v, bool one_seq,
           bool one_step) {
  return (uintptr_t)p % (v * bytes) == 0 && (seq % v == 0 || one_seq) &&
         (step % v == 0 || one_step);
}

size_t work_bytes_of(const sla_conv_shape& q) {
  if (empty(q) || q.steps == 0) return 0;
  // whichever number of channels a thread takes
  int64_t rows = 0;
  const int most = q.dtype == SLA_F64 || q.dtype == SLA_F32 ? (q.dtype == SLA_F64 ? 1 : 2) : 4;
  for (int v : {1, most}) rows = std::max(rows, cut_of(q, v, true).rows);
  return align_up((size_t)rows * (q.width + 1) * q.dim * (q.dtype == SLA_F64 ? 8 : 4));
}

// Beyond what the last-level cache holds (256 MB) packs are read past it: forward, 8 x 4096 x
// 4096 bf16 109 -> 100 us, 50003 x 768 fp32 71 -> 61 us; where the rows fit it would cost
// (reads and writes): 8 x 2048 x 2048 bf16 28 -> 30 us.
bool streams_of(const sla_conv_shape& q, bool backward) {
  const double elements = (double)(q.d_offsets ? 1 : q.n_seq) * q.steps * q.dim;
  return (backward ? 3 : 2) * elements * dtype_bytes(q.dtype) >= kMallBytes;
}

template <typename T, typename F>
sla_status in_launches(ConvArgs<T>& p, int64_t groups, F&& launch) {
  constexpr int64_t kMost = ((int64_t)1 << 32) / kWG - 1;
  for (int64_t at = 0; at < groups; at += kMost) {
    p.before = at;
    launch(dim3((unsigned)std::min(groups - at, kMost)));
    SLA_HIP(hipGetLastError());
  }
  return SLA_OK;
}

// Calls f(type, taps, channels of a thread).
template <typename F>
sla_status with_types(const sla_conv_shape& q, F&& f) {
  auto taps = [&](auto t) {
    return q.width == 2   ? f(t, std::integral_constant<int, 2>{})
           : q.width == 3 ? f(t, std::integral_constant<int, 3>{})
                          : f(t, std::integral_constant<int, 4>{});
  };
  switch (q.dtype) {
    case SLA_F64: return taps(double{});
    case SLA_F32: return taps(float{});
    case SLA_BF16: return taps(bf16_t{});
    default: return taps(f16_t{});
  }
}

template <typename T>
ConvArgs<T> args_of(const sla_conv_shape& q, const void* x, int64_t xs, int64_t xt, const void* w,
                    const void* b, const void* state) {
  using C = typename Compute<T>::type;
  ConvArgs<T> p{};
  p.x = (const T*)x, p.x_seq = q.d_offsets ? 0 : xs, p.x_step = xt;
  p.weight = (const C*)w, p.bias = (const C*)b, p.state = (const T*)state;
  p.offsets = q.d_offsets;
  p.n_seq = q.n_seq, p.steps = q.steps, p.dim = q.dim;
  p.silu = q.act == SLA_ACT_SILU;
  return p;
}
template <typename T>
void set_cut(ConvArgs<T>& p, const Cut& c) {
  p.blocks = c.blocks, p.side = c.side, p.groups = c.groups, p.run = c.run, p.runs = c.runs, p.all = c.all;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

sla_status sla_conv_sizes(const sla_conv_shape* shape, size_t* work_bytes) {
  const sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (!work_bytes) return refuse("NULL result");
  *work_bytes = work_bytes_of(*shape);
  return SLA_OK;
}

sla_status sla_rows_clear(const int64_t* d_offsets, int64_t n_seq, int64_t steps, int64_t dim,
                          sla_dtype dtype, void* d_y, void* stream) {
  if (n_seq < 0 || steps < 0 || dim < 0) return refuse("negative size");
  if (dtype != SLA_F64 && dtype != SLA_F32 && dtype != SLA_BF16 && dtype != SLA_F16)
    return refuse("unknown dtype");
  if ((__int128)steps * dim >= ((__int128)1 << 59)) {
    set_error("sizes beyond what a call can index");
    return SLA_ERR_UNSUPPORTED;
  }
  if (steps == 0 || dim == 0) return SLA_OK;
  if (!d_offsets || !d_y) return refuse("offsets or y is NULL");
  TraceRange tr("sla_rows_clear");
  const hipStream_t s = (hipStream_t)stream;
  const unsigned grid = (unsigned)std::min<int64_t>((steps * dim + kWG - 1) / kWG, 1024);
  const auto clear = [&](auto word) {
    using W = decltype(word);
    clear_rows<W><<<grid, kWG, 0, s>>>(d_offsets, n_seq, steps, dim, (W*)d_y);
  };
  if (dtype == SLA_F64) clear(uint64_t());
  else if (dtype == SLA_F32) clear(uint32_t());
  else clear(uint16_t());
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}

sla_status sla_conv_forward(const sla_conv_shape* shape, const void* d_x, int64_t x_seq_stride,
                            int64_t x_step_stride, const void* d_weight, const void* d_bias,
                            const void* d_state, void* d_y, void* d_last, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_conv_shape& q = *shape;
  if (x_seq_stride < 0 || x_step_stride < 0) return refuse("negative stride");
  if (empty(q)) return SLA_OK;
  if (q.steps && (!d_x || !d_weight || !d_y)) return refuse("x, weight or y is NULL");
  if (q.steps && (d_y == d_x || d_y == d_state || d_y == d_last || d_last == d_x))
    return refuse("an output must not be an input");
  TraceRange tr("sla_conv_forward");
  return with_types(q, [&](auto t, auto taps) -> sla_status {
    using T = decltype(t);
    constexpr int K = decltype(taps)::value, M = most_v<T>();
    const hipStream_t s = (hipStream_t)stream;
    ConvArgs<T> p = args_of<T>(q, d_x, x_seq_stride, x_step_stride, d_weight, d_bias, d_state);
    p.y = (T*)d_y, p.last = (T*)d_last;
    const size_t b = sizeof(T);
    // Packs where they leave no lane without channels.  8 x 8192 steps bf16, us, in packs and by
    // elements: 64 channels 12.2 and 7.5 (backward 31.1 and 18.3), 128 13.5 and 10.4 (32.8 and
    // 24.8), 192 14.4 and 14.8 (33.6 and 30.3), 252 15.7 and 16.3 (34.5 and 34.3).
    const bool wide =
        q.dim % M == 0 && q.dim >= kLanes * M &&
        packs(d_x, x_seq_stride, x_step_stride, b, M, q.d_offsets || q.n_seq == 1, q.steps == 1) &&
        packs(d_y, 0, 0, b, M, true, true) && packs(d_state, 0, 0, b, M, true, true) &&
        packs(d_last, 0, 0, b, M, true, true);
    const Cut c = cut_of(q, wide ? M : 1, false);
    set_cut(p, c);
    // A state updated in place is read by a sequence's first run and written by its
    // last: by one thread if they are one, else when all have read it.
    p.inlined = !q.d_offsets && q.steps && (d_last != d_state || c.runs == 1);
    sla_status e = SLA_OK;
    if (q.steps)
      e = in_launches(p, c.rows * c.groups, [&](dim3 grid) {
        if (!wide) conv_forward<T, K, 1, false><<<grid, kWG, 0, s>>>(p);
        else if (streams_of(q, false)) conv_forward<T, K, M, true><<<grid, kWG, 0, s>>>(p);
        else conv_forward<T, K, M, false><<<grid, kWG, 0, s>>>(p);
      });
    if (e != SLA_OK || !d_last || p.inlined) return e;
    return in_launches(p, (q.n_seq * (q.dim / (wide ? M : 1)) + kWG - 1) / kWG, [&](dim3 grid) {
      if (wide) conv_last<T, K, M, false><<<grid, kWG, 0, s>>>(p);
      else conv_last<T, K, 1, false><<<grid, kWG, 0, s>>>(p);
    });
  });
}

sla_status sla_conv_backward(const sla_conv_shape* shape, const void* d_x, int64_t x_seq_stride,
                             int64_t x_step_stride, const void* d_weight, const void* d_bias,
                             const void* d_state, const void* d_grad_y, int64_t grad_seq_stride,
                             int64_t grad_step_stride, const void* d_grad_last, void* d_grad_x,
                             void* d_grad_weight, void* d_grad_bias, void* d_grad_state,
                             void* d_work, size_t work_bytes, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_conv_shape& q = *shape;
  if (x_seq_stride < 0 || x_step_stride < 0 || grad_seq_stride < 0 || grad_step_stride < 0)
    return refuse("negative stride");
  if (q.dim == 0) return SLA_OK;
  if (!d_grad_weight) return refuse("the weight's gradient is NULL");
  const bool work = !empty(q) && q.steps;
  // packed rows without a sequence, whose gradients are zeros
  const bool none = q.d_offsets && !q.n_seq && q.steps;
  if (work && (!d_x || !d_weight)) return refuse("x or weight is NULL");
  if ((work || none) && !d_grad_x) return refuse("grad_x is NULL");
  if (work || none)
    for (const void* a : {d_x, d_state, d_grad_y, d_grad_last})
      if (a && (a == d_grad_x || a == d_grad_state))
        return refuse("a gradient must not be an input");
  if (d_grad_state && d_grad_state == d_grad_x)
    return refuse("the gradients must be distinct arrays");
  const size_t need = work_bytes_of(q);
  if (need && (!d_work || work_bytes < need)) return refuse("workspace too small");
  if ((uintptr_t)d_work & 255) return refuse("the workspace must be 256-byte aligned");
  TraceRange tr("sla_conv_backward");
  if (none && (st = sla_rows_clear(q.d_offsets, 0, q.steps, q.dim, q.dtype, d_grad_x, stream)) !=
                  SLA_OK)
    return st;
  return with_types(q, [&](auto t, auto taps) -> sla_status {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    constexpr int K = decltype(taps)::value, M = most_v<T>();
    const hipStream_t s = (hipStream_t)stream;
    ConvArgs<T> p = args_of<T>(q, d_x, x_seq_stride, x_step_stride, d_weight, d_bias, d_state);
    p.grad_y = (const T*)d_grad_y, p.grad_last = (const T*)d_grad_last;
    p.gy_seq = q.d_offsets ? 0 : grad_seq_stride, p.gy_step = grad_step_stride;
    p.grad_x = (T*)d_grad_x, p.grad_state = (T*)d_grad_state, p.part = (C*)d_work;
    const size_t b = sizeof(T);
    const bool one = q.d_offsets || q.n_seq == 1;
    const bool wide =
        q.dim % M == 0 && q.dim >= kLanes * M &&
        packs(d_x, x_seq_stride, x_step_stride, b, M, one, q.steps == 1) &&
        packs(d_grad_y, grad_seq_stride, grad_step_stride, b, M, one, q.steps == 1) &&
        packs(d_grad_x, 0, 0, b, M, true, true) && packs(d_state, 0, 0, b, M, true, true) &&
        packs(d_grad_last, 0, 0, b, M, true, true) && packs(d_grad_state, 0, 0, b, M, true, true);
    Cut c{};
    sla_status e = SLA_OK;
    if (work) {
      c = cut_of(q, wide ? M : 1, true);
      set_cut(p, c);
      e = in_launches(p, c.rows * c.groups, [&](dim3 grid) {
        if (!wide) conv_backward<T, K, 1, false><<<grid, kWG, 0, s>>>(p);
        else if (streams_of(q, true)) conv_backward<T, K, M, true><<<grid, kWG, 0, s>>>(p);
        else conv_backward<T, K, M, false><<<grid, kWG, 0, s>>>(p);
      });
    }
    if (e == SLA_OK && d_grad_state && q.n_seq && (q.d_offsets || !q.steps))
      e = in_launches(p, (q.n_seq * q.dim + kWG - 1) / kWG, [&](dim3 grid) {
        conv_last<T, K, 1, true><<<grid, kWG, 0, s>>>(p);
      });
    if (e != SLA_OK) return e;
    const dim3 grid((unsigned)((q.dim + kLanes - 1) / kLanes), (unsigned)q.width + 1);
    conv_sum<C><<<grid, kSumWaves * 64, 0, s>>>(p.part, c.rows, q.dim, (int)q.width, (C*)d_grad_weight,
                                     (C*)d_grad_bias);
    SLA_HIP(hipGetLastError());
    return SLA_OK;
  });
}

}  // extern "C"
