// Gated linear recurrences along a sequence and their adjoint.
//
// Forward substitution of a unit lower bidiagonal system per sequence and
// channel, h_t = a_t h_{t-1} + b_t, and back substitution of its transpose
// for the gradients, lambda_t = dh_t + a_{t+1} lambda_{t+1}.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "elem.h"
#include "internal.h"

namespace sla {
namespace {

// Steps between two kept states.
constexpr int kChunk = 64;

// The coefficient and the weight of x at one step, 1 / (1 + e^-g) and
// 1 / (1 + e^g), from e = exp(-|g|) so that neither is a difference of
// nearly equal numbers and neither overflows.
template <typename C>
__device__ __forceinline__ void sigmoid2(C g, C& a, C& keep) {
  const C e = exp(-fabs(g));
  const C big = C(1) / (C(1) + e), small = e * big;
  a = g >= C(0) ? big : small;
  keep = g >= C(0) ? small : big;
  if (g != g) a = keep = g;
}

template <int GATE, typename C>
__device__ __forceinline__ void coefficients(C g, C x, C& a, C& keep, C& b) {
  if constexpr (GATE == SLA_GATE_SIGMOID) {
    sigmoid2(g, a, keep);
    b = keep * x;
  } else {
    a = g;
    keep = C(1);
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
  C* saved;
  T* grad_x;
  T* grad_gate;
  C* grad_h0;
  const int64_t* offsets;
  int64_t x_seq, x_step, g_seq, g_step, d_seq, d_step;
  int64_t n_seq, steps, dim;
};

// Where sequence s lies: its steps in the inputs and in the dense outputs,
// and the first of its kept states.  Packed sequences number their states
// from offset / kChunk + s, which leaves each at least ceil(length / kChunk)
// rows without any sum over the lengths.
struct Span {
  int64_t in, out, len, row;
};
template <typename T>
__device__ __forceinline__ Span span_of(const Args<T>& p, int64_t s) {
  Span r;
  if (p.offsets) {
    const int64_t o0 = min(max(p.offsets[s], (int64_t)0), p.steps);
    const int64_t o1 = min(max(p.offsets[s + 1], o0), p.steps);
    r.in = r.out = o0;
    r.len = o1 - o0;
    r.row = o0 / kChunk + s;
  } else {
    r.in = 0;
    r.out = s * p.steps;
    r.len = p.steps;
    r.row = s * ((p.steps + kChunk - 1) / kChunk);
  }
  return r;
}

template <typename T, int GATE>
__global__ __launch_bounds__(kWG) void rec_forward(Args<T> p) {
  using C = typename Compute<T>::type;
  const int nb = (int)((p.dim + kWG - 1) / kWG);
  const int64_t s = blockIdx.x / nb, c = (int64_t)(blockIdx.x % nb) * kWG + threadIdx.x;
  if (c >= p.dim) return;
  const Span sp = span_of(p, s);
  const T* x = p.x + (p.offsets ? sp.in * p.x_step : s * p.x_seq) + c;
  const T* g = p.gate + (p.offsets ? sp.in * p.g_step : s * p.g_seq) + c;
  C h = p.h0 ? p.h0[s * p.dim + c] : C(0);
  for (int64_t t = 0; t < sp.len; ++t) {
    C a, keep, b;
    coefficients<GATE, C>((C)g[t * p.g_step], (C)x[t * p.x_step], a, keep, b);
    h = a * h + b;
    p.h[(sp.out + t) * p.dim + c] = (T)h;
    if (p.saved && (t + 1) % kChunk == 0) p.saved[(sp.row + t / kChunk) * p.dim + c] = h;
  }
  if (p.h_last) p.h_last[s * p.dim + c] = h;
}

template <typename T, int GATE>
__global__ __launch_bounds__(kWG) void rec_backward(Args<T> p) {
  using C = typename Compute<T>::type;
  const int nb = (int)((p.dim + kWG - 1) / kWG);
  const int64_t s = blockIdx.x / nb, c = (int64_t)(blockIdx.x % nb) * kWG + threadIdx.x;
  if (c >= p.dim) return;
  const Span sp = span_of(p, s);
  const T* x = p.x + (p.offsets ? sp.in * p.x_step : s * p.x_seq) + c;
  const T* g = p.gate + (p.offsets ? sp.in * p.g_step : s * p.g_seq) + c;
  const T* d = p.grad_h ? p.grad_h + (p.offsets ? sp.in * p.d_step : s * p.d_seq) + c : nullptr;
  C mu = p.grad_last ? p.grad_last[s * p.dim + c] : C(0);
  C hs[kChunk];  // h_{t-1} of the chunk's steps
  for (int64_t k = (sp.len + kChunk - 1) / kChunk - 1; k >= 0; --k) {
    const int64_t t0 = k * kChunk;
    const int n = (int)min((int64_t)kChunk, sp.len - t0);
    C h = k > 0 ? p.saved[(sp.row + k - 1) * p.dim + c] : p.h0 ? p.h0[s * p.dim + c] : C(0);
    for (int i = 0; i < n; ++i) {
      C a, keep, b;
      hs[i] = h;
      coefficients<GATE, C>((C)g[(t0 + i) * p.g_step], (C)x[(t0 + i) * p.x_step], a, keep, b);
      h = a * h + b;
    }
    for (int i = n - 1; i >= 0; --i) {
      const int64_t t = t0 + i;
      C a, keep, b;
      const C xv = (C)x[t * p.x_step];
      coefficients<GATE, C>((C)g[t * p.g_step], xv, a, keep, b);
      const C lam = (d ? (C)d[t * p.d_step] : C(0)) + mu;
      mu = a * lam;
      C dx = lam, dg = lam * hs[i];
      if constexpr (GATE == SLA_GATE_SIGMOID) {
        dx = lam * keep;
        dg = lam * (hs[i] - xv) * a * keep;
      }
      p.grad_x[(sp.out + t) * p.dim + c] = (T)dx;
      p.grad_gate[(sp.out + t) * p.dim + c] = (T)dg;
    }
  }
  if (p.grad_h0) p.grad_h0[s * p.dim + c] = mu;
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
      (__int128)seqs * q->steps * q->dim >= ((__int128)1 << 60) ||
      (__int128)q->n_seq * q->dim >= ((__int128)1 << 60) ||
      (__int128)(q->steps / kChunk + 1) * q->n_seq * ((q->dim + 63) / 64) >= INT32_MAX) {
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

dim3 simple_grid(const sla_linrec_shape& q) {
  return dim3((unsigned)((q.dim + kWG - 1) / kWG * q.n_seq));
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
  *work_bytes = 0;
  return SLA_OK;
}

sla_status sla_linrec_forward(const sla_linrec_shape* shape, const void* d_x,
                              int64_t x_seq_stride, int64_t x_step_stride, const void* d_gate,
                              int64_t gate_seq_stride, int64_t gate_step_stride,
                              const void* d_h0, void* d_h, void* d_h_last, void* d_saved,
                              void* d_work, size_t work_bytes, void* stream) {
  const sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (x_seq_stride < 0 || x_step_stride < 0 || gate_seq_stride < 0 || gate_step_stride < 0)
    return refuse("negative stride");
  if (empty(*shape)) return SLA_OK;
  if (!no_steps(*shape) && (!d_x || !d_gate || !d_h)) return refuse("x, gate or h is NULL");
  if (!no_steps(*shape) && (d_h == d_x || d_h == d_gate))
    return refuse("h must not be an input");
  (void)d_work;
  (void)work_bytes;
  TraceRange tr("sla_linrec_forward");
  const sla_linrec_shape& q = *shape;
  return with_types(q, [&](auto t, auto gate) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    Args<T> p{};
    p.x = (const T*)d_x;
    p.gate = (const T*)d_gate;
    p.h0 = (const C*)d_h0;
    p.h = (T*)d_h;
    p.h_last = (C*)d_h_last;
    p.saved = (C*)d_saved;
    p.offsets = q.d_offsets;
    p.x_seq = x_seq_stride;
    p.x_step = x_step_stride;
    p.g_seq = gate_seq_stride;
    p.g_step = gate_step_stride;
    p.n_seq = q.n_seq;
    p.steps = q.steps;
    p.dim = q.dim;
    rec_forward<T, decltype(gate)::value><<<simple_grid(q), kWG, 0, (hipStream_t)stream>>>(p);
    SLA_HIP(hipGetLastError());
    return SLA_OK;
  });
}

sla_status sla_linrec_backward(const sla_linrec_shape* shape, const void* d_x,
                               int64_t x_seq_stride, int64_t x_step_stride, const void* d_gate,
                               int64_t gate_seq_stride, int64_t gate_step_stride,
                               const void* d_h0, const void* d_saved, const void* d_grad_h,
                               int64_t grad_seq_stride, int64_t grad_step_stride,
                               const void* d_grad_last, void* d_grad_x, void* d_grad_gate,
                               void* d_grad_h0, void* d_work, size_t work_bytes, void* stream) {
  const sla_status st = check_shape(shape);
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
  (void)d_work;
  (void)work_bytes;
  TraceRange tr("sla_linrec_backward");
  const sla_linrec_shape& q = *shape;
  return with_types(q, [&](auto t, auto gate) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    Args<T> p{};
    p.x = (const T*)d_x;
    p.gate = (const T*)d_gate;
    p.grad_h = (const T*)d_grad_h;
    p.h0 = (const C*)d_h0;
    p.grad_last = (const C*)d_grad_last;
    p.saved = (C*)d_saved;
    p.grad_x = (T*)d_grad_x;
    p.grad_gate = (T*)d_grad_gate;
    p.grad_h0 = (C*)d_grad_h0;
    p.offsets = q.d_offsets;
    p.x_seq = x_seq_stride;
    p.x_step = x_step_stride;
    p.g_seq = gate_seq_stride;
    p.g_step = gate_step_stride;
    p.d_seq = grad_seq_stride;
    p.d_step = grad_step_stride;
    p.n_seq = q.n_seq;
    p.steps = q.steps;
    p.dim = q.dim;
    rec_backward<T, decltype(gate)::value><<<simple_grid(q), kWG, 0, (hipStream_t)stream>>>(p);
    SLA_HIP(hipGetLastError());
    return SLA_OK;
  });
}

}  // extern "C"
