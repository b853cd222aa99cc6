// The norm after a block with its gate: n = weight u / rms(u), u = x silu(gate), or
// n = weight x / rms(x) silu(gate); out = residual + scale n.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm.h"

using namespace sla;
using namespace sla::norm;

namespace {

template <typename T, typename R>
Args<T, R> args_of(const sla_norm_shape& q, sla_norm_order order, const void* x, int64_t x_row,
                   const void* gate, int64_t gate_row, const void* scale, const void* weight,
                   const void* rstd) {
  using C = typename Compute<T>::type;
  Args<T, R> p{};
  p.x = (const T*)x, p.x_row = x_row;
  p.gate = (const T*)gate, p.gate_row = gate_row;
  p.scale = (const C*)scale, p.weight = (const C*)weight, p.rstd = (C*)rstd;
  p.rows = q.rows, p.dim = q.dim, p.eps = (C)q.eps;
  p.norm_first = order == SLA_NORM_FIRST;
  return p;
}

}  // namespace

extern "C" {

sla_status sla_norm_out_forward(const sla_norm_shape* shape, sla_norm_order order, const void* d_x,
                                int64_t x_row, const void* d_gate, int64_t gate_row,
                                const void* d_residual, int64_t residual_row, const void* d_scale,
                                const void* d_weight, void* d_out, void* d_rstd, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_norm_shape& q = *shape;
  if (order != SLA_GATE_FIRST && order != SLA_NORM_FIRST) return refuse("unknown order");
  if (x_row < 0 || gate_row < 0 || residual_row < 0) return refuse("negative stride");
  if (!q.rows || !q.dim) return SLA_OK;
  if (!d_x || !d_weight || !d_out) return refuse("x, weight or out is NULL");
  if (d_out == d_x || d_out == d_gate) return refuse("an output must not be an input");
  if (d_out == d_residual && residual_row != q.dim)
    return refuse("a residual updated in place must be dense");
  TraceRange tr("sla_norm_out_forward");
  return with_types(q, [&](auto t, auto rt) -> sla_status {
    using T = decltype(t);
    using R = decltype(rt);
    constexpr int V = 16 / (int)sizeof(T);
    auto p = args_of<T, R>(q, order, d_x, x_row, d_gate, gate_row, d_scale, d_weight, d_rstd);
    p.residual = (const R*)d_residual, p.residual_row = residual_row;
    p.r = (R*)d_out;
    const bool one = q.rows == 1;
    const bool wide = q.dim % V == 0 && packs(d_x, x_row, sizeof(T), V, one) &&
                      packs(d_gate, gate_row, sizeof(T), V, one) &&
                      packs(d_residual, residual_row, sizeof(R), V, one) &&
                      packs(d_out, 0, sizeof(R), V, one);
    return run<T, R, false, false>(p, way_of(V, q.dim, wide), (hipStream_t)stream);
  });
}

sla_status sla_norm_out_backward(const sla_norm_shape* shape, sla_norm_order order,
                                 const void* d_grad_out, const void* d_x, int64_t x_row,
                                 const void* d_gate, int64_t gate_row, const void* d_scale,
                                 const void* d_weight, const void* d_rstd, void* d_grad_x,
                                 void* d_grad_gate, void* d_grad_weight, void* d_grad_scale,
                                 void* d_work, size_t work_bytes, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_norm_shape& q = *shape;
  if (order != SLA_GATE_FIRST && order != SLA_NORM_FIRST) return refuse("unknown order");
  if (x_row < 0 || gate_row < 0) return refuse("negative stride");
  if (!q.dim) return SLA_OK;
  if (!d_grad_weight) return refuse("the weight's gradient is NULL");
  if (q.rows && (!d_grad_out || !d_x || !d_weight || !d_rstd || !d_grad_x ||
                 (d_gate && !d_grad_gate)))
    return refuse("an input or a gradient is NULL");
  if (q.rows) {
    for (const void* a : {d_grad_out, d_x, d_gate})
      if (a && (a == d_grad_x || a == d_grad_gate)) return refuse("a gradient must not be an input");
    if (d_grad_x == d_grad_gate) return refuse("the gradients must be distinct arrays");
  }
  const size_t need = work_bytes_of(q);
  if (need && (!d_work || work_bytes < need)) return refuse("workspace too small");
  if ((uintptr_t)d_work & 255) return refuse("the workspace must be 256-byte aligned");
  TraceRange tr("sla_norm_out_backward");
  return with_types(q, [&](auto t, auto rt) -> sla_status {
    using T = decltype(t);
    using R = decltype(rt);
    constexpr int V = 16 / (int)sizeof(T);
    auto p = args_of<T, R>(q, order, d_x, x_row, d_gate, gate_row, d_scale, d_weight, d_rstd);
    p.grad_r = (const R*)d_grad_out;
    p.grad_x = (T*)d_grad_x, p.grad_gate = (T*)d_grad_gate;
    const bool one = q.rows == 1;
    const bool wide = q.dim % V == 0 && packs(d_x, x_row, sizeof(T), V, one) &&
                      packs(d_gate, gate_row, sizeof(T), V, one) &&
                      packs(d_grad_out, 0, sizeof(R), V, one) &&
                      packs(d_grad_x, 0, sizeof(T), V, one) &&
                      packs(d_grad_gate, 0, sizeof(T), V, one);
    return run_back<T, R, false>(q, p, wide, d_work, d_grad_weight, d_scale ? d_grad_scale : nullptr,
                                 (hipStream_t)stream);
  });
}

}  // extern "C"
