// The norm before a block, y = weight r / rms(r) with r = residual + scale x.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "norm.h"

namespace sla {
namespace norm {

sla_status refuse(const char* msg) {
  set_error(msg);
  return SLA_ERR_INVALID_ARG;
}

sla_status check_shape(const sla_norm_shape* q) {
  if (!q) return refuse("shape is NULL");
  if (q->rows < 0 || q->dim < 0) return refuse("negative size");
  if (q->dtype != SLA_F64 && q->dtype != SLA_F32 && q->dtype != SLA_BF16 && q->dtype != SLA_F16)
    return refuse("unknown dtype");
  const bool half = q->dtype == SLA_BF16 || q->dtype == SLA_F16;
  if (q->stream != q->dtype && !(half && q->stream == SLA_F32))
    return refuse("the residual has x's dtype, or fp32 where that has 16 bits");
  if (!(q->eps >= 0.0) || std::isinf(q->eps)) return refuse("eps must be finite and not negative");
  if (q->dim >= (1 << 26) || (__int128)q->rows * (q->dim + 1) >= ((__int128)1 << 58)) {
    set_error("sizes beyond what a call can index");
    return SLA_ERR_UNSUPPORTED;
  }
  return SLA_OK;
}

size_t work_bytes_of(const sla_norm_shape& q) {
  if (!q.rows || !q.dim) return 0;
  // whether a row is read in packs or not
  const int v = 16 / (int)dtype_bytes(q.dtype);
  const int64_t teams = std::max(teams_of(way_of(v, q.dim, true), q.rows),
                                 teams_of(way_of(v, q.dim, false), q.rows));
  return align_up((size_t)teams * 2 * q.dim * (q.dtype == SLA_F64 ? 8 : 4));
}

bool packs(const void* p, int64_t row, size_t bytes, int v, bool one) {
  return (uintptr_t)p % (v * bytes) == 0 && (row % v == 0 || one);
}

}  // namespace norm
}  // namespace sla

using namespace sla;
using namespace sla::norm;

extern "C" {

sla_status sla_norm_sizes(const sla_norm_shape* shape, size_t* work_bytes) {
  const sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (!work_bytes) return refuse("NULL result");
  *work_bytes = work_bytes_of(*shape);
  return SLA_OK;
}

sla_status sla_norm_in_forward(const sla_norm_shape* shape, const void* d_x, int64_t x_row,
                               const void* d_residual, int64_t residual_row, const void* d_scale,
                               const void* d_weight, void* d_y, void* d_r, void* d_rstd,
                               void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_norm_shape& q = *shape;
  if (x_row < 0 || residual_row < 0) return refuse("negative stride");
  const bool same = !d_residual && !d_scale;
  if (same && d_r) return refuse("without residual and scale r is x: it is not written");
  if (!q.rows || !q.dim) return SLA_OK;
  if (!d_x || !d_weight || !d_y || (!same && !d_r)) return refuse("x, weight, y or r is NULL");
  if (d_y == d_x || d_y == d_residual || d_r == d_x || d_y == d_r)
    return refuse("an output must not be an input");
  if (d_r && d_r == d_residual && residual_row != q.dim)
    return refuse("a residual updated in place must be dense");
  TraceRange tr("sla_norm_in_forward");
  return with_types(q, [&](auto t, auto rt) -> sla_status {
    using T = decltype(t);
    using R = decltype(rt);
    using C = typename Compute<T>::type;
    constexpr int V = 16 / (int)sizeof(T);
    Args<T, R> p{};
    p.x = (const T*)d_x, p.x_row = x_row;
    p.residual = (const R*)d_residual, p.residual_row = residual_row;
    p.scale = (const C*)d_scale, p.weight = (const C*)d_weight;
    p.y = (T*)d_y, p.r = (R*)d_r, p.rstd = (C*)d_rstd;
    p.rows = q.rows, p.dim = q.dim, p.eps = (C)q.eps;
    const bool one = q.rows == 1;
    const bool wide = q.dim % V == 0 && packs(d_x, x_row, sizeof(T), V, one) &&
                      packs(d_residual, residual_row, sizeof(R), V, one) &&
                      packs(d_y, 0, sizeof(T), V, one) && packs(d_r, 0, sizeof(R), V, one);
    return run<T, R, true, false>(p, way_of(V, q.dim, wide), (hipStream_t)stream);
  });
}

sla_status sla_norm_in_backward(const sla_norm_shape* shape, const void* d_grad_y,
                                const void* d_grad_r, const void* d_x, int64_t x_row,
                                const void* d_residual, int64_t residual_row, const void* d_scale,
                                const void* d_weight, const void* d_rstd, void* d_grad_x,
                                void* d_grad_residual, void* d_grad_weight, void* d_grad_scale,
                                void* d_work, size_t work_bytes, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_norm_shape& q = *shape;
  if (x_row < 0 || residual_row < 0) return refuse("negative stride");
  if (!q.dim) return SLA_OK;
  if (!d_grad_weight) return refuse("the weight's gradient is NULL");
  if (q.rows && (!d_grad_y || !d_x || !d_weight || !d_rstd || !d_grad_x))
    return refuse("an input or a gradient is NULL");
  if (q.rows) {
    for (const void* a : {d_grad_y, d_grad_r, d_x, d_residual})
      if (a && (a == d_grad_x || a == d_grad_residual))
        return refuse("a gradient must not be an input");
    if (d_grad_x == d_grad_residual) return refuse("the gradients must be distinct arrays");
  }
  const size_t need = work_bytes_of(q);
  if (need && (!d_work || work_bytes < need)) return refuse("workspace too small");
  if ((uintptr_t)d_work & 255) return refuse("the workspace must be 256-byte aligned");
  TraceRange tr("sla_norm_in_backward");
  return with_types(q, [&](auto t, auto rt) -> sla_status {
    using T = decltype(t);
    using R = decltype(rt);
    using C = typename Compute<T>::type;
    constexpr int V = 16 / (int)sizeof(T);
    Args<T, R> p{};
    p.grad_y = (const T*)d_grad_y, p.grad_r = (const R*)d_grad_r;
    p.x = (const T*)d_x, p.x_row = x_row;
    p.residual = (const R*)d_residual, p.residual_row = residual_row;
    p.scale = (const C*)d_scale, p.weight = (const C*)d_weight, p.rstd = (C*)d_rstd;
    p.grad_x = (T*)d_grad_x, p.grad_residual = (R*)d_grad_residual;
    p.rows = q.rows, p.dim = q.dim;
    const bool one = q.rows == 1;
    const bool wide =
        q.dim % V == 0 && packs(d_x, x_row, sizeof(T), V, one) &&
        packs(d_residual, residual_row, sizeof(R), V, one) && packs(d_grad_y, 0, sizeof(T), V, one) &&
        packs(d_grad_r, 0, sizeof(R), V, one) && packs(d_grad_x, 0, sizeof(T), V, one) &&
        packs(d_grad_residual, 0, sizeof(R), V, one);
    return run_back<T, R, true>(q, p, wide, d_work, d_grad_weight, d_grad_scale,
                                (hipStream_t)stream);
  });
}

}  // extern "C"
