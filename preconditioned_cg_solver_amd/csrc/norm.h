// Kernels of the norms before (IN) and after a block, forward and backward.
//
// Bound by bytes: each element is read once and kept in registers between the sum
// over its row and what follows.  A team of waves has a row; it walks many rows, so
// that a lane's weights stay in registers, and backward so do the sums over rows
// that are the weights' gradients.  Rows too wide for that, or not in packs, are
// read again (from the caches) where they are needed a second time.  16384 x 2048 bf16 before a
// block, fp32 stream, 70 and 107 us (5.8 and 5.7 TB/s); 16384 x 4096 bf16 after, 76 and 133
// (5.3 and 5.0).
//
// Far from that, in us, forward + backward, before a block and after it.  Wide rows, whose sums
// and next row do not fit the registers (two packs a lane of 16 waves spill 100 to 176 beside the 128
// that there are; rows read again have their sums in memory): 4096 x 16384 bf16 84 + 397 and 101 +
// 667 (bytes at 5.95 TB/s: 90 + 113 each), 4096 x 16384 fp32 248 + 464 and 241 + 586, 4000 x 8191 bf16
// 75 + 183 and 113 + 288.  Narrow rows, which leave lanes without elements: 100000 x 64 bf16 25 +
// 52 and 39 + 80 (bytes: 9 + 11 each), 100000 x 33 bf16 89 + 101 and 120 + 136.
#pragma once

#include <algorithm>

#include "rowsum.h"

namespace sla {
namespace norm {

template <typename T, typename R>
struct Args {
  using C = typename Compute<T>::type;
  const T *x, *gate, *grad_y;       // grad_y: IN
  const R *residual, *grad_r;       // grad_r: IN, of r; OUT, of out
  const C *scale, *weight;
  T *y, *grad_x, *grad_gate;
  R *r, *grad_residual;             // r: OUT, out
  C *rstd, *part_weight, *part_scale;
  int64_t rows, dim, x_row, gate_row, residual_row;
  C eps;
  bool norm_first;
};

// The sum over a team of W waves, in every lane.
template <int W, typename C>
__device__ __forceinline__ C team_sum(C v, C (&red)[2][16], int& turn) {
  v += from_lane<kXor1>(v);
  v += from_lane<kXor2>(v);
  v += from_lane<kRor4>(v);
  v += from_lane<kRor8>(v);
  v = fold_rows(v, v);
  v = fold_halves(v, v);
  if constexpr (W > 1) {
    // two buffers in turn: one barrier a sum
    if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
    lds_barrier();
    v = red[turn][0];
#pragma unroll
    for (int o = 1; o < W; ++o) v += red[turn][o];
    turn ^= 1;
  }
  return v;
}

__device__ __forceinline__ float inverse_root(float v) { return __builtin_amdgcn_rsqf(v); }
__device__ __forceinline__ double inverse_root(double v) { return 1.0 / sqrt(v); }

// The elements of a row that a lane takes together, as they were read, and what is
// worked out of them once: the normed values and the gate's sigmoid.
template <typename T, typename R, int V>
struct Cells {
  Pack<T, V> x, g;  // g: the gate, or IN backward dL/dy
  Pack<R, V> res, gr;
};
template <typename C, int V>
struct Made {
  C u[V], sig[V];
};
template <typename C, int V>
struct Weights {
  C weight[V], scale[V];
};

// W waves a row; NP packs of V elements a lane (0: as many as there are, not kept).  STREAM:
// what is written goes past the caches.
template <typename T, typename R, bool IN, bool BACK, int V, int W, int NP, bool STREAM>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_rows(Args<T, R> p) {
  using C = typename Compute<T>::type;
  using Cell = Cells<T, R, V>;
  using Make = Made<C, V>;
  using Weight = Weights<C, V>;
  constexpr int TEAMS = W == 1 ? 4 : 1, N = NP ? NP : 1, STEP = 64 * W * V;
  constexpr bool KEPT = NP > 0;
  __shared__ C red[2][16];
  int turn = 0;
  const int team = W == 1 ? threadIdx.x >> 6 : 0;
  const int first = (int)(threadIdx.x - team * 64 * W) * V;
  const int64_t slot = (int64_t)blockIdx.x * TEAMS + team, slots = (int64_t)gridDim.x * TEAMS;

  auto weights_at = [&](int64_t col) {
    Weight w;
#pragma unroll
    for (int v = 0; v < V; ++v) w.weight[v] = p.weight[col + v], w.scale[v] = C(1);
    if (p.scale)
#pragma unroll
      for (int v = 0; v < V; ++v) w.scale[v] = p.scale[col + v];
    return w;
  };
  auto load = [&](int64_t row, int64_t col) {
    Cell c{};
    c.x = *(const Pack<T, V>*)(p.x + row * p.x_row + col);
    if ((IN || !BACK) && p.residual)
      c.res = *(const Pack<R, V>*)(p.residual + row * p.residual_row + col);
    if (!IN && p.gate) c.g = *(const Pack<T, V>*)(p.gate + row * p.gate_row + col);
    if (IN && BACK) c.g = *(const Pack<T, V>*)(p.grad_y + row * p.dim + col);
    if (BACK && p.grad_r) c.gr = *(const Pack<R, V>*)(p.grad_r + row * p.dim + col);
    return c;
  };
  const bool gated = !IN && p.gate, gate_first = gated && !p.norm_first;
  auto make = [&](const Cell& c, const Weight& w) {
    Make m;
#pragma unroll
    for (int v = 0; v < V; ++v) m.u[v] = (C)c.x.v[v], m.sig[v] = C(1);
    if constexpr (IN) {
      if (p.scale)
#pragma unroll
        for (int v = 0; v < V; ++v) m.u[v] *= w.scale[v];
      if (p.residual)
#pragma unroll
        for (int v = 0; v < V; ++v) m.u[v] += (C)c.res.v[v];
    } else if (gated) {
#pragma unroll
      for (int v = 0; v < V; ++v) m.sig[v] = sigmoid((C)c.g.v[v]);
      if (gate_first)
#pragma unroll
        for (int v = 0; v < V; ++v) m.u[v] *= silu_of((C)c.g.v[v], m.sig[v]);
    }
    return m;
  };
  // backward: dL/d(u / rms), and the factor of the weight's gradient with u / rms
  auto pull = [&](const Cell& c, const Make& m, const Weight& w, int v, C& factor) {
    if constexpr (IN) {
      factor = (C)c.g.v[v];
    } else {
      factor = (C)c.gr.v[v] * w.scale[v];
      if (gated && !gate_first) factor *= silu_of((C)c.g.v[v], m.sig[v]);
    }
    return factor * w.weight[v];
  };

  Weight wr[N];
  C dw[N][V], ds[N][V];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (KEPT && first + k * STEP < p.dim) wr[k] = weights_at(first + k * STEP);
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = ds[k][v] = C(0);
  }
  C* const pw = BACK ? p.part_weight + slot * p.dim : nullptr;
  C* const ps = BACK && p.part_scale ? p.part_scale + slot * p.dim : nullptr;
  if (BACK && !KEPT)
    for (int64_t col = first; col < p.dim; col += STEP)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        pw[col + v] = C(0);
        if (ps) ps[col + v] = C(0);
      }

  // A row's packs, the next row's on their way.
  Cell ahead[N];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (first + k * STEP < p.dim) ahead[k] = load(row, first + k * STEP);
  };
  if (KEPT && slot < p.rows) fetch(slot);

  for (int64_t row = slot; row < p.rows; row += slots) {
    Cell held[N];
    Make made[N];
    if constexpr (KEPT) {
#pragma unroll
      for (int k = 0; k < N; ++k) held[k] = ahead[k];
      if (row + slots < p.rows) fetch(row + slots);
#pragma unroll
      for (int k = 0; k < N; ++k) made[k] = make(held[k], wr[k]);
    }
    // Calls f(pack, column, cells, made, weights) for each of the lane's packs.
    auto each = [&](auto&& f) {
      if constexpr (KEPT) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (first + k * STEP < p.dim) f(k, (int64_t)first + k * STEP, held[k], made[k], wr[k]);
      } else {
        for (int64_t col = first; col < p.dim; col += STEP) {
          const Cell c = load(row, col);
          const Weight w = weights_at(col);
          f(0, col, c, make(c, w), w);
        }
      }
    };
    C sum = C(0);
    if constexpr (!BACK) {
      each([&](int, int64_t, const Cell&, const Make& m, const Weight&) {
#pragma unroll
        for (int v = 0; v < V; ++v) sum += m.u[v] * m.u[v];
      });
      sum = team_sum<W>(sum, red, turn);
      const C rstd = inverse_root(sum / (C)p.dim + p.eps);
      if (first == 0 && p.rstd) p.rstd[row] = rstd;
      each([&](int, int64_t col, const Cell& c, const Make& m, const Weight& w) {
        Pack<T, V> oy;
        Pack<R, V> orr;
        C n[V];
#pragma unroll
        for (int v = 0; v < V; ++v) n[v] = m.u[v] * rstd * w.weight[v];
        if constexpr (IN) {
#pragma unroll
          for (int v = 0; v < V; ++v) oy.v[v] = (T)n[v], orr.v[v] = (R)m.u[v];
          put_pack<STREAM, V>(p.y + row * p.dim + col, oy);
        } else {
          if (gated && !gate_first)
#pragma unroll
            for (int v = 0; v < V; ++v) n[v] *= silu_of((C)c.g.v[v], m.sig[v]);
          if (p.scale)
#pragma unroll
            for (int v = 0; v < V; ++v) n[v] *= w.scale[v];
          if (p.residual)
#pragma unroll
            for (int v = 0; v < V; ++v) n[v] += (C)c.res.v[v];
#pragma unroll
          for (int v = 0; v < V; ++v) orr.v[v] = (R)n[v];
        }
        if (p.r) put_pack<STREAM, V>(p.r + row * p.dim + col, orr);
      });
    } else {
      const C rstd = p.rstd[row];
      each([&](int, int64_t, const Cell& c, const Make& m, const Weight& w) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          C factor;
          sum += pull(c, m, w, v, factor) * m.u[v];
        }
      });
      // rstd (g - hat mean(g hat)), hat = u rstd
      const C mean = team_sum<W>(sum, red, turn) / (C)p.dim * rstd * rstd;
      each([&](int k, int64_t col, const Cell& c, const Make& m, const Weight& w) {
        Pack<T, V> ox, og;
        Pack<R, V> orr;
        C aw[V], as[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          C factor;
          const C g = pull(c, m, w, v, factor), xv = (C)c.x.v[v];
          const C hat = m.u[v] * rstd;
          C du = rstd * (g - m.u[v] * mean);
          aw[v] = factor * hat;
          if constexpr (IN) {
            if (p.grad_r) du += (C)c.gr.v[v];
            orr.v[v] = (R)du;
            as[v] = du * xv;
            ox.v[v] = (T)(p.scale ? du * w.scale[v] : du);
          } else {
            const C gv = (C)c.g.v[v], s = gated ? silu_of(gv, m.sig[v]) : C(1);
            const C n = hat * w.weight[v];
            as[v] = (C)c.gr.v[v] * (gate_first ? n : n * s);
            ox.v[v] = (T)(gate_first ? du * s : du);
            if (gated) {
              const C to = gate_first ? du * xv : (C)c.gr.v[v] * w.scale[v] * n;
              og.v[v] = (T)(to * silu_slope(gv, m.sig[v]));
            }
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if constexpr (KEPT) {
            dw[k][v] += aw[v];
            ds[k][v] += as[v];
          } else {
            pw[col + v] += aw[v];
            if (ps) ps[col + v] += as[v];
          }
        }
        put_pack<STREAM, V>(p.grad_x + row * p.dim + col, ox);
        if (IN && p.grad_residual)
          put_pack<STREAM, V>(p.grad_residual + row * p.dim + col, orr);
        if (gated) put_pack<STREAM, V>(p.grad_gate + row * p.dim + col, og);
      });
    }
  }
  if constexpr (BACK && KEPT) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (first + k * STEP < p.dim)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          pw[first + k * STEP + v] = dw[k][v];
          if (ps) ps[first + k * STEP + v] = ds[k][v];
        }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

sla_status refuse(const char* msg);
sla_status check_shape(const sla_norm_shape* q);
// Workgroups at most.
constexpr int kMostGroups = 1024;
size_t work_bytes_of(const sla_norm_shape& q);
bool packs(const void* p, int64_t row, size_t bytes, int v, bool one);

// How a row is taken: elements of a pack, waves, packs of a lane (0: read again).
struct Way {
  int v, w, np;
};
// v: elements of a pack.
inline Way way_of(int v, int64_t dim, bool wide) {
  if (wide) {
    if (dim <= 64 * v) return {v, 1, 1};
    if (dim <= 256 * v) return {v, 4, 1};
    if (dim <= 512 * v) return {v, 8, 1};
    if (dim <= 1024 * v) return {v, 16, 1};
    if (dim <= 2048 * v) return {v, 16, 2};
    return {v, 16, 0};
  }
  if (dim <= 1024) return {1, 4, 4};
  if (dim <= 4096) return {1, 16, 4};
  return {1, 16, 0};
}
// Workgroups, and teams (rows of the gradients' parts).
inline int64_t groups_of(const Way& w, int64_t rows) {
  const int64_t teams = w.w == 1 ? 4 : 1;
  return std::min<int64_t>((rows + teams - 1) / teams, w.w == 16 ? kMostGroups / 2 : kMostGroups);
}
inline int64_t teams_of(const Way& w, int64_t rows) {
  return groups_of(w, rows) * (w.w == 1 ? 4 : 1);
}

template <typename T, typename R, bool IN, bool BACK>
sla_status run(Args<T, R>& p, const Way& way, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const double bytes = (double)p.rows * p.dim *
                       (sizeof(T) * (IN ? 2 + BACK : 1 + (p.gate ? 1 + BACK : 0) + BACK) +
                        sizeof(R) * ((p.residual != nullptr) + 1 + (IN && BACK)));
  // Beyond what the last-level cache holds (256 MB): 16384 x 4096 bf16 with a gate, after a
  // block, forward 81 -> 66 us, backward 144 -> 132; reads past it as well gained nothing
  // (16384 x 2048 before a block 77.5 -> 79.7).
  const bool streams = bytes >= kMallBytes;
  const unsigned grid = (unsigned)groups_of(way, p.rows);
#define SLA_NORM_CASE(v_, w_, np_, stream_)                                                 \
  if (way.v == v_ && way.w == w_ && way.np == np_ && (!stream_ || streams))                 \
    norm_rows<T, R, IN, BACK, v_, w_, np_, stream_>                                         \
        <<<grid, w_ == 1 ? 256 : w_ * 64, 0, s>>>(p)
  SLA_NORM_CASE(V, 1, 1, true);
  else SLA_NORM_CASE(V, 4, 1, true);
  else SLA_NORM_CASE(V, 8, 1, true);
  else SLA_NORM_CASE(V, 16, 1, true);
  else SLA_NORM_CASE(V, 16, 2, true);
  else SLA_NORM_CASE(V, 1, 1, false);
  else SLA_NORM_CASE(V, 4, 1, false);
  else SLA_NORM_CASE(V, 8, 1, false);
  else SLA_NORM_CASE(V, 16, 1, false);
  else SLA_NORM_CASE(V, 16, 2, false);
  else SLA_NORM_CASE(V, 16, 0, false);
  else SLA_NORM_CASE(1, 4, 4, false);
  else SLA_NORM_CASE(1, 16, 4, false);
  else SLA_NORM_CASE(1, 16, 0, false);
#undef SLA_NORM_CASE
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}

// Calls f with the types of elements and of the residual stream.
template <typename F>
sla_status with_types(const sla_norm_shape& q, F&& f) {
  switch (q.dtype) {
    case SLA_F64: return f(double{}, double{});
    case SLA_F32: return f(float{}, float{});
    case SLA_BF16: return q.stream == SLA_F32 ? f(bf16_t{}, float{}) : f(bf16_t{}, bf16_t{});
    default: return q.stream == SLA_F32 ? f(f16_t{}, float{}) : f(f16_t{}, f16_t{});
  }
}

// Runs the backward kernel, then sums the parts of the gradients of weight and scale.
template <typename T, typename R, bool IN>
sla_status run_back(const sla_norm_shape& q, Args<T, R>& p, bool wide, void* work, void* weight,
                    void* scale, hipStream_t s) {
  using C = typename Compute<T>::type;
  RowSums<C> r{};
  if (q.rows) {
    const Way way = way_of(16 / (int)sizeof(T), q.dim, wide);
    r.rows = teams_of(way, q.rows);
    p.part_weight = (C*)work;
    p.part_scale = scale ? p.part_weight + r.rows * q.dim : nullptr;
    const sla_status st = run<T, R, IN, true>(p, way, s);
    if (st != SLA_OK) return st;
  }
  r.part[0] = p.part_weight, r.part[1] = p.part_scale;
  r.out[0] = (C*)weight, r.out[1] = (C*)scale;
  r.n[0] = r.n[1] = r.stride[0] = r.stride[1] = q.dim;
  return sum_of_rows(r, s);
}

}  // namespace norm
}  // namespace sla
