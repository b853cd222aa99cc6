// Selective scans, backward.  With ds = dL/dy silu(z), backwards along a sequence:
//   g_t = ds_t C_t + mu_{t+1},  mu_t = a_t g_t,  mu after the last step = dL/dh_last,
//   dL/dC_t = sum_c ds_t h_t,   dL/dB_t = sum_c g_t delta_t x_t,
//   dL/dA = sum_t mu_t h_{t-1} delta_t,   dL/dh_0 = mu_1,
//   dL/ddelta_t = sum_n mu_t h_{t-1} A + x_t g_t B_t,  dL/dx_t = delta_t sum_n g_t B_t + D ds_t.
// (q = g a h_{t-1} = mu_t h_{t-1} needs no division and no difference.)
//
// A wave works a tile's states out again from the one saved at its start, keeps
// them and the coefficients in registers, and comes back.  Sums over a channel's
// states and over channels are folded between lanes; those over the waves of a
// workgroup go through LDS, and those over workgroups through a workspace, so that
// every sum is made in one order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "rowsum.h"
#include "selscan.h"

namespace sla {
namespace selscan {

sla_status check_in(const sla_selscan_shape& q, const sla_selscan_in* in);
sla_status check_work(size_t need, const void* work, size_t bytes);
template <typename C>
sla_status leave_empty(const sla_selscan_shape& q, const void* from, void* to, hipStream_t s);

namespace {

// Steps whose instructions are scheduled together; over more of them the compiler
// moves so many loads ahead that the states leave the registers.
constexpr int kAhead = 2;

template <typename C>
struct Drive {
  C delta, dx;  // delta_t, delta_t x_t
};
template <typename C>
struct Pull {
  C delta, ds;
};

// What a chunk leaves to the one before it, from nothing.
template <typename T, int NS, bool PAD>
__global__ __launch_bounds__(kWG) void scan_back_local(Args<T> p) {
  using C = typename Compute<T>::type;
  using R = Rows<C>;
  constexpr int TS = R::TS, EL = R::EL;
  __shared__ Pull<C> s_pull[kWavesOf][TS][kChannels];
  __shared__ C s_c[kWavesOf][TS][4 * NS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Place w = place_of<T, kWavesOf>(p);
  if (w.some <= 0) return;
  auto& pull = s_pull[wave];
  auto& cs = s_c[wave];
  const int q = lane >> 4, c = lane & 15;
  const bool live = c < w.some;
  const int64_t channel = w.channel + c;
  C a2[NS], mu[NS], total = C(0);
  get_states<NS, PAD>(a2, p.a, channel, p.states, q, live);
#pragma unroll
  for (int j = 0; j < NS; ++j) a2[j] *= C(1.4426950408889634), mu[j] = C(0);
  bool cut = false;

  const int r = lane / R::PER, cc = lane % R::PER * EL, some = w.some - cc;
  const int64_t col = w.channel + (some > 0 ? cc : 0);
  C bias[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) bias[e] = p.bias && e < some ? p.bias[col + e] : C(0);
  const T* const u0 = p.dt + w.seq * p.dt_seq + col;
  const T* const z0 = p.z ? p.z + w.seq * p.z_seq + col : nullptr;
  const T* const g0 = p.grad_y + w.seq * p.gy_seq + col;
  const T* const c0 = p.c + w.seq * p.c_seq + w.group * p.states;
  Pack<T, EL> ur, zr{}, gr;
  Pack<T, Shared<C, NS>::BL> cr;
  auto fetch = [&](int64_t t0) {
    const int n = (int)min((int64_t)TS, w.t1 - t0);
    const int64_t t = t0 + (r < n ? r : 0);
    ur = load_some<EL>(u0 + t * p.dt_step, some, p.vec);
    gr = load_some<EL>(g0 + t * p.gy_step, some, p.vec);
    if (z0) zr = load_some<EL>(z0 + t * p.z_step, some, p.vec);
    cr = load_shared<C, NS>(p, c0 + t0 * p.c_step, p.c_step, n);
  };
  const int64_t last = w.t0 + (w.t1 - 1 - w.t0) / TS * TS;
  fetch(last);
  Span now = p.offsets ? span_of(p, w, last) : Span{};
  for (int64_t t0 = last; t0 >= w.t0; t0 -= TS) {
    const int n = (int)min((int64_t)TS, w.t1 - t0);
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      C slope, delta = (C)ur.v[e] + bias[e], ds = (C)gr.v[e];
      if (p.softplus) delta = softplus(delta, slope);
      if (z0) ds *= silu((C)zr.v[e]);
      pull[r][cc + e] = {delta, ds};
    }
    keep_shared<C, NS>(cs, cr);
    if (t0 > w.t0) fetch(t0 - TS);
    unsigned starts, ends;
    edges_of<TS>(p, w, now, t0, n, starts, ends);
    wave_sync();
    C sum = C(0);
    auto step = [&](int i) {
      const Pull<C> d = pull[i][c];
#pragma unroll
      for (int j = 0; j < NS; ++j)
        mu[j] = pow2(d.delta * a2[j]) * (d.ds * cs[i][q * NS + j] + mu[j]);
      sum += d.delta;
    };
    if (n == TS && !ends) {
#pragma unroll
      for (int i = TS - 1; i >= 0; --i) step(i);
    } else {
      for (int i = n - 1; i >= 0; --i) {
        if (ends >> i & 1) {
          const int64_t s = span_of(p, w, t0 + i).seq;
          get_states<NS, PAD>(mu, p.grad_last, s * p.dim + channel, p.states, q, live);
          cut = true;
        }
        step(i);
      }
    }
    total += sum;
    wave_sync();
  }
  put_states<NS, PAD>(mu, p.ends, w.row * p.dim + channel, p.states, q, live);
  if (q == 0 && live) p.deltas[w.row * p.dim + channel] = total;
  if (threadIdx.x == 0 && w.block == 0) p.cuts[w.row] = cut;
}

template <typename T, int NS, bool PAD>
__global__ __launch_bounds__(kWG, 2) void scan_backward(Args<T> p) {
  using C = typename Compute<T>::type;
  using R = Rows<C>;
  constexpr int TS = R::TS, EL = R::EL, N4 = 4 * NS;
  __shared__ Drive<C> s_drive[kWavesOf][TS][kChannels];
  __shared__ C s_ds[kWavesOf][TS][kChannels];
  __shared__ C s_b[kWavesOf][TS][N4], s_c[kWavesOf][TS][N4];
  __shared__ C s_sum[kWavesOf][TS][3][kChannels];  // over states: C h, g B, mu h A
  __shared__ C s_bc[2][kWavesOf][TS][2][N4];       // over a wave's channels: of dB, of dC
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Place w = place_of<T, kWavesOf>(p);
  const bool idle = w.some <= 0;  // its workgroup's sums want it all the same
  auto& drive = s_drive[wave];
  auto& dss = s_ds[wave];
  auto& bs = s_b[wave];
  auto& cs = s_c[wave];
  auto& sums = s_sum[wave];

  // the lane's channel and states: the channel in bits 0, 1, 4, 5, so that most of the
  // sums over channels are made by swaps of halves and rows
  const int q = lane >> 2 & 3, c = (lane & 3) | (lane >> 4) << 2;
  const bool live = c < w.some;
  const int64_t channel = w.channel + (idle ? 0 : c);
  C a[NS], a2[NS], mu[NS], da[NS];
  get_states<NS, PAD>(a, p.a, channel, p.states, q, live);
  {
    // what enters from the chunk that follows
    const bool end = !p.offsets && w.t1 == p.steps;
    const C* from = p.chunks > 1 && !end ? p.ends : nullptr;
    get_states<NS, PAD>(mu, from, w.row * p.dim + channel, p.states, q, live);
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) a2[j] = a[j] * C(1.4426950408889634), da[j] = C(0);

  const int r = lane / R::PER, cc = lane % R::PER * EL, some = w.some - cc;
  const int64_t col = idle ? 0 : w.channel + (some > 0 ? cc : 0);
  C bias[EL], dd[EL], dbias[EL], ddd[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    bias[e] = p.bias && e < some ? p.bias[col + e] : C(0);
    dd[e] = p.d && e < some ? p.d[col + e] : C(0);
    dbias[e] = ddd[e] = C(0);
  }
  const T* const x0 = p.x + w.seq * p.x_seq + col;
  const T* const u0 = p.dt + w.seq * p.dt_seq + col;
  const T* const z0 = p.z ? p.z + w.seq * p.z_seq + col : nullptr;
  const T* const g0 = p.grad_y + w.seq * p.gy_seq + col;
  const T* const b0 = p.b + w.seq * p.b_seq + w.group * p.states;
  const T* const c0 = p.c + w.seq * p.c_seq + w.group * p.states;
  const int64_t tile0 = p.offsets ? 0 : w.seq * p.tiles;
  Pack<T, EL> xr, ur, zr{}, gr;
  Pack<T, Shared<C, NS>::BL> br, cr;
  C enter[NS];  // the state at the tile's start
  auto fetch = [&](int64_t t0) {
    const int n = (int)min((int64_t)TS, w.t1 - t0);
    const int64_t t = t0 + (r < n ? r : 0);
    xr = load_some<EL>(x0 + t * p.x_step, some, p.vec);
    ur = load_some<EL>(u0 + t * p.dt_step, some, p.vec);
    gr = load_some<EL>(g0 + t * p.gy_step, some, p.vec);
    if (z0) zr = load_some<EL>(z0 + t * p.z_step, some, p.vec);
    br = load_shared<C, NS>(p, b0 + t0 * p.b_step, p.b_step, n);
    cr = load_shared<C, NS>(p, c0 + t0 * p.c_step, p.c_step, n);
    get_states<NS, PAD>(enter, (const C*)p.saved + (tile0 + t0 / TS) * p.dim * p.states, channel,
                        p.states, q, live);
  };
  const int64_t last = w.t0 + (w.t1 - 1 - w.t0) / TS * TS;
  if (!idle) fetch(last);
  else {
    for (int i = lane; i < TS * 2 * N4; i += kLanes)
      (&s_bc[0][wave][0][0][0])[i] = (&s_bc[1][wave][0][0][0])[i] = C(0);
  }
  Span now = p.offsets ? span_of(p, w, last) : Span{};
  int turn = 0;

  for (int64_t t0 = last; t0 >= w.t0; t0 -= TS, turn ^= 1) {
    const int n = (int)min((int64_t)TS, w.t1 - t0);
    if (!idle) {
      const Pack<T, EL> x = xr, z = zr, gy = gr, u = ur;
      C delta[EL], slope[EL], ds[EL];
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        slope[e] = C(1);
        delta[e] = (C)u.v[e] + bias[e];
        if (p.softplus) delta[e] = softplus(delta[e], slope[e]);
        ds[e] = (C)gy.v[e];
        if (z0) ds[e] *= silu((C)z.v[e]);
        drive[r][cc + e] = {delta[e], delta[e] * (C)x.v[e]};
        dss[r][cc + e] = ds[e];
      }
      keep_shared<C, NS>(bs, br);
      keep_shared<C, NS>(cs, cr);
      C h0[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) h0[j] = enter[j];
      if (t0 > w.t0) fetch(t0 - TS);
      unsigned starts, ends;
      edges_of<TS>(p, w, now, t0, n, starts, ends);
      wave_sync();

      auto tile = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        C coef[TS][NS], hs[TS][NS];
        // forward again
#pragma unroll
        for (int i = 0; i < TS; ++i) {
          if (WHOLE || i < n) {
            C before[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) before[j] = i ? hs[i ? i - 1 : 0][j] : h0[j];
            if (!WHOLE && i > 0 && (starts >> i & 1))
              get_states<NS, PAD>(before, p.h0, span_of(p, w, t0 + i).seq * p.dim + channel,
                                  p.states, q, live);
            const Drive<C> d = drive[i][c];
            C s = C(0);
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              coef[i][j] = pow2(d.delta * a2[j]);
              hs[i][j] = coef[i][j] * before[j] + d.dx * bs[i][q * NS + j];
              const C v = cs[i][q * NS + j] * hs[i][j];
              s += !PAD || q * NS + j < p.states ? v : C(0);
            }
            s += from_lane<kRor8>(s);
            s += from_lane<kRor4>(s);
            sums[i][0][c] = s;
          } else {
#pragma unroll
            for (int j = 0; j < NS; ++j) coef[i][j] = hs[i][j] = C(0);
          }
          if (i % kAhead == kAhead - 1) __builtin_amdgcn_sched_barrier(0);
        }
        // and back
#pragma unroll
        for (int i = TS - 1; i >= 0; --i) {
          if (WHOLE || i < n) {
            C before[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) before[j] = i ? hs[i ? i - 1 : 0][j] : h0[j];
            if (!WHOLE) {
              const bool begins = starts >> i & 1;
              if ((ends >> i & 1) || (begins && i > 0)) {
                const int64_t s = span_of(p, w, t0 + i).seq;
                if (ends >> i & 1)
                  get_states<NS, PAD>(mu, p.grad_last, s * p.dim + channel, p.states, q, live);
                if (begins && i > 0)
                  get_states<NS, PAD>(before, p.h0, s * p.dim + channel, p.states, q, live);
              }
            }
            const Drive<C> d = drive[i][c];
            const C dsv = dss[i][c];
            C gb = C(0), qa = C(0), db[NS], dc[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              const C g = dsv * cs[i][q * NS + j] + mu[j];
              dc[j] = dsv * hs[i][j];
              db[j] = g * d.dx;
              const C v = g * bs[i][q * NS + j];
              gb += !PAD || q * NS + j < p.states ? v : C(0);
              mu[j] = coef[i][j] * g;
              const C mh = mu[j] * before[j];
              const C va = mh * a[j];
              qa += !PAD || q * NS + j < p.states ? va : C(0);
              da[j] += mh * d.delta;
            }
            if (!WHOLE && (starts >> i & 1) && p.grad_h0)
              put_states<NS, PAD>(mu, p.grad_h0, span_of(p, w, t0 + i).seq * p.dim + channel,
                                  p.states, q, live);
            gb += from_lane<kRor8>(gb);
            qa += from_lane<kRor8>(qa);
            gb += from_lane<kRor4>(gb);
            qa += from_lane<kRor4>(qa);
            sums[i][1 + (q & 1)][c] = q & 1 ? qa : gb;
            // over the channels
            const int odd = lane >> 4 & 1, high = lane >> 5;
            if constexpr (NS == 4) {
              C vb = fold_rows(fold_halves(db[0], db[1]), fold_halves(db[2], db[3]));
              C vc = fold_rows(fold_halves(dc[0], dc[1]), fold_halves(dc[2], dc[3]));
              vb += from_lane<kXor1>(vb);
              vc += from_lane<kXor1>(vc);
              C v = lane & 1 ? vc : vb;
              v += from_lane<kXor2>(v);
              if ((lane & 2) == 0) s_bc[turn][wave][i][lane & 1][q * NS + 2 * odd + high] = v;
            } else if constexpr (NS == 2) {
              C v = fold_rows(fold_halves(db[0], db[1]), fold_halves(dc[0], dc[1]));
              v += from_lane<kXor1>(v);
              v += from_lane<kXor2>(v);
              if ((lane & 3) == 0) s_bc[turn][wave][i][odd][q * NS + high] = v;
            } else {
              C v = fold_halves(db[0], dc[0]);
              v = fold_rows(v, v);
              v += from_lane<kXor1>(v);
              v += from_lane<kXor2>(v);
              if ((lane & 3) == 0 && !odd) s_bc[turn][wave][i][high][q] = v;
            }
          }
          if (i % kAhead == 0) __builtin_amdgcn_sched_barrier(0);
        }
      };
      if (n == TS && !starts && !ends) tile(std::true_type{});
      else tile(std::false_type{});
      wave_sync();

      if (r < n) {
        Pack<T, EL> ox, ou, oz;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const C xv = (C)x.v[e], gb = sums[r][1][cc + e], qa = sums[r][2][cc + e];
          const C du = (qa + xv * gb) * slope[e];
          ou.v[e] = (T)du;
          dbias[e] += du;
          C gx = delta[e] * gb;
          if (p.d) gx += dd[e] * ds[e];
          ddd[e] += ds[e] * xv;
          ox.v[e] = (T)gx;
          if (z0) {
            C zs, s = sums[r][0][cc + e];
            if (p.d) s += dd[e] * xv;
            silu((C)z.v[e], zs);
            oz.v[e] = (T)((C)gy.v[e] * s * zs);
          }
        }
        const int64_t to = (w.at + t0 + r) * p.dim + col;
        store_some<EL>(p.grad_x + to, ox, some, p.vec);
        store_some<EL>(p.grad_dt + to, ou, some, p.vec);
        if (z0) store_some<EL>(p.grad_z + to, oz, some, p.vec);
      }
    }
    // One barrier a tile: the other half of s_bc is written next, and read by a
    // wave only after the barrier that follows.
    __syncthreads();
    C* const to = p.part_bc + ((int64_t)w.block * (p.offsets ? p.steps : p.n_seq * p.steps) +
                               w.at + t0) * 2 * p.states;
    for (int k = threadIdx.x; k < n * 2 * N4; k += kWG) {
      const int i = k / (2 * N4), of = k / N4 & 1, st = k % N4;
      C v = s_bc[turn][0][i][of][st];
#pragma unroll
      for (int o = 1; o < kWavesOf; ++o) v += s_bc[turn][o][i][of][st];
      if (st < p.states) to[(i * 2 + of) * p.states + st] = v;
    }
  }
  if (idle) return;
  put_states<NS, PAD>(da, p.part_a, w.row * p.dim + channel, p.states, q, live);
  // over the rows' lanes
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    for (int o = R::PER; o < kLanes; o <<= 1) {
      dbias[e] += __shfl_xor(dbias[e], o);
      ddd[e] += __shfl_xor(ddd[e], o);
    }
    if (r == 0 && e < some) {
      p.part_bias[w.row * p.dim + col + e] = dbias[e];
      p.part_d[w.row * p.dim + col + e] = ddd[e];
    }
  }
}

// dB and dC: sums over the channel blocks of a group.
template <typename T>
__global__ __launch_bounds__(kWG) void sum_blocks(Args<T> p, T* grad_b, T* grad_c, int64_t all) {
  using C = typename Compute<T>::type;
  const int64_t k = (p.before + blockIdx.x) * kWG + threadIdx.x;
  const int64_t row = (int64_t)p.groups * p.states;
  const int64_t step = k / (2 * row);
  if (step >= all) return;
  const int in = (int)(k % (2 * row)), of = in / (int)row, at = in % (int)row;
  const int g = at / p.states, st = at % p.states, per = p.blocks / p.groups;
  const int64_t plane = all * 2 * p.states;
  const C* from = p.part_bc + g * per * plane + (step * 2 + of) * p.states + st;
  C s = C(0);
#pragma unroll 8
  for (int b = 0; b < per; ++b) s += from[b * plane];
  (of ? grad_c : grad_b)[step * row + at] = (T)s;
}

}  // namespace
}  // namespace selscan
}  // namespace sla

using namespace sla;
using namespace sla::selscan;

extern "C" sla_status sla_selscan_backward(const sla_selscan_shape* shape, const sla_selscan_in* in,
                                           const void* d_saved, const void* d_grad_y,
                                           int64_t grad_seq, int64_t grad_step,
                                           const void* d_grad_last, const sla_selscan_grads* grads,
                                           void* d_work, size_t work_bytes, void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_selscan_shape& q = *shape;
  if ((st = check_in(q, in)) != SLA_OK) return st;
  if (!grads) return refuse("gradients are NULL");
  if (grad_seq < 0 || grad_step < 0) return refuse("negative stride");
  if (empty(q)) return SLA_OK;
  const sla_selscan_grads& o = *grads;
  if (!o.d_a) return refuse("a gradient is NULL");
  if (!no_steps(q)) {
    if (!d_saved || !d_grad_y) return refuse("the saved states or grad_y is NULL");
    if (!o.d_x || !o.d_dt || !o.d_b || !o.d_c || (in->d_z && !o.d_z))
      return refuse("a gradient is NULL");
    const void* outs[] = {o.d_x, o.d_dt, in->d_z ? o.d_z : nullptr, o.d_b, o.d_c};
    for (int i = 0; i < 5; ++i) {
      for (const void* a : {in->d_x, in->d_dt, in->d_z, in->d_b, in->d_c, d_grad_y, d_saved})
        if (a && a == outs[i]) return refuse("a gradient must not be an input");
      for (int j = 0; j < i; ++j)
        if (outs[i] && outs[i] == outs[j]) return refuse("the gradients must be distinct arrays");
    }
  }
  const Work w = work_of(q, true);
  if ((st = check_work(w.bytes, d_work, work_bytes)) != SLA_OK) return st;
  TraceRange tr("sla_selscan_backward");
  const hipStream_t s = (hipStream_t)stream;
  void* const h0 = in->d_h0 ? o.d_h0 : nullptr;
  if (h0 && (q.d_offsets || q.steps == 0)) {
    st = q.dtype == SLA_F64 ? leave_empty<double>(q, d_grad_last, h0, s)
                            : leave_empty<float>(q, d_grad_last, h0, s);
    if (st != SLA_OK) return st;
  }
  const Plan plan = plan_of(q, true);
  return with_type(q, [&](auto t) -> sla_status {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    Args<T> p = args_of<T>(q, *in, plan, w, d_work);
    p.grad_y = (const T*)d_grad_y;
    p.gy_seq = q.d_offsets ? 0 : grad_seq, p.gy_step = grad_step;
    p.grad_last = (const C*)d_grad_last;
    p.saved = (C*)d_saved;
    p.grad_x = (T*)o.d_x, p.grad_dt = (T*)o.d_dt, p.grad_z = (T*)o.d_z;
    p.grad_h0 = (C*)h0;
    const int el = tile_steps(q) / 4;
    p.vec = p.vec && packs(d_grad_y, grad_seq, grad_step, sizeof(T), el, q.d_offsets || q.n_seq == 1,
                           q.steps == 1) &&
            packs(o.d_x, 0, 0, sizeof(T), el, true, true) &&
            packs(o.d_dt, 0, 0, sizeof(T), el, true, true) &&
            (!in->d_z || packs(o.d_z, 0, 0, sizeof(T), el, true, true));
    if (!no_steps(q)) {
      const int64_t groups = plan.rows * plan.blocks;
      sla_status e = with_states(q.n_state, [&](auto ns, auto pad) -> sla_status {
        constexpr int NS = decltype(ns)::value;
        constexpr bool PAD = decltype(pad)::value;
        if (plan.chunks > 1) {
          sla_status e = in_launches(p, groups, [&](dim3 grid) {
            scan_back_local<T, NS, PAD><<<grid, kWG, 0, s>>>(p);
          });
          if (e == SLA_OK) e = join(p, plan, true, s);
          if (e != SLA_OK) return e;
        }
        return in_launches(p, groups, [&](dim3 grid) {
          scan_backward<T, NS, PAD><<<grid, kWG, 0, s>>>(p);
        });
      });
      if (e != SLA_OK) return e;
      const int64_t all = (q.d_offsets ? 1 : q.n_seq) * q.steps;
      const int64_t n = all * 2 * q.groups * q.n_state;
      e = in_launches(p, (n + kWG - 1) / kWG, [&](dim3 grid) {
        sum_blocks<T><<<grid, kWG, 0, s>>>(p, (T*)o.d_b, (T*)o.d_c, all);
      });
      if (e != SLA_OK) return e;
    }
    RowSums<C> r{};
    r.rows = plan.rows;
    const C* parts[] = {p.part_a, p.part_d, p.part_bias};
    void* const outs[] = {o.d_a, o.d_d, o.d_dt_bias};
    for (int k = 0; k < 3; ++k) {
      r.part[k] = parts[k];
      r.out[k] = (C*)outs[k];
      r.n[k] = r.stride[k] = q.dim * (k ? 1 : q.n_state);
    }
    return sum_of_rows(r, s);
  });
}
