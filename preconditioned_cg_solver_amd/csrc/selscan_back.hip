// Selective scans, backward.  With ds = dL/dy silu(z), backwards along a sequence:
//   g_t = ds_t C_t + mu_{t+1},  mu_t = a_t g_t,  mu after the last step = dL/dh_last,
//   dL/dC_t = sum_c ds_t h_t,   dL/dB_t = sum_c g_t delta_t x_t,
//   dL/dA = sum_t mu_t h_{t-1} delta_t,   dL/dh_0 = mu_1,
//   dL/ddelta_t = sum_n mu_t h_{t-1} A + x_t g_t B_t,  dL/dx_t = delta_t sum_n g_t B_t + D ds_t.
// (q = g a h_{t-1} = mu_t h_{t-1} needs no division and no difference.)
//
// A wave works a tile's states out again from the one saved at its start, keeps
// them in registers, with the coefficients of the last steps (the others' are worked
// out twice), and comes back.  Sums over a channel's states and over channels are folded
// between lanes; those over the waves of a workgroup go through LDS, with one barrier a
// tile, and those over workgroups through a workspace, so that every sum is made in one
// order.  Bound by arithmetic: a tile takes 1634 vector instructions; 8 x 2048 x 2048 x 16
// states bf16, cut to two waves a SIMD, 490 us with the vector unit at work 86% of them, after
// a first pass of 106.  fp64, a wave a SIMD: 8 x 2048 x 1024 x 16 states 1395 us the whole
// call, fp32 361.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "rowsum.h"
#include "selscan.h"

namespace sla {
namespace selscan {

sla_status check_in(const sla_selscan_shape& q, const sla_selscan_in* in);
sla_status check_work(size_t need, const void* work, size_t bytes);
template <typename C>
sla_status leave_empty(const sla_selscan_shape& q, const void* from, void* to, hipStream_t s);

namespace {

// Steps whose instructions may mix, while the operands of as many more are on their
// way from LDS: the barriers to the scheduler put those loads first, where it would
// put them last, and keep it from taking so many ahead that the states leave the
// registers.
constexpr int kAhead = 2;
// The last steps of a tile, whose coefficients there are registers for until the way back.
template <typename T>
constexpr int kept_steps() {
  return sizeof(T) == 8 ? 1 : sizeof(T) == 4 ? 2 : 4;
}

template <typename C>
struct Drive {
  C delta, dx;  // delta_t, delta_t x_t
};
template <typename C>
struct Pull {
  C delta, ds;
};

// What a chunk leaves to the one before it, from nothing.
template <typename T, int NS, bool FAST>
__global__ __launch_bounds__(kWG) void scan_back_local(Args<T> p) {
  using C = typename Compute<T>::type;
  using R = Rows<C>;
  constexpr int TS = R::TS, EL = R::EL;
  __shared__ Pull<C> s_pull[kWavesOf][TS][kChannels];
  __shared__ C s_c[kWavesOf][TS][4 * NS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Place w = place_of<T, kWavesOf>(p);
  if (w.some <= 0 || w.part == 0) return;  // what the first leaves is not asked
  auto& pull = s_pull[wave];
  auto& cs = s_c[wave];
  const int q = lane >> 4, c = lane & 15;
  const bool live = c < w.some;
  const int64_t channel = w.channel + c;
  C a2[NS], mu[NS], total = C(0);
  enter_states<NS, FAST>(a2, p.a, channel, p.states, q, live);
#pragma unroll
  for (int j = 0; j < NS; ++j) a2[j] *= C(1.4426950408889634), mu[j] = C(0);
  bool cut = false;

  const int r = lane / R::PER, cc = lane % R::PER * EL, some = w.some - cc;
  const int64_t col = w.channel + (some > 0 ? cc : 0);
  C bias[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) bias[e] = p.bias && e < some ? p.bias[col + e] : C(0);
  settle(bias);
  const int64_t last = w.t0 + (w.t1 - 1 - w.t0) / TS * TS;
  using Row = Stream<FAST, EL, T>;
  Row us(p.dt + w.seq * p.dt_seq + col, p.dt_step, last, r, some, -TS);
  Row zs(p.z + w.seq * p.z_seq + col, p.z_step, last, r, some, -TS);
  Row gs(p.grad_y + w.seq * p.gy_seq + col, p.gy_step, last, r, some, -TS);
  auto ct = shared_stream<FAST, C, NS>(p, p.c + w.seq * p.c_seq + w.group * p.states, p.c_step,
                                       last, -TS);
  const bool gated = p.z != nullptr;
  Pack<T, EL> ur, zr{}, gr;
  Pack<T, Shared<C, NS>::BL> cr;
  auto fetch = [&](int n) {
    ur = us.load(n, TS);
    gr = gs.load(n, TS);
    if (gated) zr = zs.load(n, TS);
    cr = ct.load(n, TS);
    us.move(), gs.move(), zs.move(), ct.move();
  };
  fetch((int)(w.t1 - last));
  Span now = p.offsets ? waited_for(span_of(p, w, last)) : Span{};
  for (int64_t t0 = last; t0 >= w.t0; t0 -= TS) {
    const int n = (int)min((int64_t)TS, w.t1 - t0);
    C delta[EL], ds[EL], slope;
#pragma unroll
    for (int e = 0; e < EL; ++e) delta[e] = (C)ur.v[e] + bias[e], ds[e] = (C)gr.v[e];
    if (p.softplus)
#pragma unroll
      for (int e = 0; e < EL; ++e) delta[e] = softplus(delta[e], slope);
    if (gated)
#pragma unroll
      for (int e = 0; e < EL; ++e) ds[e] *= silu((C)zr.v[e]);
    const unsigned inside = inside_of(w, t0, TS);
    const bool is = inside >> r & 1;
#pragma unroll
    for (int e = 0; e < EL; ++e) pull[r][cc + e] = {is ? delta[e] : C(0), is ? ds[e] : C(0)};
    keep_shared<C, NS>(cs, cr, inside);
    if (t0 > w.t0) fetch(TS);
    unsigned starts, ends;
    int64_t mine;
    edges_of<TS, true>(p, w, now, t0, n, starts, ends, mine);
    wave_sync();
    C sum = C(0);
    struct Step {
      Pull<C> d;
      C c[NS];
    };
    auto read = [&](int i) {
      Step v;
      v.d = pull[i][c];
#pragma unroll
      for (int j = 0; j < NS; ++j) v.c[j] = cs[i][q * NS + j];
      return v;
    };
    auto step = [&](const Step& v) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
        mu[j] = pow2(v.d.delta * a2[j]) * (v.d.ds * v.c[j] + mu[j]);
      sum += v.d.delta;
    };
    if (n == TS && !ends) {
      constexpr int G = 4;
      Step ahead[G];
#pragma unroll
      for (int k = 0; k < G; ++k) ahead[k] = read(TS - 1 - k);
#pragma unroll
      for (int i = TS - 1; i >= 0; i -= G) {
        Step at[G];
#pragma unroll
        for (int k = 0; k < G; ++k) at[k] = ahead[k];
        if (i >= G)
#pragma unroll
          for (int k = 0; k < G; ++k) ahead[k] = read(i - G - k);
#pragma unroll
        for (int k = 0; k < G; ++k) step(at[k]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      for (int i = n - 1; i >= 0; --i) {
        if (ends >> i & 1) {
          const int64_t s = from_lane_of(mine, i);
          enter_states<NS, FAST>(mu, p.grad_last, s * p.dim + channel, p.states, q, live);
          cut = true;
        }
        step(read(i));
      }
    }
    total += sum;
    wave_sync();
  }
  put_states<NS, FAST>(mu, p.ends, w.row * p.dim + channel, p.states, q, live);
  if (q == 0 && live) p.deltas[w.row * p.dim + channel] = total;
  if (threadIdx.x == 0 && w.block == 0) p.cuts[w.row] = cut;
}

// Two waves a SIMD; in fp64 one, with all of its registers.
template <typename T, int NS, bool FAST>
__global__ __launch_bounds__(kWG, sizeof(T) == 8 ? 1 : 2) void scan_backward(Args<T> p) {
  using C = typename Compute<T>::type;
  using R = Rows<C>;
  constexpr int TS = R::TS, EL = R::EL, N4 = 4 * NS;
  __shared__ Drive<C> s_drive[kWavesOf][TS][kChannels];
  __shared__ C s_ds[kWavesOf][TS][kChannels], s_slope[kWavesOf][TS][kChannels];
  __shared__ C s_bias[kWavesOf][kChannels], s_d[kWavesOf][kChannels];
  __shared__ C s_b[kWavesOf][TS][N4], s_c[kWavesOf][TS][N4];
  __shared__ C s_sum[kWavesOf][TS][3][kChannels];  // over states: C h, g B, mu h A / ln 2
  __shared__ C s_bc[2][kWavesOf][TS][2][N4];       // over a wave's channels: of dB, of dC
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Place w = place_of<T, kWavesOf>(p);
  const bool idle = w.some <= 0;  // its workgroup's sums want it all the same
  auto& drive = s_drive[wave];
  auto& dss = s_ds[wave];
  auto& slopes = s_slope[wave];
  auto& bs = s_b[wave];
  auto& cs = s_c[wave];
  auto& sums = s_sum[wave];

  // the lane's channel and states: the channel in bits 0, 1, 4, 5, so that most of the
  // sums over channels are made by swaps of halves and rows
  const int q = lane >> 2 & 3, c = (lane & 3) | (lane >> 4) << 2;
  const bool live = c < w.some;
  const int64_t channel = w.channel + (idle ? 0 : c);
  C a2[NS], mu[NS], da[NS];
  enter_states<NS, FAST>(a2, p.a, channel, p.states, q, live);
  {
    // what enters from the chunk that follows
    const bool end = !p.offsets && w.t1 == p.steps;
    const C* from = p.chunks > 1 && !end ? p.ends : nullptr;
    enter_states<NS, FAST>(mu, from, w.row * p.dim + channel, p.states, q, live);
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) a2[j] *= C(1.4426950408889634), da[j] = C(0);

  const int r = lane / R::PER, cc = lane % R::PER * EL, some = w.some - cc;
  const int64_t col = idle ? 0 : w.channel + (some > 0 ? cc : 0);
  C dbias[EL], ddd[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) dbias[e] = ddd[e] = C(0);
  if (lane < kChannels) {
    s_bias[wave][lane] = p.bias && lane < w.some ? p.bias[w.channel + lane] : C(0);
    s_d[wave][lane] = p.d && lane < w.some ? p.d[w.channel + lane] : C(0);
  }
  if (FAST && some <= 0)
#pragma unroll
    for (int e = 0; e < EL; ++e) drive[r][cc + e] = {C(0), C(0)}, dss[r][cc + e] = C(0);
  wave_sync();
  const int64_t last = w.t0 + (w.t1 - 1 - w.t0) / TS * TS;
  using Row = Stream<FAST, EL, T>;
  Row xs(p.x + w.seq * p.x_seq + col, p.x_step, last, r, some, -TS);
  Row us(p.dt + w.seq * p.dt_seq + col, p.dt_step, last, r, some, -TS);
  Row zs(p.z + w.seq * p.z_seq + col, p.z_step, last, r, some, -TS);
  Row gs(p.grad_y + w.seq * p.gy_seq + col, p.gy_step, last, r, some, -TS);
  auto bt = shared_stream<FAST, C, NS>(p, p.b + w.seq * p.b_seq + w.group * p.states, p.b_step,
                                       last, -TS);
  auto ct = shared_stream<FAST, C, NS>(p, p.c + w.seq * p.c_seq + w.group * p.states, p.c_step,
                                       last, -TS);
  const bool gated = p.z != nullptr;
  const int64_t tile = p.dim * p.states;
  const C* saved = (const C*)p.saved + ((p.offsets ? 0 : w.seq * p.tiles) + last / TS) * tile;
  int64_t to = (w.at + last + r) * p.dim + col;
  Pack<T, EL> xr, ur, zr{}, gr;
  Pack<T, Shared<C, NS>::BL> br, cr;
  C enter[NS];  // the state at the tile's start
  auto fetch = [&](int n) {
    xr = xs.load(n, TS);
    ur = us.load(n, TS);
    gr = gs.load(n, TS);
    if (gated) zr = zs.load(n, TS);
    br = bt.load(n, TS);
    cr = ct.load(n, TS);
    get_states<NS, FAST>(enter, saved, channel, p.states, q, live);
    xs.move(), us.move(), gs.move(), zs.move(), bt.move(), ct.move();
    saved -= tile;
  };
  if (!idle) fetch((int)(w.t1 - last));
  else {
    for (int i = lane; i < TS * 2 * N4; i += kLanes)
      (&s_bc[0][wave][0][0][0])[i] = (&s_bc[1][wave][0][0][0])[i] = C(0);
  }
  Span now = p.offsets ? waited_for(span_of(p, w, last)) : Span{};
  int turn = 0;

  for (int64_t t0 = last; t0 >= w.t0; t0 -= TS, turn ^= 1) {
    const int n = (int)min((int64_t)TS, w.t1 - t0);
    // Steps of a sequence: the others' rows may hold anything, and have gradients of zero.
    const unsigned inside = inside_of(w, t0, TS);
    if (!idle) {
      const Pack<T, EL> x = xr, z = zr, gy = gr;
      const bool is = inside >> r & 1;
      C zsig[EL];
      {
        C delta[EL], slope[EL], ds[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e)
          delta[e] = (C)ur.v[e] + s_bias[wave][cc + e], ds[e] = (C)gy.v[e];
        if (p.softplus)
#pragma unroll
          for (int e = 0; e < EL; ++e) {
            delta[e] = softplus(delta[e], slope[e]);
            slopes[r][cc + e] = slope[e];
          }
        if (gated)
#pragma unroll
          for (int e = 0; e < EL; ++e) {
            zsig[e] = sigmoid((C)z.v[e]);
            ds[e] *= silu_of((C)z.v[e], zsig[e]);
          }
        if (!FAST || some > 0)  // else they stay 0, as what does not exist adds nothing to sums
#pragma unroll
          for (int e = 0; e < EL; ++e) {
            drive[r][cc + e] = {delta[e], delta[e] * (C)x.v[e]};
            dss[r][cc + e] = ds[e];
          }
      }
      keep_shared<C, NS>(bs, br);
      keep_shared<C, NS>(cs, cr);
      C h0[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) h0[j] = enter[j];
      settle(h0);
      if (t0 > w.t0) fetch(TS);
      unsigned starts, ends;
      int64_t mine;
      edges_of<TS, true>(p, w, now, t0, n, starts, ends, mine);
      // In the upper half the steps of no sequence, which are left out (a word of its own, and a
      // test for it, cost registers in all tiles: 8 x 2048 x 2048 bf16 both ways 845 and 873 us).
      starts |= (~inside & 0xffffu) << 16;
      wave_sync();

      struct Step {
        Drive<C> d;
        C ds, b[NS], c[NS];
      };
      auto read = [&](int i) {
        Step v;
        v.d = drive[i][c];
        v.ds = dss[i][c];
#pragma unroll
        for (int j = 0; j < NS; ++j) v.b[j] = bs[i][q * NS + j], v.c[j] = cs[i][q * NS + j];
        return v;
      };
      // A step forward, from `before` to `now`, and back.
      auto coefficients = [&](const Step& v, C (&coef)[NS]) {
#pragma unroll
        for (int j = 0; j < NS; ++j) coef[j] = pow2(v.d.delta * a2[j]);
      };
      auto advance = [&](const Step& v, int i, const C (&coef)[NS], const C (&before)[NS],
                         C (&now)[NS]) {
        C s = C(0);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          now[j] = coef[j] * before[j] + v.d.dx * v.b[j];
          const C m = v.c[j] * now[j];
          s += FAST || q * NS + j < p.states ? m : C(0);
        }
        s += from_lane<kRor8>(s);
        s += from_lane<kRor4>(s);
        sums[i][0][c] = s;
      };
      auto retreat = [&](const Step& v, int i, const C (&coef)[NS], const C (&before)[NS],
                         const C (&now)[NS]) {
        C gb = C(0), qa = C(0), db[NS], dc[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const C g = v.ds * v.c[j] + mu[j];
          dc[j] = v.ds * now[j];
          db[j] = g * v.d.dx;
          const C m = g * v.b[j];
          gb += FAST || q * NS + j < p.states ? m : C(0);
          mu[j] = coef[j] * g;
          const C mh = mu[j] * before[j];
          const C ma = mh * a2[j];
          qa += FAST || q * NS + j < p.states ? ma : C(0);
          da[j] += mh * v.d.delta;
        }
        // lanes of even q end with the sum of one, those of odd q with the other's
        C two = (q & 1 ? qa : gb) + from_lane<kRor4>(q & 1 ? gb : qa);
        two += from_lane<kRor8>(two);
        sums[i][1 + (q & 1)][c] = two;
        // over the channels (lanes that hold the same sum write it to the same place)
        const int odd = lane >> 4 & 1, high = lane >> 5;
        if constexpr (NS == 4) {
          C vb = fold_rows(fold_halves(db[0], db[1]), fold_halves(db[2], db[3]));
          C vc = fold_rows(fold_halves(dc[0], dc[1]), fold_halves(dc[2], dc[3]));
          vb += from_lane<kXor1>(vb);
          vc += from_lane<kXor1>(vc);
          C o = lane & 1 ? vc : vb;
          o += from_lane<kXor2>(o);
          s_bc[turn][wave][i][lane & 1][q * NS + 2 * odd + high] = o;
        } else if constexpr (NS == 2) {
          C o = fold_rows(fold_halves(db[0], db[1]), fold_halves(dc[0], dc[1]));
          o += from_lane<kXor1>(o);
          o += from_lane<kXor2>(o);
          s_bc[turn][wave][i][odd][q * NS + high] = o;
        } else {
          C o = fold_halves(db[0], dc[0]);
          o = fold_rows(o, o);
          o += from_lane<kXor1>(o);
          o += from_lane<kXor2>(o);
          s_bc[turn][wave][i][high][q] = o;
        }
      };
      if (n == TS && !starts && !ends) {
        constexpr int G = kAhead, KEPT = kept_steps<T>();
        C hs[TS][NS], kept[KEPT][NS];
        Step at[G], ahead[G];
#pragma unroll
        for (int k = 0; k < G; ++k) ahead[k] = read(k);
#pragma unroll
        for (int i = 0; i < TS; i += G) {
#pragma unroll
          for (int k = 0; k < G; ++k) {
            at[k] = ahead[k];
            if (i + G < TS) ahead[k] = read(i + G + k);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < G; ++k) {
            C coef[NS];
            coefficients(at[k], coef);
            advance(at[k], i + k, coef, i + k ? hs[i + k ? i + k - 1 : 0] : h0, hs[i + k]);
            if (i + k >= TS - KEPT)
#pragma unroll
              for (int j = 0; j < NS; ++j) kept[i + k - (TS - KEPT)][j] = coef[j];
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int k = 0; k < G; ++k) ahead[k] = read(TS - 1 - k);
#pragma unroll
        for (int i = TS - 1; i >= 0; i -= G) {
#pragma unroll
          for (int k = 0; k < G; ++k) {
            at[k] = ahead[k];
            if (i >= G) ahead[k] = read(i - G - k);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < G; ++k) {
            C coef[NS];
            if (i - k >= TS - KEPT)
#pragma unroll
              for (int j = 0; j < NS; ++j) coef[j] = kept[i - k - (TS - KEPT)][j];
            else
              coefficients(at[k], coef);
            retreat(at[k], i - k, coef, i - k ? hs[i - k ? i - k - 1 : 0] : h0, hs[i - k]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        // Tiles in which a sequence begins or ends, step by step; the states are in memory.
        // (Counting steps of no sequence as zeros would not do: a state or gradient beside them
        // that is not finite makes NaN of a product with 0.)
        C hs[TS + 1][NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) hs[0][j] = h0[j];
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          C before[NS], now[NS];
#pragma unroll
          for (int j = 0; j < NS; ++j) before[j] = now[j] = hs[i][j];
          if (!(starts >> (16 + i) & 1)) {
            if (i > 0 && (starts >> i & 1))
              enter_states<NS, FAST>(before, p.h0, from_lane_of(mine, i) * p.dim + channel,
                                     p.states, q, live);
            const Step v = read(i);
            C coef[NS];
            coefficients(v, coef);
            advance(v, i, coef, before, now);
          }
#pragma unroll
          for (int j = 0; j < NS; ++j) hs[i + 1][j] = now[j];
        }
#pragma unroll 1
        for (int i = n - 1; i >= 0; --i) {
          if (starts >> (16 + i) & 1) {
            for (int k = lane; k < 2 * N4; k += kLanes) (&s_bc[turn][wave][i][0][0])[k] = C(0);
            continue;
          }
          const bool begins = starts >> i & 1, stops = ends >> i & 1;
          const int64_t s = from_lane_of(mine, i);
          C before[NS], now[NS];
#pragma unroll
          for (int j = 0; j < NS; ++j) before[j] = hs[i][j], now[j] = hs[i + 1][j];
          if (stops)
            enter_states<NS, FAST>(mu, p.grad_last, s * p.dim + channel, p.states, q, live);
          if (begins && i > 0)
            enter_states<NS, FAST>(before, p.h0, s * p.dim + channel, p.states, q, live);
          const Step v = read(i);
          C coef[NS];
          coefficients(v, coef);
          retreat(v, i, coef, before, now);
          if (begins && p.grad_h0)
            put_states<NS, FAST>(mu, p.grad_h0, s * p.dim + channel, p.states, q, live);
        }
      }
      wave_sync();

      if (r < n) {
        C gx[EL], gb[EL], du[EL], dsv[EL], xv[EL];
        Pack<T, EL> ox, ou, oz{};
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          xv[e] = (C)x.v[e], gb[e] = sums[r][1][cc + e], dsv[e] = dss[r][cc + e];
          du[e] = sums[r][2][cc + e] * C(0.69314718055994531) + xv[e] * gb[e];
          gx[e] = drive[r][cc + e].delta * gb[e];
          ddd[e] += is ? dsv[e] * xv[e] : C(0);
        }
        if (p.softplus)
#pragma unroll
          for (int e = 0; e < EL; ++e) du[e] *= slopes[r][cc + e];
#pragma unroll
        for (int e = 0; e < EL; ++e) du[e] = is ? du[e] : C(0);
        C skip[EL];
        if (p.d)
#pragma unroll
          for (int e = 0; e < EL; ++e) skip[e] = s_d[wave][cc + e], gx[e] += skip[e] * dsv[e];
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          dbias[e] += du[e];
          ou.v[e] = (T)du[e], ox.v[e] = is ? (T)gx[e] : T(0);
        }
        if (gated) {
          C total[EL];
#pragma unroll
          for (int e = 0; e < EL; ++e) total[e] = sums[r][0][cc + e];
          if (p.d)
#pragma unroll
            for (int e = 0; e < EL; ++e) total[e] += skip[e] * xv[e];
#pragma unroll
          for (int e = 0; e < EL; ++e)
            oz.v[e] = is ? (T)((C)gy.v[e] * total[e] * silu_slope((C)z.v[e], zsig[e])) : T(0);
        }
        store_some<FAST, EL>(p.grad_x + to, ox, some);
        store_some<FAST, EL>(p.grad_dt + to, ou, some);
        if (gated) store_some<FAST, EL>(p.grad_z + to, oz, some);
      }
      to -= TS * p.dim;
    }
    // One barrier a tile: the other half of s_bc is written next, and read by a
    // wave only after the barrier that follows.
    lds_barrier();
    C* const out = p.part_bc + ((int64_t)w.block * (p.offsets ? p.steps : p.n_seq * p.steps) +
                                w.at + t0) * 2 * p.states;
    for (int k = threadIdx.x; k < n * 2 * N4; k += kWG) {
      const int i = k / (2 * N4), of = k / N4 & 1, st = k % N4;
      C v = s_bc[turn][0][i][of][st];
#pragma unroll
      for (int o = 1; o < kWavesOf; ++o) v += s_bc[turn][o][i][of][st];
      if (st < p.states) out[(i * 2 + of) * p.states + st] = v;
    }
  }
  if (idle) return;
  put_states<NS, FAST>(da, p.part_a, w.row * p.dim + channel, p.states, q, live);
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
  if (!q.dim) return SLA_OK;
  const sla_selscan_grads& o = *grads;
  if (!o.d_a) return refuse("a gradient is NULL");
  // packed rows without a sequence, whose gradients are zeros
  const bool none = q.d_offsets && !q.n_seq && q.steps;
  if (!no_steps(q) || none) {
    if (!none && (!d_saved || !d_grad_y)) return refuse("the saved states or grad_y is NULL");
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
  if (none) {
    const int64_t shared = q.groups * q.n_state;
    for (auto [to, width] : {std::pair{o.d_x, q.dim}, {o.d_dt, q.dim},
                             {in->d_z ? o.d_z : nullptr, q.dim}, {o.d_b, shared}, {o.d_c, shared}})
      if (to && (st = sla_rows_clear(q.d_offsets, 0, q.steps, width, q.dtype, to, stream)) != SLA_OK)
        return st;
  }
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
    p.fast = p.fast && packs(d_grad_y, grad_seq, grad_step, sizeof(T), el, q.d_offsets || q.n_seq == 1,
                           q.steps == 1) &&
            packs(o.d_x, 0, 0, sizeof(T), el, true, true) &&
            packs(o.d_dt, 0, 0, sizeof(T), el, true, true) &&
            (!in->d_z || packs(o.d_z, 0, 0, sizeof(T), el, true, true));
    if (!no_steps(q)) {
      const int64_t groups = plan.rows * plan.blocks;
      sla_status e = with_states(q.n_state, p.fast, [&](auto ns, auto fast) -> sla_status {
        constexpr int NS = decltype(ns)::value;
        constexpr bool FAST = decltype(fast)::value;
        if (plan.chunks > 1) {
          sla_status e = in_launches(p, groups, [&](dim3 grid) {
            scan_back_local<T, NS, FAST><<<grid, kWG, 0, s>>>(p);
          });
          if (e == SLA_OK) e = join(p, plan, true, s);
          if (e != SLA_OK) return e;
        }
        return in_launches(p, groups, [&](dim3 grid) {
          scan_backward<T, NS, FAST><<<grid, kWG, 0, s>>>(p);
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
