// Selective scans, forward: h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t per
// channel and state, y_t = C_t . h_t + D x_t, gated by z.
//
// Per state and step the scan takes a product, an exponential, a product and two
// fused sums, so with 16 states it is bound by arithmetic, not bytes.  A lane keeps
// its states in registers through all steps; what depends on the channel alone
// (softplus, the gate) is worked out once per element in another sharing of the
// tile among the lanes, and handed over through LDS of the wave.  A tile takes 486 vector
// instructions; 8 x 2048 x 2048 x 16 states bf16, a wave a SIMD, 212 us with the vector unit
// at work 60% of them, 16 x 2048 x 2048 332.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "selscan.h"

namespace sla {
namespace selscan {
namespace {

template <typename C>
struct Drive {
  C delta, dx;  // delta_t, delta_t x_t
};

// FULL writes the outputs from the state that enters the chunk; otherwise what
// the chunk leaves from nothing, for the joining.
template <typename T, int NS, bool FAST, bool FULL>
__global__ __launch_bounds__(kWG) void scan_forward(Args<T> p) {
  using C = typename Compute<T>::type;
  using R = Rows<C>;
  constexpr int TS = R::TS, EL = R::EL;
  __shared__ Drive<C> s_drive[kWavesOf][TS][kChannels];
  __shared__ C s_b[kWavesOf][TS][4 * NS], s_c[FULL ? kWavesOf : 1][TS][4 * NS];
  __shared__ C s_sum[FULL ? kWavesOf : 1][TS][kChannels];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Place w = place_of<T, kWavesOf>(p);
  // what the last chunk leaves is not asked
  if (w.some <= 0 || (!FULL && w.part == p.chunks - 1)) return;
  auto& drive = s_drive[wave];
  auto& bs = s_b[wave];
  auto& cs = s_c[FULL ? wave : 0];
  auto& sums = s_sum[FULL ? wave : 0];

  // the lane's channel and states
  const int q = lane >> 4, c = lane & 15;
  const bool live = c < w.some;
  const int64_t channel = w.channel + c;
  C a2[NS], h[NS], total = C(0);
  enter_states<NS, FAST>(a2, p.a, channel, p.states, q, live);
#pragma unroll
  for (int j = 0; j < NS; ++j) a2[j] *= C(1.4426950408889634);
  bool cut = false;
  {
    const bool first = !p.offsets && w.t0 == 0;
    const C* from = FULL ? (p.chunks > 1 ? p.ends : first ? p.h0 : nullptr)
                         : (first ? p.h0 : nullptr);
    const int64_t row = FULL && p.chunks > 1 ? w.row : w.seq;
    enter_states<NS, FAST>(h, from, row * p.dim + channel, p.states, q, live);
    cut = first;
  }

  // its share of the rows
  const int r = lane / R::PER, cc = lane % R::PER * EL, some = w.some - cc;
  const int64_t col = w.channel + (some > 0 ? cc : 0);
  C bias[EL], dd[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    bias[e] = p.bias && e < some ? p.bias[col + e] : C(0);
    dd[e] = FULL && p.d && e < some ? p.d[col + e] : C(0);
  }
  settle(bias);
  settle(dd);
  using Row = Stream<FAST, EL, T>;
  Row xs(p.x + w.seq * p.x_seq + col, p.x_step, w.t0, r, some, TS);
  Row us(p.dt + w.seq * p.dt_seq + col, p.dt_step, w.t0, r, some, TS);
  Row zs(p.z + w.seq * p.z_seq + col, p.z_step, w.t0, r, some, TS);
  auto bt = shared_stream<FAST, C, NS>(p, p.b + w.seq * p.b_seq + w.group * p.states, p.b_step,
                                       w.t0, TS);
  auto ct = shared_stream<FAST, C, NS>(p, p.c + w.seq * p.c_seq + w.group * p.states, p.c_step,
                                       w.t0, TS);
  const bool gated = FULL && p.z;
  T* y = FULL ? p.y + (w.at + w.t0 + r) * p.dim + col : nullptr;
  const int64_t tile = p.dim * p.states;
  C* saved = FULL && p.saved ? p.saved + ((p.offsets ? 0 : w.seq * p.tiles) + w.t0 / TS) * tile
                             : nullptr;
  Pack<T, EL> xr, ur, zr{};
  Pack<T, Shared<C, NS>::BL> br, cr{};
  auto fetch = [&](int n) {
    xr = xs.load(n, TS);
    ur = us.load(n, TS);
    br = bt.load(n, TS);
    xs.move(), us.move(), bt.move();
    if constexpr (FULL) {
      if (gated) zr = zs.load(n, TS);
      cr = ct.load(n, TS);
      zs.move(), ct.move();
    }
  };
  int left = (int)(w.t1 - w.t0);  // steps
  fetch(min(left, TS));
  Span now = p.offsets ? waited_for(span_of(p, w, w.t0)) : Span{};

  for (int64_t t0 = w.t0; left > 0; t0 += TS, left -= TS) {
    const int n = min(left, TS);
    const Pack<T, EL> x = xr, z = zr;
    C delta[EL], slope;
#pragma unroll
    for (int e = 0; e < EL; ++e) delta[e] = (C)ur.v[e] + bias[e];
    if (p.softplus)
#pragma unroll
      for (int e = 0; e < EL; ++e) delta[e] = softplus(delta[e], slope);
#pragma unroll
    for (int e = 0; e < EL; ++e) drive[r][cc + e] = {delta[e], delta[e] * (C)x.v[e]};
    keep_shared<C, NS>(bs, br);
    if constexpr (FULL) keep_shared<C, NS>(cs, cr);
    if (left > TS) fetch(min(left - TS, TS));
    unsigned starts, ends;
    int64_t mine;
    edges_of<TS, false>(p, w, now, t0, n, starts, ends, mine);
    if (!p.offsets) starts = 0;  // h holds what enters
    auto begin = [&](int i) {
      const int64_t s = from_lane_of(mine, i);
      enter_states<NS, FAST>(h, p.h0, s * p.dim + channel, p.states, q, live);
      cut = true;
    };
    if (starts & 1) begin(0);
    if (FULL && saved) {
      put_states<NS, FAST>(h, saved, channel, p.states, q, live);
      saved += tile;
    }
    wave_sync();
    C sum = C(0);
    struct Step {
      Drive<C> d;
      C b[NS], c[FULL ? NS : 1];
    };
    auto read = [&](int i) {
      Step v;
      v.d = drive[i][c];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        v.b[j] = bs[i][q * NS + j];
        if constexpr (FULL) v.c[j] = cs[i][q * NS + j];
      }
      return v;
    };
    auto step = [&](const Step& v) {
      C s = C(0);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        h[j] = pow2(v.d.delta * a2[j]) * h[j] + v.d.dx * v.b[j];
        if constexpr (FULL) {
          const C m = v.c[j] * h[j];
          s += FAST || q * NS + j < p.states ? m : C(0);
        }
      }
      if constexpr (!FULL) sum += v.d.delta;
      return s;
    };
    if (n == TS && !starts && !ends) {
      // groups of steps, the next one's operands on their way from LDS
      constexpr int G = 4;
      Step ahead[G];
#pragma unroll
      for (int k = 0; k < G; ++k) ahead[k] = read(k);
#pragma unroll
      for (int i = 0; i < TS; i += G) {
        Step at[G];
        C s[G];
#pragma unroll
        for (int k = 0; k < G; ++k) at[k] = ahead[k];
        if (i + G < TS)
#pragma unroll
          for (int k = 0; k < G; ++k) ahead[k] = read(i + G + k);
#pragma unroll
        for (int k = 0; k < G; ++k) s[k] = step(at[k]);
        if constexpr (FULL)
          sums[i + ((q >> 1) | ((q & 1) << 1))][c] =
              fold_rows(fold_halves(s[0], s[1]), fold_halves(s[2], s[3]));
      }
    } else {
      for (int i = 0; i < n; ++i) {
        if (i > 0 && (starts >> i & 1)) begin(i);
        C s = step(read(i));
        if constexpr (FULL) {
          s = fold_halves(s, s);
          sums[i][c] = fold_rows(s, s);
          if (ends >> i & 1) {
            const int64_t at = from_lane_of(mine, i);
            put_states<NS, FAST>(h, p.h_last, at * p.dim + channel, p.states, q, live);
          }
        }
      }
    }
    total += sum;
    wave_sync();
    if constexpr (FULL) {
      if (r < n && t0 + r >= w.lo && t0 + r < w.hi) {
        C v[EL];
        Pack<T, EL> o;
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = sums[r][cc + e];
        if (p.d)
#pragma unroll
          for (int e = 0; e < EL; ++e) v[e] += dd[e] * (C)x.v[e];
        if (gated)
#pragma unroll
          for (int e = 0; e < EL; ++e) v[e] *= silu((C)z.v[e]);
#pragma unroll
        for (int e = 0; e < EL; ++e) o.v[e] = (T)v[e];
        store_some<FAST, EL>(y, o, some);
      }
      y += TS * p.dim;
      wave_sync();
    }
  }
  if constexpr (!FULL) {
    put_states<NS, FAST>(h, p.ends, w.row * p.dim + channel, p.states, q, live);
    if (q == 0 && live) p.deltas[w.row * p.dim + channel] = total;
    if (threadIdx.x == 0 && w.block == 0) p.cuts[w.row] = cut;
  }
}

// Sequences of a few steps, a serving step above all: 4 lanes take a channel from the
// first step to the last, its states among them, without LDS.  n x steps x 4096 x 16
// states bf16, here and in tiles, us: 16 x 1 4.8 and 8.6, 16 x 4 7.1 and 9.9, 16 x 8 10.1 and
// 11.4, 16 x 16 15.9 and 14.3; 64 x 1 10.5 and 22.6, 64 x 8 25.3 and 29.7, 64 x 16 45.7 and 38.5.
constexpr int kFew = 8;
template <typename T, int NS, bool FAST>
__global__ __launch_bounds__(kWG) void scan_few(Args<T> p) {
  using C = typename Compute<T>::type;
  const int64_t k = (p.before + blockIdx.x) * kWG + threadIdx.x;
  const int q = (int)(k & 3);
  const int64_t s = (k >> 2) / p.dim, channel = (k >> 2) % p.dim;
  if (s >= p.n_seq) return;
  const int g = (int)(channel / p.group_dim), at = q * NS;
  const T* x = p.x + s * p.x_seq + channel;
  const T* u = p.dt + s * p.dt_seq + channel;
  const T* z = p.z ? p.z + s * p.z_seq + channel : nullptr;
  const T* b = p.b + s * p.b_seq + (int64_t)g * p.states + (FAST ? at : 0);
  const T* c = p.c + s * p.c_seq + (int64_t)g * p.states + (FAST ? at : 0);
  T* y = p.y + s * p.steps * p.dim + channel;
  C a2[NS], h[NS];
  get_states<NS, FAST>(a2, p.a, channel, p.states, q, true);
  get_states<NS, FAST>(h, p.h0, s * p.dim + channel, p.states, q, true);
#pragma unroll
  for (int j = 0; j < NS; ++j) a2[j] *= C(1.4426950408889634);
  const C bias = p.bias ? p.bias[channel] : C(0), d = p.d ? p.d[channel] : C(0);
  for (int64_t t = 0; t < p.steps; ++t) {
    C bv[NS], cv[NS];
    if constexpr (FAST) {
      const auto bp = *(const Pack<T, NS>*)b, cp = *(const Pack<T, NS>*)c;
#pragma unroll
      for (int j = 0; j < NS; ++j) bv[j] = (C)bp.v[j], cv[j] = (C)cp.v[j];
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const bool in = at + j < p.states;
        bv[j] = in ? (C)b[at + j] : C(0), cv[j] = in ? (C)c[at + j] : C(0);
      }
    }
    const C xv = (C)*x;
    C delta = (C)*u + bias, slope, sum = C(0);
    if (p.softplus) delta = softplus(delta, slope);
    const C dx = delta * xv;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      h[j] = pow2(delta * a2[j]) * h[j] + dx * bv[j];
      const C m = cv[j] * h[j];
      sum += FAST || at + j < p.states ? m : C(0);
    }
    sum += from_lane<kXor1>(sum);
    sum += from_lane<kXor2>(sum);
    if (p.d) sum += d * xv;
    if (z) {
      sum *= silu((C)*z);
      z += p.z_step;
    }
    if (q == 0) *y = (T)sum;
    x += p.x_step, u += p.dt_step, b += p.b_step, c += p.c_step, y += p.dim;
  }
  put_states<NS, FAST>(h, p.h_last, s * p.dim + channel, p.states, q, true);
}

// h e^(a sum), for exponents whose power leaves the range where the product does
// not: in four factors, none of them 0, so that a state that is not finite
// stays so; one that is 0 stays 0.
template <typename C>
__device__ __forceinline__ C factor(C a, C sum) {
  constexpr C kLow = sizeof(C) == 8 ? C(-1022) : C(-126);
  const C e = a == C(0) ? C(0) : a * sum * C(1.4426950408889634 / 4);
  return pow2(max(e, kLow));
}
template <typename C>
__device__ __forceinline__ C carried(C h, C f) {
  return h == C(0) ? C(0) : h * f * f * f * f;
}

// Follows each state through the chunks, in place: what a chunk leaves from
// nothing becomes what enters it.  A thread has one state of a sequence (packed: of
// all); the loads of sixteen chunks are on their way together.
template <typename T, bool BACKWARD>
__global__ __launch_bounds__(kLanes) void scan_join(Args<T> p) {
  using C = typename Compute<T>::type;
  const int64_t per = p.dim * p.states;
  const int64_t k = (p.before + blockIdx.x) * kLanes + threadIdx.x;
  const int64_t seq = k / per, at = k % per;
  if (seq >= (p.offsets ? 1 : p.n_seq)) return;
  const int64_t channel = at / p.states;
  const C a = p.a[at];
  const C* start = BACKWARD ? p.grad_last : p.h0;
  C h = !p.offsets && start ? start[seq * per + at] : C(0);
  constexpr int U = 16;
  const int64_t first = seq * p.chunks + (BACKWARD ? p.chunks - 1 : 0), step = BACKWARD ? -1 : 1;
  C* ends = p.ends + first * per + at;
  const C* from = ends;
  const C* sums = p.deltas + first * p.dim + channel;
  const int* cuts = p.cuts + first;
  for (int left = p.chunks; left > 0; left -= U) {
    C end[U], sum[U];
    int cut[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      end[u] = *from;
      sum[u] = *sums;
      cut[u] = *cuts;
      const int64_t hop = u + 1 < left ? step : 0;
      from += hop * per, sums += hop * p.dim, cuts += hop;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const C f = factor(a, sum[u]);
      if (u < left) *ends = h;
      ends += step * per;
      h = cut[u] ? end[u] : carried(h, f) + end[u];
    }
  }
}

// Sequences without steps leave the state that they began with: a workgroup takes
// kWG elements of a state, of one sequence after the other.
template <typename C>
__global__ __launch_bounds__(kWG) void scan_empty(const int64_t* offsets, int64_t n_seq,
                                                  int64_t per, const C* from, C* to) {
  const int64_t i = (int64_t)blockIdx.x * kWG + threadIdx.x;
  for (int64_t s = blockIdx.y; s < n_seq; s += gridDim.y) {
    if (offsets && offsets[s + 1] > offsets[s]) continue;
    if (i < per) to[s * per + i] = from ? from[s * per + i] : C(0);
  }
}

}  // namespace

sla_status refuse(const char* msg) {
  set_error(msg);
  return SLA_ERR_INVALID_ARG;
}
bool empty(const sla_selscan_shape& q) { return q.n_seq == 0 || q.dim == 0; }
bool no_steps(const sla_selscan_shape& q) { return empty(q) || q.steps == 0; }

sla_status check_shape(const sla_selscan_shape* q) {
  if (!q) return refuse("shape is NULL");
  if (q->n_seq < 0 || q->steps < 0 || q->dim < 0) return refuse("negative size");
  if (q->dtype != SLA_F64 && q->dtype != SLA_F32 && q->dtype != SLA_BF16 && q->dtype != SLA_F16)
    return refuse("unknown dtype");
  if (q->softplus != 0 && q->softplus != 1) return refuse("softplus must be 0 or 1");
  if (q->groups < 1 || q->dim % q->groups) return refuse("the groups must divide the channels");
  if (q->n_state < 1) return refuse("a channel needs a state");
  const int64_t seqs = q->d_offsets ? 1 : q->n_seq;
  if (q->n_state > 16) {
    set_error("at most 16 states a channel");
    return SLA_ERR_UNSUPPORTED;
  }
  if (q->n_seq >= INT32_MAX || q->dim >= (1 << 23) || q->steps >= ((int64_t)1 << 40) ||
      (__int128)seqs * (q->steps + 16) * (q->dim + 64) * 16 >= ((__int128)1 << 59) ||
      (__int128)q->n_seq * q->dim * 16 >= ((__int128)1 << 59)) {
    set_error("sizes beyond what a call can index");
    return SLA_ERR_UNSUPPORTED;
  }
  return SLA_OK;
}

Plan plan_of(const sla_selscan_shape& q, bool backward) {
  Plan p;
  if (no_steps(q)) return p;
  const bool packed = q.d_offsets != nullptr;
  const int64_t per = q.dim / q.groups, seqs = packed ? 1 : q.n_seq;
  const int ts = tile_steps(q);
  p.blocks = (int)(q.groups * ((per + kChannels * kWavesOf - 1) / (kChannels * kWavesOf)));
  p.tiles = (q.steps + ts - 1) / ts;
  const int64_t waves = seqs * q.groups * ((per + kChannels - 1) / kChannels);
  // Waves that leave SIMDs idle have their sequences cut, which costs a pass over the
  // steps that writes nothing.  With 16 states, us, whole and cut to 4096 waves: forward 2 x
  // 2048 x 2048 bf16 (256 waves) 201 and 73, 4 x 2048 x 2048 200 and 128, 8 x 2048 x 2048 (a wave
  // a SIMD) 215 and 239, 16 x 2048 x 2048 330 and 437; backward 695 and 176, 707 and 335, 717 and
  // 628, 1026 and 1168.  Packed sequences make chunks of uneven work: 30011 x 1000 fp16 cut
  // to 4096 355 and 720, to 8192 320 and 689.
  int64_t chunks = 1;
  if (waves < (backward ? 1536 : 768))
    chunks = std::min(((packed ? 8192 : 4096) + waves - 1) / waves, (p.tiles + 3) / 4);
  // 2^31 steps of a chunk are more than any chunk has, also of one a sequence
  const int64_t least = (q.steps >> 30) + 1;
  chunks = std::max(chunks, least);
  const int64_t tiles = (p.tiles + chunks - 1) / chunks;
  p.chunk = (int)(tiles * ts);
  p.chunks = (int)((p.tiles + tiles - 1) / tiles);
  p.rows = seqs * p.chunks;
  return p;
}

Work work_of(const sla_selscan_shape& q, bool backward) {
  Work w;
  if (no_steps(q)) return w;
  const Plan p = plan_of(q, backward);
  const size_t size = q.dtype == SLA_F64 ? 8 : 4, rows = (size_t)p.rows;
  const size_t states = align_up(rows * q.dim * q.n_state * size);
  const size_t channels = align_up(rows * q.dim * size);
  if (p.chunks > 1) {
    w.deltas_at = states;
    w.cuts_at = w.deltas_at + channels;
    w.bytes = w.cuts_at + align_up(rows * sizeof(int));
  }
  if (backward) {
    const size_t all = (size_t)(q.d_offsets ? 1 : q.n_seq) * q.steps;
    w.a_at = w.bytes;
    w.d_at = w.a_at + states;
    w.bias_at = w.d_at + channels;
    w.bc_at = w.bias_at + channels;
    w.bytes = w.bc_at + align_up((size_t)p.blocks * all * 2 * q.n_state * size);
  }
  return w;
}

bool packs(const void* p, int64_t seq, int64_t step, size_t bytes, int v, bool one_seq,
           bool one_step) {
  return (uintptr_t)p % (v * bytes) == 0 && (seq % v == 0 || one_seq) &&
         (step % v == 0 || one_step);
}

template <typename T>
Args<T> args_of(const sla_selscan_shape& q, const sla_selscan_in& in, const Plan& plan,
                const Work& w, void* work) {
  using C = typename Compute<T>::type;
  Args<T> p{};
  const bool packed = q.d_offsets != nullptr;
  p.x = (const T*)in.d_x, p.x_seq = packed ? 0 : in.x_seq, p.x_step = in.x_step;
  p.dt = (const T*)in.d_dt, p.dt_seq = packed ? 0 : in.dt_seq, p.dt_step = in.dt_step;
  p.z = (const T*)in.d_z, p.z_seq = packed ? 0 : in.z_seq, p.z_step = in.z_step;
  p.b = (const T*)in.d_b, p.b_seq = packed ? 0 : in.b_seq, p.b_step = in.b_step;
  p.c = (const T*)in.d_c, p.c_seq = packed ? 0 : in.c_seq, p.c_step = in.c_step;
  p.a = (const C*)in.d_a, p.d = (const C*)in.d_d, p.bias = (const C*)in.d_dt_bias;
  p.h0 = (const C*)in.d_h0;
  p.offsets = q.d_offsets;
  p.n_seq = q.n_seq, p.steps = q.steps, p.dim = q.dim;
  p.states = (int)q.n_state, p.groups = (int)q.groups, p.group_dim = q.dim / q.groups;
  p.blocks = plan.blocks, p.chunk = plan.chunk, p.chunks = plan.chunks, p.tiles = plan.tiles;
  p.softplus = q.softplus;
  const bool one = packed || q.n_seq == 1, step = q.steps == 1;
  const int el = tile_steps(q) * kChannels / kLanes, ns = q.n_state <= 4 ? 1 : q.n_state <= 8 ? 2 : 4;
  const int bl = ns;  // what a lane takes of B and C, or more
  const size_t b = sizeof(T);
  p.fast = p.group_dim % el == 0 && packs(in.d_x, in.x_seq, in.x_step, b, el, one, step) &&
          packs(in.d_dt, in.dt_seq, in.dt_step, b, el, one, step) &&
          (!in.d_z || packs(in.d_z, in.z_seq, in.z_step, b, el, one, step));
  p.fast = p.fast && p.states == 4 * ns && packs(in.d_b, in.b_seq, in.b_step, b, bl, one, step) &&
           packs(in.d_c, in.c_seq, in.c_step, b, bl, one, step);
  char* base = (char*)work;
  p.ends = (C*)base, p.deltas = (C*)(base + w.deltas_at), p.cuts = (int*)(base + w.cuts_at);
  p.part_a = (C*)(base + w.a_at), p.part_d = (C*)(base + w.d_at);
  p.part_bias = (C*)(base + w.bias_at), p.part_bc = (C*)(base + w.bc_at);
  return p;
}

template <typename T>
sla_status join(const Args<T>& p, const Plan& plan, bool backward, hipStream_t s) {
  if (plan.chunks < 2) return SLA_OK;
  Args<T> a = p;
  const int64_t n = (p.offsets ? 1 : p.n_seq) * p.dim * p.states;
  return in_launches(a, (n + kLanes - 1) / kLanes, [&](dim3 grid) {
    if (backward) scan_join<T, true><<<grid, kLanes, 0, s>>>(a);
    else scan_join<T, false><<<grid, kLanes, 0, s>>>(a);
  });
}

template <typename C>
sla_status leave_empty(const sla_selscan_shape& q, const void* from, void* to, hipStream_t s) {
  const int64_t per = q.dim * q.n_state;
  if (!q.n_seq) return SLA_OK;
  const dim3 grid((unsigned)((per + kWG - 1) / kWG), (unsigned)std::min<int64_t>(q.n_seq, 256));
  scan_empty<C><<<grid, kWG, 0, s>>>(q.d_offsets, q.n_seq, per, (const C*)from, (C*)to);
  SLA_HIP(hipGetLastError());
  return SLA_OK;
}
template sla_status leave_empty<float>(const sla_selscan_shape&, const void*, void*, hipStream_t);
template sla_status leave_empty<double>(const sla_selscan_shape&, const void*, void*, hipStream_t);

#define SLA_SELSCAN_TYPES(T)                                                                   \
  template Args<T> args_of<T>(const sla_selscan_shape&, const sla_selscan_in&, const Plan&,    \
                              const Work&, void*);                                             \
  template sla_status join<T>(const Args<T>&, const Plan&, bool, hipStream_t);
SLA_SELSCAN_TYPES(double)
SLA_SELSCAN_TYPES(float)
SLA_SELSCAN_TYPES(bf16_t)
SLA_SELSCAN_TYPES(f16_t)

sla_status check_in(const sla_selscan_shape& q, const sla_selscan_in* in) {
  if (!in) return refuse("inputs are NULL");
  for (int64_t s : {in->x_seq, in->x_step, in->dt_seq, in->dt_step, in->z_seq, in->z_step,
                    in->b_seq, in->b_step, in->c_seq, in->c_step})
    if (s < 0) return refuse("negative stride");
  if (!no_steps(q) && (!in->d_x || !in->d_dt || !in->d_a || !in->d_b || !in->d_c))
    return refuse("x, dt, A, B or C is NULL");
  return SLA_OK;
}

sla_status check_work(size_t need, const void* work, size_t bytes) {
  if (need && (!work || bytes < need)) return refuse("workspace too small");
  if ((uintptr_t)work & 255) return refuse("the workspace must be 256-byte aligned");
  return SLA_OK;
}

}  // namespace selscan
}  // namespace sla

using namespace sla;
using namespace sla::selscan;

extern "C" {

sla_status sla_selscan_sizes(const sla_selscan_shape* shape, size_t* saved_bytes,
                             size_t* forward_bytes, size_t* backward_bytes) {
  const sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  if (!saved_bytes || !forward_bytes || !backward_bytes) return refuse("NULL result");
  const sla_selscan_shape& q = *shape;
  const size_t tiles = no_steps(q) ? 0 : (size_t)(q.d_offsets ? 1 : q.n_seq) *
                                             plan_of(q, false).tiles;
  *saved_bytes = tiles * q.dim * q.n_state * (q.dtype == SLA_F64 ? 8 : 4);
  *forward_bytes = work_of(q, false).bytes;
  *backward_bytes = work_of(q, true).bytes;
  return SLA_OK;
}

sla_status sla_selscan_forward(const sla_selscan_shape* shape, const sla_selscan_in* in, void* d_y,
                               void* d_h_last, void* d_saved, void* d_work, size_t work_bytes,
                               void* stream) {
  sla_status st = check_shape(shape);
  if (st != SLA_OK) return st;
  const sla_selscan_shape& q = *shape;
  if ((st = check_in(q, in)) != SLA_OK) return st;
  if (empty(q)) return SLA_OK;
  if (!no_steps(q)) {
    if (!d_y) return refuse("y is NULL");
    for (const void* a : {in->d_x, in->d_dt, in->d_z, in->d_b, in->d_c})
      if (a == d_y) return refuse("y must not be an input");
  }
  if (q.d_offsets && d_h_last && d_h_last == in->d_h0)
    return refuse("packed sequences' states cannot be updated in place");
  const Work w = work_of(q, false);
  if ((st = check_work(w.bytes, d_work, work_bytes)) != SLA_OK) return st;
  TraceRange tr("sla_selscan_forward");
  const hipStream_t s = (hipStream_t)stream;
  if (d_h_last && (q.d_offsets || q.steps == 0) && d_h_last != in->d_h0) {
    st = q.dtype == SLA_F64 ? leave_empty<double>(q, in->d_h0, d_h_last, s)
                            : leave_empty<float>(q, in->d_h0, d_h_last, s);
    if (st != SLA_OK) return st;
  }
  if (no_steps(q)) return SLA_OK;
  const Plan plan = plan_of(q, false);
  return with_type(q, [&](auto t) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    Args<T> p = args_of<T>(q, *in, plan, w, d_work);
    p.y = (T*)d_y;
    p.fast = p.fast && packs(d_y, 0, 0, sizeof(T), tile_steps(q) / 4, true, true);
    p.h_last = (C*)d_h_last;
    p.saved = (C*)d_saved;
    return with_states(q.n_state, p.fast, [&](auto ns, auto fast) -> sla_status {
      constexpr int NS = decltype(ns)::value;
      constexpr bool FAST = decltype(fast)::value;
      if (q.steps <= kFew && !q.d_offsets && !d_saved) {
        const int64_t lanes = q.n_seq * q.dim * 4;
        return in_launches(p, (lanes + kWG - 1) / kWG, [&](dim3 grid) {
          scan_few<T, NS, FAST><<<grid, kWG, 0, s>>>(p);
        });
      }
      const int64_t groups = plan.rows * plan.blocks;
      if (plan.chunks > 1) {
        sla_status e = in_launches(p, groups, [&](dim3 grid) {
          scan_forward<T, NS, FAST, false><<<grid, kWG, 0, s>>>(p);
        });
        if (e == SLA_OK) e = join(p, plan, false, s);
        if (e != SLA_OK) return e;
      }
      return in_launches(p, groups, [&](dim3 grid) {
        scan_forward<T, NS, FAST, true><<<grid, kWG, 0, s>>>(p);
      });
    });
  });
}

}  // extern "C"
