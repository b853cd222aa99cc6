// Selective scans: what the forward and the backward kernels share.
//
// A wave takes 16 channels of a chunk of steps, tile by tile.  A lane has one
// channel and NS of its states, so the states of a channel lie in 4 lanes; the
// products that sum over them are folded between those lanes.
// A wave exchanges data through LDS of its own, without barriers; but for one thing, the
// sums over channels of the backward pass, nothing is shared between waves but the caches.
#pragma once

#include <type_traits>

#include "seq.h"

namespace sla {
namespace selscan {

constexpr int kChannels = 16;  // of a wave
constexpr int kLanes = 64;
// Steps of a tile: the backward pass holds NS states of each of them in registers (16
// steps of 4 states: 64 registers in fp32), and the coefficients of the last few.  A
// state is saved at every tile.
template <typename C>
constexpr int tile_steps() {
  return sizeof(C) == 8 ? 8 : 16;
}
inline int tile_steps(const sla_selscan_shape& q) { return q.dtype == SLA_F64 ? 8 : 16; }

template <typename T>
struct Args {
  using C = typename Compute<T>::type;
  const T *x, *dt, *z, *b, *c, *grad_y;
  int64_t x_seq, x_step, dt_seq, dt_step, z_seq, z_step, b_seq, b_step, c_seq, c_step, gy_seq,
      gy_step;
  const C *a, *d, *bias, *h0, *grad_last;
  T* y;
  C *h_last, *saved;
  T *grad_x, *grad_dt, *grad_z;
  C* grad_h0;
  const int64_t* offsets;
  int64_t n_seq, steps, dim;
  int states, groups;
  int64_t group_dim;  // channels of a group
  int blocks;         // of channels, of all groups
  int chunk, chunks;  // steps of a chunk; chunks of a sequence (packed: of all)
  int64_t tiles;      // of a sequence (packed: of all)
  int64_t before;     // workgroups of earlier launches of the call
  bool softplus;
  bool fast;          // whole packs, 4, 8 or 16 states: see with_states
  // joining the chunks, [row][channel][state] and [row][channel]: what a chunk
  // leaves from nothing, then what enters it; the sum of its deltas; whether
  // what enters it does not reach its end
  C* ends;
  C* deltas;
  int* cuts;
  // parts of gradients that are sums
  C *part_a, *part_d, *part_bias;  // [row][channel][state], [row][channel]
  C* part_bc;                      // [block][step of all][2][states]
};

// Where a wave works: its row of chunks, sequence, steps and channels.
struct Place {
  int64_t row, seq, t0, t1;  // steps t0 <= t < t1 (packed: of all sequences)
  int64_t part;              // which chunk of the sequence (packed: of all)
  int64_t at;                // the step that x's row 0 of this sequence is (packed: 0)
  int64_t channel;           // the first of the wave
  int64_t lo, hi;            // steps of sequences: packed rows before and behind are of none
  int group, block, some;    // channels that exist, of the wave's 16
};
template <typename T, int WAVES>
__device__ __forceinline__ Place place_of(const Args<T>& p) {
  Place w;
  const int64_t k = p.before + blockIdx.x;
  w.row = k / p.blocks;
  w.block = (int)(k % p.blocks);
  const int per = p.blocks / p.groups;
  w.group = w.block / per;
  const int64_t first = (int64_t)(w.block % per) * (kChannels * WAVES) +
                        __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kChannels;
  w.some = (int)min(max(p.group_dim - first, (int64_t)0), (int64_t)kChannels);
  w.channel = w.group * p.group_dim + first;
  w.seq = p.offsets ? 0 : w.row / p.chunks;
  w.part = p.offsets ? w.row : w.row % p.chunks;
  w.t0 = w.part * p.chunk;
  w.t1 = min(w.t0 + p.chunk, p.steps);
  w.at = p.offsets ? 0 : w.seq * p.steps;
  w.lo = p.offsets ? row_at(p.offsets[0], 0, p.steps) : 0;
  w.hi = p.offsets ? row_at(p.offsets[p.n_seq], w.lo, p.steps) : p.steps;
  return w;
}

// The sequence that holds a step, and where it begins and ends.
struct Span {
  int64_t seq, begin, end;
};
template <typename T>
__device__ __forceinline__ Span span_of(const Args<T>& p, const Place& w, int64_t t) {
  if (!p.offsets) return {w.seq, 0, p.steps};
  const int64_t s = sequence_of(p.offsets, p.n_seq, t);
  return {s, p.offsets[s], p.offsets[s + 1]};
}
__device__ __forceinline__ int64_t from_lane_of(int64_t v, int lane) {
  const unsigned lo = __builtin_amdgcn_readlane((int)v, lane);
  const unsigned hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
// The same in all lanes, and waited for here (see settle).
__device__ __forceinline__ Span waited_for(const Span& s) {
  return {from_lane_of(s.seq, 0), from_lane_of(s.begin, 0), from_lane_of(s.end, 0)};
}
// Which steps of a tile are the first, and the last, of a sequence (bits); then lane i
// knows the sequence of step i (`mine`).  `now` is the sequence of a step near by, where
// the tiles are walked from (BACK: to their start).  Most tiles are inside one; else
// 64 offsets around are read at once, and only if those do not reach is there a
// search: 12 loads one after the other among 3000 sequences, at each end and beginning,
// were two thirds of the time of 3000 sequences of 33 steps.
template <int TS, bool BACK, typename T>
__device__ __forceinline__ void edges_of(const Args<T>& p, const Place& w, Span& now, int64_t t0,
                                         int n, unsigned& starts, unsigned& ends, int64_t& mine) {
  starts = ends = 0;
  mine = w.seq;
  if (!p.offsets) {
    if (t0 == 0) starts = 1u;
    if (t0 + n == p.steps) ends = 1u << (n - 1);
    return;
  }
  if (now.begin < t0 && t0 + n < now.end) return;
  const int lane = threadIdx.x & 63;
  const int64_t base = BACK ? max(now.seq - (kLanes - 3), (int64_t)0) : now.seq;
  const int64_t k = base + lane;
  const int64_t at = k <= p.n_seq ? p.offsets[k] : INT64_MAX;
  const int64_t first = from_lane_of(at, 0), last = from_lane_of(at, kLanes - 1);
  unsigned inside = 0;
  if (first <= t0 && last > t0 + n) {
    for (int i = 0; i < n; ++i) {
      const int64_t t = t0 + i;
      const int64_t s = base + __popcll(__ballot(at <= t)) - 1;
      if (lane == i) mine = min(s, p.n_seq - 1);
      if (__ballot(at == t && k < p.n_seq)) starts |= 1u << i;
      if (__ballot(at == t + 1 && k > 0)) ends |= 1u << i;
      if (t >= w.lo && t < w.hi) inside |= 1u << i;
    }
  } else {
    const int64_t t = t0 + lane;
    const bool in = lane < n;
    const Span s = in ? span_of(p, w, t) : Span{0, -1, -1};
    mine = s.seq;
    starts = (unsigned)__ballot(in && s.begin == t);
    ends = (unsigned)__ballot(in && s.end == t + 1);
    inside = (unsigned)__ballot(in && t >= w.lo && t < w.hi);
  }
  starts &= inside, ends &= inside;
  now.seq = from_lane_of(mine, BACK ? 0 : n - 1);
  now = waited_for({now.seq, p.offsets[now.seq], p.offsets[now.seq + 1]});
}

// How lanes share a tile's rows when they read and write them: EL neighbouring
// channels of one step each.
template <typename C>
struct Rows {
  static constexpr int TS = tile_steps<C>();
  static constexpr int EL = TS * kChannels / kLanes;
  static constexpr int PER = kChannels / EL;  // lanes of a row
};

// EL elements from p, of which `some` exist.  FAST: all of them or none, in a pack; p
// is then valid in any case, and what is read where none exist is not used.
template <bool FAST, int EL, typename T>
__device__ __forceinline__ Pack<T, EL> load_some(const T* p, int some) {
  if constexpr (FAST) return *(const Pack<T, EL>*)p;
  Pack<T, EL> r;
#pragma unroll
  for (int e = 0; e < EL; ++e) r.v[e] = e < some ? p[e] : T(0);
  return r;
}
template <bool FAST, int EL, typename T>
__device__ __forceinline__ void store_some(T* p, const Pack<T, EL>& v, int some) {
  if constexpr (FAST) {
    if (some > 0) *(Pack<T, EL>*)p = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < EL; ++e)
    if (e < some) p[e] = v.v[e];
}

// B or C of a tile: a lane takes BL neighbouring states of one step.
template <typename C, int NS>
struct Shared {
  static constexpr int TS = tile_steps<C>();
  static constexpr int BL = NS * 4 * TS >= kLanes ? NS * 4 * TS / kLanes : 1;
  static constexpr int PER = 4 * NS / BL;  // lanes of a step
};
// `steps` (bits): those that are not 0 whatever was read.
template <typename C, int NS, typename T>
__device__ __forceinline__ void keep_shared(C (*to)[4 * NS], const Pack<T, Shared<C, NS>::BL>& v,
                                            unsigned steps = ~0u) {
  using S = Shared<C, NS>;
  const int lane = threadIdx.x & 63, t = lane / S::PER, at = lane % S::PER * S::BL;
  if (S::TS * S::PER < kLanes && t >= S::TS) return;
  const bool is = steps >> t & 1;
#pragma unroll
  for (int e = 0; e < S::BL; ++e) to[t][at + e] = is ? (C)v.v[e] : C(0);
}
// Steps of a tile that are of a sequence (bits).
__device__ __forceinline__ unsigned inside_of(const Place& w, int64_t t0, int ts) {
  if (t0 >= w.lo && t0 + ts <= w.hi) return ~0u;
  const int a = (int)min(max(w.lo - t0, (int64_t)0), (int64_t)ts);
  const int b = (int)min(max(w.hi - t0, (int64_t)0), (int64_t)ts);
  return ((1u << b) - 1) & ~((1u << a) - 1);
}

// A lane's place in the rows of an array of steps; it moves from tile to tile.  In a
// tile of n < TS steps, lanes of the others read the last.
template <bool FAST, int EL, typename T>
struct Stream {
  const T* at;
  int64_t step, hop;
  int row, some;
  // `base`: the lane's first element of step 0; t0: the first tile's step.
  __device__ __forceinline__ Stream(const T* base, int64_t step_, int64_t t0, int row_, int some_,
                                    int hop_)
      : at(base + (t0 + row_) * step_), step(step_), hop(hop_ * step_), row(row_), some(some_) {}
  __device__ __forceinline__ Pack<T, EL> load(int n, int ts) const {
    const T* p = at;
    if (n < ts) p -= max(row - (n - 1), 0) * step;
    return load_some<FAST, EL>(p, some);
  }
  __device__ __forceinline__ void move() { at += hop; }
};
template <bool FAST, typename C, int NS, typename T>
__device__ __forceinline__ Stream<FAST, Shared<C, NS>::BL, T> shared_stream(
    const Args<T>& p, const T* base, int64_t step, int64_t t0, int hop) {
  using S = Shared<C, NS>;
  const int lane = threadIdx.x & 63, at = lane % S::PER * S::BL, some = p.states - at;
  return {base + (some > 0 ? at : 0), step, t0, min(lane / S::PER, S::TS - 1), some, hop};
}

// A lane's NS states in an array [..][channel][state].
template <int NS, bool FAST, typename C>
__device__ __forceinline__ void get_states(C (&h)[NS], const C* base, int64_t channel, int states,
                                           int q, bool live) {
#pragma unroll
  for (int j = 0; j < NS; ++j) h[j] = C(0);
  if (!base || !live) return;
  const C* at = base + channel * states + q * NS;
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (FAST || q * NS + j < states) h[j] = at[j];
}
// The same, waited for.
template <int NS, bool FAST, typename C>
__device__ __forceinline__ void enter_states(C (&h)[NS], const C* base, int64_t channel,
                                             int states, int q, bool live) {
  get_states<NS, FAST>(h, base, channel, states, q, live);
  settle(h);
}
template <int NS, bool FAST, typename C>
__device__ __forceinline__ void put_states(const C (&h)[NS], C* base, int64_t channel, int states,
                                           int q, bool live) {
  if (!base || !live) return;
  C* at = base + channel * states + q * NS;
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (FAST || q * NS + j < states) at[j] = h[j];
}

sla_status check_shape(const sla_selscan_shape* q);
sla_status refuse(const char* msg);
bool empty(const sla_selscan_shape& q);
bool no_steps(const sla_selscan_shape& q);

// How a call is cut: see plan_of.
struct Plan {
  int chunk = 0, chunks = 1, blocks = 1;
  int64_t rows = 0, tiles = 0;
};
Plan plan_of(const sla_selscan_shape& q, bool backward);
constexpr int kWavesOf = 4;  // waves of a workgroup, side by side in the channels

// The workspace: what joins the chunks, and the parts of summed gradients.
struct Work {
  size_t deltas_at = 0, cuts_at = 0, a_at = 0, d_at = 0, bias_at = 0, bc_at = 0, bytes = 0;
};
Work work_of(const sla_selscan_shape& q, bool backward);

template <typename T>
sla_status join(const Args<T>& p, const Plan& plan, bool backward, hipStream_t s);

// A launch has less than 2^32 threads.
template <typename T, typename F>
sla_status in_launches(Args<T>& p, int64_t groups, F&& launch) {
  constexpr int64_t kMost = ((int64_t)1 << 32) / kWG - 1;
  for (int64_t at = 0; at < groups; at += kMost) {
    p.before = at;
    launch(dim3((unsigned)std::min(groups - at, kMost)));
    SLA_HIP(hipGetLastError());
  }
  return SLA_OK;
}

// Calls f with the storage type, then with the states of a lane and whether all of
// them exist and every array can be read in packs, as most models' can: then no
// lane asks what exists, and the loads of the next tile stay on their way through
// the present one.
template <typename F>
sla_status with_type(const sla_selscan_shape& q, F&& f) {
  switch (q.dtype) {
    case SLA_F64: return f(double{});
    case SLA_F32: return f(float{});
    case SLA_BF16: return f(bf16_t{});
    default: return f(f16_t{});
  }
}
template <typename F>
sla_status with_states(int64_t n, bool fast, F&& f) {
  auto pick = [&](auto ns) {
    return fast ? f(ns, std::true_type{}) : f(ns, std::false_type{});
  };
  if (n <= 4) return pick(std::integral_constant<int, 1>{});
  if (n <= 8) return pick(std::integral_constant<int, 2>{});
  return pick(std::integral_constant<int, 4>{});
}

bool packs(const void* p, int64_t seq, int64_t step, size_t bytes, int v, bool one_seq,
           bool one_step);
template <typename T>
Args<T> args_of(const sla_selscan_shape& q, const sla_selscan_in& in, const Plan& plan,
                const Work& w, void* work);

}  // namespace selscan
}  // namespace sla
