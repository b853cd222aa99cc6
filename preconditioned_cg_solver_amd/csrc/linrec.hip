// Gated linear recurrences along a sequence and their adjoint.
//
// Forward substitution of a unit lower bidiagonal system per sequence and
// channel, h_t = a_t h_{t-1} + b_t, and back substitution of its transpose
// for the gradients, lambda_t = dh_t + a_{t+1} lambda_{t+1}.
//
// A step is the map h -> a h + b, and maps compose: two in a row are
// h -> (a2 a1) h + (a2 b1 + b2).  A workgroup reads a chunk of steps, composes
// them and publishes the result, takes what enters the chunk from the one
// before it and only then writes its rows, from registers: every row is read
// and written once, in one launch.  What enters is folded one chunk at a time
// from the same side whichever way it was found, so the bits do not depend
// on timing.
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

// A workgroup takes a chunk: W channels of as many steps as its registers
// hold.  A thread has V neighbouring channels of consecutive steps.  The
// backward pass holds more per element, in chunks of 128 steps for every type.
constexpr int kThreads = 512;
// The channels of narrow chunks, and of the forward pass's wide ones (see
// width_of).
constexpr int kNarrow = 64, kWide = 128;
constexpr int chunk_of(size_t size, int width, bool backward) {
  return (size == 8 || backward ? 8192 : 16384) / width;
}
template <typename T, int W, bool BACKWARD>
constexpr int chunk_steps() {
  return chunk_of(sizeof(T), W, BACKWARD);
}
// The steps from one saved state to the next: a chunk of the backward pass.
constexpr int kSave = chunk_of(2, kNarrow, true);
static_assert(kSave == chunk_of(8, kNarrow, true), "of any type");
// Whether the forward pass keeps the coefficients between its two passes over
// a chunk, or the rows as they were loaded, which in 16 bits take half the
// registers and let half the threads hold a chunk.
constexpr bool keeps(size_t size, int width) { return size > 2 || width != kNarrow; }
// Rows that are kept as loaded but not in pairs take a register an element.
template <typename T, int W, int V>
constexpr int forward_threads() {
  return keeps(sizeof(T), W) || V == 1 ? kThreads : kThreads / 2;
}

// Products of coefficients can leave the range of their type where the states
// that they carry do not: 300 steps that double a state of zero, a coefficient
// of zero after very large ones, a large state that shrinks by more than the
// type can express, an infinite one that stays infinite.
//
// A product is therefore zero only where a coefficient is, and the least number
// where it underflowed.  The sigmoid's coefficients, at most 1 (UNIT), lose no
// more than that.  With linear gates
//  - a part (a thread's steps) whose product lost more has NaN in its place;
//  - a chunk whose map (a, m) is not finite, or whose product lost more, does
//    not offer it: what leaves it is taken from part to part;
//  - a small product is not applied where what it lost shows (loses);
//  - where the parts' maps fail, the steps of the channel in the chunk are taken
//    one by one, from memory, by the wave that joins the parts.
// Forward, 65536 x 512 fp32, where an ordinary call takes 93 us: chunks without
// maps throughout 0.43 ms, every step one by one 17 ms (8 x 2048 x 2048: 0.63 ms).
template <typename C>
struct Range {
  static constexpr bool k64 = sizeof(C) == 8;
  static constexpr C kNormal = k64 ? C(0x1p-1022) : C(0x1p-126f);
  static constexpr C kLeast = k64 ? C(0x1p-1074) : C(0x1p-149f);
  // A product that underflowed and then grows by kGrowth at most is known to
  // kLeast kGrowth, which is a rounding error of kSmall.
  static constexpr C kGrowth = k64 ? C(0x1p64) : C(0x1p24);
  static constexpr C kSmall = k64 ? C(0x1p-950) : C(0x1p-100);
};
template <typename C>
__device__ __forceinline__ bool infinite(C v) {
  return fabs(v) == C(INFINITY);
}
// A product whose smallest factor is `least`.
template <typename C>
__device__ __forceinline__ C not_zero(C product, C least) {
  return ((product == C(0)) & (least != C(0))) ? copysign(Range<C>::kLeast, product) : product;
}
// Whether a h + m loses what it should hold of the state h: a may be off by
// kLeast kGrowth, and m does not hide it.
template <typename C>
__device__ __forceinline__ bool loses(C a, C h, C m) {
  const C shows = fabs(h) * Range<C>::kSmall;
  const bool small = fabs(a) < Range<C>::kSmall, hidden = !(fabs(m) < shows);
  return small & !hidden & (a != C(0)) & (shows < C(INFINITY));
}

// Follows the coefficients of a part and their product.
template <bool UNIT, typename C>
struct Factors {
  C least = C(1), low = C(1), most = C(0);  // smallest coefficient, product; largest coefficient
  __device__ __forceinline__ void take(C a, C product) {
    least = min(least, fabs(a));
    if constexpr (!UNIT) low = min(low, fabs(product)), most = max(most, fabs(a));
  }
  // The product, unless it grew after it had underflowed and matters, for no
  // coefficient is zero.  (No branches: the compiler would move the pass over
  // the rows into them.)
  __device__ __forceinline__ C checked(C product) const {
    const C a = not_zero(product, least);
    if constexpr (UNIT) return a;
    return ((low < Range<C>::kNormal) & (most > C(1)) & (least != C(0))) ? C(NAN) : a;
  }
};
// Follows the parts of a chunk and their product.
template <bool UNIT, typename C>
struct Joined {
  C least = C(1), low = C(1), growth = C(1);  // smallest part, product; all growth
  __device__ __forceinline__ void take(C part, C product) {
    least = min(least, fabs(part));
    if constexpr (!UNIT) low = min(low, fabs(product)), growth *= max(fabs(part), C(1));
  }
  // Whether the map (product, m) stands for the chunk.
  __device__ __forceinline__ bool whole(C& product, C m) const {
    product = not_zero(product, least);
    if constexpr (UNIT) return true;
    return __builtin_isfinite(product) && __builtin_isfinite(m) &&
           (min(low, least) >= Range<C>::kNormal || growth <= Range<C>::kGrowth);
  }
};

// 1 / (1 + e^-g), the coefficient, and 1 / (1 + e^g), the weight of x, neither
// as a difference of nearly equal numbers.
__device__ __forceinline__ void sigmoid2(float g, float& a, float& keep) {
  const float e = __builtin_amdgcn_exp2f(-1.44269504f * g);
  a = __builtin_amdgcn_rcpf(1.0f + e);
  keep = e > 0x1p60f ? 1.0f : e * a;  // e may be infinite, and then a is 0
}
__device__ __forceinline__ void sigmoid2(double g, double& a, double& keep) {
  const double e = exp(-fabs(g)), big = 1.0 / (1.0 + e), small = e * big;
  a = g >= 0.0 ? big : small;
  keep = g >= 0.0 ? small : big;
}
// Both in one number: the smaller, negative where that is the weight; the
// larger is 1 less it, to half a unit in the last place.
template <typename C>
__device__ __forceinline__ C fold(C a, C keep) {
  return a > keep ? -keep : a;
}
template <typename C>
__device__ __forceinline__ void unfold(C s, C& a, C& keep) {
  const C m = fabs(s), big = C(1) - m;
  const bool neg = signbit(s);
  a = neg ? big : m;
  keep = neg ? m : big;
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
  C* saved;      // the state after each chunk of the backward pass
  T* grad_x;
  T* grad_gate;
  C* grad_h0;
  const int64_t* offsets;
  int64_t x_seq, x_step, g_seq, g_step, d_seq, d_step;
  int64_t n_seq, steps, dim;
  int chunks;        // dense: of each sequence
  int chains, links, counters;  // chains of chunks, chunks of each, counters of tickets
  int blocks;        // channel blocks
  int64_t rows;      // chunks of all sequences (packed: at most)
  unsigned before;   // workgroups of earlier launches of the call
  bool streams;      // the rows go past the caches
  // joining the chunks of a sequence
  int* ticket;
  int* progress;     // [chain][64 channels of it][link]
  C* sums;           // [row][2][channel]: a chunk's product of a and its sum from a zero start
  C* ends;           // [row][channel]: what leaves the chunk (forward: h; backward: mu)
  const int* row_seq;  // packed: the sequence of a row
};

// A packed sequence's first row.  Rows offset / chunk + s are distinct and
// leave each sequence at least ceil(length / chunk) of them, without any sum
// over the lengths.
__device__ __forceinline__ int64_t first_row(const int64_t* offsets, int64_t steps, int chunk,
                                             int64_t s) {
  return min(max(offsets[s], (int64_t)0), steps) / chunk + s;
}

// A chunk: its sequence, place and length.
struct Where {
  int64_t s, row;
  int64_t first;         // packed: the sequence's first step
  int64_t x, g, d, out;  // element offsets of the sequence's first step
  int64_t len;           // of the sequence
  int64_t c, after;      // chunks before and after it
  int64_t mark;          // its place in `progress`
};

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Chunk `row` of a packed sequence or of the dense sequence s.  Whatever the
// offsets hold, the steps lie in [0, p.steps) and 0 <= c.
template <int kChunk, typename T>
__device__ __forceinline__ Where locate(const Args<T>& p, int64_t s, int64_t row) {
  Where w;
  w.s = s;
  w.row = row;
  if (p.offsets) {
    const int64_t o0 = min(max(uniform(p.offsets[s]), (int64_t)0), p.steps);
    const int64_t o1 = min(max(uniform(p.offsets[s + 1]), o0), p.steps);
    w.first = o0;
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
// Addresses are a uniform array and a lane's byte offset within it.
template <typename C>
__device__ __forceinline__ C* lane_ptr(C* base, uint32_t bytes) {
  return (C*)((char*)base + bytes);
}
template <typename C>
__device__ __forceinline__ const C* lane_ptr(const C* base, uint32_t bytes) {
  return (const C*)((const char*)base + bytes);
}
template <typename C>
__device__ __forceinline__ void publish(C* base, uint32_t bytes, C v) {
  Word<C> u = __builtin_bit_cast(Word<C>, v);
  if (u == ~Word<C>(0)) u = __builtin_bit_cast(Word<C>, C(NAN));
  __hip_atomic_store((Word<C>*)lane_ptr(base, bytes), u, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
template <typename C>
__device__ __forceinline__ C look(const C* base, uint32_t bytes) {
  return __builtin_bit_cast(C, __hip_atomic_load((const Word<C>*)lane_ptr(base, bytes),
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// How far a chunk is, per 64 of its channels: a hint of which words are worth
// reading, so that waiting costs one cache line per look.
enum Progress { kNothing = 0, kSums = 1, kEnd = 2 };

// What enters a chunk, from the chunks before it (forward: STEP = -1) or
// after it (backward: STEP = 1), `have` of them in the sequence, channel by
// lane: the end of the nearest one whose end is known, carried over the sums
// of those between.  The sums are applied one by one from the far end, as
// each chunk's own end is computed, so the bits do not depend on how far the
// look went.  progress, ends and sums point at the nearest chunk's.

// Nothing is carried over a sum that does not stand for its chunk: a chunk
// without a map publishes none, and one whose map loses what it should carry is
// not used; then that chunk's end is waited for.

// The nearest two, in one trip to memory (the backward pass with four: 8 x 4096 x
// 1024 bf16 104 -> 124 us, for what is read in vain; forward 45.8 -> 47.6 us).
constexpr int kNear = 2;
template <int STEP, bool UNIT, typename C>
__device__ __forceinline__ bool near_carry(const C* ends, const C* sums, uint32_t bytes,
                                           int64_t dim, int have, C& carry) {
  C e[kNear], a[kNear], m[kNear];
#pragma unroll
  for (int j = 0; j < kNear; ++j) {
    const int64_t off = STEP * min(j, have - 1) * dim;
    e[j] = look(ends + off, bytes);
    if (j + 1 < kNear) {
      a[j] = look(sums + 2 * off, bytes);
      m[j] = look(sums + 2 * off + dim, bytes);
    }
  }
  int at = -1;
  bool open = true;  // the sums so far are all known
#pragma unroll
  for (int j = 0; j < kNear; ++j) {
    if (open && at < 0 && j < have && __all(written(e[j]))) at = j;
    if (j + 1 < kNear) open = open && __all(written(a[j]) && written(m[j]));
  }
  if (at < 0) return false;
  carry = e[0];
  bool ok = true;
#pragma unroll
  for (int j = kNear - 1; j >= 0; --j) {
    if (j == at) carry = e[j];
    if (j + 1 < kNear && j < at) {
      ok = ok && (UNIT || !loses(a[j], carry, m[j]));
      carry = a[j] * carry + m[j];
    }
  }
  return __all(ok);
}

// Every chunk publishes its sums, if it has any, before it waits for anything,
// and a chunk waits only for chunks whose tickets were drawn before its own, by
// workgroups that therefore run already: the wait ends.
constexpr int kReach = 32, kBatch = 8;
template <int STEP, bool UNIT, typename C>
__device__ __forceinline__ C wait_carry(const int* progress, const C* ends, const C* sums,
                                        uint32_t bytes, int64_t dim, int64_t have) {
  const int n = (int)min(have, (int64_t)kReach), lane = threadIdx.x & 63;
  C near = C(0);
  if (near_carry<STEP, UNIT>(ends, sums, bytes, dim, n, near)) return near;
  for (;; __builtin_amdgcn_s_sleep(1)) {
    int f = kNothing;
    if (lane < n)
      f = __hip_atomic_load(progress + STEP * lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t done = __ballot(f >= kEnd), some = __ballot(f >= kSums);
    if (done == 0) continue;
    const int j = __builtin_ctzll(done);
    const uint64_t between = (1ull << j) - 1;
    if ((some & between) != between) continue;
    C h = look(ends + STEP * j * dim, bytes);
    bool ok = true;
    for (int top = j; top > 0; top -= kBatch) {
      C a[kBatch], m[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int64_t off = STEP * max(top - 1 - q, 0) * 2 * dim;
        a[q] = look(sums + off, bytes);
        m[q] = look(sums + off + dim, bytes);
      }
      if (top == j) ok = written(h);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (top - 1 - q >= 0) {
          ok = ok && written(a[q]) && written(m[q]) && (UNIT || !loses(a[q], h, m[q]));
          h = a[q] * h + m[q];
        }
      }
    }
    if (j == 0) ok = written(h);
    if (__all(ok)) return h;
  }
}
__device__ __forceinline__ void tell(int* progress, Progress v) {
  if ((threadIdx.x & 63) == 0)
    __hip_atomic_store(progress, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Tickets are drawn from two counters, kTicketStep bytes apart.  One serves
// its atomics one after the other (forward, 4 x 4096 x 1024 bf16: 38.1 us
// against 35.8), but keeps all chains at the same step, whose row is one piece of
// memory; with many they drift apart (65536 x 512 fp32, counters 1, 2, 8, 64:
// 89.8, 89.6, 109, 109 us; backward, 131072 x 2048 bf16: 551, 576, 647, 649 us).
constexpr int kCounters = 2, kTicketStep = 64;

// Marks every word as not written, zeroes the tickets and finds each row's
// sequence: the last one that begins at or before it.  2 to 6 us of a call; a
// launch of its own, since a chunk may look at any word.
template <typename C>
__global__ __launch_bounds__(kWG) void rec_begin(Word<C>* sums, int64_t n_sums, Word<C>* ends,
                                                 int64_t n_ends, int* ticket, int* progress,
                                                 int64_t n_progress, int* row_seq,
                                                 int64_t rows, const int64_t* offsets,
                                                 int64_t n_seq, int64_t steps, int chunk) {
  const int64_t i0 = (int64_t)blockIdx.x * kWG + threadIdx.x, n = (int64_t)gridDim.x * kWG;
  if (i0 < kCounters) ticket[i0 * (kTicketStep / sizeof(int))] = 0;
  for (int64_t i = i0; i < n_sums; i += n) sums[i] = ~Word<C>(0);
  for (int64_t i = i0; i < n_ends; i += n) ends[i] = ~Word<C>(0);
  for (int64_t i = i0; i < n_progress; i += n) progress[i] = kNothing;
  if (!row_seq) return;
  for (int64_t r = i0; r < rows; r += n) {
    int64_t lo = 0, hi = n_seq;  // first_row(lo) <= r < first_row(hi)
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (first_row(offsets, steps, chunk, mid) <= r) lo = mid;
      else hi = mid;
    }
    row_seq[r] = (int)lo;
  }
}

// This workgroup's chunk and channel block; false if there is none for it.
// CHAIN: the chunks of a sequence and channel block (packed: of a channel
// block) form a chain, each handed out by ticket before those that wait for
// it (REVERSE: from the last chunk on); a counter serves every
// p.counters-th chain.
template <int W, bool CHAIN, bool REVERSE, typename T>
__device__ __forceinline__ bool my_chunk(const Args<T>& p, Where& w, int& block) {
  if constexpr (!CHAIN) {
    const unsigned group = p.before + blockIdx.x;
    const int64_t s = group / (unsigned)p.blocks;
    block = group % (unsigned)p.blocks;
    w = locate<chunk_steps<T, W, REVERSE>()>(p, s, p.offsets ? 0 : s * p.chunks);
    return true;
  } else {
    __shared__ int drawn;
    const unsigned J = p.counters, j = blockIdx.x % J;  // (p.before is even)
    if (threadIdx.x == 0)
      drawn = __hip_atomic_fetch_add(p.ticket + j * (kTicketStep / sizeof(int)), 1,
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const unsigned k = __builtin_amdgcn_readfirstlane(drawn);
    const unsigned chains = (p.chains - j + J - 1) / J;  // of this counter
    unsigned c = k / chains;
    const unsigned chain = j + k % chains * J;
    if (c >= (unsigned)p.links) return false;
    if (REVERSE) c = p.links - 1 - c;
    block = chain % (unsigned)p.blocks;
    const int64_t s = p.offsets ? __builtin_amdgcn_readfirstlane(p.row_seq[c])
                                : chain / (unsigned)p.blocks;
    w = locate<chunk_steps<T, W, REVERSE>()>(p, s, p.offsets ? (int64_t)c : s * p.chunks + c);
    w.mark = (int64_t)chain * (W / 64) * p.links + c;
    return true;
  }
}

// A row past its packed sequence's end: none of valid offsets waits for it,
// and the end it publishes keeps those of any others from waiting for ever.
template <int W, int kChunk, typename T>
__device__ __forceinline__ bool unused_row(const Args<T>& p, const Where& w, int block) {
  using C = typename Compute<T>::type;
  if (!p.offsets || w.c == 0 || w.c * kChunk < w.len) return false;
  const int64_t ch0 = (int64_t)block * W;
  if (threadIdx.x < W) {
    if (ch0 + threadIdx.x < p.dim)
      publish(p.ends + w.row * p.dim + ch0, threadIdx.x * (uint32_t)sizeof(C), C(0));
    tell(p.progress + w.mark + (int64_t)(threadIdx.x >> 6) * p.links, kEnd);
  }
  return true;
}

// A thread's part of a chunk: V channels of S steps.
template <typename T, int W, int V, int N, bool BACKWARD>
struct Part {
  static constexpr int kChunk = chunk_steps<T, W, BACKWARD>();
  static constexpr int kWidth = W, kPer = V;
  static constexpr int kLanes = W / V;         // per row
  static constexpr int kSubs = N / kLanes;         // parts along the steps
  static constexpr int S = kChunk / kSubs;
  int sub, c0;       // its place among them, its first channel within the block
  bool act;          // it has channels
  int64_t at;        // the first one (0 where it has none)
  int64_t t0;        // first step
  int nv;            // steps
  bool full;         // the whole chunk has all its steps
};
template <typename P, typename T>
__device__ __forceinline__ P my_part(const Args<T>& p, const Where& w, int block) {
  constexpr int kChunk = P::kChunk;
  P r;
  r.sub = threadIdx.x / P::kLanes;
  r.c0 = threadIdx.x % P::kLanes * P::kPer;
  const int64_t ch = (int64_t)block * P::kWidth + r.c0;
  r.act = ch < p.dim;
  r.at = r.act ? ch : 0;
  r.full = w.len - w.c * kChunk >= kChunk;
  r.t0 = w.c * kChunk + r.sub * P::S;
  r.nv = (int)min(max(w.len - r.t0, (int64_t)0), (int64_t)P::S);
  return r;
}

// Rows past the caches (`streams`) or through them.
template <typename Q>
using Words = unsigned __attribute__((ext_vector_type(sizeof(Q) / 4)));
template <typename Q>
__device__ __forceinline__ Q read_row(const Q* p, bool streams) {
  if constexpr (sizeof(Q) >= 4) {
    if (streams) {
      const Words<Q> w = __builtin_nontemporal_load((const Words<Q>*)p);
      return __builtin_bit_cast(Q, w);
    }
  }
  return *p;
}
template <typename Q>
__device__ __forceinline__ void write_row(Q* p, const Q& v, bool streams) {
  if constexpr (sizeof(Q) >= 4) {
    if (streams) {
      __builtin_nontemporal_store(__builtin_bit_cast(Words<Q>, v), (Words<Q>*)p);
      return;
    }
  }
  *p = v;
}

// A thread's rows of an input; steps past the sequence's end hold `none`.
template <int S, int V, typename T>
__device__ __forceinline__ void load_part(const T* first, int64_t step, int64_t t0, int nv,
                                          bool full, bool streams, T none,
                                          Pack<T, V> (&r)[S]) {
  const T* row = first + t0 * step;
  if (full && streams) {
#pragma unroll
    for (int i = 0; i < S; ++i) r[i] = read_row((const Pack<T, V>*)(row + i * step), true);
  } else if (full) {
#pragma unroll
    for (int i = 0; i < S; ++i) r[i] = *(const Pack<T, V>*)(row + i * step);
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) r[i].v[v] = none;
      if (i < nv) r[i] = *(const Pack<T, V>*)row;
      row += step;
    }
  }
}
// The gate of a step that does nothing (with x = 0): coefficient 1, weight 0.
template <int GATE, typename T>
__device__ __forceinline__ T idle_gate() {
  return (T)(GATE == SLA_GATE_SIGMOID ? INFINITY : 1.0f);
}

// Keeps the compiler from carrying over what it derived from these elements.
template <typename T, int V>
__device__ __forceinline__ void forget(Pack<T, V>& p) {
  if constexpr (sizeof(p) < 4) {
    uint16_t u;
    __builtin_memcpy(&u, &p, 2);
    asm volatile("" : "+v"(u));
    __builtin_memcpy(&p, &u, 2);
  } else {
    uint32_t u[sizeof(p) / 4];
    __builtin_memcpy(u, &p, sizeof(p));
#pragma unroll
    for (size_t k = 0; k < sizeof(p) / 4; ++k) asm volatile("" : "+v"(u[k]));
    __builtin_memcpy(&p, u, sizeof(p));
  }
}

// Keeps a pass over the rows in their order, four elements at a time: taken
// together, the rows' intermediate values would not fit the registers.
template <int V>
__device__ __forceinline__ void row_fence(int i) {
  if ((i + 1) * V % 4 == 0) __builtin_amdgcn_sched_barrier(0);
}

// The linear steps of a lane's channel, ch0 + lane, in a chunk one by one, from
// memory, where the parts' maps do not stand for them; `enter` takes what enters
// part q (and, of states, what leaves the last).
template <typename P, typename C, typename T, typename F>
__device__ __forceinline__ C walk_states(const Args<T>& p, const Where& w, int64_t ch0, C h,
                                         F enter) {
  const int64_t t0 = w.c * P::kChunk;
  const T* g = p.gate + w.g + t0 * p.g_step + ch0;
  const T* x = p.x + w.x + t0 * p.x_step + ch0;
  const uint32_t lane = threadIdx.x * (uint32_t)sizeof(T);
  int n = (int)min(w.len - t0, (int64_t)P::kChunk);
#pragma unroll 1
  for (int q = 0; q < P::kSubs; ++q) {
    enter(q, h);
#pragma unroll 1
    for (int i = 0; i < P::S && n > 0; ++i, --n) {
      h = (C)*lane_ptr(g, lane) * h + (C)*lane_ptr(x, lane);
      g += p.g_step, x += p.x_step;
    }
  }
  enter(P::kSubs, h);
  return h;
}
// The adjoint, from the chunk's end to its beginning.
template <typename P, typename C, typename T, typename F>
__device__ __forceinline__ C walk_adjoint(const Args<T>& p, const Where& w, int64_t ch0, C mu,
                                          F enter) {
  const int64_t t0 = w.c * P::kChunk;
  const int n = (int)min(w.len - t0, (int64_t)P::kChunk);
  const T* g = p.gate + w.g + (t0 + n) * p.g_step + ch0;
  const T* d = p.grad_h + w.d + (t0 + n) * p.d_step + ch0;
  const uint32_t lane = threadIdx.x * (uint32_t)sizeof(T);
#pragma unroll 1
  for (int q = P::kSubs - 1; q >= 0; --q) {
    enter(q, mu);
#pragma unroll 1
    for (int i = min(n - q * P::S, P::S); i > 0; --i) {
      g -= p.g_step, d -= p.d_step;
      mu = (C)*lane_ptr(g, lane) * ((p.grad_h ? (C)*lane_ptr(d, lane) : C(0)) + mu);
    }
  }
  return mu;
}
// Whether that is needed: `from` entered the chunk and the parts' maps, part(0)
// the first taken, made `to` of it, by way of state(0) = from, state(1) ...,
// `high` the largest.  Once not finite, a state stays so, so its last value tells.
template <int N, typename C, typename F, typename G>
__device__ __forceinline__ bool went_wrong(C from, C to, C high, F part, G state) {
  bool wrong = to != to || (infinite(to) && !infinite(from));
  if (high > Range<C>::kGrowth) {
#pragma unroll 1
    for (int k = 0; k < N; ++k) {
      const C a = fabs(part(k)), after = k + 1 < N ? state(k + 1) : to;
      wrong = wrong || (a < Range<C>::kNormal && a != C(0) &&
                        fabs(after) < fabs(state(k)) * Range<C>::kSmall);
    }
  }
  return wrong && from == from;
}

// One chunk of a sequence.  CHAIN: sequences may have several, joined by the
// look-back; otherwise each has one.
//
// Bound by the bytes of x, gate and h, at the rate at which rows are reached in
// pieces of 128 or 256 bytes, and by the latency of the joining: 4 x 4096 x 4096
// bf16 84 to 88 us (4.6 to 4.8 TB/s; the chunks without the joining 78 us), 8 x 2048
// x 2048 bf16 48 us (37 us), 65536 x 512 fp32 88 us (4.6 TB/s), 262144 x 1024 fp16 331
// to 343 us (4.7 to 4.9 TB/s; in chunks of twice the steps and threads 349 us), 120
// packed sequences of 833 x 1024 bf16 150 us (4.1 TB/s).  A quarter-rate exponential
// and reciprocal an element leave no room to work the coefficients out twice
// where registers hold them.
// Workgroups that stay and fetch the next chunk's rows while they join one
// took 148 us for the first of these: two fit a compute unit, and neither
// hides the other's wait.
template <typename T, int GATE, int W, int V, bool CHAIN>
__global__ __launch_bounds__((forward_threads<T, W, V>()), 4) void rec_forward(Args<T> p) {
  using C = typename Compute<T>::type;
  using P = Part<T, W, V, forward_threads<T, W, V>(), false>;
  constexpr bool kSig = GATE == SLA_GATE_SIGMOID;
  constexpr int S = P::S, kSubs = P::kSubs;
  __shared__ C s_a[kSubs][W], s_m[kSubs][W];
  int block;
  Where w;
  if (!my_chunk<W, CHAIN, false>(p, w, block)) return;
  if (CHAIN && unused_row<W, P::kChunk>(p, w, block)) return;
  static_assert(kSave % S == 0, "saved states fall between parts");
  const P r = my_part<P>(p, w, block);

  // The rows as loaded or, where they fit, the coefficients they give; else
  // each of the two passes over them works those out.
  constexpr bool kKeep = keeps(sizeof(T), W);
  Pack<T, V> x[S], g[S];
  C ka[kKeep ? S : 1][V], kb[kKeep ? S : 1][V];
  load_part<S, V>(p.gate + w.g + r.at, p.g_step, r.t0, r.nv, r.full, p.streams,
                  idle_gate<GATE, T>(), g);
  load_part<S, V>(p.x + w.x + r.at, p.x_step, r.t0, r.nv, r.full, p.streams, (T)0.0f, x);
  auto coefficients = [&](int i, int v, C& a, C& b) {
    b = (C)x[i].v[v];
    a = (C)g[i].v[v];
    if constexpr (kSig) {
      C keep;
      sigmoid2((C)g[i].v[v], a, keep);
      b *= keep;
    }
  };
  {
    // Where the registers are full of rows, a product that came out as zero is
    // looked into afterwards: 262144 x 1024 fp16 343 us, 350 with every
    // coefficient followed (120 packed sequences of 833 x 1024 bf16 154 and 164).
    constexpr bool kFollow = !kSig || kKeep || V == 1;
    C pa[V], pm[V];
    Factors<kSig, C> f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pa[v] = C(1), pm[v] = C(0);
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        C a, b;
        coefficients(i, v, a, b);
        if constexpr (kKeep) ka[i][v] = a, kb[i][v] = b;
        pm[v] = a * pm[v] + b;
        pa[v] *= a;
        if constexpr (kFollow) f[v].take(a, pa[v]);
      }
      row_fence<V>(i);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (kFollow) {
        pa[v] = f[v].checked(pa[v]);
      } else if (pa[v] == C(0)) {
        C least = (C)g[0].v[v], keep;
#pragma unroll
        for (int i = 1; i < S; ++i) least = min(least, (C)g[i].v[v]);
        sigmoid2(least, least, keep);
        pa[v] = not_zero(pa[v], least);
      }
      s_a[r.sub][r.c0 + v] = pa[v], s_m[r.sub][r.c0 + v] = pm[v];
    }
  }
  __syncthreads();
  // From here a lane has a channel, in the first W / 64 waves.
  const int64_t ch0 = (int64_t)block * W, row0 = w.row * p.dim + ch0;
  const int channels = (int)min((int64_t)W, p.dim - ch0);
  const bool join = threadIdx.x < W, act = (int)threadIdx.x < channels;
  const uint32_t at = act ? threadIdx.x * (uint32_t)sizeof(C) : 0;
  C *ends = p.ends + row0, *sums = p.sums + row0 + w.row * p.dim;
  int* mark = p.progress + w.mark + (int64_t)(threadIdx.x >> 6) * p.links;
  C ca = C(1), cm = C(0), h = C(0);
  bool whole = true;  // the chunk's map stands for it
  if (CHAIN && join) {
    Joined<kSig, C> f;
#pragma unroll 4
    for (int q = 0; q < kSubs; ++q) {
      const C pa = s_a[q][threadIdx.x];
      cm = pa * cm + s_m[q][threadIdx.x];
      ca *= pa;
      f.take(pa, ca);
    }
    whole = f.whole(ca, cm);
    if (kSig || __all(whole || !act)) {
      if (act) {
        publish(sums, at, ca);
        publish(sums + p.dim, at, cm);
      }
      tell(mark, kSums);
    }
  }
  if (join) {
    if (w.c == 0) {
      if (p.h0) h = *lane_ptr(p.h0 + w.s * p.dim + ch0, at);
    } else if constexpr (CHAIN) {
      h = wait_carry<-1, kSig>(mark - 1, ends - p.dim, sums - 2 * p.dim, at, p.dim, w.c);
    }
    whole = whole && (kSig || !loses(ca, h, cm));
    const bool now = CHAIN && (kSig || __all(whole || !act));
    const C from = h, end = ca * h + cm;
    if (now) {
      if (act) publish(ends, at, end);
      tell(mark, kEnd);
    }
    if (w.len == 0 && w.c == 0 && act && p.h_last)
      *lane_ptr(p.h_last + w.s * p.dim + ch0, at) = h;
    // the state where a chunk of the backward pass ends and another follows
    auto save = [&](int q, C h) {
      const int64_t t = w.c * P::kChunk + q * S;
      if (p.saved && t % kSave == 0 && t < w.len && act) {
        const int64_t row = p.offsets ? w.first / kSave + w.s
                                      : w.s * ((p.steps + kSave - 1) / kSave);
        *lane_ptr(p.saved + (row + t / kSave - 1) * p.dim + ch0, at) = h;
      }
    };
    // what enters each part, in the place of its sum
    C high = C(0);
#pragma unroll 4
    for (int q = 0; q < kSubs; ++q) {
      const C next = s_a[q][threadIdx.x] * h + s_m[q][threadIdx.x];
      if constexpr (!kSig) high = max(high, fabs(h));
      s_m[q][threadIdx.x] = h;
      h = next;
      save(q + 1, h);
    }
    if (!kSig && act &&
        went_wrong<kSubs>(from, h, high, [&](int q) { return s_a[q][threadIdx.x]; },
                          [&](int q) { return s_m[q][threadIdx.x]; }))
      h = walk_states<P>(p, w, ch0, from, [&](int q, C h) {
        if (q < kSubs) s_m[q][threadIdx.x] = h;
        if (q > 0) save(q, h);
      });
    if (CHAIN && !kSig && !now) {
      if (act) publish(ends, at, whole ? end : h);
      tell(mark, kEnd);
    }
  }
  __syncthreads();
  if (r.nv == 0 || !r.act) return;
  if constexpr (!kKeep) {
#pragma unroll
    for (int i = 0; i < S; ++i) forget(x[i]), forget(g[i]);
  }
  C hv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) hv[v] = s_m[r.sub][r.c0 + v];
  T* out = p.h + w.out + r.t0 * p.dim + r.at;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    Pack<T, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C a, b;
      if constexpr (kKeep) a = ka[i][v], b = kb[i][v];
      else coefficients(i, v, a, b);
      hv[v] = a * hv[v] + b;
      o.v[v] = (T)hv[v];
    }
    if (i < r.nv) write_row((Pack<T, V>*)(out + i * p.dim), o, p.streams);
    row_fence<V>(i);
  }
  if (r.t0 + r.nv == w.len && p.h_last) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.h_last[w.s * p.dim + r.at + v] = hv[v];
  }
}

// One chunk of the adjoint, from the saved state before it.  The composed maps
// of the forward pass are needed again, for h, beside those of mu.  The sum of a
// part's map of mu is taken from the part's end, in a pass of its own over the
// registers: taken with the product of the coefficients before each step, in
// the pass that loads them, it would be NaN where that product leaves its range
// (and 8 x 2048 x 2048 bf16 took 89 us instead of 86, fp64 4 x 2048 x 1024 101 instead
// of 85, for the registers that the products held; where most steps of a part lie
// past the sequence's end it costs, 256 x 32 x 4096 bf16 130 and 135 us).
//
// Bound as the forward pass, by the bytes of x, gate, dh and the two gradients,
// and by registers: in 16 bits a thread has 64 of them for its 16 elements, so
// that four workgroups share a compute unit: 8 x 2048 x 2048 bf16 79 us (4.3 TB/s),
// 65536 x 512 fp32 140 us (4.8 TB/s), 120 packed sequences of 833 x 1024 bf16 266 us
// (3.8 TB/s).
template <typename T, int GATE, int V, bool CHAIN>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 4) void rec_backward(Args<T> p) {
  using C = typename Compute<T>::type;
  constexpr int W = kNarrow;
  using P = Part<T, W, V, kThreads, true>;
  constexpr bool kSig = GATE == SLA_GATE_SIGMOID;
  constexpr int S = P::S, kSubs = P::kSubs;
  __shared__ C s_a[kSubs][W], s_m[kSubs][W], s_u[kSubs][W];
  __shared__ Pack<T, V> s_d[S][kThreads];
  int block;
  Where w;
  if (!my_chunk<W, CHAIN, true>(p, w, block)) return;
  if (CHAIN && unused_row<W, P::kChunk>(p, w, block)) return;
  const P r = my_part<P>(p, w, block);

  // f: the coefficient, for the sigmoid folded with the weight of x: held
  // apart, the two would not fit the registers, so the compiler is kept from
  // carrying them over from pass to pass.  dL/dh waits in LDS.
  C f[S][V];
  Pack<T, V> x[S];
  auto step = [&](int i, int v, C& a, C& keep) {
    if constexpr (kSig) {
      asm volatile("" : "+v"(f[i][v]));
      unfold(f[i][v], a, keep);
    } else {
      a = f[i][v], keep = C(1);
    }
  };
  {
    C pa[V], pm[V], pu[V];
    Factors<kSig, C> k[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pa[v] = C(1), pm[v] = C(0), pu[v] = C(0);
    // Room to keep the coefficients for the second pass, beside f: 8 x 2048 x 2048
    // fp32 142 us, 145 with those worked out from f; in fp64 the registers overflow
    // (99 us for 86).
    constexpr bool kRoom = sizeof(T) == 4;
    C ka[kRoom ? S : 1][V];
    Pack<T, V> g[S], d[S];
    load_part<S, V>(p.gate + w.g + r.at, p.g_step, r.t0, r.nv, r.full, p.streams,
                    idle_gate<GATE, T>(), g);
    load_part<S, V>(p.x + w.x + r.at, p.x_step, r.t0, r.nv, r.full, p.streams, (T)0.0f, x);
    load_part<S, V>(p.grad_h + w.d + r.at, p.d_step, r.t0, p.grad_h ? r.nv : 0,
                    r.full && p.grad_h, p.streams, (T)0.0f, d);
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        C a = (C)g[i].v[v], keep, b = (C)x[i].v[v];
        f[i][v] = a;
        if constexpr (kSig) {
          sigmoid2((C)g[i].v[v], a, keep);
          f[i][v] = fold(a, keep);
          b *= keep;
        }
        if constexpr (kRoom) ka[i][v] = a;
        pm[v] = a * pm[v] + b;
        pa[v] *= a;
        k[v].take(a, pa[v]);
      }
      s_d[i][threadIdx.x] = d[i];
      forget(x[i]);
      row_fence<V>(i);
    }
    // mu leaving the part, from a zero start; from its end, so that no product
    // of coefficients comes in
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      const Pack<T, V> d = s_d[i][threadIdx.x];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        C a, keep;
        if constexpr (kRoom) a = ka[i][v];
        else step(i, v, a, keep);
        pu[v] = a * ((C)d.v[v] + pu[v]);
      }
      row_fence<V>(i);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      pa[v] = k[v].checked(pa[v]);
      s_a[r.sub][r.c0 + v] = pa[v];
      s_m[r.sub][r.c0 + v] = pm[v];
      s_u[r.sub][r.c0 + v] = pu[v];
    }
  }
  __syncthreads();
  const int64_t ch0 = (int64_t)block * W, row0 = w.row * p.dim + ch0;
  const int64_t state0 = w.s * p.dim + ch0;
  const int channels = (int)min((int64_t)W, p.dim - ch0);
  const bool join = threadIdx.x < W, act = (int)threadIdx.x < channels;
  const uint32_t at = act ? threadIdx.x * (uint32_t)sizeof(C) : 0;
  C *ends = p.ends + row0, *sums = p.sums + row0 + w.row * p.dim;
  int* mark = p.progress + w.mark;
  C ca = C(1), cu = C(0), mu = C(0);
  if (join) {
    bool whole = true;  // the chunk's map of mu stands for it
    if constexpr (CHAIN) {
      Joined<kSig, C> k;
#pragma unroll 4
      for (int q = kSubs - 1; q >= 0; --q) {
        const C pa = s_a[q][threadIdx.x];
        cu = pa * cu + s_u[q][threadIdx.x];
        ca *= pa;
        k.take(pa, ca);
      }
      whole = k.whole(ca, cu);
      if (kSig || __all(whole || !act)) {
        if (act) {
          publish(sums, at, ca);
          publish(sums + p.dim, at, cu);
        }
        tell(mark, kSums);
      }
    }
    C h = C(0);
    if (w.c > 0) h = *lane_ptr(p.saved + row0 - p.dim, at);
    else if (p.h0) h = *lane_ptr(p.h0 + state0, at);
    const C h_from = h;
    // what enters each part from before, in the place of its sum
    C high = C(0);
#pragma unroll 4
    for (int q = 0; q < kSubs; ++q) {
      const C next = s_a[q][threadIdx.x] * h + s_m[q][threadIdx.x];
      if constexpr (!kSig) high = max(high, fabs(h));
      s_m[q][threadIdx.x] = h;
      h = next;
    }
    if (!kSig && act &&
        went_wrong<kSubs>(h_from, h, high, [&](int q) { return s_a[q][threadIdx.x]; },
                          [&](int q) { return s_m[q][threadIdx.x]; }))
      walk_states<P>(p, w, ch0, h_from, [&](int q, C h) {
        if (q < kSubs) s_m[q][threadIdx.x] = h;
      });
    if (w.after == 0) {
      if (p.grad_last) mu = *lane_ptr(p.grad_last + state0, at);
    } else if constexpr (CHAIN) {
      mu = wait_carry<1, kSig>(mark + 1, ends + p.dim, sums + 2 * p.dim, at, p.dim, w.after);
    }
    whole = whole && (kSig || !loses(ca, mu, cu));
    const bool now = CHAIN && (kSig || __all(whole || !act));
    const C from = mu, end = ca * mu + cu;
    if (now) {
      if (act) publish(ends, at, end);
      tell(mark, kEnd);
    }
    if (w.len == 0 && w.c == 0 && act && p.grad_h0) *lane_ptr(p.grad_h0 + state0, at) = mu;
    high = C(0);
#pragma unroll 4
    for (int q = kSubs - 1; q >= 0; --q) {
      const C next = s_a[q][threadIdx.x] * mu + s_u[q][threadIdx.x];
      if constexpr (!kSig) high = max(high, fabs(mu));
      s_u[q][threadIdx.x] = mu;
      mu = next;
    }
    if (!kSig && act &&
        went_wrong<kSubs>(from, mu, high,
                          [&](int k) { return s_a[kSubs - 1 - k][threadIdx.x]; },
                          [&](int k) { return s_u[kSubs - 1 - k][threadIdx.x]; }))
      mu = walk_adjoint<P>(p, w, ch0, from, [&](int q, C mu) { s_u[q][threadIdx.x] = mu; });
    if (CHAIN && !kSig && !now) {
      if (act) publish(ends, at, whole ? end : mu);
      tell(mark, kEnd);
    }
  }
  __syncthreads();
  if (r.nv == 0 || !r.act) return;
  C h[V], mv[V], z[S][V];  // z: h_{t-1} - x (linear: h_{t-1})
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = s_m[r.sub][r.c0 + v], mv[v] = s_u[r.sub][r.c0 + v];
#pragma unroll
  for (int i = 0; i < S; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C a, keep;
      step(i, v, a, keep);
      const C xv = (C)x[i].v[v];
      z[i][v] = kSig ? h[v] - xv : h[v];
      h[v] = a * h[v] + (kSig ? keep * xv : xv);
    }
    row_fence<V>(i);
  }
  T* ox = p.grad_x + w.out + r.t0 * p.dim + r.at;
  T* og = p.grad_gate + w.out + r.t0 * p.dim + r.at;
#pragma unroll
  for (int i = S - 1; i >= 0; --i) {
    Pack<T, V> rx, rg;
    const Pack<T, V> d = s_d[i][threadIdx.x];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C a, keep;
      step(i, v, a, keep);
      const C lam = (C)d.v[v] + mv[v];
      mv[v] = a * lam;
      rx.v[v] = (T)(kSig ? lam * keep : lam);
      rg.v[v] = (T)(kSig ? mv[v] * z[i][v] * keep : lam * z[i][v]);
    }
    if (i < r.nv) {
      write_row((Pack<T, V>*)(ox + i * p.dim), rx, p.streams);
      write_row((Pack<T, V>*)(og + i * p.dim), rg, p.streams);
    }
    row_fence<V>(i);
  }
  // mu has passed the first step
  if (r.t0 == 0 && p.grad_h0) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.grad_h0[w.s * p.dim + r.at + v] = mv[v];
  }
}

// Sequences of a few steps, a serving step above all: a thread takes V
// channels from the first step to the last.  Bound by the launch for a step (16 x
// 4096 bf16: 3.0 us, the chunks' kernel 7.0), by latency or bytes beyond: 256 x 32 x
// 4096 bf16 34 us a call, in chunks 91; up to 32 steps it was never the slower.
constexpr int kFew = 32;
template <typename T, int GATE, int V>
__global__ __launch_bounds__(kWG) void few_forward(Args<T> p) {
  using C = typename Compute<T>::type;
  const int64_t k = ((int64_t)p.before + blockIdx.x) * kWG + threadIdx.x, per = p.dim / V;
  if (k >= p.n_seq * per) return;
  const int64_t s = k / per, at = k % per * V;
  int64_t first = 0, len = p.steps;
  if (p.offsets) {
    first = min(max(p.offsets[s], (int64_t)0), p.steps);
    len = min(max(p.offsets[s + 1], first), p.steps) - first;
  }
  const int64_t out = p.offsets ? first : s * p.steps;
  const T* g0 = p.gate + s * p.g_seq + first * p.g_step + at;
  const T* x0 = p.x + s * p.x_seq + first * p.x_step + at;
  C h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = p.h0 ? p.h0[s * p.dim + at + v] : C(0);
  for (int64_t t = 0; t < len; ++t) {
    const auto g = *(const Pack<T, V>*)(g0 + t * p.g_step);
    const auto x = *(const Pack<T, V>*)(x0 + t * p.x_step);
    Pack<T, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      C a = (C)g.v[v], b = (C)x.v[v];
      if constexpr (GATE == SLA_GATE_SIGMOID) {
        C keep;
        sigmoid2((C)g.v[v], a, keep);
        b *= keep;
      }
      h[v] = a * h[v] + b;
      o.v[v] = (T)h[v];
    }
    *(Pack<T, V>*)(p.h + (out + t) * p.dim + at) = o;
  }
  if (p.h_last) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.h_last[s * p.dim + at + v] = h[v];
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

sla_status refuse(const char* msg) {
  set_error(msg);
  return SLA_ERR_INVALID_ARG;
}

// Channels of a chunk.  Narrow chunks have more steps, so fewer of them are
// joined one after the other; wide ones reach longer pieces of a row, which
// pays where many sequences and channels stand side by side.  Forward, narrow and
// wide, us: dense bf16 8 x 4096 x 1024 56, 50, 1000 x 300 x 256 130, 117, 1 x 65536 x 512
// fp32 93, 119; packed bf16 x 1024, 12 sequences of 8333 151, 180, 120 of 833 161,
// 187, 800 of 125 220, 246 (fp32 x 512: 156, 136).  The backward pass, narrow and
// with chunks of 256 channels, which are not here any more: 92 and 129, 193 and
// 221, 144 and 296; 264 and 600, 269 and 453, 276 and 407; for sequences of some 32
// steps the wide ones were the faster.
int width_of(const sla_linrec_shape& q, bool backward) {
  if (backward || q.d_offsets || q.n_seq * q.dim < 8192) return kNarrow;
  // under a quarter of the lanes without a channel: 1000 x 300 x 64 bf16, forward, 36
  // us narrow and 54 wide
  return (q.dim + kWide - 1) / kWide * kWide * 3 > q.dim * 4 ? kNarrow : kWide;
}
int chunk_of(const sla_linrec_shape& q, bool backward) {
  return chunk_of(dtype_bytes(q.dtype), width_of(q, backward), backward);
}

// Rows of chunks (see first_row).
int64_t rows_of(const sla_linrec_shape& q, bool backward) {
  const int chunk = chunk_of(q, backward);
  if (q.d_offsets) return q.steps / chunk + q.n_seq;
  return q.n_seq * ((q.steps + chunk - 1) / chunk);
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
  if (q->n_seq >= INT32_MAX || q->dim >= (1 << 28) || q->steps >= ((int64_t)1 << 40) ||
      (__int128)(q->steps / 32 + 1) * q->n_seq >= ((__int128)1 << 60) ||
      (__int128)seqs * q->steps * q->dim >= ((__int128)1 << 60) ||
      (__int128)q->n_seq * q->dim >= ((__int128)1 << 60) ||
      (__int128)(std::max(rows_of(*q, false), rows_of(*q, true)) + 2 * q->n_seq + 64) *
              (q->dim / 64 + 64) >= INT32_MAX) {
    set_error("sizes beyond what a call can index");
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
bool one_chunk(const sla_linrec_shape& q, bool backward) {
  return q.steps <= chunk_of(q, backward);
}

// One per 64 channels of each chunk.
int64_t progress_words(const sla_linrec_shape& q, bool backward) {
  const int width = width_of(q, backward);
  return rows_of(q, backward) * ((q.dim + width - 1) / width) * (width / 64);
}

// The workspace of a call that joins chunks: the tickets, the progress, the
// rows' sequences, the chunks' sums and ends; enough for either direction.
struct Work {
  size_t progress_at = 0, rows_at = 0, sums_at = 0, ends_at = 0, bytes = 0;
};
Work work_of(const sla_linrec_shape& q) {
  Work w;
  if (no_steps(q) || (one_chunk(q, false) && one_chunk(q, true))) return w;
  const size_t rows = (size_t)std::max(rows_of(q, false), rows_of(q, true));
  const size_t marks = (size_t)std::max(progress_words(q, false), progress_words(q, true));
  const size_t words = rows * q.dim * state_bytes(q);
  w.progress_at = kCounters * kTicketStep;
  w.rows_at = w.progress_at + align_up(marks * sizeof(int));
  w.sums_at = w.rows_at + (q.d_offsets ? align_up(rows * sizeof(int)) : 0);
  w.ends_at = w.sums_at + align_up(2 * words);
  w.bytes = w.ends_at + align_up(words);
  return w;
}

// Whether an array's rows allow access by `v` channels at a time, anywhere.
bool packs(const sla_linrec_shape& q, const void* p, int64_t seq, int64_t step, int v) {
  return (uintptr_t)p % (v * dtype_bytes(q.dtype)) == 0 &&
         (seq % v == 0 || q.d_offsets || q.n_seq == 1) && (step % v == 0 || q.steps == 1);
}

template <typename T>
Args<T> common_args(const sla_linrec_shape& q, const void* x, int64_t xs, int64_t xt,
                    const void* g, int64_t gs, int64_t gt, const void* h0, bool backward) {
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
  const int chunk = chunk_of(q, backward);
  p.chunks = (int)std::max<int64_t>(1, (q.steps + chunk - 1) / chunk);
  p.rows = rows_of(q, backward);
  // 16-bit rows beyond what the last-level cache holds (256 MB) go past it:
  // forward, 4 x 4096 x 4096 bf16 90.9 -> 87.9 us, 262144 x 1024 fp16 352 -> 345 us.
  // In 32 bits it does not pay: 65536 x 512, both directions, 224 us through it and
  // 226 us past it.
  const double elements = (double)(q.d_offsets ? 1 : q.n_seq) * q.steps * q.dim;
  p.streams = sizeof(T) == 2 && (backward ? 5 : 3) * elements * sizeof(T) > 256 << 20;
  return p;
}

// Channels per thread, where every array's rows allow it: what 8 bytes hold
// forward (4 x 4096 x 4096 bf16 88.5 us a call, with 4 bytes 91.8), 4 bytes backward
// (both directions of 8 x 2048 x 2048 143 us, with 8 bytes 175: twice as many
// parts to join, half as many steps in each).
template <typename T>
constexpr int most_v(bool backward) {
  return std::max(1, (backward ? 4 : 8) / (int)sizeof(T));
}

// A launch has less than 2^32 threads: calls launch(grid) for `groups`
// workgroups in as many launches as they need.  (A chunk waits for tickets drawn
// before its own, in the same launch or an earlier one.)
template <typename T, typename F>
sla_status in_launches(Args<T>& p, int64_t groups, F&& launch) {
  constexpr int64_t kMost = (((int64_t)1 << 32) - 1) / kThreads & ~(int64_t)1;
  for (int64_t at = 0; at < groups; at += kMost) {
    p.before = (unsigned)at;
    launch(dim3((unsigned)std::min(groups - at, kMost)));
    SLA_HIP(hipGetLastError());
  }
  return SLA_OK;
}

// Sets up the chunks' joining and calls launch(W, V, CHAIN, grid), the first
// three as types.
template <int M, typename T, typename F>
sla_status run_chunks(const sla_linrec_shape& q, Args<T>& p, bool packed_v, void* work,
                      bool backward, hipStream_t s, F&& launch) {
  using C = typename Compute<T>::type;
  const bool chain = !no_steps(q) && !one_chunk(q, backward);
  const int width = width_of(q, backward);
  p.blocks = (int)((q.dim + width - 1) / width);
  int64_t grid = q.n_seq * p.blocks;
  if (chain) {
    p.chains = (int)(q.d_offsets ? p.blocks : q.n_seq * p.blocks);
    p.links = (int)(q.d_offsets ? p.rows : p.chunks);
    p.counters = p.chains % kCounters ? 1 : kCounters;
    grid = (int64_t)p.chains * p.links;
    const Work w = work_of(q);
    char* base = (char*)work;
    p.ticket = (int*)base;
    p.progress = (int*)(base + w.progress_at);
    int* row_seq = q.d_offsets ? (int*)(base + w.rows_at) : nullptr;
    p.row_seq = row_seq;
    p.sums = (C*)(base + w.sums_at);
    p.ends = (C*)(base + w.ends_at);
    const int64_t words = p.rows * p.dim;
    const int64_t want = (2 * words / 4 + kWG - 1) / kWG;
    const dim3 begin((unsigned)std::min<int64_t>(std::max<int64_t>(want, 1), 2048));
    rec_begin<C><<<begin, kWG, 0, s>>>((Word<C>*)p.sums, 2 * words, (Word<C>*)p.ends, words,
                                       p.ticket, p.progress, progress_words(q, backward),
                                       row_seq, p.rows, q.d_offsets, q.n_seq, q.steps,
                                       chunk_of(q, backward));
    SLA_HIP(hipGetLastError());
  }
  auto with_v = [&](auto w, auto v) {
    return in_launches(p, grid, [&](dim3 g) {
      if (chain) launch(w, v, std::true_type{}, g);
      else launch(w, v, std::false_type{}, g);
    });
  };
  auto with_w = [&](auto w) {
    return packed_v ? with_v(w, std::integral_constant<int, M>{})
                    : with_v(w, std::integral_constant<int, 1>{});
  };
  return width == kNarrow ? with_w(std::integral_constant<int, kNarrow>{})
                          : with_w(std::integral_constant<int, kWide>{});
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
  *saved_bytes =
      no_steps(*shape) ? 0 : (size_t)rows_of(*shape, true) * shape->dim * state_bytes(*shape);
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
  return with_types(q, [&](auto t, auto gate) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    constexpr int GATE = decltype(gate)::value, M = most_v<T>(false);
    const bool wide = q.dim % M == 0 && packs(q, d_x, x_seq_stride, x_step_stride, M) &&
                      packs(q, d_gate, gate_seq_stride, gate_step_stride, M) &&
                      packs(q, d_h, 0, 0, M);
    const hipStream_t s = (hipStream_t)stream;
    Args<T> p = common_args<T>(q, d_x, x_seq_stride, x_step_stride, d_gate, gate_seq_stride,
                               gate_step_stride, d_h0, false);
    p.h = (T*)d_h;
    p.h_last = (C*)d_h_last;
    p.saved = (C*)d_saved;
    if (q.steps <= kFew) {
      const int64_t n = q.n_seq * (q.dim / (wide ? M : 1));
      return in_launches(p, (n + kWG - 1) / kWG, [&](dim3 grid) {
        if (wide) few_forward<T, GATE, M><<<grid, kWG, 0, s>>>(p);
        else few_forward<T, GATE, 1><<<grid, kWG, 0, s>>>(p);
      });
    }
    return run_chunks<M>(q, p, wide, d_work, false, s, [&](auto w, auto v, auto chain, dim3 grid) {
      constexpr int W = decltype(w)::value, V = decltype(v)::value;
      rec_forward<T, GATE, W, V, decltype(chain)::value>
          <<<grid, (forward_threads<T, W, V>()), 0, s>>>(p);
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
  return with_types(q, [&](auto t, auto gate) {
    using T = decltype(t);
    using C = typename Compute<T>::type;
    constexpr int GATE = decltype(gate)::value, M = most_v<T>(true);
    const bool wide = q.dim % M == 0 && packs(q, d_x, x_seq_stride, x_step_stride, M) &&
                      packs(q, d_gate, gate_seq_stride, gate_step_stride, M) &&
                      packs(q, d_grad_h, grad_seq_stride, grad_step_stride, M) &&
                      packs(q, d_grad_x, 0, 0, M) && packs(q, d_grad_gate, 0, 0, M);
    const hipStream_t s = (hipStream_t)stream;
    Args<T> p = common_args<T>(q, d_x, x_seq_stride, x_step_stride, d_gate, gate_seq_stride,
                               gate_step_stride, d_h0, true);
    p.grad_h = (const T*)d_grad_h;
    p.d_seq = q.d_offsets ? 0 : grad_seq_stride;
    p.d_step = grad_step_stride;
    p.grad_last = (const C*)d_grad_last;
    p.saved = (C*)d_saved;
    p.grad_x = (T*)d_grad_x;
    p.grad_gate = (T*)d_grad_gate;
    p.grad_h0 = (C*)d_grad_h0;
    return run_chunks<M>(q, p, wide, d_work, true, s, [&](auto w, auto v, auto chain, dim3 grid) {
      if constexpr (decltype(w)::value == kNarrow)
        rec_backward<T, GATE, decltype(v)::value, decltype(chain)::value>
            <<<grid, kThreads, 0, s>>>(p);
    });
  });
}

}  // extern "C"
