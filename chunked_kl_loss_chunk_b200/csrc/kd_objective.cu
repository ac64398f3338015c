// kd_objective.cu -- the objectives of post-training over token
// log-probabilities: the clipped policy loss with a KL term, and the paired
// preference loss, each with its gradient for every token.
//
// Both read a few fp32 arrays over the batch's tokens once and write one, so
// memory bounds them when the batch is large and launch latency when it is
// small.  A batch is S sequences of tokens that lie one after the other: rows of
// L tokens, or sequence b at [cu[b], cu[b + 1]).  Work is split over the tokens
// and not over the sequences, so that one long sequence among short ones
// costs no more than its tokens.
#include <limits.h>
#include <math.h>

#include "kd_common.cuh"
#include "kd_internal.h"

namespace kd {

// ----------------------------------------------------------------------------
// Sequences over the token axis
// ----------------------------------------------------------------------------
// First token of sequence b, 0 <= b <= S, clamped into the batch: cu is the
// caller's data, and a bad entry must not take a loop out of bounds.
__device__ __forceinline__ int32_t seq_begin(const SeqLayout& q, int32_t b) {
  if (!q.cu) return b * q.L;
  return min(max(__ldg(q.cu + b), 0), q.N);
}

// t / L for 0 <= t < 2^31 by a multiplication (Granlund and Montgomery, "Division
// by invariant integers using multiplication", 1994): the host gives ceil(2^p / L).
__device__ __forceinline__ int32_t row_of(const SeqLayout& q, int32_t t) {
  if (q.L == 1) return t;
  return static_cast<int32_t>(__umulhi(static_cast<uint32_t>(t), q.div_mul) >> q.div_shift);
}

// Sequence of token t: the last b with begin(b) <= t, so that empty sequences
// are passed over.  -1 before the first sequence, S behind the last.
__device__ __forceinline__ int32_t seq_of(const SeqLayout& q, int32_t t) {
  if (!q.cu) return row_of(q, t);
  int32_t lo = -1, hi = q.S;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (__ldg(q.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The same for one token by a whole warp: 32 probes a step, so that a batch of
// 1000 sequences takes two dependent loads and not ten.
__device__ __forceinline__ int32_t seq_of_warp(const SeqLayout& q, int32_t t, int lane) {
  if (!q.cu) return row_of(q, t);
  int32_t lo = -1, n = q.S + 2;            // the answer is one of lo .. lo + n - 1
  while (n > 1) {
    const int32_t step = (n + 31) / 32;
    const int64_t at = static_cast<int64_t>(lo) + static_cast<int64_t>(lane + 1) * step;
    const bool before = at <= q.S && __ldg(q.cu + at) <= t;
    // an ascending cu sets the lowest lanes; of any other, the run of them is taken
    const int k = __ffs(~__ballot_sync(0xffffffffu, before)) - 1;
    const int32_t skip = (k < 0 ? 32 : k) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

// A token's sequence and where that sequence ends.
struct Cursor {
  int32_t b, e;
};
__device__ __forceinline__ Cursor cursor_of(const SeqLayout& q, int32_t b) {
  // b == -1 ends where the first sequence begins
  return Cursor{b, b >= q.S ? INT_MAX : seq_begin(q, b + 1)};
}
__device__ __forceinline__ Cursor cursor_at(const SeqLayout& q, int32_t t) {
  return cursor_of(q, seq_of(q, t));
}
__device__ __forceinline__ Cursor cursor_at_warp(const SeqLayout& q, int32_t t, int lane) {
  return cursor_of(q, seq_of_warp(q, t, lane));
}

// The sequence of token t, which c ends at or before: the next, unless that is empty.
__device__ __forceinline__ Cursor cursor_after(const SeqLayout& q, const Cursor& c, int32_t t) {
  if (c.b + 1 < q.S) {
    const int32_t e = seq_begin(q, c.b + 2);
    if (e > t) return Cursor{c.b + 1, e};
  }
  return cursor_at(q, t);
}

// Sequences of a lane's four tokens of a row in which c, its first token's, ends:
// the beginnings of the next 32 are loaded once and searched by shuffles; only a
// row with more has each lane search cu.
__device__ __forceinline__ void row_sequences(const SeqLayout& q, const Cursor& c, int32_t row0,
                                              int lane, int32_t (&b)[4]) {
  const int32_t last = min(row0 + 127, q.N - 1), t0 = row0 + 4 * lane;
  if (!q.cu) {
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = row_of(q, min(t0 + j, last));
    return;
  }
  const int64_t next = static_cast<int64_t>(c.b) + 1 + lane;
  const int32_t start = next <= q.S ? seq_begin(q, static_cast<int32_t>(next)) : INT_MAX;
  const bool few = __shfl_sync(0xffffffffu, start, 31) > last;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int32_t t = min(t0 + j, last);
    if (few) {
      int k = 0;                           // beginnings at or before t
#pragma unroll
      for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xffffffffu, start, k + step - 1) <= t) k += step;
      b[j] = c.b + k;
    } else {
      b[j] = seq_of(q, t);
    }
  }
}

// Records KD_ERR_BAD_INDEX unless 0 <= cu[0] <= cu[1] <= ... <= cu[S] <= N; true where this
// thread has seen that it is not so.  The loss of such a batch is NaN, for callers that
// do not read the status.
__device__ __forceinline__ bool check_layout(const SeqLayout& q, uint32_t* status) {
  bool bad = false;
  if (!q.cu) return false;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; b <= q.S;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int32_t x = __ldg(q.cu + b);
    const int32_t y = b < q.S ? __ldg(q.cu + b + 1) : q.N;
    if (x < 0 || x > y || x > q.N) bad = true;
  }
  if (bad) set_status(status, KD_ERR_BAD_INDEX);
  return bad;
}
// The same for a block that checks by itself, in every thread (a barrier).
__device__ __forceinline__ bool check_layout_block(const SeqLayout& q, uint32_t* status) {
  return q.cu && __syncthreads_or(check_layout(q, status));
}
// What the blocks of this grid, all of which have checked, or of an earlier one have seen.
__device__ __forceinline__ bool layout_bad(const SeqLayout& q, const uint32_t* status) {
  return q.cu && __ldcg(status) != 0u;
}
__device__ __forceinline__ float loss_out(double loss, bool bad) {
  return bad ? __int_as_float(0x7FC00000) : static_cast<float>(loss);
}

// ----------------------------------------------------------------------------
// Rows of 128 tokens, four a lane, copied asynchronously into shared memory some
// rows ahead of their use.  A lane copies its own tokens, and as a rule reads no
// others, so the copies need no barrier.  With the loads of the next row held in registers
// instead, the sums of the preference loss over 4.2M tokens took 15 us, waiting for
// memory at 28 warps an SM; they take 10 us.  The mask is loaded one row further
// ahead, into registers, and a row in which no token counts (a prompt, padding) is
// not copied at all.
// ----------------------------------------------------------------------------
template <int ARRAYS, int DEPTH>
struct RowQueue {
  static constexpr int ROW = ARRAYS * 512;            // bytes of a row
  static constexpr int WARP = DEPTH * ROW;
  unsigned char* at;                                  // this lane's places

  // The four values from p, of which the first `left` lie in the array; 0 in the places of
  // the others.  vec: p is 16-byte aligned.
  __device__ __forceinline__ void copy(int slot, int k, const float* p, int left, bool vec) const {
    const uint32_t to = smem_u32(at + slot * ROW + k * 512);
    if (vec) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p),
                   "r"(left < 4 ? 4 * left : 16)
                   : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * j),
                     "l"(j < left ? p + j : p), "r"(j < left ? 4 : 0)
                     : "memory");
    }
  }
  __device__ __forceinline__ void commit() const {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // No copy is under way (a walk may end before it has used all that it asked for).
  __device__ __forceinline__ void drain() const {
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  // The oldest row of DEPTH committed ones has arrived.
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
  }
  __device__ __forceinline__ void read(int slot, int k, float (&v)[4]) const {
    const float4 q = *reinterpret_cast<const float4*>(at + slot * ROW + k * 512);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  }
};

// Mask bytes with those outside [first, last) cleared.
__device__ __forceinline__ uint32_t inside(uint32_t m, int32_t t, int32_t first, int32_t last) {
  if (t >= first && t + 4 <= last) return m;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (t + j < first || t + j >= last) m &= ~(0xFFu << (8 * j));
  return m;
}
__device__ __forceinline__ bool mask_byte(uint32_t m, int j) { return m & (0xFFu << (8 * j)); }
// 0x80 in each byte that is not 0.
__device__ __forceinline__ uint32_t byte_flags(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w) & 0x80808080u;
}

// Mask bytes of four tokens, straight from memory.  vec: p is 4-byte aligned.
__device__ __forceinline__ uint32_t load_mask4(const uint8_t* p, int32_t t, int32_t N, bool vec) {
  if (t >= N) return 0u;
  if (!p) return t + 4 <= N ? 0x01010101u : 0x01010101u >> (8 * (4 - (N - t)));
  if (vec && t + 4 <= N) return __ldg(reinterpret_cast<const uint32_t*>(p + t));
  uint32_t m = 0;
  for (int j = 0; j < min(N - t, 4); ++j) m |= static_cast<uint32_t>(__ldg(p + t + j)) << (8 * j);
  return m;
}

__device__ __forceinline__ int32_t rows_of(const SeqLayout& q) { return (q.N + 127) / 128; }

// Four tokens' values to p + t.  vec: p is 16-byte aligned.
__device__ __forceinline__ void store4(float* p, int32_t t, int32_t N, const float (&v)[4],
                                       bool vec) {
  if (vec && t + 4 <= N) {
    *reinterpret_cast<float4*>(p + t) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t + j < N) p[t + j] = v[j];
  }
}

// True in every thread of the block that arrives last at `ticket` (zero before
// the grid); what the other blocks wrote before is then visible.
__device__ __forceinline__ bool last_block(uint32_t* ticket, uint32_t* sm_flag) {
  if (threadIdx.x == 0) {
    __threadfence();
    *sm_flag = atomicAdd(ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  return *sm_flag != 0;
}

// ----------------------------------------------------------------------------
// Clipped policy loss with a KL term.  Per token, with d = logp - old,
// r = e^d and q = ref - logp:
//   term  = -(clipped ? A bound : A r) + beta (e^q - 1 - q)
//   grad  = -(clipped ?    0    : A r) + beta (1 - e^q)
//   clipped: A > 0 and r > 1 + hi, or A < 0 and r < 1 - lo
// weighted by 1 / sum m, 1 / (S n_b) or 1 / denom.  The weight needs the counts
// of the mask first: a pass over the mask alone (1 byte a token) runs before
// the main one.
// ----------------------------------------------------------------------------
constexpr int OBJ_THREADS = 256;
constexpr int POLICY_STATS = OBJ_PARTIALS;   // sums: loss, tokens, r, clipped, KL
// Blocks of the main pass and of the preference loss's sums that an SM holds at once,
// which is also their grid: 2, 3, 4 and 5 of the first took 50, 42, 44 and 53 us at
// 8.4M tokens (more blocks leave too few registers); 4 and 5 of the second the same.
constexpr int POLICY_BLOCKS_PER_SM = 3, PREF_BLOCKS_PER_SM = 4;
constexpr int PREF_SHORT_MEAN = 30;   // tokens a sequence, on average, below which it is short

// Two fp32 values that one instruction works on (fma.rn.f32x2 and its like): the
// main pass is bound by the instructions it issues once its rows arrive in time.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void f2_get(const F2& a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(const F2& a, const F2& b, const F2& c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(const F2& a, const F2& b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(const F2& a, const F2& b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// e^x as 2^(x log2 e), with the hardware's 2^y (2^-22 of the value): the error of
// the product adds |x| 2^-24, as much as the rounding of x itself.
__device__ __forceinline__ F2 exp2v(const F2& x) {
  float lo, hi;
  f2_get(mul2(x, f2(1.44269504088896341f)), lo, hi);
  return f2(ex2_approx(lo), ex2_approx(hi));
}

// k = e^q - 1 - q without the cancellation of small q: q^2 times the Taylor series
// of (e^q - 1 - q) / q^2, whose first left-out term is below 2^-20 of it for
// |q| < 1/2.  Both forms are computed: a warp's tokens would take both branches as
// a rule.  em1: e^q - 1, which for a large -q (or an infinite one: the reference holds
// the token impossible) is not to be had as k + q any more.
__device__ __forceinline__ F2 exp_minus_linear(const F2& q, F2& em1) {
  F2 s = f2(1.f / 5040.f);
  s = fma2(s, q, f2(1.f / 720.f));
  s = fma2(s, q, f2(1.f / 120.f));
  s = fma2(s, q, f2(1.f / 24.f));
  s = fma2(s, q, f2(1.f / 6.f));
  s = fma2(s, q, f2(0.5f));
  s = mul2(mul2(q, q), s);
  const F2 far1 = add2(exp2v(q), f2(-1.f)), far = fma2(q, f2(-1.f), far1);
  float q0, q1, s0, s1, f0, f1, m0, m1, g0, g1;
  f2_get(q, q0, q1);
  f2_get(s, s0, s1);
  f2_get(far, f0, f1);
  f2_get(add2(s, q), m0, m1);
  f2_get(far1, g0, g1);
  const bool near0 = fabsf(q0) < 0.5f, near1 = fabsf(q1) < 0.5f;
  em1 = f2(near0 ? m0 : g0, near1 ? m1 : g1);
  return f2(near0 ? s0 : f0, near1 ? s1 : f1);
}

// Which of the 16 tokens from t0 the mask keeps, as bits.
__device__ __forceinline__ uint32_t mask_bits16(const PolicyArgs& a, int32_t t0) {
  uint32_t m = 0;
  if (a.mask_vec && t0 + 16 <= a.seq.N) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.mask + t0));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the four bytes' flags, gathered into four bits
      m |= ((byte_flags(w[i]) >> 7) * 0x10204080u >> 28) << (4 * i);
    }
  } else {
    for (int j = 0; j < 16; ++j)
      if (t0 + j < a.seq.N && __ldg(a.mask + t0 + j)) m |= 1u << j;
  }
  return m;
}

// Unmasked tokens of all sequences among this thread's 16-token pieces.
__device__ __forceinline__ uint32_t policy_count_all(const PolicyArgs& a, int64_t thread,
                                                     int64_t n_threads) {
  const int32_t first = seq_begin(a.seq, 0), last = seq_begin(a.seq, a.seq.S);
  uint32_t total = 0;
  for (int64_t i = thread * 16; i < a.seq.N; i += n_threads * 16) {
    const int32_t t0 = static_cast<int32_t>(i);
    uint32_t m = mask_bits16(a, t0);
    if (t0 < first || t0 + 16 > last)
      for (int j = 0; j < 16; ++j)
        if (t0 + j < first || t0 + j >= last) m &= ~(1u << j);
    total += __popc(m);
  }
  return total;
}

// Sum of a count over the block, in every thread.
__device__ __forceinline__ uint32_t block_count(uint32_t n, uint32_t* sm) {
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) n += sm[i];
  __syncthreads();
  return n;
}

__device__ __forceinline__ void policy_count_flush(const PolicyArgs& a, int32_t b, uint32_t n,
                                                   int lane) {
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n && b >= 0 && b < a.seq.S) atomicAdd(a.count + b, n);
}

// Unmasked tokens of each sequence, added to count[b] (zero before).  A warp takes
// 512 tokens at a time, and holds its count while the sequence stays the same: atomics
// on one address queue up.  (They are integer ones; their order does not matter.)
__device__ __forceinline__ void policy_count_each(const PolicyArgs& a, int32_t warp,
                                                  int32_t n_warps, int lane) {
  const SeqLayout& q = a.seq;
  int32_t held_b = -1;
  uint32_t held = 0;
  bool waited = false;               // for the kernel that clears the counts
  for (int64_t row = static_cast<int64_t>(warp) * 512; row < q.N;
       row += static_cast<int64_t>(n_warps) * 512) {
    const int32_t r0 = static_cast<int32_t>(row), t0 = r0 + lane * 16;   // below N + 512 < 2^31
    const uint32_t m = mask_bits16(a, t0);
    const Cursor first = cursor_at_warp(q, r0, lane);
    if (first.e >= min(r0 + 512, q.N)) {       // one sequence holds the 512
      if (first.b != held_b) {
        if (held_b >= 0 && !waited) {
          griddep_wait();
          waited = true;
        }
        policy_count_flush(a, held_b, held, lane);
        held_b = first.b;
        held = 0;
      }
      held += __popc(m);
      continue;
    }
    if (!waited) griddep_wait();
    waited = true;
    Cursor c = first;
    if (t0 >= c.e && t0 < q.N) c = cursor_at(q, t0);
    int32_t pos = t0;
    const int32_t end = min(t0 + 16, q.N);
    while (pos < end) {
      const int32_t stop = max(min(c.e, end), pos + 1);   // a bad cu still moves on
      const uint32_t n = __popc((m >> (pos - t0)) & ((1u << (stop - pos)) - 1u));
      if (n && c.b >= 0 && c.b < q.S) atomicAdd(a.count + c.b, n);
      pos = stop;
      if (pos < end) c = cursor_after(q, c, pos);
    }
  }
  if (!waited) griddep_wait();
  policy_count_flush(a, held_b, held, lane);
}

// Advantage (where it is the sequence's) and weight of the tokens of sequence b.
__device__ __forceinline__ void policy_look(const PolicyArgs& a, int32_t b, float seqs, float& adv,
                                            float& w) {
  const SeqLayout& q = a.seq;
  b = min(max(b, 0), q.S - 1);
  if (!a.adv_per_token) adv = __ldg(a.adv + b);
  if (a.reduction == KD_REDUCE_SEQUENCE) {
    const int32_t n = a.mask ? static_cast<int32_t>(__ldcg(a.count + b))
                             : seq_begin(q, b + 1) - seq_begin(q, b);
    // at least 1: the weight of a token that does not count is multiplied, too
    w = 1.f / (seqs * static_cast<float>(max(n, 1)));
  }
}

constexpr int POLICY_DEPTH = 2;
using PolicyQueue = RowQueue<4, POLICY_DEPTH>;

// Mask of a lane's tokens of a row: 0 beyond the batch and outside every sequence.
__device__ __forceinline__ uint32_t policy_mask(const PolicyArgs& a, int32_t row, int32_t n_rows,
                                                int32_t first, int32_t last, int lane) {
  if (row >= n_rows) return 0u;
  const int32_t t = row * 128 + 4 * lane;
  const uint32_t m = load_mask4(a.mask, t, a.seq.N, a.mask_vec);
  return a.seq.cu ? inside(m, t, first, last) : m;
}

// Starts the copies of a row with mask m, if any of its tokens counts.
template <bool OLD, bool REF>
__device__ __forceinline__ void policy_fetch(const PolicyArgs& a, const PolicyQueue& rows, int slot,
                                             int32_t row, uint32_t m, int lane) {
  if (__any_sync(0xffffffffu, m != 0)) {
    const int32_t t = row * 128 + 4 * lane, left = a.seq.N - t;
    if (left > 0) {
      rows.copy(slot, 0, a.logp + t, left, a.vec);
      if (OLD) rows.copy(slot, 1, a.old_logp + t, left, a.vec);
      if (REF) rows.copy(slot, 2, a.ref_logp + t, left, a.vec);
      if (a.adv_per_token) rows.copy(slot, 3, a.adv + t, left, a.vec);
    }
  }
  rows.commit();
}

// The masks of a warp's next rows, and the copies of those but the last under way.
struct PolicyAhead {
  uint32_t m[POLICY_DEPTH + 1];
  Cursor c;                         // of the next row, where sequences matter
};
__device__ __forceinline__ bool policy_by_sequence(const PolicyArgs& a) {
  return a.reduction == KD_REDUCE_SEQUENCE || !a.adv_per_token;
}
template <bool OLD, bool REF>
__device__ __forceinline__ void policy_start(const PolicyArgs& a, const PolicyQueue& rows,
                                             int32_t row, int32_t n_warps, PolicyAhead& ahead,
                                             int lane) {
  const int32_t n_rows = rows_of(a.seq), first = seq_begin(a.seq, 0);
  const int32_t last = seq_begin(a.seq, a.seq.S);
#pragma unroll
  for (int k = 0; k <= POLICY_DEPTH; ++k)
    ahead.m[k] = policy_mask(a, row + k * n_warps, n_rows, first, last, lane);
#pragma unroll
  for (int k = 0; k < POLICY_DEPTH; ++k)
    policy_fetch<OLD, REF>(a, rows, k, row + k * n_warps, ahead.m[k], lane);
  ahead.c = Cursor{0, INT_MAX};
  if (policy_by_sequence(a) && row < n_rows) ahead.c = cursor_at_warp(a.seq, row * 128, lane);
}

__device__ __forceinline__ void policy_add(double (&v)[POLICY_STATS], const F2& loss,
                                           const F2& ratio, const F2& kl) {
  float x, y;
  f2_get(loss, x, y);
  v[0] += x + y;
  f2_get(ratio, x, y);
  v[2] += x + y;
  f2_get(kl, x, y);
  v[4] += x + y;
}

// The main pass.  A warp takes rows of 128 tokens, `row` and every n_warps-th
// after it, the first of them under way (policy_start).  Sums go to v:
// fp32 over at most 16 rows of a lane's tokens, then fp64 (conversions to fp64 are
// slow: see the gradients' sums).  n_all: the tokens that count, for
// KD_REDUCE_TOKEN.
template <bool OLD, bool REF>
__device__ __forceinline__ void policy_tokens(const PolicyArgs& a, const PolicyQueue& queue,
                                              int32_t row, int32_t n_warps, uint32_t n_all,
                                              PolicyAhead& ahead, int lane,
                                              double (&v)[POLICY_STATS]) {
  const SeqLayout& q = a.seq;
  const bool need_seq = policy_by_sequence(a);
  const int32_t first = seq_begin(q, 0), last = seq_begin(q, q.S), n_rows = rows_of(q);
  float w = a.inv_denom;
  if (a.reduction == KD_REDUCE_TOKEN) {
    const uint32_t n = a.mask ? n_all : static_cast<uint32_t>(max(last - first, 0));
    w = n ? 1.f / static_cast<float>(n) : 0.f;
  }
  const float seqs = static_cast<float>(q.S);
  uint32_t n_tok = 0, n_clip = 0;
  F2 s_loss = f2(0.f), s_ratio = f2(0.f), s_kl = f2(0.f);
  int held = 0;
  for (int slot = 0; row < n_rows; row += n_warps, slot = slot + 1 == POLICY_DEPTH ? 0 : slot + 1) {
    const int32_t t0 = row * 128 + 4 * lane;
    const uint32_t m = ahead.m[0];
#pragma unroll
    for (int k = 0; k < POLICY_DEPTH; ++k) ahead.m[k] = ahead.m[k + 1];
    ahead.m[POLICY_DEPTH] =
        policy_mask(a, row + (POLICY_DEPTH + 1) * n_warps, n_rows, first, last, lane);
    queue.wait();
    float out[4] = {0.f, 0.f, 0.f, 0.f};
    if (__any_sync(0xffffffffu, m != 0)) {
      float lp[4], od[4], rf[4], at[4], wt[4];
      queue.read(slot, 0, lp);
      if (OLD) queue.read(slot, 1, od);
      if (REF) queue.read(slot, 2, rf);
      if (a.adv_per_token) queue.read(slot, 3, at);
#pragma unroll
      for (int j = 0; j < 4; ++j) wt[j] = w;
      if (need_seq) {
        const Cursor c = ahead.c;
        if (c.e >= row * 128 + 128) {          // one sequence holds the row
          policy_look(a, c.b, seqs, at[0], wt[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) {
            if (!a.adv_per_token) at[j] = at[0];
            wt[j] = wt[0];
          }
        } else {
          int32_t b[4];
          row_sequences(q, c, row * 128, lane, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) policy_look(a, b[j], seqs, at[j], wt[j]);
        }
      }
      // What a token that does not count holds is replaced before it is used: with its A and x at
      // 0 and its d at -inf, every term below and its ratio are 0 (a ratio of 1, to be taken off
      // at the end, would cost ratios far below one their digits).
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const bool on0 = mask_byte(m, j), on1 = mask_byte(m, j + 1);
        const float A0 = on0 ? at[j] : 0.f, A1 = on1 ? at[j + 1] : 0.f;
        const F2 A = f2(A0, A1), nlp = mul2(f2(lp[j], lp[j + 1]), f2(-1.f));
        float d0 = 0.f, d1 = 0.f;
        F2 ratio = f2(1.f);
        if (OLD) {
          f2_get(add2(f2(od[j], od[j + 1]), nlp), d0, d1);      // -d
          d0 = on0 ? -d0 : -INFINITY;
          d1 = on1 ? -d1 : -INFINITY;
          ratio = exp2v(f2(d0, d1));
          s_ratio = add2(s_ratio, ratio);
        }
        // r against the border in the logarithm.  d is the rounded difference, and rounding
        // keeps order: only d equal to the rounded border needs the exact difference.
        // (For A < 0 both sides are negated; an A of 0 or NaN is not clipped.)
        const bool up0 = A0 > 0.f, up1 = A1 > 0.f;
        const float border0 = up0 ? a.log_hi : -a.log_lo, border1 = up1 ? a.log_hi : -a.log_lo;
        const float e0 = up0 ? d0 : -d0, e1 = up1 ? d1 : -d1;
        bool clip0 = e0 > border0 && fabsf(A0) > 0.f, clip1 = e1 > border1 && fabsf(A1) > 0.f;
        if (e0 == border0 || e1 == border1) {
          const double x0 = OLD && on0 ? static_cast<double>(lp[j]) - od[j] : 0.0;
          const double x1 = OLD && on1 ? static_cast<double>(lp[j + 1]) - od[j + 1] : 0.0;
          clip0 = fabsf(A0) > 0.f && (up0 ? x0 > a.log_hi64 : x0 < a.log_lo64);
          clip1 = fabsf(A1) > 0.f && (up1 ? x1 > a.log_hi64 : x1 < a.log_lo64);
        }
        float r0, r1, t0_, t1_;
        f2_get(ratio, r0, r1);
        r0 = clip0 ? (up0 ? a.bound_hi : a.bound_lo) : r0;
        r1 = clip1 ? (up1 ? a.bound_hi : a.bound_lo) : r1;
        F2 term = mul2(A, f2(r0, r1));
        f2_get(term, t0_, t1_);
        F2 grad = f2(clip0 ? 0.f : t0_, clip1 ? 0.f : t1_);
        if (REF) {
          float x0, x1;
          f2_get(add2(f2(rf[j], rf[j + 1]), nlp), x0, x1);
          const F2 x = f2(on0 ? x0 : 0.f, on1 ? x1 : 0.f);
          F2 em1;
          const F2 k = exp_minus_linear(x, em1);
          s_kl = add2(s_kl, k);
          if (a.kl_coef != 0.f) {                      // 0 times an infinite k stays out
            term = fma2(f2(-a.kl_coef), k, term);
            grad = fma2(f2(a.kl_coef), em1, grad);
          }
        }
        const F2 nw = f2(-wt[j], -wt[j + 1]);
        s_loss = fma2(nw, term, s_loss);
        n_clip += (clip0 ? 1u : 0u) + (clip1 ? 1u : 0u);
        f2_get(mul2(nw, grad), out[j], out[j + 1]);
      }
      n_tok += __popc(byte_flags(m));
      if (++held == 16) {
        policy_add(v, s_loss, s_ratio, s_kl);
        s_loss = s_ratio = s_kl = f2(0.f);
        held = 0;
      }
    }
    if (a.dlogp && t0 < q.N) store4(a.dlogp, t0, q.N, out, a.vec);
    policy_fetch<OLD, REF>(a, queue, slot, row + POLICY_DEPTH * n_warps, ahead.m[POLICY_DEPTH - 1],
                           lane);
    if (need_seq && row + n_warps < n_rows && __any_sync(0xffffffffu, ahead.m[0] != 0))
      ahead.c = cursor_at_warp(q, (row + n_warps) * 128, lane);
  }
  policy_add(v, s_loss, s_ratio, s_kl);
  v[1] = n_tok;
  if (!OLD) v[2] = n_tok;
  v[3] = n_clip;
}

__device__ __forceinline__ void policy_write(const PolicyArgs& a, const double (&v)[POLICY_STATS],
                                             bool bad) {
  const double n = v[1] > 0.0 ? v[1] : 1.0;
  *a.loss = loss_out(v[0], bad);
  a.stats[0] = static_cast<float>(v[1]);
  a.stats[1] = static_cast<float>(v[2] / n);
  a.stats[2] = static_cast<float>(v[3] / n);
  a.stats[3] = static_cast<float>(v[4] / n);
}

// KD_REDUCE_TOKEN: a count for each block, which the main kernel adds.
__global__ void __launch_bounds__(OBJ_THREADS) policy_count_all_kernel(const PolicyArgs a) {
  __shared__ uint32_t sm[OBJ_THREADS / 32];
  griddep_launch_dependents();
  const uint32_t n =
      block_count(policy_count_all(a, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                                   static_cast<int64_t>(gridDim.x) * blockDim.x),
                  sm);
  if (threadIdx.x == 0) {
    a.count[blockIdx.x] = n;
    if (blockIdx.x == 0) {
      clear_status(a.status);
      *a.ticket = 0u;
    }
  }
}

// Status, ticket and, for KD_REDUCE_SEQUENCE with a mask, the sequences' counts: a
// kernel and not a memset, so that the next one can start under it.
__global__ void __launch_bounds__(OBJ_THREADS) policy_clear_kernel(const PolicyArgs a,
                                                                   int32_t counts) {
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * OBJ_THREADS + threadIdx.x;
  if (i == 0) {
    clear_status(a.status);
    *a.ticket = 0u;
  }
  if (i < counts) a.count[i] = 0u;
}

__global__ void __launch_bounds__(OBJ_THREADS) policy_count_each_kernel(const PolicyArgs a) {
  griddep_launch_dependents();
  policy_count_each(a, (blockIdx.x * blockDim.x + threadIdx.x) >> 5,
                    (gridDim.x * blockDim.x) >> 5, threadIdx.x & 31);
}

// 8.4M tokens, a third of them counting, advantages per token and a reference: 27 us,
// 6.1 TB/s of what a call has to read and write at most, and 197 instructions a row
// (0.6 of the issue slots).  0.8M packed tokens: 15 us, of which most is latency: the
// first loads, the look-ups, and the reduction over the blocks at the end.
template <bool OLD, bool REF>
__global__ void __launch_bounds__(OBJ_THREADS, POLICY_BLOCKS_PER_SM)
policy_main_kernel(const PolicyArgs a) {
  __shared__ __align__(16) unsigned char rows[OBJ_THREADS / 32 * PolicyQueue::WARP];
  __shared__ double sm[OBJ_THREADS / 32 * POLICY_STATS];
  __shared__ uint32_t flag, counts[OBJ_THREADS / 32];
  const int lane = threadIdx.x & 31;
  const int32_t row = (blockIdx.x * OBJ_THREADS + threadIdx.x) >> 5;
  const int32_t n_warps = (gridDim.x * OBJ_THREADS) >> 5;
  const PolicyQueue queue{rows + (threadIdx.x >> 5) * PolicyQueue::WARP + 16 * lane};
  PolicyAhead ahead;
  // the first rows do not wait for the counts
  policy_start<OLD, REF>(a, queue, row, n_warps, ahead, lane);
  griddep_wait();
  uint32_t n_all = 0;
  if (a.n_counts) {
    for (int i = threadIdx.x; i < a.n_counts; i += OBJ_THREADS) n_all += __ldcg(a.count + i);
    n_all = block_count(n_all, counts);
  }
  check_layout(a.seq, a.status);
  double v[POLICY_STATS] = {};
  policy_tokens<OLD, REF>(a, queue, row, n_warps, n_all, ahead, lane, v);
  block_sum(v, sm);
  if (threadIdx.x == 0)
#pragma unroll
    for (int i = 0; i < POLICY_STATS; ++i) a.partials[blockIdx.x * POLICY_STATS + i] = v[i];
  if (!last_block(a.ticket, &flag)) return;
  const bool bad = layout_bad(a.seq, a.status);
#pragma unroll
  for (int i = 0; i < POLICY_STATS; ++i) v[i] = 0.0;
  for (uint32_t k = threadIdx.x; k < gridDim.x; k += blockDim.x)
#pragma unroll
    for (int i = 0; i < POLICY_STATS; ++i) v[i] += __ldcg(a.partials + k * POLICY_STATS + i);
  block_sum(v, sm);
  if (threadIdx.x == 0) policy_write(a, v, bad);
}

// The whole loss in one block, for batches where launches cost more than the
// tokens: the counts, then the tokens.
template <bool OLD, bool REF>
__global__ void __launch_bounds__(OBJ_THREADS, 1) policy_one_kernel(const PolicyArgs a) {
  __shared__ __align__(16) unsigned char rows[OBJ_THREADS / 32 * PolicyQueue::WARP];
  __shared__ double sm[OBJ_THREADS / 32 * POLICY_STATS];
  __shared__ uint32_t counts[OBJ_THREADS / 32];
  constexpr int NW = OBJ_THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PolicyQueue queue{rows + warp * PolicyQueue::WARP + 16 * lane};
  PolicyAhead ahead;
  policy_start<OLD, REF>(a, queue, warp, NW, ahead, lane);
  if (threadIdx.x == 0) clear_status(a.status);
  uint32_t n_all = 0;
  if (a.mask && a.reduction == KD_REDUCE_SEQUENCE) {
    for (int32_t b = threadIdx.x; b < a.seq.S; b += OBJ_THREADS) a.count[b] = 0u;
    __syncthreads();
    policy_count_each(a, warp, NW, lane);
  } else if (a.mask && a.reduction == KD_REDUCE_TOKEN) {
    n_all = block_count(policy_count_all(a, threadIdx.x, OBJ_THREADS), counts);
  }
  __syncthreads();
  const bool bad = check_layout_block(a.seq, a.status);
  double v[POLICY_STATS] = {};
  policy_tokens<OLD, REF>(a, queue, warp, NW, n_all, ahead, lane, v);
  block_sum(v, sm);
  if (threadIdx.x == 0) policy_write(a, v, bad);
}

// ----------------------------------------------------------------------------
// Paired preference loss.
//   s_b = sum_t m_t (logp_t - ref_t) [/ n_b],  D = s_chosen - s_rejected,
//   z = beta D - margin
//   sigmoid  -(1 - e) log s(z) - e log s(-z);  hinge  max(0, 1 - z);
//   ipo      (D - 1 / (2 beta))^2
// Three steps: sums over every sequence; the pairs, a warp each or, where there are
// more of them than warps, a lane; the gradient, one value per sequence, spread over
// its tokens.
//
// The sums.  A warp walks a span of tokens, 128 at a time, adding each lane's
// four tokens in fp64 (a sum of 100,000 log-probabilities would lose 1e-2 of a
// unit in fp32), and reduces over the lanes where a sequence ends.  What it
// holds of a sequence goes to whole[b] if the sequence lies inside the span, to
// tail[span] if it begins there and goes on, and to head[span] if it began
// before; so every sum is added in one order, without atomics.
// ----------------------------------------------------------------------------
__device__ __forceinline__ void flush_part(SeqPart* to, double sum, uint32_t n, int lane) {
  sum = warp_sum(sum);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) *to = SeqPart{sum, static_cast<double>(n)};
}

// The same as cursor_after, by a whole warp.
__device__ __forceinline__ Cursor cursor_after_warp(const SeqLayout& q, const Cursor& c, int32_t t,
                                                    int lane) {
  if (c.b + 1 < q.S) {
    const int32_t e = seq_begin(q, c.b + 2);
    if (e > t) return Cursor{c.b + 1, e};
  }
  return cursor_at_warp(q, t, lane);
}

constexpr int PREF_DEPTH = 4;
using PrefQueue = RowQueue<2, PREF_DEPTH>;
constexpr int PREF_SMEM = PrefQueue::WARP + 128;     // bytes of a warp: its rows, a row's mask

__device__ __forceinline__ void pref_fetch(const PrefArgs& a, const PrefQueue& rows, int slot,
                                           int32_t t, int32_t s1, uint32_t m) {
  if (__any_sync(0xffffffffu, m != 0)) {
    if (t < s1) {
      rows.copy(slot, 0, a.logp + t, s1 - t, a.vec);
      if (a.ref_logp) rows.copy(slot, 1, a.ref_logp + t, s1 - t, a.vec);
    }
  }
  rows.commit();
}

// Sequences [b0, b1), all inside the row [r, r1) that lies in `row` (arrived, mask in
// `masks`): one lane for each.
__device__ __forceinline__ void pref_short(const PrefArgs& a, const unsigned char* row,
                                           const uint8_t* masks, int32_t b0, int32_t b1, int32_t r,
                                           int32_t r1, int lane) {
  for (int64_t b = static_cast<int64_t>(b0) + lane; b < b1; b += 32) {
    const int32_t begin = max(seq_begin(a.seq, static_cast<int32_t>(b)), r);
    const int32_t end = min(seq_begin(a.seq, static_cast<int32_t>(b) + 1), r1);
    double sum = 0.0;
    int n = 0;
    for (int i = begin - r; i < end - r; ++i) {
      if (!masks[i]) continue;
      const float x = reinterpret_cast<const float*>(row)[i];
      const float y = a.ref_logp ? reinterpret_cast<const float*>(row + 512)[i] : 0.f;
      sum += static_cast<double>(x) - static_cast<double>(y);
      ++n;
    }
    a.whole[b] = SeqPart{sum, static_cast<double>(n)};
  }
}

// smem: PREF_SMEM bytes of this warp.  SHORT: sequences that lie inside a row are taken
// a lane each, where a row holds several, and not one after the other by the warp.
// The code for it slows the walk over long ones, so batches choose by their mean
// length.
template <bool SHORT>
__device__ __forceinline__ void pref_sums(const PrefArgs& a, unsigned char* smem, int32_t span_i,
                                          int lane) {
  const SeqLayout& q = a.seq;
  const PrefQueue queue{smem + 16 * lane};
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + PrefQueue::WARP);
  const int32_t s0 = span_i * a.span, s1 = q.N - s0 < a.span ? q.N : s0 + a.span;
  uint32_t ahead[PREF_DEPTH + 1];            // masks of the next rows
#pragma unroll
  for (int k = 0; k <= PREF_DEPTH; ++k)
    ahead[k] = load_mask4(a.mask, s0 + 128 * k + 4 * lane, s1, a.mask_vec);
#pragma unroll
  for (int k = 0; k < PREF_DEPTH; ++k)
    pref_fetch(a, queue, k, s0 + 128 * k + 4 * lane, s1, ahead[k]);
  Cursor c = cursor_at_warp(q, s0, lane);
  bool begun = c.b >= 0 && c.b < q.S && seq_begin(q, c.b) >= s0;
  double sum = 0.0;
  uint32_t n = 0;
  int slot = 0;
  for (int32_t r = s0; r < s1 && c.b < q.S; r += 128) {
    const int32_t r1 = min(r + 128, s1), t = r + 4 * lane;
    const uint32_t m = ahead[0];
#pragma unroll
    for (int k = 0; k < PREF_DEPTH; ++k) ahead[k] = ahead[k + 1];
    ahead[PREF_DEPTH] = load_mask4(a.mask, t + 128 * (PREF_DEPTH + 1), s1, a.mask_vec);
    queue.wait();
    const bool any = __any_sync(0xffffffffu, m != 0);
    float x[4] = {}, y[4] = {};
    if (any) {
      queue.read(slot, 0, x);
      if (a.ref_logp) queue.read(slot, 1, y);
    }
    double d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double ref = a.ref_logp ? static_cast<double>(y[j]) : 0.0;
      d[j] = mask_byte(m, j) ? static_cast<double>(x[j]) - ref : 0.0;
    }
    if (!SHORT) pref_fetch(a, queue, slot, t + 128 * PREF_DEPTH, s1, ahead[PREF_DEPTH - 1]);
    if (c.e >= r1 && c.b >= 0) {             // the whole row belongs to one sequence
      if (any) {
        sum += (d[0] + d[1]) + (d[2] + d[3]);
        n += __popc(byte_flags(m));
      }
    } else {
      int32_t pos = r;
      while (pos < r1) {
        const int32_t stop = min(c.e, r1);
        if (c.b >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (t + j >= pos && t + j < stop) {
              sum += d[j];
              n += mask_byte(m, j) ? 1u : 0u;
            }
        }
        if (c.e >= r1) break;                // the row's rest is taken
        if (c.b >= 0) flush_part(begun ? a.whole + c.b : a.head + span_i, sum, n, lane);
        sum = 0.0;
        n = 0;
        begun = true;
        pos = max(stop, pos + 1);            // a bad cu still moves on
        c = cursor_after_warp(q, c, pos, lane);
        if (SHORT && c.b < q.S && c.e < r1) {    // it ends in the row as well, and others may
          const Cursor l = cursor_at_warp(q, r1 - 1, lane);
          masks[lane] = m;
          __syncwarp();                      // the lanes' copies and masks, for all lanes
          pref_short(a, smem + slot * PrefQueue::ROW, reinterpret_cast<const uint8_t*>(masks),
                     max(c.b, 0), min(l.b, q.S), r, r1, lane);
          __syncwarp();
          c = l;
          if (c.b < q.S) pos = max(seq_begin(q, max(c.b, 0)), pos);
        }
        if (c.b >= q.S) break;               // behind the last sequence
      }
      if (c.b >= q.S) break;
    }
    if (c.e == r1) {                         // ends with the row
      if (c.b >= 0) flush_part(begun ? a.whole + c.b : a.head + span_i, sum, n, lane);
      sum = 0.0;
      n = 0;
      if (r1 >= s1) break;
      c = cursor_after_warp(q, c, r1, lane);
      begun = true;
    }
    // (a row is overwritten after all lanes have read it)
    if (SHORT) pref_fetch(a, queue, slot, t + 128 * PREF_DEPTH, s1, ahead[PREF_DEPTH - 1]);
    if (++slot == PREF_DEPTH) slot = 0;
  }
  if (c.b >= 0 && c.b < q.S && c.e > s1)
    flush_part(begun ? a.tail + span_i : a.head + span_i, sum, n, lane);
  queue.drain();
}

// Sum and count of each lane's sequence b (-1: none) from its parts.  Called by a
// whole warp, which adds the many parts of a long sequence together.
__device__ __forceinline__ SeqPart pref_join(const PrefArgs& a, int32_t b, int lane) {
  constexpr int ALONE = 4;                   // parts that a lane adds by itself
  SeqPart p{0.0, 0.0};
  int32_t i0 = 0, i1 = -1;
  if (b >= 0) {
    const int32_t t0 = seq_begin(a.seq, b), t1 = seq_begin(a.seq, b + 1);
    if (t1 > t0) {
      i0 = t0 / a.span;
      i1 = (t1 - 1) / a.span;
    }
    if (i1 == i0) {
      p = SeqPart{__ldcg(&a.whole[b].sum), __ldcg(&a.whole[b].n)};
    } else if (i1 - i0 < ALONE) {
      SeqPart part[ALONE];
#pragma unroll
      for (int k = 0; k < ALONE; ++k) {
        part[k] = SeqPart{0.0, 0.0};
        if (i0 + k > i1) continue;
        const SeqPart* s = k == 0 ? a.tail + i0 : a.head + i0 + k;
        part[k] = SeqPart{__ldcg(&s->sum), __ldcg(&s->n)};
      }
#pragma unroll
      for (int k = 0; k < ALONE; ++k) {
        p.sum += part[k].sum;
        p.n += part[k].n;
      }
    }
  }
  uint32_t many = __ballot_sync(0xffffffffu, i1 - i0 >= ALONE);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    const int32_t j0 = __shfl_sync(0xffffffffu, i0, src), j1 = __shfl_sync(0xffffffffu, i1, src);
    SeqPart part{0.0, 0.0};
    if (lane == 0) part = SeqPart{__ldcg(&a.tail[j0].sum), __ldcg(&a.tail[j0].n)};
#pragma unroll 8
    for (int32_t i = j0 + 1 + lane; i <= j1; i += 32) {
      const double2 h = __ldcg(reinterpret_cast<const double2*>(a.head + i));
      part.sum += h.x;
      part.n += h.y;
    }
    part.sum = warp_sum(part.sum);
    part.n = warp_sum(part.n);
    if (lane == src) p = part;
  }
  return p;
}

// Pairs from i on, a lane for each of a warp's a.pairs_per_warp: the rewards and the
// gradient of each of the two sequences' tokens.  Returns the lane's pair's loss.
__device__ __forceinline__ double pref_pair(const PrefArgs& a, int32_t i, int lane) {
  const int32_t B = a.seq.S / 2;
  const bool mine = lane < a.pairs_per_warp && i + lane < B;
  i = mine ? i + lane : -1;
  const SeqPart c = pref_join(a, i, lane), r = pref_join(a, mine ? i + B : -1, lane);
  if (!mine) return 0.0;
  const double per_c = a.normalize ? 1.0 / fmax(c.n, 1.0) : 1.0;
  const double per_r = a.normalize ? 1.0 / fmax(r.n, 1.0) : 1.0;
  const double sc = c.sum * per_c, sr = r.sum * per_r, D = sc - sr;
  const double z = a.beta * D - a.margin;
  double loss, slope;
  if (a.kind == KD_PREF_IPO) {
    const double u = D - 0.5 / a.beta;
    loss = u * u;
    slope = 2.0 * u;
  } else if (a.kind == KD_PREF_HINGE) {
    loss = z < 1.0 ? 1.0 - z : (z >= 1.0 ? 0.0 : z);       // NaN stays NaN
    slope = z < 1.0 ? -a.beta : (z >= 1.0 ? 0.0 : z);
  } else {
    const double soft = log1p(exp(-fabs(z)));
    loss = (1.0 - a.smoothing) * (fmax(-z, 0.0) + soft);
    if (a.smoothing > 0.0) loss += a.smoothing * (fmax(z, 0.0) + soft);   // z may be infinite
    if (z != z) loss = z;
    slope = a.beta * (a.smoothing - 1.0 / (1.0 + exp(z)));
  }
  a.rewards[i] = static_cast<float>(a.beta * sc);
  a.rewards[i + B] = static_cast<float>(a.beta * sr);
  a.coef[i] = static_cast<float>(slope * per_c * a.inv_pairs);
  a.coef[i + B] = static_cast<float>(-slope * per_r * a.inv_pairs);
  return loss;
}

// This warp's groups of pairs; returns the sum of the lane's losses.
__device__ __forceinline__ double pref_pairs(const PrefArgs& a, int32_t warp, int32_t n_warps,
                                             int lane) {
  const int64_t step = static_cast<int64_t>(n_warps) * a.pairs_per_warp;
  double sum = 0.0;
  for (int64_t i = static_cast<int64_t>(warp) * a.pairs_per_warp; i < a.seq.S / 2; i += step)
    sum += pref_pair(a, static_cast<int32_t>(i), lane);
  return sum;
}

// The gradient of rows of 128 tokens, `row` and every n_warps-th after it;
// m_next is the mask of the first.
__device__ __forceinline__ void pref_tokens(const PrefArgs& a, int32_t row, int32_t n_warps,
                                            uint32_t m_next, int lane) {
  const SeqLayout& q = a.seq;
  const int32_t n_rows = rows_of(q);
  for (; row < n_rows; row += n_warps) {
    const uint32_t m = m_next;
    const int32_t row0 = row * 128, t0 = row0 + 4 * lane;
    if (row + n_warps < n_rows)
      m_next = load_mask4(a.mask, (row + n_warps) * 128 + 4 * lane, q.N, a.mask_vec);
    const Cursor c = cursor_at_warp(q, row0, lane);
    float out[4];
    if (c.e >= row0 + 128) {
      const float k = c.b >= 0 && c.b < q.S ? __ldcg(a.coef + c.b) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = mask_byte(m, j) ? k : 0.f;
    } else {
      int32_t b[4];
      row_sequences(q, c, row0, lane, b);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out[j] = mask_byte(m, j) && b[j] >= 0 && b[j] < q.S ? __ldcg(a.coef + b[j]) : 0.f;
    }
    if (t0 < q.N) store4(a.dlogp, t0, q.N, out, a.vec);
  }
}

// 4.2M tokens with a reference: 11 us (3.4 TB/s; 7 rows a warp leave little after the
// first loads' latency), then the pairs 4 and the tokens 5 (17 MB written).
template <bool SHORT>
__global__ void __launch_bounds__(OBJ_THREADS, PREF_BLOCKS_PER_SM)
pref_sums_kernel(const PrefArgs a) {
  __shared__ __align__(16) unsigned char rows[OBJ_THREADS / 32 * PREF_SMEM];
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) clear_status(a.status);
  const int warp = threadIdx.x >> 5;
  const int32_t i = blockIdx.x * (OBJ_THREADS / 32) + warp;
  if (i < a.n_spans) pref_sums<SHORT>(a, rows + warp * PREF_SMEM, i, threadIdx.x & 31);
}

__global__ void __launch_bounds__(OBJ_THREADS) pref_pair_kernel(const PrefArgs a) {
  __shared__ double sm[OBJ_THREADS / 32];
  griddep_launch_dependents();
  griddep_wait();                            // the sums
  check_layout(a.seq, a.status);
  double v[1] = {pref_pairs(a, (blockIdx.x * OBJ_THREADS + threadIdx.x) >> 5,
                            (gridDim.x * OBJ_THREADS) >> 5, threadIdx.x & 31)};
  block_sum(v, sm);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = v[0];
}

// The tokens' gradients, and in the last block the sum of the pairs' losses
// (n_partials blocks of the kernel before), which the gradients do not need.
__global__ void __launch_bounds__(OBJ_THREADS) pref_tokens_kernel(const PrefArgs a,
                                                                  int n_partials) {
  __shared__ double sm[OBJ_THREADS / 32];
  const int lane = threadIdx.x & 31;
  const int32_t row = (blockIdx.x * OBJ_THREADS + threadIdx.x) >> 5;
  const uint32_t m =
      row < rows_of(a.seq) ? load_mask4(a.mask, row * 128 + 4 * lane, a.seq.N, a.mask_vec) : 0u;
  griddep_wait();                            // the pairs
  if (a.dlogp) pref_tokens(a, row, (gridDim.x * OBJ_THREADS) >> 5, m, lane);
  if (blockIdx.x != gridDim.x - 1) return;
  const bool bad = layout_bad(a.seq, a.status);
  double v[1] = {0.0};
  for (int k = threadIdx.x; k < n_partials; k += OBJ_THREADS) v[0] += __ldcg(a.partials + k);
  block_sum(v, sm);
  if (threadIdx.x == 0) *a.loss = loss_out(v[0] * a.inv_pairs, bad);
}

// The three steps in one block, for batches where launches cost more than the
// tokens.
template <bool SHORT>
__global__ void __launch_bounds__(OBJ_THREADS, 1) pref_one_kernel(const PrefArgs a) {
  __shared__ __align__(16) unsigned char rows[OBJ_THREADS / 32 * PREF_SMEM];
  __shared__ double sm[OBJ_THREADS / 32];
  constexpr int NW = OBJ_THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) clear_status(a.status);
  for (int32_t i = warp; i < a.n_spans; i += NW)
    pref_sums<SHORT>(a, rows + warp * PREF_SMEM, i, lane);
  __syncthreads();
  const bool bad = check_layout_block(a.seq, a.status);
  double v[1] = {pref_pairs(a, warp, NW, lane)};
  block_sum(v, sm);                          // its barriers also publish the gradients
  if (threadIdx.x == 0) *a.loss = loss_out(v[0] * a.inv_pairs, bad);
  if (a.dlogp)
    pref_tokens(a, warp, NW, load_mask4(a.mask, 4 * threadIdx.x, a.seq.N, a.mask_vec), lane);
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

// Batches of at most this many tokens and sequences run in one block.  (8, 2048 and 4096
// tokens: policy 4.3, 4.8 to 5.2 and 7 to 7.5 us in one block, 6.6 to 6.8 in several;
// 8, 512, 1024 and 2048 tokens: preference 5.2, 5.3 to 6.2, 6.3 and 7.2 to 10 against 6.3,
// 6.4 to 7.5, 8.1 and 6.7 to 7.8.)
constexpr int64_t POLICY_ONE_BLOCK = 2048, PREF_ONE_BLOCK = 1024;

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), int64_t blocks, int threads, cudaStream_t s, bool pdl,
                   const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

int64_t at_most(int64_t x, int64_t cap) { return x < cap ? (x > 0 ? x : 1) : cap; }

}  // namespace

namespace {

template <bool OLD, bool REF>
kd_status policy_launch(PolicyArgs a, cudaStream_t s, int num_sms) {
  const SeqLayout& q = a.seq;
  if (q.N <= POLICY_ONE_BLOCK && q.S <= POLICY_ONE_BLOCK)
    return launch(policy_one_kernel<OLD, REF>, 1, OBJ_THREADS, s, false, a) == cudaSuccess
               ? KD_OK
               : KD_ERR_CUDA;
  const bool all = a.mask && a.reduction == KD_REDUCE_TOKEN;
  const bool each = a.mask && a.reduction == KD_REDUCE_SEQUENCE;
  cudaError_t e = cudaSuccess;
  if (all) {
    a.n_counts = static_cast<int32_t>(
        at_most((static_cast<int64_t>(q.N) + 16 * OBJ_THREADS - 1) / (16 * OBJ_THREADS),
                at_most(4 * num_sms, OBJ_MAX_COUNTS)));
    e = launch(policy_count_all_kernel, a.n_counts, OBJ_THREADS, s, false, a);
  } else {
    const int32_t counts = each ? q.S : 0;
    e = launch(policy_clear_kernel, (static_cast<int64_t>(counts) + OBJ_THREADS) / OBJ_THREADS,
               OBJ_THREADS, s, false, a, counts);
    if (e == cudaSuccess && each)
      e = launch(policy_count_each_kernel,
                 at_most((static_cast<int64_t>(q.N) + 4095) / 4096, 4 * num_sms), OBJ_THREADS, s,
                 true, a);
  }
  if (e != cudaSuccess) return KD_ERR_CUDA;
  const int64_t per_block = 4 * OBJ_THREADS;
  const int64_t cap = at_most(POLICY_BLOCKS_PER_SM * num_sms, OBJ_MAX_BLOCKS);
  e = launch(policy_main_kernel<OLD, REF>, at_most((q.N + per_block - 1) / per_block, cap),
             OBJ_THREADS, s, true, a);
  return e == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

}  // namespace

kd_status policy_loss(const PolicyArgs& a, cudaStream_t s, int num_sms) {
  if (a.old_logp)
    return a.ref_logp ? policy_launch<true, true>(a, s, num_sms)
                      : policy_launch<true, false>(a, s, num_sms);
  return a.ref_logp ? policy_launch<false, true>(a, s, num_sms)
                    : policy_launch<false, false>(a, s, num_sms);
}

kd_status preference_loss(PrefArgs a, cudaStream_t s, int num_sms) {
  const SeqLayout& q = a.seq;
  constexpr int W = OBJ_THREADS / 32;
  // a warp for each pair as long as they last, then a lane
  const bool one = q.N <= PREF_ONE_BLOCK && q.S <= PREF_ONE_BLOCK;
  const int64_t pairs = q.S / 2, warps = one ? W : static_cast<int64_t>(W) * 4 * num_sms;
  a.pairs_per_warp = static_cast<int32_t>(at_most((pairs + warps - 1) / warps, 32));
  // (2048 sequences of 8 tokens: 9 us with a lane each, 12 without; of 30: 10.4 and 10.3)
  const bool few_tokens = static_cast<int64_t>(q.N) < static_cast<int64_t>(PREF_SHORT_MEAN) * q.S;
  if (one)
    return launch(few_tokens ? pref_one_kernel<true> : pref_one_kernel<false>, 1, OBJ_THREADS, s,
                  false, a) == cudaSuccess
               ? KD_OK
               : KD_ERR_CUDA;
  if (launch(few_tokens ? pref_sums_kernel<true> : pref_sums_kernel<false>,
             (a.n_spans + W - 1) / W, OBJ_THREADS, s, false, a) != cudaSuccess)
    return KD_ERR_CUDA;
  const int64_t cap = at_most(8 * num_sms, OBJ_MAX_BLOCKS);
  const int64_t groups = (pairs + a.pairs_per_warp - 1) / a.pairs_per_warp;
  const int64_t pair_blocks = at_most((groups + W - 1) / W, cap);
  if (launch(pref_pair_kernel, pair_blocks, OBJ_THREADS, s, true, a) != cudaSuccess)
    return KD_ERR_CUDA;
  const int64_t per_block = 4 * OBJ_THREADS;
  const int64_t blocks = a.dlogp ? at_most((q.N + per_block - 1) / per_block, cap) : 1;
  if (launch(pref_tokens_kernel, blocks, OBJ_THREADS, s, true, a, static_cast<int>(pair_blocks)) !=
      cudaSuccess)
    return KD_ERR_CUDA;
  return KD_OK;
}

}  // namespace kd
