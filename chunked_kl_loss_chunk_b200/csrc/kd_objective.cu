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

// Sequence of token t: the last b with begin(b) <= t, so that empty sequences
// are passed over.  -1 before the first sequence, S behind the last.
__device__ __forceinline__ int32_t seq_of(const SeqLayout& q, int32_t t) {
  if (!q.cu) return static_cast<int32_t>(static_cast<uint32_t>(t) / static_cast<uint32_t>(q.L));
  int32_t lo = -1, hi = q.S;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (__ldg(q.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A token's sequence and where that sequence ends.
struct Cursor {
  int32_t b, e;
};
__device__ __forceinline__ Cursor cursor_at(const SeqLayout& q, int32_t t) {
  Cursor c;
  c.b = seq_of(q, t);
  c.e = c.b >= q.S ? INT_MAX : seq_begin(q, c.b + 1);   // b == -1: the first sequence's begin
  return c;
}

// Records KD_ERR_BAD_INDEX unless 0 <= cu[0] <= cu[1] <= ... <= cu[S] <= N.
__device__ __forceinline__ void check_layout(const SeqLayout& q, uint32_t* status) {
  if (!q.cu) return;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; b <= q.S;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int32_t x = __ldg(q.cu + b);
    const int32_t y = b < q.S ? __ldg(q.cu + b + 1) : q.N;
    if (x < 0 || x > y || x > q.N) set_status(status, KD_ERR_BAD_INDEX);
  }
}

// Four consecutive tokens from t (a multiple of 4): values, or `fill` beyond N.
__device__ __forceinline__ void load4(const float* p, int32_t t, int32_t N, float fill,
                                      float (&v)[4]) {
  if (t + 4 <= N) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p + t));
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = t + j < N ? __ldg(p + t + j) : fill;
  }
}

// Bit j: token t + j lies in the batch and its mask byte is not 0.
__device__ __forceinline__ uint32_t load_mask4(const uint8_t* p, int32_t t, int32_t N) {
  if (!p) return t + 4 <= N ? 0xFu : (t < N ? (1u << (N - t)) - 1u : 0u);
  uint32_t m = 0;
  if (t + 4 <= N) {
    const uchar4 q = __ldg(reinterpret_cast<const uchar4*>(p + t));
    m = (q.x ? 1u : 0u) | (q.y ? 2u : 0u) | (q.z ? 4u : 0u) | (q.w ? 8u : 0u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t + j < N && __ldg(p + t + j)) m |= 1u << j;
  }
  return m;
}

__device__ __forceinline__ void store4(float* p, int32_t t, int32_t N, const float (&v)[4]) {
  if (t + 4 <= N) {
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
// the main one.  Integer atomics add the counts, whose order does not matter.
// ----------------------------------------------------------------------------
constexpr int OBJ_THREADS = 256;
constexpr int POLICY_STATS = 5;   // loss, tokens, ratios, clipped, KL

// e^q - 1 - q without the cancellation of small q: q^2 times the Taylor series of
// (e^q - 1 - q) / q^2, whose first left-out term is below 2^-24 of it for |q| < 1/2.
__device__ __forceinline__ float exp_minus_linear(float q) {
  if (fabsf(q) < 0.5f) {
    float s = 1.f / 362880.f;
    s = fmaf(s, q, 1.f / 40320.f);
    s = fmaf(s, q, 1.f / 5040.f);
    s = fmaf(s, q, 1.f / 720.f);
    s = fmaf(s, q, 1.f / 120.f);
    s = fmaf(s, q, 1.f / 24.f);
    s = fmaf(s, q, 1.f / 6.f);
    s = fmaf(s, q, 0.5f);
    return q * q * s;
  }
  return expf(q) - 1.f - q;
}

// Mask counts, into count[0] (all sequences) or count[b].
__device__ __forceinline__ void policy_count(const PolicyArgs& a, int32_t warp, int32_t n_warps,
                                             int lane) {
  const SeqLayout& q = a.seq;
  const bool per_seq = a.reduction == KD_REDUCE_SEQUENCE;
  const int32_t first = seq_begin(q, 0), last = seq_begin(q, q.S);
  uint32_t total = 0;
  for (int64_t row = static_cast<int64_t>(warp) * 512; row < q.N;
       row += static_cast<int64_t>(n_warps) * 512) {
    const int32_t t0 = static_cast<int32_t>(row) + lane * 16;    // row + 512 <= N + 511 < 2^31
    uint32_t m = 0;
    if (t0 + 16 <= q.N) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.mask + t0));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((w[i] >> (8 * j)) & 0xFFu) m |= 1u << (4 * i + j);
    } else {
      for (int j = 0; j < 16; ++j)
        if (t0 + j < q.N && __ldg(a.mask + t0 + j)) m |= 1u << j;
    }
    if (!per_seq) {
      if (q.cu && (t0 < first || t0 + 16 > last)) {
        for (int j = 0; j < 16; ++j)
          if (t0 + j < first || t0 + j >= last) m &= ~(1u << j);
      }
      total += __popc(m);
      continue;
    }
    Cursor c{q.S, INT_MAX};
    if (t0 < q.N) c = cursor_at(q, t0);
    int same;
    __match_all_sync(0xffffffffu, c.e >= t0 + 16 ? c.b : -2 - lane, &same);
    if (same) {
      const uint32_t n = __reduce_add_sync(0xffffffffu, __popc(m));
      if (lane == 0 && n && c.b >= 0 && c.b < q.S) atomicAdd(a.count + c.b, n);
    } else {
      int32_t pos = t0;
      const int32_t end = min(t0 + 16, q.N);
      while (pos < end) {
        const int32_t stop = max(min(c.e, end), pos + 1);   // a bad cu still moves on
        const uint32_t n = __popc((m >> (pos - t0)) & ((1u << (stop - pos)) - 1u));
        if (n && c.b >= 0 && c.b < q.S) atomicAdd(a.count + c.b, n);
        pos = stop;
        if (pos < end) c = cursor_at(q, pos);
      }
    }
  }
  if (!per_seq) {
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0 && total) atomicAdd(a.count, total);
  }
}

// The main pass over this thread's groups of four tokens; sums into v.
__device__ __forceinline__ void policy_tokens(const PolicyArgs& a, int64_t thread,
                                              int64_t n_threads, double (&v)[POLICY_STATS]) {
  const SeqLayout& q = a.seq;
  const bool per_seq = a.reduction == KD_REDUCE_SEQUENCE;
  const int32_t first = seq_begin(q, 0), last = seq_begin(q, q.S);
  float w = a.inv_denom;
  if (a.reduction == KD_REDUCE_TOKEN) {
    const uint32_t n = a.mask ? __ldcg(a.count) : static_cast<uint32_t>(max(last - first, 0));
    w = n ? 1.f / static_cast<float>(n) : 0.f;
  }
  const bool need_seq = per_seq || !a.adv_per_token;
  uint32_t n_tok = 0, n_clip = 0;
  const int64_t groups = (static_cast<int64_t>(q.N) + 3) / 4;
  for (int64_t g = thread; g < groups; g += n_threads) {
    const int32_t t0 = static_cast<int32_t>(4 * g);
    float lp[4], od[4], rf[4], av[4], out[4];
    uint32_t m = load_mask4(a.mask, t0, q.N);
    load4(a.logp, t0, q.N, 0.f, lp);
    if (a.old_logp) load4(a.old_logp, t0, q.N, 0.f, od);
    if (a.ref_logp) load4(a.ref_logp, t0, q.N, 0.f, rf);
    if (a.adv_per_token) load4(a.adv, t0, q.N, 0.f, av);
    if (q.cu && (t0 < first || t0 + 4 > last)) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t0 + j < first || t0 + j >= last) m &= ~(1u << j);
    }
    Cursor c{-1, INT_MIN};
    float adv = 0.f, s_loss = 0.f, s_ratio = 0.f, s_kl = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[j] = 0.f;
      if (!((m >> j) & 1u)) continue;       // values of masked tokens are never used
      if (need_seq && t0 + j >= c.e) {
        c = cursor_at(q, t0 + j);
        const int32_t b = min(max(c.b, 0), q.S - 1);
        if (!a.adv_per_token) adv = __ldg(a.adv + b);
        if (per_seq) {
          const uint32_t n = a.mask ? __ldcg(a.count + b)
                                    : static_cast<uint32_t>(max(c.e - seq_begin(q, b), 1));
          w = 1.f / (static_cast<float>(q.S) * static_cast<float>(n));
        }
      }
      const float A = a.adv_per_token ? av[j] : adv;
      float d = 0.f, r = 1.f;
      bool clip = false;
      if (a.old_logp) {
        d = lp[j] - od[j];
        r = expf(d);
      }
      // r against the border in the logarithm.  d is the rounded difference, and rounding
      // keeps order: only d equal to the rounded border needs the exact difference.
      if (A > 0.f) {
        clip = d > a.log_hi || (d == a.log_hi && (a.old_logp ? static_cast<double>(lp[j]) - od[j]
                                                             : 0.0) > a.log_hi64);
      } else if (A < 0.f) {
        clip = d < a.log_lo || (d == a.log_lo && (a.old_logp ? static_cast<double>(lp[j]) - od[j]
                                                             : 0.0) < a.log_lo64);
      }
      const float Ar = A * r;
      float term = clip ? -A * (A > 0.f ? a.bound_hi : a.bound_lo) : -Ar;
      float grad = clip ? 0.f : -Ar;
      if (a.ref_logp) {
        const float x = rf[j] - lp[j];
        const float k = exp_minus_linear(x);
        s_kl += k;
        if (a.kl_coef != 0.f) {
          term = fmaf(a.kl_coef, k, term);
          grad = fmaf(-a.kl_coef, k + x, grad);      // 1 - e^x = -(k + x)
        }
      }
      s_loss = fmaf(w, term, s_loss);
      s_ratio += r;
      ++n_tok;
      n_clip += clip ? 1u : 0u;
      out[j] = w * grad;
    }
    v[0] += s_loss;
    v[2] += s_ratio;
    v[4] += s_kl;
    if (a.dlogp) store4(a.dlogp, t0, q.N, out);
  }
  v[1] = n_tok;
  v[3] = n_clip;
}

__device__ __forceinline__ void policy_write(const PolicyArgs& a, const double (&v)[POLICY_STATS]) {
  const double n = v[1] > 0.0 ? v[1] : 1.0;
  *a.loss = static_cast<float>(v[0]);
  a.stats[0] = static_cast<float>(v[1]);
  a.stats[1] = static_cast<float>(v[2] / n);
  a.stats[2] = static_cast<float>(v[3] / n);
  a.stats[3] = static_cast<float>(v[4] / n);
}

__global__ void __launch_bounds__(OBJ_THREADS) policy_count_kernel(const PolicyArgs a) {
  griddep_launch_dependents();
  policy_count(a, (blockIdx.x * blockDim.x + threadIdx.x) >> 5, (gridDim.x * blockDim.x) >> 5,
               threadIdx.x & 31);
}

__global__ void __launch_bounds__(OBJ_THREADS) policy_main_kernel(const PolicyArgs a) {
  __shared__ double sm[32 * POLICY_STATS];
  __shared__ uint32_t flag;
  griddep_wait();                            // the counts
  check_layout(a.seq, a.status);
  double v[POLICY_STATS] = {};
  policy_tokens(a, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                static_cast<int64_t>(gridDim.x) * blockDim.x, v);
  block_sum(v, sm);
  if (threadIdx.x == 0)
#pragma unroll
    for (int i = 0; i < POLICY_STATS; ++i) a.partials[blockIdx.x * POLICY_STATS + i] = v[i];
  if (!last_block(a.ticket, &flag)) return;
#pragma unroll
  for (int i = 0; i < POLICY_STATS; ++i) v[i] = 0.0;
  for (uint32_t k = threadIdx.x; k < gridDim.x; k += blockDim.x)
#pragma unroll
    for (int i = 0; i < POLICY_STATS; ++i) v[i] += __ldcg(a.partials + k * POLICY_STATS + i);
  block_sum(v, sm);
  if (threadIdx.x == 0) policy_write(a, v);
}

// The whole loss in one block, for batches where launches cost more than the
// tokens: the counts, then the tokens.
__global__ void __launch_bounds__(1024) policy_one_kernel(const PolicyArgs a) {
  __shared__ double sm[32 * POLICY_STATS];
  if (threadIdx.x == 0) *a.status = 0u;
  if (a.mask && a.reduction != KD_REDUCE_FIXED) {
    const int32_t n = a.reduction == KD_REDUCE_SEQUENCE ? a.seq.S : 1;
    for (int32_t b = threadIdx.x; b < n; b += blockDim.x) a.count[b] = 0u;
    __syncthreads();
    policy_count(a, threadIdx.x >> 5, blockDim.x >> 5, threadIdx.x & 31);
  }
  __syncthreads();
  check_layout(a.seq, a.status);
  double v[POLICY_STATS] = {};
  policy_tokens(a, threadIdx.x, blockDim.x, v);
  block_sum(v, sm);
  if (threadIdx.x == 0) policy_write(a, v);
}

// ----------------------------------------------------------------------------
// Paired preference loss.
//   s_b = sum_t m_t (logp_t - ref_t) [/ n_b],  D = s_chosen - s_rejected,
//   z = beta D - margin
//   sigmoid  -(1 - e) log s(z) - e log s(-z);  hinge  max(0, 1 - z);
//   ipo      (D - 1 / (2 beta))^2
// Three steps: sums over every sequence; one warp for each pair; the gradient,
// one value per sequence, spread over its tokens.
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

__device__ __forceinline__ void pref_sums(const PrefArgs& a, int64_t span_i, int lane) {
  const SeqLayout& q = a.seq;
  const int32_t s0 = static_cast<int32_t>(span_i * a.span);
  const int32_t s1 = static_cast<int32_t>(min(static_cast<int64_t>(s0) + a.span,
                                              static_cast<int64_t>(q.N)));
  Cursor c = cursor_at(q, s0);
  bool begun = c.b >= 0 && c.b < q.S && seq_begin(q, c.b) >= s0;
  double sum = 0.0;
  uint32_t n = 0;
  for (int32_t r = s0; r < s1 && c.b < q.S; r += 128) {
    const int32_t r1 = min(r + 128, s1), t = r + 4 * lane;
    float x[4], y[4];
    uint32_t m = 0;
    if (t < s1) {
      m = load_mask4(a.mask, t, q.N);
      load4(a.logp, t, q.N, 0.f, x);
      if (a.ref_logp) load4(a.ref_logp, t, q.N, 0.f, y);
    }
    double d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      d[j] = (m >> j) & 1u ? static_cast<double>(x[j]) - (a.ref_logp ? static_cast<double>(y[j]) : 0.0)
                           : 0.0;
    if (c.e >= r1 && c.b >= 0) {             // the whole row belongs to one sequence
      sum += (d[0] + d[1]) + (d[2] + d[3]);
      n += __popc(m);
    } else {
      int32_t pos = r;
      while (pos < r1) {
        const int32_t stop = min(c.e, r1);
        if (c.b >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (t + j >= pos && t + j < stop) {
              sum += d[j];
              n += (m >> j) & 1u;
            }
        }
        if (c.e >= r1) break;                // the row's rest is taken
        if (c.b >= 0) flush_part(begun ? a.whole + c.b : a.head + span_i, sum, n, lane);
        sum = 0.0;
        n = 0;
        pos = max(stop, pos + 1);            // a bad cu still moves on
        c = cursor_at(q, pos);
        begun = true;
        if (c.b >= q.S) break;               // behind the last sequence
      }
      if (c.b >= q.S) break;
    }
    if (c.e == r1) {                         // ends with the row
      if (c.b >= 0) flush_part(begun ? a.whole + c.b : a.head + span_i, sum, n, lane);
      sum = 0.0;
      n = 0;
      if (r1 >= s1) return;
      c = cursor_at(q, r1);
      begun = true;
    }
  }
  if (c.b >= 0 && c.b < q.S && c.e > s1)
    flush_part(begun ? a.tail + span_i : a.head + span_i, sum, n, lane);
}

// Sum and count of sequence b from its parts.  Called by a whole warp.
__device__ __forceinline__ SeqPart pref_join(const PrefArgs& a, int32_t b, int lane) {
  const int32_t t0 = seq_begin(a.seq, b), t1 = seq_begin(a.seq, b + 1);
  if (t1 <= t0) return SeqPart{0.0, 0.0};
  const int32_t i0 = t0 / a.span, i1 = (t1 - 1) / a.span;
  if (i0 == i1) return SeqPart{__ldcg(&a.whole[b].sum), __ldcg(&a.whole[b].n)};
  SeqPart p{0.0, 0.0};
  for (int32_t i = i0 + lane; i <= i1; i += 32) {
    const SeqPart* s = i == i0 ? a.tail + i : a.head + i;
    p.sum += __ldcg(&s->sum);
    p.n += __ldcg(&s->n);
  }
  return SeqPart{warp_sum(p.sum), warp_sum(p.n)};
}

// One warp for each pair: the loss of the pair (returned in every lane), the
// rewards and the gradient of each of its two sequences' tokens.
__device__ __forceinline__ double pref_pair(const PrefArgs& a, int32_t i, int lane) {
  const int32_t B = a.seq.S / 2;
  SeqPart c = pref_join(a, i, lane), r = pref_join(a, i + B, lane);
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
    loss = (1.0 - a.smoothing) * (fmax(-z, 0.0) + soft) + a.smoothing * (fmax(z, 0.0) + soft);
    if (z != z) loss = z;
    slope = a.beta * (a.smoothing - 1.0 / (1.0 + exp(z)));
  }
  if (lane == 0) {
    a.rewards[i] = static_cast<float>(a.beta * sc);
    a.rewards[i + B] = static_cast<float>(a.beta * sr);
    a.coef[i] = static_cast<float>(slope * per_c * a.inv_pairs);
    a.coef[i + B] = static_cast<float>(-slope * per_r * a.inv_pairs);
  }
  return loss;
}

// The gradient of this thread's groups of four tokens.
__device__ __forceinline__ void pref_tokens(const PrefArgs& a, int64_t thread, int64_t n_threads) {
  const SeqLayout& q = a.seq;
  const int64_t groups = (static_cast<int64_t>(q.N) + 3) / 4;
  for (int64_t g = thread; g < groups; g += n_threads) {
    const int32_t t0 = static_cast<int32_t>(4 * g);
    const uint32_t m = load_mask4(a.mask, t0, q.N);
    float out[4], k = 0.f;
    Cursor c{-1, INT_MIN};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[j] = 0.f;
      if (!((m >> j) & 1u)) continue;
      if (t0 + j >= c.e) {
        c = cursor_at(q, t0 + j);
        k = c.b >= 0 && c.b < q.S ? __ldcg(a.coef + c.b) : 0.f;
      }
      out[j] = k;
    }
    store4(a.dlogp, t0, q.N, out);
  }
}

__global__ void __launch_bounds__(OBJ_THREADS) pref_sums_kernel(const PrefArgs a) {
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.status = 0u;
    *a.ticket = 0u;
  }
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (OBJ_THREADS / 32) + (threadIdx.x >> 5);
  if (i < a.n_spans) pref_sums(a, i, threadIdx.x & 31);
}

__global__ void __launch_bounds__(OBJ_THREADS) pref_pair_kernel(const PrefArgs a) {
  __shared__ double sm[32];
  __shared__ uint32_t flag;
  griddep_launch_dependents();
  griddep_wait();                            // the sums
  check_layout(a.seq, a.status);
  const int lane = threadIdx.x & 31;
  double v[1] = {0.0};
  for (int32_t i = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < a.seq.S / 2;
       i += (gridDim.x * blockDim.x) >> 5) {
    const double l = pref_pair(a, i, lane);
    if (lane == 0) v[0] += l;
  }
  block_sum(v, sm);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = v[0];
  if (!last_block(a.ticket, &flag)) return;
  v[0] = 0.0;
  for (uint32_t k = threadIdx.x; k < gridDim.x; k += blockDim.x) v[0] += __ldcg(a.partials + k);
  block_sum(v, sm);
  if (threadIdx.x == 0) *a.loss = static_cast<float>(v[0] * a.inv_pairs);
}

__global__ void __launch_bounds__(OBJ_THREADS) pref_tokens_kernel(const PrefArgs a) {
  griddep_wait();                            // the pairs' gradients
  pref_tokens(a, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// The three steps in one block, for batches where launches cost more than the
// tokens.
__global__ void __launch_bounds__(1024) pref_one_kernel(const PrefArgs a) {
  __shared__ double sm[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (threadIdx.x == 0) *a.status = 0u;
  for (int64_t i = warp; i < a.n_spans; i += nw) pref_sums(a, i, lane);
  __syncthreads();
  check_layout(a.seq, a.status);
  double v[1] = {0.0};
  for (int32_t i = warp; i < a.seq.S / 2; i += nw) {
    const double l = pref_pair(a, i, lane);
    if (lane == 0) v[0] += l;
  }
  block_sum(v, sm);                          // its barriers also publish the gradients
  if (threadIdx.x == 0) *a.loss = static_cast<float>(v[0] * a.inv_pairs);
  if (a.dlogp) pref_tokens(a, threadIdx.x, blockDim.x);
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

// Batches of at most this many tokens (and sequences) run in one block.
constexpr int64_t ONE_BLOCK_TOKENS = 8192;

template <typename Args>
cudaError_t launch(void (*kern)(Args), int64_t blocks, int threads, cudaStream_t s,
                   const Args& a, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

int64_t at_most(int64_t x, int64_t cap) { return x < cap ? (x > 0 ? x : 1) : cap; }

}  // namespace

kd_status policy_loss(const PolicyArgs& a, cudaStream_t s, int num_sms) {
  const SeqLayout& q = a.seq;
  if (q.N <= ONE_BLOCK_TOKENS && q.S <= ONE_BLOCK_TOKENS)
    return launch(policy_one_kernel, 1, 1024, s, a, false) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  const bool counts = a.mask && a.reduction != KD_REDUCE_FIXED;
  const size_t clear = OBJ_HEADER + (counts && a.reduction == KD_REDUCE_SEQUENCE
                                         ? sizeof(uint32_t) * static_cast<size_t>(q.S) : 0);
  if (cudaMemsetAsync(a.status, 0, clear, s) != cudaSuccess) return KD_ERR_CUDA;
  if (counts) {
    const int64_t blocks = (static_cast<int64_t>(q.N) + 4095) / 4096;
    if (launch(policy_count_kernel, at_most(blocks, 4 * num_sms), OBJ_THREADS, s, a, false) !=
        cudaSuccess)
      return KD_ERR_CUDA;
  }
  const int64_t groups = (static_cast<int64_t>(q.N) + 3) / 4;
  const int64_t cap = at_most(6 * num_sms, OBJ_MAX_BLOCKS);
  if (launch(policy_main_kernel, at_most((groups + OBJ_THREADS - 1) / OBJ_THREADS, cap),
             OBJ_THREADS, s, a, counts) != cudaSuccess)
    return KD_ERR_CUDA;
  return KD_OK;
}

kd_status preference_loss(const PrefArgs& a, cudaStream_t s, int num_sms) {
  const SeqLayout& q = a.seq;
  if (q.N <= ONE_BLOCK_TOKENS && q.S <= ONE_BLOCK_TOKENS)
    return launch(pref_one_kernel, 1, 1024, s, a, false) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  constexpr int W = OBJ_THREADS / 32;
  if (launch(pref_sums_kernel, (a.n_spans + W - 1) / W, OBJ_THREADS, s, a, false) != cudaSuccess)
    return KD_ERR_CUDA;
  const int64_t pairs = q.S / 2, cap = at_most(8 * num_sms, OBJ_MAX_BLOCKS);
  if (launch(pref_pair_kernel, at_most((pairs + W - 1) / W, cap), OBJ_THREADS, s, a, true) !=
      cudaSuccess)
    return KD_ERR_CUDA;
  if (!a.dlogp) return KD_OK;
  const int64_t groups = (static_cast<int64_t>(q.N) + 3) / 4;
  if (launch(pref_tokens_kernel, at_most((groups + OBJ_THREADS - 1) / OBJ_THREADS, cap),
             OBJ_THREADS, s, a, true) != cudaSuccess)
    return KD_ERR_CUDA;
  return KD_OK;
}

}  // namespace kd
