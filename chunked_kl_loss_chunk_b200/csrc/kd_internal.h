// kd_internal.h -- declarations shared by the translation units of libkd.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kd.h"

namespace kd {

// Header of every workspace, in 32-bit words: the status at 0, a counter or ticket at 2,
// the label of what a keeping forward of the head left (64 bits), whether the backward
// found the label that it needs, and the status before its own.
constexpr int WS_LABEL_WORD = 4, WS_FOUND_WORD = 6, WS_BEFORE_WORD = 7, WS_HEADER_BYTES = 32;

// Largest number of K-splits used for dH = dz W (its fp32 partials live in
// the workspace).
constexpr int KD_DH_MAX_SPLIT = 4;

// Consecutive chunks whose dz the backward keeps side by side, so that dW is
// updated once per group (its read-modify-write traffic falls by this factor).
constexpr int KD_DW_GROUP = 2;

// Largest number of cached teacher entries per position (the prep kernel
// sorts a row's entries in shared memory, and the top-K build keeps up to this
// many in its selection buffer).
constexpr int KD_MAX_K = 1024;

// Alignment of every region of a fused-loss workspace, and of its base: the
// tensor maps encoded over the dz scratch and the dH partials need at least
// 16 bytes, and the regions are placed at multiples of this.
constexpr size_t KD_WS_ALIGN = 1024;

// Byte offsets of the regions of a fused-loss workspace.
// Every size is computed with overflow checks: when a byte count does not fit
// in size_t, `ok` is false and every offset from that point on, and `total`,
// read SIZE_MAX, so no finite workspace is ever accepted for such sizes.
struct WsLayout {
  size_t p_sorted = 0, idx_sorted = 0, stats = 0, kl = 0, scratch = 0, hpart = 0, total = 0;
  size_t fwd_end = 0;    // end of the forward's partials (the forward uses nothing beyond)
  int64_t ldz = 0;       // row pitch (elements) of the dz scratch
  int64_t rows_pad = 0;  // chunk rows rounded up to 256 (rows per dH partial)
  bool ok = true;
};

WsLayout ws_layout(int64_t T, int64_t d, int64_t V, int K, int64_t chunk, int dtype);

// Workspace of a head log-probability forward that keeps its exponentials for the
// backward: ws_layout(T, d, V, 1, chunk), whose dz they lie in, then the forward's
// partials (of fwd_chunk rows; in the backward the copy of h for dW) and the reference of each block of 32 exponentials.
struct KeepLayout {
  size_t part = 0, block_max = 0, total = 0;
  int64_t ld_max = 0;
  bool ok = true;
};
KeepLayout keep_layout(int64_t T, int64_t d, int64_t V, int64_t chunk, int64_t fwd_chunk, int dtype);

// Host validation shared by every fused-loss entry point, for everything but
// the workspace and the outputs: non-null, 16-byte-aligned inputs; positive
// sizes with K <= V; a finite tau > 0 (KD_ERR_INVALID_ARG); a supported dtype,
// d % 8 == 0, K <= KD_MAX_K, V < 2^31 - 256, d < 2^31, T < 2^40 and
// min(chunk, T) <= 2^30 (KD_ERR_UNSUPPORTED).  Makes no CUDA call.
kd_status validate_loss_inputs(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                               int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                               int64_t chunk, float tau);

// What a row of the head's logits is reduced to: the KL against K cached
// teacher entries, or (targets non-null, K == 1) the log-probability of one
// target, whose backward takes the gradient of each row's log-probability.
struct RowTerms {
  const float* t_vals = nullptr;
  const int32_t* t_idx = nullptr;
  int K = 1;
  uint32_t flags = 0;
  const int32_t* targets = nullptr;
  const float* grad_rows = nullptr;
  // The forward keeps its exponentials (T <= KD_DW_GROUP of the backward's chunk, which
  // keep_chunk then is); the backward makes dz of them when kept_logp, the forward's logp,
  // is given (keep_chunk is then the forward's chunk).
  int64_t keep_chunk = 0;
  const float* kept_logp = nullptr;
  // Of what the forward keeps: written by it, looked for by the backward (0 for neither).
  uint64_t keep_label = 0;
};

// The fused loss over T positions whose loss and gradients are normalised by
// T_norm >= T: T_norm == T for a whole batch, the batch's total positions when
// these T rows are one data-parallel shard of it (then the shards' losses and
// dW contributions sum to the batch's).  dW is fp32, or for bf16 operands, with
// T <= KD_DW_GROUP chunk and accumulate == 0, dW_dtype KD_DTYPE_BF16.  Log-probabilities of targets pass
// T_norm == 1, and loss == null (no mean is taken).  row_out: KL_t or logp_t.
kd_status fused_fwd(const void* h, const void* W, int dtype, int64_t T, int64_t T_norm, int64_t d,
                    int64_t V, const RowTerms& rt, int64_t chunk, float tau, float* loss,
                    float* lse, float* row_out, void* ws, cudaStream_t s, int num_sms,
                    uint64_t limit_ns);

kd_status fused_bwd(const void* h, const void* W, int dtype, int64_t T, int64_t T_norm, int64_t d,
                    int64_t V, const RowTerms& rt, int64_t chunk, float tau, const float* lse,
                    const float* grad_loss, void* dH, void* dW, int dW_dtype, int accumulate,
                    void* ws, cudaStream_t s, int num_sms, uint64_t limit_ns);

// Rows that one launch of the head's log-probability forward takes at least: what
// it keeps of a row is 16 bytes per 256 vocabulary entries (17 MB at this many
// rows and V = 131072), so a smaller chunk, which bounds the backward's dz, would
// only cost launches.
constexpr int64_t KD_HEAD_FWD_ROWS = 2048;
// Rows that its backward takes at least, of a chunk: those of one GEMM tile, which
// fewer would leave partly empty.
constexpr int64_t KD_HEAD_BWD_ROWS = 256;

// The top-K build's row counter (zero before each build) in the workspace's header.
constexpr size_t KD_TOPK_COUNTER_OFFSET = 8;
cudaError_t launch_topk_bf16(const void* logits, int64_t T, int64_t V, int K, float* out_vals,
                             int32_t* out_idx, uint32_t* status, unsigned long long* row_counter,
                             cudaStream_t stream, int num_sms);

// ---- objectives over token log-probabilities (kd_objective.cu) ----

// Sequences of tokens that lie one after the other: sequence b at
// [cu[b], cu[b + 1]), or (cu null) rows of L tokens with N == S L.
struct SeqLayout {
  const int32_t* cu;
  int32_t S, N, L;
  uint32_t div_mul, div_shift;      // t / L == umulhi(t, div_mul) >> div_shift, for L > 1
};

// Largest number of tokens or sequences: the kernels' token offsets, with what
// they read ahead of one, stay below 2^31.
constexpr int64_t OBJ_MAX_TOKENS = (int64_t(1) << 31) - 1024;
// First region of an objective's workspace: status word at byte 0, ticket of
// the last block at byte 8.
constexpr size_t OBJ_HEADER = 1024;
constexpr int64_t OBJ_MAX_COUNTS = 1024;   // counts of the mask, one a block
constexpr int64_t OBJ_MAX_BLOCKS = 2048;   // blocks that leave partial sums
constexpr int OBJ_PARTIALS = 5;            // sums a block of the policy loss leaves

struct PolicyArgs {
  SeqLayout seq;
  const float *logp, *old_logp, *ref_logp, *adv;
  const uint8_t* mask;
  int adv_per_token, reduction;
  int vec, mask_vec;                // float arrays and mask 16-byte aligned
  float bound_hi, bound_lo;         // 1 + clip_high, 1 - clip_low
  float log_hi, log_lo;             // their logarithms, rounded, and exact:
  double log_hi64, log_lo64;
  float kl_coef, inv_denom;
  float *loss, *stats, *dlogp;
  uint32_t *status, *ticket;
  uint32_t* count;                  // unmasked tokens of each sequence, or of each block's part
  int32_t n_counts;                 // of the second kind
  double* partials;
};

kd_status policy_loss(const PolicyArgs& a, cudaStream_t s, int num_sms);

// What a span of tokens holds of a sequence: the sum and the number of its
// unmasked tokens.
struct SeqPart {
  double sum, n;
};

struct PrefArgs {
  SeqLayout seq;                    // S == 2 pairs: the chosen, then the rejected
  const float *logp, *ref_logp;
  const uint8_t* mask;
  int kind, normalize;
  int vec, mask_vec;                // float arrays and mask 16-byte aligned
  double beta, margin, smoothing, inv_pairs;
  int32_t span;                     // tokens a warp sums, a multiple of 128
  int32_t n_spans;
  int32_t pairs_per_warp;
  float *loss, *rewards, *dlogp;
  uint32_t* status;
  SeqPart *whole, *head, *tail;     // [S], [n_spans], [n_spans]
  float* coef;                      // [S] gradient of each of a sequence's tokens
  double* partials;
};

kd_status preference_loss(PrefArgs a, cudaStream_t s, int num_sms);

// Tokens a warp sums: one span for each of the warps that are resident at once
// (32 an SM), in whole rows of 128.
constexpr int64_t PREF_WARPS = 148 * 32;
inline int64_t pref_span(int64_t n_tokens) {
  const int64_t rows = (n_tokens + 127) / 128;
  return 128 * ((rows + PREF_WARPS - 1) / PREF_WARPS);
}

// ---- gradient norm and clipping (kd_gradnorm.cu) ----

// Host arrays of n tensors; outs may be null where nothing is written.
struct GradList {
  const void* const* grads;
  void* const* outs;
  const int64_t* numels;
  const int* dtypes;
  int n;
};
constexpr int64_t GRAD_MAX_BLOCKS = 1024;      // sums that one launch leaves
constexpr int GRAD_MIN_TENSORS = 1000;         // tensors a launch takes at least, but for the last

kd_status check_grads(const GradList& l, bool writes);   // makes no CUDA call
kd_status grad_sumsq(const GradList& l, double* sumsq, uint32_t* status, double* partials,
                     cudaStream_t s, int num_sms);
kd_status grad_clip(const GradList& l, double max_norm, const double* sumsq, float* norm,
                    uint32_t* status, double* partials, cudaStream_t s, int num_sms);

cudaError_t launch_wait_probe(uint32_t* status, uint64_t limit_ns, cudaStream_t s);

// Current time limit of device-side waits (kd_set_wait_limit_ns).
uint64_t wait_limit_ns();

// Launch accounting and optional per-GEMM event recording.
void count_launch();
void profile_before(int kind, double flops, cudaStream_t s);
void profile_after(cudaStream_t s);

}  // namespace kd
