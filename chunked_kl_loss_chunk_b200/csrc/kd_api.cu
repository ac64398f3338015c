// kd_api.cu -- the C ABI declared in include/kd.h: argument validation,
// workspace sizing, device status, and dispatch to the kernels.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "kd_internal.h"

namespace {

std::atomic<uint64_t> g_wait_limit_ns{4000000000ull};  // 4 s; set from any host thread
std::atomic<uint64_t> g_launches{0};

struct Profile {
  void* const* start = nullptr;
  void* const* end = nullptr;
  int* kinds = nullptr;
  double* flops = nullptr;
  int capacity = 0, mask = 0, n = 0;
  bool armed = false;   // set between profile_before and profile_after
} g_prof;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int num_sms_current() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

using kd::KD_MAX_K;

}  // namespace

namespace kd {

void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

uint64_t wait_limit_ns() { return g_wait_limit_ns.load(std::memory_order_relaxed); }

// While `s` is being captured into a CUDA graph the record must be external to
// become an event node of the graph (timed on every replay); outside capture
// it is a plain record.  A failed record is cleared so that it can never be
// reported as the failure of the launch it brackets.
static void record_profile_event(void* ev, cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) cs = cudaStreamCaptureStatusNone;
  const cudaError_t e =
      cs == cudaStreamCaptureStatusActive
          ? cudaEventRecordWithFlags(static_cast<cudaEvent_t>(ev), s, cudaEventRecordExternal)
          : cudaEventRecord(static_cast<cudaEvent_t>(ev), s);
  if (e != cudaSuccess) cudaGetLastError();
}

void profile_before(int kind, double flops, cudaStream_t s) {
  g_prof.armed = false;
  if (!g_prof.start || !(g_prof.mask & kind) || g_prof.n >= g_prof.capacity) return;
  record_profile_event(g_prof.start[g_prof.n], s);
  if (g_prof.kinds) g_prof.kinds[g_prof.n] = kind;
  if (g_prof.flops) g_prof.flops[g_prof.n] = flops;
  g_prof.armed = true;
}

void profile_after(cudaStream_t s) {
  if (!g_prof.armed) return;
  record_profile_event(g_prof.end[g_prof.n], s);
  ++g_prof.n;
  g_prof.armed = false;
}

kd_status validate_loss_inputs(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                               int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                               int64_t chunk, float tau) {
  if (!h || !W || !t_vals || !t_idx) return KD_ERR_INVALID_ARG;
  if (T < 1 || d < 1 || V < 1 || K < 1 || K > V || chunk < 1) return KD_ERR_INVALID_ARG;
  if (!(tau > 0.f) || !isfinite(tau)) return KD_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(t_vals, 16) || !aligned(t_idx, 16))
    return KD_ERR_INVALID_ARG;
  if (dtype != KD_DTYPE_BF16 && dtype != KD_DTYPE_F32) return KD_ERR_UNSUPPORTED;
  if (d % 8 != 0 || K > KD_MAX_K || V >= (int64_t(1) << 31) - 256 ||
      d >= (int64_t(1) << 31) || T >= (int64_t(1) << 40))
    return KD_ERR_UNSUPPORTED;
  // Rows per chunk: the backward contracts dW over two chunks' rows in one
  // 32-bit GEMM extent.
  if ((chunk < T ? chunk : T) > (int64_t(1) << 30)) return KD_ERR_UNSUPPORTED;
  return KD_OK;
}

}  // namespace kd

extern "C" {

const char* kd_status_string(int status) {
  switch (status) {
    case KD_OK: return "KD_OK";
    case KD_ERR_INVALID_ARG: return "KD_ERR_INVALID_ARG";
    case KD_ERR_UNSUPPORTED: return "KD_ERR_UNSUPPORTED";
    case KD_ERR_WORKSPACE: return "KD_ERR_WORKSPACE";
    case KD_ERR_BAD_INDEX: return "KD_ERR_BAD_INDEX";
    case KD_ERR_TIMEOUT: return "KD_ERR_TIMEOUT";
    case KD_ERR_CUDA: return "KD_ERR_CUDA";
    case KD_ERR_INTERNAL: return "KD_ERR_INTERNAL";
    default: return "KD_ERR_UNKNOWN";
  }
}

int kd_version(void) { return (1 << 16) | 1; }

size_t kd_topk_workspace_size(int64_t T, int64_t V, int K) {
  (void)T;
  (void)V;
  (void)K;
  return 1024;
}

kd_status kd_topk_build(const void* logits, int dtype, int64_t T, int64_t V, int K,
                        float* out_vals, int32_t* out_idx, void* ws, size_t ws_bytes,
                        void* stream) {
  if (!logits || !out_vals || !out_idx || !ws) return KD_ERR_INVALID_ARG;
  if (T < 1 || V < 1 || K < 1 || K > V) return KD_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(out_vals, 16) || !aligned(out_idx, 16) ||
      !aligned(ws, 1024))
    return KD_ERR_INVALID_ARG;
  if (dtype != KD_DTYPE_BF16) return KD_ERR_UNSUPPORTED;
  if (K > KD_MAX_K || V >= (int64_t(1) << 31)) return KD_ERR_UNSUPPORTED;
  if (ws_bytes < kd_topk_workspace_size(T, V, K)) return KD_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  // status word and row counter, both zero before the build
  if (cudaMemsetAsync(ws, 0, kd::WS_HEADER_BYTES, s) != cudaSuccess) return KD_ERR_CUDA;
  unsigned long long* row_counter = reinterpret_cast<unsigned long long*>(
      static_cast<char*>(ws) + kd::KD_TOPK_COUNTER_OFFSET);
  if (kd::launch_topk_bf16(logits, T, V, K, out_vals, out_idx, static_cast<uint32_t*>(ws),
                           row_counter, s, sms) != cudaSuccess)
    return KD_ERR_CUDA;
  return KD_OK;
}

size_t kd_fused_kl_workspace_size(int64_t T, int64_t d, int64_t V, int K, int64_t chunk,
                                  int dtype) {
  if (T < 1 || d < 1 || V < 1 || K < 1 || chunk < 1) return 0;
  const kd::WsLayout L = kd::ws_layout(T, d, V, K, chunk, dtype);
  return L.ok ? L.total : 0;
}

static kd_status validate_loss(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                               int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                               int64_t chunk, float tau, void* ws, size_t ws_bytes) {
  const kd_status st = kd::validate_loss_inputs(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, tau);
  if (st != KD_OK) return st;
  if (!ws || !aligned(ws, kd::KD_WS_ALIGN)) return KD_ERR_INVALID_ARG;
  const kd::WsLayout L = kd::ws_layout(T, d, V, K, chunk, dtype);
  if (!L.ok || ws_bytes < L.total) return KD_ERR_WORKSPACE;
  return KD_OK;
}

}  // extern "C"

// The forward and backward behind every fused-loss entry point; T_norm is the
// count the loss and gradients are normalised by (T, or a whole batch's
// positions for a data-parallel shard of it).
static kd_status fwd_entry(const void* h, const void* W, int dtype, int64_t T, int64_t T_norm,
                           int64_t d, int64_t V, const float* t_vals, const int32_t* t_idx,
                           int K, int64_t chunk, float temperature, uint32_t flags, float* loss,
                           float* lse, float* kl_rows, void* ws, size_t ws_bytes, void* stream) {
  kd_status st =
      validate_loss(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, ws, ws_bytes);
  if (st != KD_OK) return st;
  if ((flags & ~KD_KL_KNOWN_FLAGS) != 0u) return KD_ERR_INVALID_ARG;
  if (T_norm < T) return KD_ERR_INVALID_ARG;
  if (T_norm >= (int64_t(1) << 40)) return KD_ERR_UNSUPPORTED;
  if (!loss || !lse) return KD_ERR_INVALID_ARG;
  if (!aligned(loss, 4) || !aligned(lse, 16) || (kl_rows && !aligned(kl_rows, 16)))
    return KD_ERR_INVALID_ARG;
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  kd::RowTerms rt;
  rt.t_vals = t_vals;
  rt.t_idx = t_idx;
  rt.K = K;
  rt.flags = flags;
  return kd::fused_fwd(h, W, dtype, T, T_norm, d, V, rt, chunk, temperature, loss, lse, kl_rows, ws,
                       static_cast<cudaStream_t>(stream), sms, kd::wait_limit_ns());
}

static kd_status bwd_entry(const void* h, const void* W, int dtype, int64_t T, int64_t T_norm,
                           int64_t d, int64_t V, const float* t_vals, const int32_t* t_idx,
                           int K, int64_t chunk, float temperature, uint32_t flags,
                           const float* lse, const float* grad_loss, void* dH, float* dW,
                           int accumulate_dW, void* ws, size_t ws_bytes, void* stream) {
  kd_status st =
      validate_loss(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, ws, ws_bytes);
  if (st != KD_OK) return st;
  if ((flags & ~KD_KL_KNOWN_FLAGS) != 0u) return KD_ERR_INVALID_ARG;
  if (T_norm < T) return KD_ERR_INVALID_ARG;
  if (T_norm >= (int64_t(1) << 40)) return KD_ERR_UNSUPPORTED;
  if (!lse || !dH || !dW) return KD_ERR_INVALID_ARG;
  if (!aligned(lse, 16) || !aligned(dH, 16) || !aligned(dW, 16) ||
      (grad_loss && !aligned(grad_loss, 4)))
    return KD_ERR_INVALID_ARG;
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  kd::RowTerms rt;
  rt.t_vals = t_vals;
  rt.t_idx = t_idx;
  rt.K = K;
  rt.flags = flags;
  return kd::fused_bwd(h, W, dtype, T, T_norm, d, V, rt, chunk, temperature, lse, grad_loss, dH, dW,
                       KD_DTYPE_F32, accumulate_dW, ws, static_cast<cudaStream_t>(stream), sms,
                       kd::wait_limit_ns());
}

extern "C" {

kd_status kd_fused_kl_fwd_ex(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                             int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                             int64_t chunk, float temperature, uint32_t flags, float* loss,
                             float* lse, float* kl_rows, void* ws, size_t ws_bytes,
                             void* stream) {
  return fwd_entry(h, W, dtype, T, T, d, V, t_vals, t_idx, K, chunk, temperature, flags, loss, lse,
                   kl_rows, ws, ws_bytes, stream);
}

kd_status kd_fused_kl_fwd(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                          int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                          int64_t chunk, float temperature, float* loss, float* lse,
                          float* kl_rows, void* ws, size_t ws_bytes, void* stream) {
  return fwd_entry(h, W, dtype, T, T, d, V, t_vals, t_idx, K, chunk, temperature, 0u, loss, lse,
                   kl_rows, ws, ws_bytes, stream);
}

kd_status kd_fused_kl_fwd_shard(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                                int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                                int64_t chunk, float temperature, uint32_t flags, int64_t T_total,
                                float* loss, float* lse, float* kl_rows, void* ws,
                                size_t ws_bytes, void* stream) {
  return fwd_entry(h, W, dtype, T, T_total, d, V, t_vals, t_idx, K, chunk, temperature, flags,
                   loss, lse, kl_rows, ws, ws_bytes, stream);
}

kd_status kd_fused_kl_bwd_ex(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                             int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                             int64_t chunk, float temperature, uint32_t flags, const float* lse,
                             const float* grad_loss, void* dH, float* dW, int accumulate_dW,
                             void* ws, size_t ws_bytes, void* stream) {
  return bwd_entry(h, W, dtype, T, T, d, V, t_vals, t_idx, K, chunk, temperature, flags, lse,
                   grad_loss, dH, dW, accumulate_dW, ws, ws_bytes, stream);
}

kd_status kd_fused_kl_bwd(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                          int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                          int64_t chunk, float temperature, const float* lse,
                          const float* grad_loss, void* dH, float* dW, int accumulate_dW,
                          void* ws, size_t ws_bytes, void* stream) {
  return bwd_entry(h, W, dtype, T, T, d, V, t_vals, t_idx, K, chunk, temperature, 0u, lse,
                   grad_loss, dH, dW, accumulate_dW, ws, ws_bytes, stream);
}

kd_status kd_fused_kl_bwd_shard(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                                int64_t V, const float* t_vals, const int32_t* t_idx, int K,
                                int64_t chunk, float temperature, uint32_t flags, int64_t T_total,
                                const float* lse, const float* grad_loss, void* dH, float* dW,
                                int accumulate_dW, void* ws, size_t ws_bytes, void* stream) {
  return bwd_entry(h, W, dtype, T, T_total, d, V, t_vals, t_idx, K, chunk, temperature, flags, lse,
                   grad_loss, dH, dW, accumulate_dW, ws, ws_bytes, stream);
}

static int64_t head_fwd_chunk(int64_t chunk) {
  return chunk > kd::KD_HEAD_FWD_ROWS ? chunk : kd::KD_HEAD_FWD_ROWS;
}

static int64_t head_bwd_chunk(int64_t chunk) {
  return chunk > kd::KD_HEAD_BWD_ROWS ? chunk : kd::KD_HEAD_BWD_ROWS;
}

// Whether the backward forms dz of all T rows at once.
static bool one_group(int64_t T, int64_t chunk) {
  return (T + kd::KD_DW_GROUP - 1) / kd::KD_DW_GROUP <= head_bwd_chunk(chunk);
}

size_t kd_head_logprob_workspace_size(int64_t T, int64_t d, int64_t V, int64_t chunk, int dtype,
                                      int use) {
  if (T < 1 || d < 1 || V < 1 || chunk < 1) return 0;
  if (use == KD_HEAD_KEEP) {
    if (!one_group(T, chunk)) return 0;
    const kd::KeepLayout K = kd::keep_layout(T, d, V, head_bwd_chunk(chunk), head_fwd_chunk(chunk), dtype);
    return K.ok ? K.total : 0;
  }
  const kd::WsLayout F = kd::ws_layout(T, d, V, 1, head_fwd_chunk(chunk), dtype);
  if (!F.ok) return 0;
  if (use == KD_HEAD_FWD) return F.fwd_end;
  const kd::WsLayout L = kd::ws_layout(T, d, V, 1, head_bwd_chunk(chunk), dtype);
  if (!L.ok) return 0;
  return L.total > F.fwd_end ? L.total : F.fwd_end;
}

// Label of what a forward keeps for a backward of the same sizes, temperature and type, and
// of chunks that place it alike: FNV-1a (Fowler, Noll and Vo) over these numbers, never 0.
static uint64_t keep_label(int dtype, int64_t T, int64_t d, int64_t V, int64_t chunk, float tau) {
  uint32_t tau_bits;
  memcpy(&tau_bits, &tau, 4);
  const int64_t bwd = head_bwd_chunk(chunk), fwd = head_fwd_chunk(chunk);
  const uint64_t of[] = {static_cast<uint64_t>(dtype), static_cast<uint64_t>(T),
                         static_cast<uint64_t>(d),     static_cast<uint64_t>(V),
                         static_cast<uint64_t>(bwd < T ? bwd : T),
                         static_cast<uint64_t>(fwd < T ? fwd : T), tau_bits};
  uint64_t x = 14695981039346656037ull;
  for (uint64_t v : of)
    for (int i = 0; i < 8; ++i, v >>= 8) x = (x ^ (v & 0xFF)) * 1099511628211ull;
  return x ? x : 1;
}

// Checks shared by the two calls below.
static kd_status validate_head(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                               int64_t V, const int32_t* targets, int64_t chunk, float tau,
                               void* ws, size_t ws_bytes, bool backward, bool keep) {
  if (!targets || !aligned(targets, 4)) return KD_ERR_INVALID_ARG;
  // the head's own checks, with h in the places of the two arrays of a cache with K = 1
  const kd_status st =
      kd::validate_loss_inputs(h, W, dtype, T, d, V, static_cast<const float*>(h),
                               static_cast<const int32_t*>(h), 1, chunk, tau);
  if (st != KD_OK) return st;
  if (!ws || !aligned(ws, kd::KD_WS_ALIGN)) return KD_ERR_INVALID_ARG;
  if (keep) {
    if (!one_group(T, chunk)) return KD_ERR_UNSUPPORTED;
    const kd::KeepLayout K = kd::keep_layout(T, d, V, head_bwd_chunk(chunk), head_fwd_chunk(chunk), dtype);
    return K.ok && ws_bytes >= K.total ? KD_OK : KD_ERR_WORKSPACE;
  }
  const kd::WsLayout L =
      kd::ws_layout(T, d, V, 1, backward ? head_bwd_chunk(chunk) : head_fwd_chunk(chunk), dtype);
  if (!L.ok || ws_bytes < (backward ? L.total : L.fwd_end)) return KD_ERR_WORKSPACE;
  return KD_OK;
}

kd_status kd_head_logprob_fwd(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                              int64_t V, const int32_t* targets, int64_t chunk, float temperature,
                              int keep, float* logp, float* lse, void* ws, size_t ws_bytes,
                              void* stream) {
  const kd_status st = validate_head(h, W, dtype, T, d, V, targets, chunk, temperature, ws,
                                     ws_bytes, false, keep != 0);
  if (st != KD_OK) return st;
  if (!logp || !lse || !aligned(logp, 4) || !aligned(lse, 4)) return KD_ERR_INVALID_ARG;
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  kd::RowTerms rt;
  rt.targets = targets;
  rt.keep_chunk = keep ? head_bwd_chunk(chunk) : 0;
  rt.keep_label = keep ? keep_label(dtype, T, d, V, chunk, temperature) : 0;
  return kd::fused_fwd(h, W, dtype, T, 1, d, V, rt, head_fwd_chunk(chunk), temperature, nullptr,
                       lse, logp, ws, static_cast<cudaStream_t>(stream), sms, kd::wait_limit_ns());
}

kd_status kd_head_logprob_bwd(const void* h, const void* W, int dtype, int64_t T, int64_t d,
                              int64_t V, const int32_t* targets, int64_t chunk, float temperature,
                              const float* lse, const float* kept_logp, const float* grad_logp,
                              const float* grad_loss, void* dH, void* dW, int dW_dtype, int accumulate_dW, void* ws,
                              size_t ws_bytes, void* stream) {
  const kd_status st = validate_head(h, W, dtype, T, d, V, targets, chunk, temperature, ws,
                                     ws_bytes, true, kept_logp != nullptr);
  if (st != KD_OK) return st;
  if (!lse || !grad_logp || (!dH && !dW)) return KD_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(kept_logp, 4) || !aligned(grad_logp, 4) || !aligned(dH, 16) || !aligned(dW, 16) ||
      !aligned(grad_loss, 4))
    return KD_ERR_INVALID_ARG;
  if (dW && dW_dtype != KD_DTYPE_F32 &&
      (dW_dtype != KD_DTYPE_BF16 || dtype != KD_DTYPE_BF16 || accumulate_dW ||
       !one_group(T, chunk)))
    return KD_ERR_UNSUPPORTED;
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  kd::RowTerms rt;
  rt.targets = targets;
  rt.grad_rows = grad_logp;
  rt.kept_logp = kept_logp;
  rt.keep_chunk = kept_logp ? head_fwd_chunk(chunk) : 0;
  rt.keep_label = kept_logp ? keep_label(dtype, T, d, V, chunk, temperature) : 0;
  return kd::fused_bwd(h, W, dtype, T, 1, d, V, rt, head_bwd_chunk(chunk), temperature, lse, grad_loss, dH, dW,
                       dW ? dW_dtype : KD_DTYPE_F32, accumulate_dW, ws, static_cast<cudaStream_t>(stream), sms,
                       kd::wait_limit_ns());
}

// Layout checks shared by the objectives.
static kd_status validate_layout(const int32_t* cu, int64_t n_seqs, int64_t n_tokens,
                                 kd::SeqLayout* q) {
  if (n_seqs < 1 || n_tokens < 1) return KD_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || (!cu && n_tokens % n_seqs != 0)) return KD_ERR_INVALID_ARG;
  if (n_seqs > kd::OBJ_MAX_TOKENS || n_tokens > kd::OBJ_MAX_TOKENS) return KD_ERR_UNSUPPORTED;
  q->cu = cu;
  q->S = static_cast<int32_t>(n_seqs);
  q->N = static_cast<int32_t>(n_tokens);
  q->L = cu ? 0 : static_cast<int32_t>(n_tokens / n_seqs);
  if (q->L > 1) {
    int log = 0;                                     // ceil(log2 L), at most 31
    while ((int64_t(1) << log) < q->L) ++log;
    q->div_mul = static_cast<uint32_t>(((uint64_t(1) << (31 + log)) + q->L - 1) / q->L);
    q->div_shift = static_cast<uint32_t>(log - 1);
  }
  return KD_OK;
}

static size_t up1024(size_t x) { return (x + 1023) & ~size_t(1023); }

// Bytes for the counts of the mask, of each sequence or of each block's part.
static size_t policy_counts(int64_t n_seqs) {
  return up1024(4 * static_cast<size_t>(n_seqs > kd::OBJ_MAX_COUNTS ? n_seqs : kd::OBJ_MAX_COUNTS));
}

size_t kd_policy_loss_workspace_size(int64_t n_seqs, int64_t n_tokens) {
  if (n_seqs < 1 || n_tokens < 1 || n_seqs > kd::OBJ_MAX_TOKENS || n_tokens > kd::OBJ_MAX_TOKENS)
    return 0;
  return kd::OBJ_HEADER + policy_counts(n_seqs) +
         kd::OBJ_MAX_BLOCKS * kd::OBJ_PARTIALS * sizeof(double);
}

kd_status kd_policy_loss(const float* logp, const float* old_logp, const float* ref_logp,
                         const float* advantages, int advantages_per_token, const uint8_t* mask,
                         const int32_t* cu_seqlens, int64_t n_seqs, int64_t n_tokens,
                         double clip_low, double clip_high, double kl_coef, int reduction,
                         double denom, float* loss, float* stats, float* dlogp, void* ws,
                         size_t ws_bytes, void* stream) {
  if (!logp || !advantages || !loss || !stats || !ws) return KD_ERR_INVALID_ARG;
  if (!aligned(logp, 4) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) ||
      !aligned(advantages, 4) || !aligned(loss, 4) || !aligned(stats, 4) || !aligned(dlogp, 4) ||
      !aligned(ws, 1024))
    return KD_ERR_INVALID_ARG;
  if (!(clip_low >= 0.0 && clip_low <= 1.0) || !(clip_high >= 0.0) ||
      !isfinite(static_cast<float>(kl_coef)) ||
      (kl_coef != 0.0 && !ref_logp))
    return KD_ERR_INVALID_ARG;
  if (reduction != KD_REDUCE_TOKEN && reduction != KD_REDUCE_SEQUENCE &&
      reduction != KD_REDUCE_FIXED)
    return KD_ERR_INVALID_ARG;
  // (an infinite weight would make the zeros of tokens that do not count NaN)
  if (reduction == KD_REDUCE_FIXED &&
      !(denom > 0.0 && isfinite(denom) && isfinite(static_cast<float>(1.0 / denom))))
    return KD_ERR_INVALID_ARG;
  kd::PolicyArgs a = {};
  const kd_status st = validate_layout(cu_seqlens, n_seqs, n_tokens, &a.seq);
  if (st != KD_OK) return st;
  if (ws_bytes < kd_policy_loss_workspace_size(n_seqs, n_tokens)) return KD_ERR_WORKSPACE;
  a.logp = logp;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.adv = advantages;
  a.mask = mask;
  a.adv_per_token = advantages_per_token != 0;
  a.vec = aligned(logp, 16) && aligned(old_logp, 16) && aligned(ref_logp, 16) &&
          (!a.adv_per_token || aligned(advantages, 16)) && aligned(dlogp, 16);
  a.mask_vec = aligned(mask, 16);
  a.reduction = reduction;
  a.bound_hi = static_cast<float>(1.0 + clip_high);
  a.bound_lo = static_cast<float>(1.0 - clip_low);
  a.log_hi64 = log1p(clip_high);
  a.log_lo64 = log1p(-clip_low);
  a.log_hi = static_cast<float>(a.log_hi64);
  a.log_lo = static_cast<float>(a.log_lo64);
  a.kl_coef = static_cast<float>(kl_coef);
  a.inv_denom = reduction == KD_REDUCE_FIXED ? static_cast<float>(1.0 / denom) : 0.f;
  a.loss = loss;
  a.stats = stats;
  a.dlogp = dlogp;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.status = reinterpret_cast<uint32_t*>(w);
  a.ticket = reinterpret_cast<uint32_t*>(w + 8);
  a.count = reinterpret_cast<uint32_t*>(w + kd::OBJ_HEADER);
  a.partials = reinterpret_cast<double*>(w + kd::OBJ_HEADER + policy_counts(n_seqs));
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  return kd::policy_loss(a, static_cast<cudaStream_t>(stream), sms);
}

size_t kd_preference_loss_workspace_size(int64_t n_pairs, int64_t n_tokens) {
  if (n_pairs < 1 || n_tokens < 1 || n_pairs > kd::OBJ_MAX_TOKENS / 2 ||
      n_tokens > kd::OBJ_MAX_TOKENS)
    return 0;
  const int64_t span = kd::pref_span(n_tokens);
  const size_t spans = static_cast<size_t>((n_tokens + span - 1) / span);
  const size_t S = 2 * static_cast<size_t>(n_pairs);
  return kd::OBJ_HEADER + up1024(S * sizeof(kd::SeqPart)) + 2 * up1024(spans * sizeof(kd::SeqPart)) +
         up1024(S * sizeof(float)) + kd::OBJ_MAX_BLOCKS * sizeof(double);
}

kd_status kd_preference_loss(const float* logp, const float* ref_logp, const uint8_t* mask,
                             const int32_t* cu_seqlens, int64_t n_pairs, int64_t n_tokens,
                             int kind, double beta, double margin, double label_smoothing,
                             int length_normalize, int64_t pairs_total, float* loss,
                             float* rewards, float* dlogp, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!logp || !loss || !rewards || !ws) return KD_ERR_INVALID_ARG;
  if (!aligned(logp, 4) || !aligned(ref_logp, 4) || !aligned(loss, 4) || !aligned(rewards, 4) ||
      !aligned(dlogp, 4) || !aligned(ws, 1024))
    return KD_ERR_INVALID_ARG;
  if (kind != KD_PREF_SIGMOID && kind != KD_PREF_HINGE && kind != KD_PREF_IPO)
    return KD_ERR_INVALID_ARG;
  if (!(beta > 0.0 && isfinite(beta)) || !isfinite(margin) ||
      !(label_smoothing >= 0.0 && label_smoothing < 0.5))
    return KD_ERR_INVALID_ARG;
  // a margin has no place in the squared form, label smoothing only in the logistic one
  if ((kind == KD_PREF_IPO && margin != 0.0) || (kind != KD_PREF_SIGMOID && label_smoothing != 0.0))
    return KD_ERR_INVALID_ARG;
  if (n_pairs < 1 || pairs_total < n_pairs) return KD_ERR_INVALID_ARG;
  if (n_pairs > kd::OBJ_MAX_TOKENS / 2) return KD_ERR_UNSUPPORTED;
  kd::PrefArgs a = {};
  const kd_status st = validate_layout(cu_seqlens, 2 * n_pairs, n_tokens, &a.seq);
  if (st != KD_OK) return st;
  if (ws_bytes < kd_preference_loss_workspace_size(n_pairs, n_tokens)) return KD_ERR_WORKSPACE;
  a.logp = logp;
  a.ref_logp = ref_logp;
  a.mask = mask;
  a.kind = kind;
  a.normalize = length_normalize != 0;
  a.vec = aligned(logp, 16) && aligned(ref_logp, 16) && aligned(dlogp, 16);
  a.mask_vec = aligned(mask, 16);
  a.beta = beta;
  a.margin = margin;
  a.smoothing = label_smoothing;
  a.inv_pairs = 1.0 / static_cast<double>(pairs_total);
  a.span = static_cast<int32_t>(kd::pref_span(n_tokens));
  a.n_spans = static_cast<int32_t>((n_tokens + a.span - 1) / a.span);
  a.loss = loss;
  a.rewards = rewards;
  a.dlogp = dlogp;
  unsigned char* w = static_cast<unsigned char*>(ws);
  const size_t S = 2 * static_cast<size_t>(n_pairs), part = sizeof(kd::SeqPart);
  a.status = reinterpret_cast<uint32_t*>(w);
  w += kd::OBJ_HEADER;
  a.whole = reinterpret_cast<kd::SeqPart*>(w);
  w += up1024(S * part);
  a.head = reinterpret_cast<kd::SeqPart*>(w);
  w += up1024(static_cast<size_t>(a.n_spans) * part);
  a.tail = reinterpret_cast<kd::SeqPart*>(w);
  w += up1024(static_cast<size_t>(a.n_spans) * part);
  a.coef = reinterpret_cast<float*>(w);
  w += up1024(S * sizeof(float));
  a.partials = reinterpret_cast<double*>(w);
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  return kd::preference_loss(a, static_cast<cudaStream_t>(stream), sms);
}

size_t kd_grad_clip_workspace_size(int n_tensors) {
  if (n_tensors < 1) return 0;
  return 1024 + (static_cast<size_t>(n_tensors) / kd::GRAD_MIN_TENSORS + 1) *
                    static_cast<size_t>(kd::GRAD_MAX_BLOCKS) * sizeof(double);
}

kd_status kd_grad_sumsq(const void* const* grads, const int64_t* numels, const int* dtypes,
                        int n_tensors, double* sumsq, void* ws, size_t ws_bytes, void* stream) {
  if (!sumsq || !aligned(sumsq, 8) || !ws || !aligned(ws, 1024)) return KD_ERR_INVALID_ARG;
  const kd::GradList l{grads, nullptr, numels, dtypes, n_tensors};
  const kd_status st = kd::check_grads(l, false);
  if (st != KD_OK) return st;
  if (ws_bytes < kd_grad_clip_workspace_size(n_tensors)) return KD_ERR_WORKSPACE;
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  unsigned char* w = static_cast<unsigned char*>(ws);
  return kd::grad_sumsq(l, sumsq, reinterpret_cast<uint32_t*>(w),
                        reinterpret_cast<double*>(w + 1024), static_cast<cudaStream_t>(stream),
                        sms);
}

kd_status kd_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                       const int* dtypes, int n_tensors, double max_norm, const double* sumsq,
                       float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (!norm || !aligned(norm, 4) || !aligned(sumsq, 8) || !ws || !aligned(ws, 1024) ||
      !(max_norm >= 0.0))
    return KD_ERR_INVALID_ARG;
  const kd::GradList l{grads, outs, numels, dtypes, n_tensors};
  const kd_status st = kd::check_grads(l, true);
  if (st != KD_OK) return st;
  if (ws_bytes < kd_grad_clip_workspace_size(n_tensors)) return KD_ERR_WORKSPACE;
  const int sms = num_sms_current();
  if (sms <= 0) return KD_ERR_CUDA;
  unsigned char* w = static_cast<unsigned char*>(ws);
  return kd::grad_clip(l, max_norm, sumsq, norm, reinterpret_cast<uint32_t*>(w),
                       reinterpret_cast<double*>(w + 1024), static_cast<cudaStream_t>(stream),
                       sms);
}

kd_status kd_read_device_status(const void* ws, void* stream) {
  if (!ws) return KD_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, ws, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess) return KD_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return KD_ERR_CUDA;
  return static_cast<kd_status>(v);
}

uint64_t kd_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

kd_status kd_profile_attach(void* const* start_events, void* const* end_events, int* kinds,
                            double* flops, int capacity, int kind_mask) {
  if (!start_events || !end_events || capacity < 1) return KD_ERR_INVALID_ARG;
  g_prof.start = start_events;
  g_prof.end = end_events;
  g_prof.kinds = kinds;
  g_prof.flops = flops;
  g_prof.capacity = capacity;
  g_prof.mask = kind_mask;
  g_prof.n = 0;
  g_prof.armed = false;
  return KD_OK;
}

int kd_profile_detach(void) {
  const int n = g_prof.n;
  g_prof = Profile{};
  return n;
}

kd_status kd_set_wait_limit_ns(uint64_t limit_ns) {
  if (limit_ns < 1000) return KD_ERR_INVALID_ARG;
  g_wait_limit_ns.store(limit_ns, std::memory_order_relaxed);
  return KD_OK;
}

kd_status kd_debug_wait_probe(void* ws, size_t ws_bytes, uint64_t limit_ns, void* stream) {
  if (!ws || ws_bytes < 1024 || !aligned(ws, 1024)) return KD_ERR_INVALID_ARG;
  if (limit_ns < 1000 || limit_ns > 10000000000ull) return KD_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, 4, s) != cudaSuccess) return KD_ERR_CUDA;
  if (kd::launch_wait_probe(static_cast<uint32_t*>(ws), limit_ns, s) != cudaSuccess)
    return KD_ERR_CUDA;
  return KD_OK;
}

}  // extern "C"
