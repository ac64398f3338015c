"""Thin Python binding of libkd (the C ABI in include/kd.h).

Argument marshalling only: every step of the top-K build and of the fused
chunked KL loss runs in the library's CUDA kernels.  PyTorch supplies device
memory and the current stream.  There is no CPU fallback: if libkd.so is
missing or fails to load, every call raises.

Low-level functions carry the C names (``kd_topk_build``, ``kd_fused_kl_fwd``,
``kd_fused_kl_bwd`` ...) and take raw integers (device pointers, sizes, stream
handle).  ``topk_build``, ``fused_kl_fwd``, ``fused_kl_bwd`` and
``FusedTopKKLLoss`` wrap them for torch tensors, and so do ``head_logprobs``,
``head_logprobs_bwd`` and ``HeadLogprobs`` for the log-probabilities of given
tokens, and ``policy_loss``, ``PolicyLoss``, ``preference_loss`` and
``PreferenceLoss`` for the objectives over them, ``grad_sumsq`` and
``clip_grad_norm`` for the gradients of the whole step.
"""

from __future__ import annotations

import array
import contextlib
import ctypes
import operator
import os
import re
import warnings

import torch
from torch.autograd.function import once_differentiable

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libkd.so")
DEBUG_LIB_PATH = os.path.join(_PKG_DIR, "libkd_debug.so")   # built with -DKD_DEBUG=1
HEADER_PATH = os.path.join(os.path.dirname(_PKG_DIR), "include", "kd.h")

KD_OK, KD_ERR_INVALID_ARG, KD_ERR_UNSUPPORTED, KD_ERR_WORKSPACE = 0, 1, 2, 3
KD_ERR_BAD_INDEX, KD_ERR_TIMEOUT, KD_ERR_CUDA, KD_ERR_INTERNAL = 4, 5, 6, 7
KD_DTYPE_F32, KD_DTYPE_BF16 = 0, 1
KD_KL_LOGPROB_CACHE, KD_KL_TAU_SQUARED = 0x1, 0x2
KD_TARGET_IGNORE = -100
KD_HEAD_FWD, KD_HEAD_BOTH, KD_HEAD_KEEP = 0, 1, 2
KD_REDUCE_TOKEN, KD_REDUCE_SEQUENCE, KD_REDUCE_FIXED = 0, 1, 2
KD_PREF_SIGMOID, KD_PREF_HINGE, KD_PREF_IPO = 0, 1, 2
REDUCTIONS = {"token": KD_REDUCE_TOKEN, "sequence": KD_REDUCE_SEQUENCE, "fixed": KD_REDUCE_FIXED}
PREFERENCE_KINDS = {"sigmoid": KD_PREF_SIGMOID, "hinge": KD_PREF_HINGE, "ipo": KD_PREF_IPO}
ADVANTAGES_PER = ("sequence", "token")
CACHE_KINDS = ("logits", "logprobs")

_c_i64, _c_int, _c_sz, _c_vp, _c_u64 = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_uint64
_c_u32, _c_f64 = ctypes.c_uint32, ctypes.c_double

_SIGNATURES = {
    "kd_status_string": (ctypes.c_char_p, [_c_int]),
    "kd_version": (_c_int, []),
    "kd_topk_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_int]),
    "kd_topk_build": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "kd_fused_kl_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_int, _c_i64, _c_int]),
    "kd_fused_kl_fwd": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_int,
                                 _c_i64, ctypes.c_float, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "kd_fused_kl_bwd": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_int,
                                 _c_i64, ctypes.c_float, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp,
                                 _c_sz, _c_vp]),
    "kd_fused_kl_fwd_ex": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_int,
                                    _c_i64, ctypes.c_float, _c_u32, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz,
                                    _c_vp]),
    "kd_fused_kl_bwd_ex": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_int,
                                    _c_i64, ctypes.c_float, _c_u32, _c_vp, _c_vp, _c_vp, _c_vp, _c_int,
                                    _c_vp, _c_sz, _c_vp]),
    "kd_fused_kl_fwd_shard": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp,
                                       _c_int, _c_i64, ctypes.c_float, _c_u32, _c_i64, _c_vp, _c_vp,
                                       _c_vp, _c_vp, _c_sz, _c_vp]),
    "kd_fused_kl_bwd_shard": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp,
                                       _c_int, _c_i64, ctypes.c_float, _c_u32, _c_i64, _c_vp, _c_vp,
                                       _c_vp, _c_vp, _c_int, _c_vp, _c_sz, _c_vp]),
    "kd_head_logprob_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_int]),
    "kd_head_logprob_fwd": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64,
                                     ctypes.c_float, _c_int, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "kd_head_logprob_bwd": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64,
                                     ctypes.c_float, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int,
                                     _c_vp, _c_sz, _c_vp]),
    "kd_policy_loss_workspace_size": (_c_sz, [_c_i64, _c_i64]),
    "kd_policy_loss": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_i64, _c_i64, _c_f64,
                                _c_f64, _c_f64, _c_int, _c_f64, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz,
                                _c_vp]),
    "kd_preference_loss_workspace_size": (_c_sz, [_c_i64, _c_i64]),
    "kd_preference_loss": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_f64, _c_f64,
                                    _c_f64, _c_int, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "kd_grad_clip_workspace_size": (_c_sz, [_c_int]),
    "kd_grad_sumsq": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_sz, _c_vp]),
    "kd_grad_clip": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_f64, _c_vp, _c_vp, _c_vp, _c_sz,
                              _c_vp]),
    "kd_read_device_status": (_c_int, [_c_vp, _c_vp]),
    "kd_set_wait_limit_ns": (_c_int, [_c_u64]),
    "kd_debug_wait_probe": (_c_int, [_c_vp, _c_sz, _c_u64, _c_vp]),
    "kd_launch_count": (_c_u64, []),
    "kd_fused_kl_fwd_noalloc": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp,
                                         _c_int, _c_i64, ctypes.c_float, _c_vp, _c_vp, _c_vp, _c_vp]),
    "kd_profile_attach": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int]),
    "kd_profile_detach": (_c_int, []),
}

KD_GEMM_FWD_LSE, KD_GEMM_BWD_DZ, KD_GEMM_DH, KD_GEMM_DW = 1, 2, 4, 8
GEMM_KIND_NAMES = {1: "fwd_lse", 2: "bwd_dz", 4: "dH", 8: "dW", 12: "dH+dW"}

_lib = None
_native = None
# the entry points that _kd_native calls, in the order of its bind()
_NATIVE_CALLS = ("kd_head_logprob_workspace_size", "kd_head_logprob_fwd", "kd_head_logprob_bwd",
                 "kd_policy_loss_workspace_size", "kd_policy_loss",
                 "kd_preference_loss_workspace_size", "kd_preference_loss",
                 "kd_grad_clip_workspace_size", "kd_grad_clip")


def header_symbols():
    """Names of the functions declared in include/kd.h."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kd_[a-z0-9_]+)\s*\(", text)))


def load():
    """Load libkd.so (raises if it is missing: there is no fallback), and
    _kd_native.so, the short way to the post-training calls.  Where that one is
    not to be had (only the library was built, or for another torch), a warning
    says so once and those calls are made through ctypes: the same kernels, and
    some 10 us more of host time a call."""
    global _lib, _native
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libkd.so not built ({LIB_PATH}); run chunked_kl_loss_chunk_b200.build")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    try:
        from chunked_kl_loss_chunk_b200 import _kd_native
    except ImportError as e:
        warnings.warn(f"_kd_native.so not built or not loadable ({e}): post-training calls go through ctypes; "
                      "run chunked_kl_loss_chunk_b200.build", RuntimeWarning, stacklevel=2)
        _native = None
    else:
        _kd_native.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _NATIVE_CALLS))
        _native = _kd_native
    _lib = lib
    return lib


def use_library(path: str):
    """Route every later call to the library at `path` (e.g. DEBUG_LIB_PATH,
    whose kernels also check internal invariants); returns the previous path."""
    global _lib, LIB_PATH
    prev = LIB_PATH
    LIB_PATH = path
    _lib = None
    load()
    return prev


class KDError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def status_string(status: int) -> str:
    return load().kd_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != KD_OK:
        raise KDError(status, where)


# ---------------------------------------------------------------- raw C names

def kd_topk_workspace_size(T, V, K):
    return load().kd_topk_workspace_size(T, V, K)


def kd_topk_build(logits, dtype, T, V, K, out_vals, out_idx, ws, ws_bytes, stream):
    return load().kd_topk_build(logits, dtype, T, V, K, out_vals, out_idx, ws, ws_bytes, stream)


def kd_fused_kl_workspace_size(T, d, V, K, chunk, dtype):
    return load().kd_fused_kl_workspace_size(T, d, V, K, chunk, dtype)


def kd_fused_kl_fwd(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, loss, lse, kl_rows,
                    ws, ws_bytes, stream):
    return load().kd_fused_kl_fwd(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, loss,
                                  lse, kl_rows, ws, ws_bytes, stream)


def kd_fused_kl_bwd(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, lse, grad_loss, dH,
                    dW, accumulate_dW, ws, ws_bytes, stream):
    return load().kd_fused_kl_bwd(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, lse,
                                  grad_loss, dH, dW, accumulate_dW, ws, ws_bytes, stream)


def kd_fused_kl_fwd_ex(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, flags, loss, lse,
                       kl_rows, ws, ws_bytes, stream):
    return load().kd_fused_kl_fwd_ex(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature,
                                     flags, loss, lse, kl_rows, ws, ws_bytes, stream)


def kd_fused_kl_bwd_ex(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, flags, lse,
                       grad_loss, dH, dW, accumulate_dW, ws, ws_bytes, stream):
    return load().kd_fused_kl_bwd_ex(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature,
                                     flags, lse, grad_loss, dH, dW, accumulate_dW, ws, ws_bytes,
                                     stream)


def kd_fused_kl_fwd_shard(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, flags,
                          T_total, loss, lse, kl_rows, ws, ws_bytes, stream):
    return load().kd_fused_kl_fwd_shard(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature,
                                        flags, T_total, loss, lse, kl_rows, ws, ws_bytes, stream)


def kd_fused_kl_bwd_shard(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, flags,
                          T_total, lse, grad_loss, dH, dW, accumulate_dW, ws, ws_bytes, stream):
    return load().kd_fused_kl_bwd_shard(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature,
                                        flags, T_total, lse, grad_loss, dH, dW, accumulate_dW, ws,
                                        ws_bytes, stream)


def kd_fused_kl_fwd_noalloc(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature, loss, lse,
                            kl_rows, stream):
    """Forward for callers that cannot provide a workspace (scratch is a fixed
    array inside the library; see include/kd.h for its limit and caveats)."""
    return load().kd_fused_kl_fwd_noalloc(h, W, dtype, T, d, V, t_vals, t_idx, K, chunk, temperature,
                                          loss, lse, kl_rows, stream)


def kd_head_logprob_workspace_size(T, d, V, chunk, dtype, use):
    return load().kd_head_logprob_workspace_size(T, d, V, chunk, dtype, use)


def kd_head_logprob_fwd(h, W, dtype, T, d, V, targets, chunk, temperature, keep, logp, lse, ws,
                        ws_bytes, stream):
    return load().kd_head_logprob_fwd(h, W, dtype, T, d, V, targets, chunk, temperature, keep, logp,
                                      lse, ws, ws_bytes, stream)


def kd_head_logprob_bwd(h, W, dtype, T, d, V, targets, chunk, temperature, lse, kept_logp, grad_logp,
                        grad_loss, dH, dW, dW_dtype, accumulate_dW, ws, ws_bytes, stream):
    return load().kd_head_logprob_bwd(h, W, dtype, T, d, V, targets, chunk, temperature, lse,
                                      kept_logp, grad_logp, grad_loss, dH, dW, dW_dtype,
                                      accumulate_dW, ws, ws_bytes, stream)


def kd_policy_loss_workspace_size(n_seqs, n_tokens):
    return load().kd_policy_loss_workspace_size(n_seqs, n_tokens)


def kd_policy_loss(logp, old_logp, ref_logp, advantages, advantages_per_token, mask, cu_seqlens,
                   n_seqs, n_tokens, clip_low, clip_high, kl_coef, reduction, denom, loss, stats,
                   dlogp, ws, ws_bytes, stream):
    return load().kd_policy_loss(logp, old_logp, ref_logp, advantages, advantages_per_token, mask,
                                 cu_seqlens, n_seqs, n_tokens, clip_low, clip_high, kl_coef,
                                 reduction, denom, loss, stats, dlogp, ws, ws_bytes, stream)


def kd_preference_loss_workspace_size(n_pairs, n_tokens):
    return load().kd_preference_loss_workspace_size(n_pairs, n_tokens)


def kd_preference_loss(logp, ref_logp, mask, cu_seqlens, n_pairs, n_tokens, kind, beta, margin,
                       label_smoothing, length_normalize, pairs_total, loss, rewards, dlogp, ws,
                       ws_bytes, stream):
    return load().kd_preference_loss(logp, ref_logp, mask, cu_seqlens, n_pairs, n_tokens, kind, beta,
                                     margin, label_smoothing, length_normalize, pairs_total, loss,
                                     rewards, dlogp, ws, ws_bytes, stream)


def kd_grad_clip_workspace_size(n_tensors):
    return load().kd_grad_clip_workspace_size(n_tensors)


def kd_grad_sumsq(grads, numels, dtypes, n_tensors, sumsq, ws, ws_bytes, stream):
    return load().kd_grad_sumsq(grads, numels, dtypes, n_tensors, sumsq, ws, ws_bytes, stream)


def kd_grad_clip(grads, outs, numels, dtypes, n_tensors, max_norm, sumsq, norm, ws, ws_bytes, stream):
    return load().kd_grad_clip(grads, outs, numels, dtypes, n_tensors, max_norm, sumsq, norm, ws,
                               ws_bytes, stream)


def kd_read_device_status(ws, stream):
    return load().kd_read_device_status(ws, stream)


def kd_set_wait_limit_ns(limit_ns):
    return load().kd_set_wait_limit_ns(limit_ns)


def kd_debug_wait_probe(ws, ws_bytes, limit_ns, stream):
    return load().kd_debug_wait_probe(ws, ws_bytes, limit_ns, stream)


def kd_launch_count():
    return load().kd_launch_count()


def kd_profile_attach(start_events, end_events, kinds, flops, capacity, kind_mask):
    return load().kd_profile_attach(start_events, end_events, kinds, flops, capacity, kind_mask)


def kd_profile_detach():
    return load().kd_profile_detach()


class GemmProfiler:
    """Records CUDA events around every tensor-core GEMM launch (per kind)
    while active; ``results()`` gives (kind, flops, ms) per launch."""

    def __init__(self, capacity: int = 4096, kind_mask: int = 15):
        self.capacity = capacity
        self.kind_mask = kind_mask
        self.start = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        self.end = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        for e in self.start + self.end:      # materialise the event handles
            e.record()
        torch.cuda.synchronize()
        self._s = (ctypes.c_void_p * capacity)(*[e.cuda_event for e in self.start])
        self._e = (ctypes.c_void_p * capacity)(*[e.cuda_event for e in self.end])
        self._k = (ctypes.c_int * capacity)()
        self._f = (ctypes.c_double * capacity)()
        self.n = 0

    def __enter__(self):
        _check(kd_profile_attach(self._s, self._e, self._k, self._f, self.capacity, self.kind_mask),
               "kd_profile_attach")
        return self

    def __exit__(self, *exc):
        self.n = kd_profile_detach()
        return False

    def results(self):
        torch.cuda.synchronize()
        return [(int(self._k[i]), float(self._f[i]), self.start[i].elapsed_time(self.end[i]))
                for i in range(self.n)]


# ---------------------------------------------------------------- torch helpers

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KD_DTYPE_BF16
    if t.dtype == torch.float32:
        return KD_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """Caller-owned workspace: a 1024-byte-aligned uint8 view of ``nbytes``."""
    n = max(int(nbytes), 1024)
    buf = torch.empty(n + 1024, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 1024
    ws = buf[off:off + n]
    assert ws.data_ptr() % 1024 == 0
    return ws


def read_device_status(ws: torch.Tensor, stream=None) -> int:
    return kd_read_device_status(ws.data_ptr(), _stream(stream))


def topk_build(logits: torch.Tensor, K: int, ws: torch.Tensor | None = None, stream=None):
    """Top-K cache of bf16 teacher logits [T, V] -> (vals f32 [T,K], idx i32 [T,K])."""
    assert logits.is_cuda and logits.is_contiguous() and logits.dim() == 2
    T, V = logits.shape
    vals = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    idx = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    need = kd_topk_workspace_size(T, V, K)
    if ws is None:
        ws = alloc_workspace(need, logits.device)
    _check(kd_topk_build(logits.data_ptr(), _dtype_code(logits), T, V, K, vals.data_ptr(),
                         idx.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
           "kd_topk_build")
    return vals, idx


def workspace_for(h: torch.Tensor, W: torch.Tensor, K: int, chunk: int) -> torch.Tensor:
    T, d = h.shape
    V = W.shape[0]
    return alloc_workspace(kd_fused_kl_workspace_size(T, d, V, K, chunk, _dtype_code(h)), h.device)


def kl_flags(cache: str = "logits", tau_squared: bool = False) -> int:
    """The C ABI's flag bits for a cache kind ("logits": renormalised top-K
    logits; "logprobs": full-vocabulary teacher log-probabilities, S <= 1) and
    the optional tau^2 factor."""
    if cache not in CACHE_KINDS:
        raise ValueError(f"cache must be one of {CACHE_KINDS}")
    return (KD_KL_LOGPROB_CACHE if cache == "logprobs" else 0) | (KD_KL_TAU_SQUARED if tau_squared else 0)


def fused_kl_fwd(h, W, t_vals, t_idx, chunk: int, temperature: float = 1.0, ws=None,
                 kl_rows: bool = False, stream=None, cache: str = "logits",
                 tau_squared: bool = False, T_total: int | None = None):
    """Returns (loss [] f32, lse [T] f32, kl [T] f32 or None, ws).  With
    ``T_total`` the rows are one data-parallel shard of a batch of T_total
    positions (kd_fused_kl_fwd_shard): the loss is this shard's part of the
    batch's mean."""
    for t in (h, W, t_vals, t_idx):
        assert t.is_cuda and t.is_contiguous()
    T, d = h.shape
    V = W.shape[0]
    K = t_vals.shape[1]
    flags = kl_flags(cache, tau_squared)
    if ws is None:
        ws = workspace_for(h, W, K, chunk)
    loss = torch.empty((), dtype=torch.float32, device=h.device)
    lse = torch.empty((T,), dtype=torch.float32, device=h.device)
    kl = torch.empty((T,), dtype=torch.float32, device=h.device) if kl_rows else None
    if T_total is None:
        _check(kd_fused_kl_fwd_ex(h.data_ptr(), W.data_ptr(), _dtype_code(h), T, d, V,
                                  t_vals.data_ptr(), t_idx.data_ptr(), K, chunk, float(temperature),
                                  flags, loss.data_ptr(), lse.data_ptr(), _ptr(kl), ws.data_ptr(),
                                  ws.numel(), _stream(stream)),
               "kd_fused_kl_fwd_ex")
    else:
        _check(kd_fused_kl_fwd_shard(h.data_ptr(), W.data_ptr(), _dtype_code(h), T, d, V,
                                     t_vals.data_ptr(), t_idx.data_ptr(), K, chunk,
                                     float(temperature), flags, int(T_total), loss.data_ptr(),
                                     lse.data_ptr(), _ptr(kl), ws.data_ptr(), ws.numel(),
                                     _stream(stream)),
               "kd_fused_kl_fwd_shard")
    return loss, lse, kl, ws


def fused_kl_bwd(h, W, t_vals, t_idx, lse, chunk: int, temperature: float = 1.0, grad_loss=None,
                 ws=None, dH=None, dW=None, accumulate_dW: bool = False, stream=None,
                 cache: str = "logits", tau_squared: bool = False, T_total: int | None = None):
    """Returns (dH [T,d] dtype of h, dW [V,d] f32, ws).  With ``T_total`` the
    rows are one data-parallel shard of a batch of T_total positions
    (kd_fused_kl_bwd_shard): dH is the batch gradient's rows of this shard and
    dW this shard's term of the batch's dW."""
    T, d = h.shape
    V = W.shape[0]
    K = t_vals.shape[1]
    flags = kl_flags(cache, tau_squared)
    if ws is None:
        ws = workspace_for(h, W, K, chunk)
    if dH is None:
        dH = torch.empty_like(h)
    if dW is None:
        dW = torch.empty((V, d), dtype=torch.float32, device=h.device)
    if T_total is None:
        _check(kd_fused_kl_bwd_ex(h.data_ptr(), W.data_ptr(), _dtype_code(h), T, d, V,
                                  t_vals.data_ptr(), t_idx.data_ptr(), K, chunk, float(temperature),
                                  flags, lse.data_ptr(), _ptr(grad_loss), dH.data_ptr(),
                                  dW.data_ptr(), int(accumulate_dW), ws.data_ptr(), ws.numel(),
                                  _stream(stream)),
               "kd_fused_kl_bwd_ex")
    else:
        _check(kd_fused_kl_bwd_shard(h.data_ptr(), W.data_ptr(), _dtype_code(h), T, d, V,
                                     t_vals.data_ptr(), t_idx.data_ptr(), K, chunk,
                                     float(temperature), flags, int(T_total), lse.data_ptr(),
                                     _ptr(grad_loss), dH.data_ptr(), dW.data_ptr(),
                                     int(accumulate_dW), ws.data_ptr(), ws.numel(),
                                     _stream(stream)),
               "kd_fused_kl_bwd_shard")
    return dH, dW, ws


class FusedTopKKLLoss(torch.autograd.Function):
    """Drop-in loss: forward = kd_fused_kl_fwd_ex, backward = kd_fused_kl_bwd_ex.

    ``loss = FusedTopKKLLoss.apply(h, W, t_vals, t_idx, chunk, temperature)``,
    optionally followed by ``cache`` ("logits" or "logprobs") and
    ``tau_squared``; gradients flow to h and W (W's gradient is returned in
    W's dtype).
    """

    @staticmethod
    def forward(ctx, h, W, t_vals, t_idx, chunk, temperature, cache="logits", tau_squared=False):
        loss, lse, _, ws = fused_kl_fwd(h, W, t_vals, t_idx, chunk, temperature, cache=cache,
                                        tau_squared=tau_squared)
        ctx.save_for_backward(h, W, t_vals, t_idx, lse)
        ctx.chunk, ctx.temperature, ctx.ws = chunk, temperature, ws
        ctx.cache, ctx.tau_squared = cache, tau_squared
        return loss

    @staticmethod
    def backward(ctx, g):
        h, W, t_vals, t_idx, lse = ctx.saved_tensors
        g = g.to(torch.float32).contiguous()
        dH, dW, _ = fused_kl_bwd(h, W, t_vals, t_idx, lse, ctx.chunk, ctx.temperature,
                                 grad_loss=g, ws=ctx.ws, cache=ctx.cache,
                                 tau_squared=ctx.tau_squared)
        return dH, dW.to(W.dtype), None, None, None, None, None, None


# ------------------------------------------------- log-probabilities of given tokens

def _require(name: str, t, dtype, shape, device):
    """Checks one tensor argument: a dense CUDA tensor of this type and shape on
    this device.  (The usual case first: these checks are a good part of what a
    call on a small batch costs.)"""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a torch tensor is needed")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} is needed, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} is needed, not {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, not on the CUDA device {device} of the call")
    raise ValueError(f"{name}: must be contiguous")


_HERE = contextlib.nullcontext()


def _use_stream(device, stream):
    """Context in which a call's outputs and workspace are allocated and its
    kernels launched: the given stream, or the device's current one."""
    if stream is None:
        index = device.index
        return _HERE if torch.cuda.current_device() == index else torch.cuda.device(index)
    if stream.device != device:
        raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _used_on(stream, tensors):
    """Tells the allocator that a given stream reads or writes these tensors, so
    that their memory is not handed out again before that stream is done."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _current_stream(device) -> int:
    # the raw handle: building a torch.cuda.Stream for it costs as much as the launch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(ws, nbytes: int, like):
    """(what to keep alive, address, bytes) of a call's workspace: the given one,
    or one allocated on the device of the fp32 or bf16 tensor `like`."""
    if ws is not None:
        _require("ws", ws, torch.uint8, (ws.numel(),), like.device)
        return ws, ws.data_ptr(), ws.numel()
    n = max(nbytes, 1024)
    buf = like.new_empty((n + 1024) // 2)
    return buf, (buf.data_ptr() + 1023) & ~1023, n


def _native_result(out, where: str):
    """Outputs of a call made by _kd_native, or the error that it returned."""
    if out.__class__ is int:
        raise KDError(out, where)
    return out


def _head_sizes(h, W, targets):
    if not (isinstance(h, torch.Tensor) and isinstance(W, torch.Tensor)) or h.dim() != 2 or W.dim() != 2:
        raise ValueError("h [T, d] and W [V, d] are needed")
    T, d = h.shape
    V = W.shape[0]
    code = _dtype_code(h)
    _require("h", h, h.dtype, (T, d), h.device)
    _require("W", W, h.dtype, (V, d), h.device)
    _require("targets", targets, torch.int32, (T,), h.device)
    return T, d, V, code


def _one_group(T: int, chunk: int) -> bool:
    """Whether the backward forms dz of all T positions at once: two chunks of them,
    each of at least a GEMM tile's 256 rows."""
    return T <= 2 * max(chunk, 256)


def head_logprobs(h, W, targets, chunk: int, temperature: float = 1.0, ws=None, stream=None,
                  backward: bool = False, keep: bool = False):
    """Log-probabilities of one token per position through the output head, the
    [T, V] logits never materialised: (logp f32 [T], lse f32 [T], ws).

    ``targets`` int32 [T]; KD_TARGET_IGNORE (-100) marks positions without a
    token (logp 0, no gradient).  Any other target outside [0, V) gives a logp of
    NaN and no gradient, and KD_ERR_BAD_INDEX in ``ws``.  ``backward=True`` sizes the workspace for
    ``head_logprobs_bwd`` as well, which takes ``lse`` and may take ``ws``.
    ``keep=True`` (T <= 2 chunks, of at least 256 positions each) leaves in ``ws`` what one backward needs of the
    logits, which then does not project again: hand it ``ws`` and
    ``kept_logp=logp``, and let nothing else use ``ws`` in between."""
    use = KD_HEAD_KEEP if keep else (KD_HEAD_BOTH if backward else KD_HEAD_FWD)
    load()
    if stream is None and _native is not None:
        out = _native.head_logprobs(h, W, targets, chunk, temperature, use, ws)
        if out is not None:
            return _native_result(out, "kd_head_logprob_fwd")
    T, d, V, code = _head_sizes(h, W, targets)
    with _use_stream(h.device, stream):
        if ws is None:
            ws = alloc_workspace(kd_head_logprob_workspace_size(T, d, V, chunk, code, use), h.device)
        else:
            _require("ws", ws, torch.uint8, (ws.numel(),), h.device)
        logp = torch.empty((T,), dtype=torch.float32, device=h.device)
        lse = torch.empty_like(logp)
        _check(kd_head_logprob_fwd(h.data_ptr(), W.data_ptr(), code, T, d, V, targets.data_ptr(),
                                   chunk, float(temperature), bool(keep), logp.data_ptr(),
                                   lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                   _current_stream(h.device)),
               "kd_head_logprob_fwd")
    _used_on(stream, (h, W, targets, ws))
    return logp, lse, ws


def head_logprobs_bwd(h, W, targets, lse, grad_logp, chunk: int, temperature: float = 1.0,
                      grad_loss=None, ws=None, dH=None, dW=None, accumulate_dW: bool = False,
                      stream=None, need=(True, True), dW_dtype=torch.float32, kept_logp=None):
    """Gradients of sum_t grad_logp[t] * logp[t] (times the device scalar
    ``grad_loss``): (dH [T, d] dtype of h, dW [V, d] f32, ws).  The logits are
    recomputed chunk by chunk; ``accumulate_dW=True`` adds into a given dW;
    ``dW_dtype=torch.bfloat16`` gives a bf16 dW where T <= 2 chunks (of at least
    256 positions each).
    ``need=(dH, dW)`` leaves out a gradient that is not wanted (None in its
    place).  ``kept_logp`` and ``ws`` of a forward with ``keep=True``: its
    exponentials take the place of recomputed logits, and are used up.  A ``ws`` that
    does not hold them (any more) gives NaN, and KD_ERR_WORKSPACE in it."""
    load()
    if stream is None and _native is not None and dH is None and dW is None and not accumulate_dW and any(need) and \
            (dW_dtype is torch.float32 or dW_dtype is torch.bfloat16):
        out = _native.head_logprobs_bwd(h, W, targets, lse, kept_logp, grad_logp, grad_loss, chunk, temperature,
                                        need[0], need[1], dW_dtype is torch.bfloat16, ws)
        if out is not None:
            return _native_result(out, "kd_head_logprob_bwd")
    T, d, V, code = _head_sizes(h, W, targets)
    _require("lse", lse, torch.float32, (T,), h.device)
    _require("grad_logp", grad_logp, torch.float32, (T,), h.device)
    if grad_loss is not None:
        _require("grad_loss", grad_loss, torch.float32, grad_loss.shape, h.device)
        if grad_loss.numel() != 1:
            raise ValueError("grad_loss: one value is needed")
    if kept_logp is not None:
        _require("kept_logp", kept_logp, torch.float32, (T,), h.device)
        if ws is None:
            raise ValueError("kept_logp: needs the workspace of its forward")
    if accumulate_dW and dW is None:
        raise ValueError("accumulate_dW: needs the dW to add to")
    if dW_dtype is not torch.float32 and dW_dtype is not torch.bfloat16:
        raise TypeError(f"dW_dtype: float32 or bfloat16 is needed, not {dW_dtype}")
    if not any(need):
        raise ValueError("need: at least one gradient")
    with _use_stream(h.device, stream):
        if ws is None:
            ws = alloc_workspace(kd_head_logprob_workspace_size(T, d, V, chunk, code, KD_HEAD_BOTH),
                                 h.device)
        else:
            _require("ws", ws, torch.uint8, (ws.numel(),), h.device)
        if not need[0]:
            dH = None
        elif dH is None:
            dH = torch.empty_like(h)
        else:
            _require("dH", dH, h.dtype, (T, d), h.device)
        if not need[1]:
            dW = None
        elif dW is None:
            dW = torch.empty((V, d), dtype=dW_dtype, device=h.device)
        else:
            _require("dW", dW, dW_dtype, (V, d), h.device)
        _check(kd_head_logprob_bwd(h.data_ptr(), W.data_ptr(), code, T, d, V, targets.data_ptr(),
                                   chunk, float(temperature), lse.data_ptr(), _ptr(kept_logp),
                                   grad_logp.data_ptr(),
                                   _ptr(grad_loss), _ptr(dH), _ptr(dW),
                                   KD_DTYPE_BF16 if dW_dtype is torch.bfloat16 else KD_DTYPE_F32,
                                   int(accumulate_dW), ws.data_ptr(), ws.numel(), _current_stream(h.device)),
               "kd_head_logprob_bwd")
    _used_on(stream, (h, W, targets, lse, grad_logp, grad_loss, kept_logp, dH, dW, ws))
    return dH, dW, ws


class HeadLogprobs(torch.autograd.Function):
    """``logp = HeadLogprobs.apply(h, W, targets, chunk, temperature=1.0, keep=None)``:
    the log-probabilities of ``head_logprobs`` (NaN for a target that is neither a token
    nor KD_TARGET_IGNORE) with gradients to h and W (W's in W's dtype).

    ``keep=True`` (up to two chunks of positions, of at least 256 each): the forward
    holds a workspace of kd_head_logprob_workspace_size(..., KD_HEAD_KEEP) bytes until
    its backward, one for each such forward of a graph, and the backward does not
    project again.  That is two chunks of exponentials in the operands' type, also where
    T is one chunk (4 V bytes per position then, for bf16, and 2 V for T of two chunks),
    V / 8 bytes per position of their references, and 16 d bytes per position of a chunk
    for the partials of dH: 1.26 GB at T = chunk = 2048, d = 4096, V = 131072.  The kept
    exponentials are rounded to the operands' type, one rounding more of each dz entry.
    ``keep=False``: nothing is held, and the backward recomputes the logits chunk by
    chunk, as it does beyond two chunks.  None keeps where that is possible."""

    @classmethod
    def apply(cls, h, W, targets, chunk, temperature=1.0, keep=None):
        if not torch.is_grad_enabled():          # nothing will ask for what a forward keeps
            return head_logprobs(h.detach(), W.detach(), targets, chunk, temperature)[0]
        return super().apply(h, W, targets, chunk, temperature, keep)

    @staticmethod
    def forward(ctx, h, W, targets, chunk, temperature, keep):
        if keep is None:
            keep = _one_group(h.shape[0], chunk)
        keep = bool(keep) and any(ctx.needs_input_grad[:2])
        logp, lse, ws = head_logprobs(h, W, targets, chunk, temperature, keep=keep)
        ctx.save_for_backward(h, W, targets, lse, logp if keep else None)
        ctx.chunk, ctx.temperature = chunk, temperature
        ctx.ws = ws if keep else None
        return logp

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        h, W, targets, lse, kept = ctx.saved_tensors
        ws, ctx.ws = ctx.ws, None        # used up: a second backward recomputes
        # dW leaves the kernel in W's type where it is formed in one go, and is added up in fp32
        # and rounded afterwards otherwise
        direct = _one_group(h.shape[0], ctx.chunk)
        dH, dW, _ = head_logprobs_bwd(h, W, targets, lse, g.contiguous(), ctx.chunk, ctx.temperature,
                                      need=ctx.needs_input_grad[:2], ws=ws,
                                      kept_logp=None if ws is None else kept,
                                      dW_dtype=W.dtype if direct else torch.float32)
        return dH, None if dW is None else dW.to(W.dtype), None, None, None, None


# ------------------------------------------------- objectives over token log-probabilities

def _sequences(logp, cu_seqlens, mask):
    """(number of sequences, number of tokens) of a batch of token
    log-probabilities: rows of a 2-D ``logp``, or ``cu_seqlens`` over a 1-D one."""
    if not isinstance(logp, torch.Tensor):
        raise TypeError("logp: a torch tensor is needed")
    dev = logp.device
    _require("logp", logp, torch.float32, logp.shape, dev)
    if cu_seqlens is None:
        if logp.dim() != 2:
            raise ValueError("logp: [sequences, tokens] is needed, or cu_seqlens with one axis of tokens")
        n_seqs = logp.shape[0]
    else:
        if logp.dim() != 1 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens: [sequences + 1] over one axis of tokens is needed")
        _require("cu_seqlens", cu_seqlens, torch.int32, cu_seqlens.shape, dev)
        n_seqs = cu_seqlens.shape[0] - 1
    if mask is not None:
        if mask.dtype is not torch.bool and mask.dtype is not torch.uint8:
            raise TypeError(f"mask: bool or uint8 is needed, not {mask.dtype}")
        _require("mask", mask, mask.dtype, logp.shape, dev)
    return n_seqs, logp.numel()


def policy_loss(logp, old_logp, advantages, *, mask=None, ref_logp=None, cu_seqlens=None,
                advantages_per: str = "sequence", clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, reduction: str = "token", denom: float | None = None,
                grad: bool = True, ws=None, stream=None):
    """Clipped policy loss with a KL term: (loss f32 [], stats f32 [4], dlogp f32
    like logp, or None with ``grad=False``).

    ``logp`` f32 [sequences, tokens], or [tokens] with ``cu_seqlens`` int32
    [sequences + 1]; ``old_logp`` (None: on-policy, ratio 1) and ``ref_logp``
    (None: no KL) like it; ``mask`` bool or uint8 like it; ``advantages`` f32
    [sequences], or like ``logp`` with ``advantages_per="token"``.
    ``reduction``: "token", "sequence" or "fixed" (with ``denom``).  ``stats``:
    tokens that count, and over them the means of the ratio, of "clipped" and
    of the KL estimate.  ``dlogp`` is what ``head_logprobs_bwd`` takes.  A
    ``cu_seqlens`` that does not ascend within the tokens makes the loss NaN (and
    KD_ERR_BAD_INDEX in a given ``ws``)."""
    lib = load()
    if stream is None and _native is not None and reduction in REDUCTIONS and advantages_per in ADVANTAGES_PER and \
            (reduction == "fixed") == (denom is not None):
        out = _native.policy_loss(logp, old_logp, ref_logp, advantages, advantages_per == "token", mask,
                                  cu_seqlens, clip_low, clip_high, kl_coef, REDUCTIONS[reduction],
                                  0.0 if denom is None else denom, grad, ws)
        if out is not None:
            return _native_result(out, "kd_policy_loss")
    n_seqs, n = _sequences(logp, cu_seqlens, mask)
    dev = logp.device
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {tuple(REDUCTIONS)}")
    if (reduction == "fixed") != (denom is not None):
        raise ValueError("denom: belongs to reduction=\"fixed\" and to no other")
    if advantages_per not in ADVANTAGES_PER:
        raise ValueError(f"advantages_per must be one of {ADVANTAGES_PER}")
    per_token = advantages_per == "token"
    _require("advantages", advantages, torch.float32, logp.shape if per_token else (n_seqs,), dev)
    if old_logp is not None:
        _require("old_logp", old_logp, torch.float32, logp.shape, dev)
    if ref_logp is not None:
        _require("ref_logp", ref_logp, torch.float32, logp.shape, dev)
    with _use_stream(dev, stream):
        keep, at, nbytes = _workspace(ws, lib.kd_policy_loss_workspace_size(n_seqs, n), logp)
        loss = logp.new_empty(())
        stats = logp.new_empty(4)
        dlogp = torch.empty_like(logp) if grad else None
        _check(lib.kd_policy_loss(logp.data_ptr(), _ptr(old_logp), _ptr(ref_logp),
                                  advantages.data_ptr(), per_token, _ptr(mask), _ptr(cu_seqlens),
                                  n_seqs, n, clip_low, clip_high, kl_coef, REDUCTIONS[reduction],
                                  0.0 if denom is None else denom, loss.data_ptr(),
                                  stats.data_ptr(), _ptr(dlogp), at, nbytes, _current_stream(dev)),
               "kd_policy_loss")
    _used_on(stream, (logp, old_logp, ref_logp, advantages, mask, cu_seqlens, ws))
    return loss, stats, dlogp


class PolicyLoss(torch.autograd.Function):
    """``loss, stats = PolicyLoss.apply(logp, old_logp, advantages, options)``: the
    loss of ``policy_loss`` with a gradient to ``logp``; ``options`` is a dict of
    its keyword arguments."""

    @staticmethod
    def forward(ctx, logp, old_logp, advantages, options=None):
        loss, stats, dlogp = policy_loss(logp, old_logp, advantages, **{
            **(options or {}), "grad": ctx.needs_input_grad[0]})
        ctx.save_for_backward(dlogp)
        ctx.mark_non_differentiable(stats)
        return loss, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        (dlogp,) = ctx.saved_tensors
        return dlogp * g, None, None, None


def preference_loss(logp, *, ref_logp=None, mask=None, cu_seqlens=None, kind: str = "sigmoid",
                    beta: float = 0.1, margin: float = 0.0, label_smoothing: float = 0.0,
                    length_normalize: bool = False, pairs_total: int | None = None,
                    grad: bool = True, ws=None, stream=None):
    """Paired preference loss: (loss f32 [], rewards f32 [2 pairs], dlogp f32 like
    logp, or None with ``grad=False``).

    ``logp`` f32 [2 pairs, tokens], or [tokens] with ``cu_seqlens`` int32
    [2 pairs + 1]: first every pair's chosen sequence, then every pair's rejected
    one.  ``ref_logp`` (None: no reference) and ``mask`` like ``logp``.  ``kind``:
    "sigmoid" (with ``label_smoothing``), "hinge" or "ipo".  ``pairs_total``: the
    pairs of the whole batch when these are a part of it.  A bad ``cu_seqlens``
    as for ``policy_loss``."""
    lib = load()
    if stream is None and _native is not None and kind in PREFERENCE_KINDS:
        out = _native.preference_loss(logp, ref_logp, mask, cu_seqlens, PREFERENCE_KINDS[kind], beta, margin,
                                      label_smoothing, length_normalize, pairs_total, grad, ws)
        if out is not None:
            return _native_result(out, "kd_preference_loss")
    n_seqs, n = _sequences(logp, cu_seqlens, mask)
    dev = logp.device
    if n_seqs % 2:
        raise ValueError(f"{n_seqs} sequences: chosen and rejected ones come in pairs")
    if kind not in PREFERENCE_KINDS:
        raise ValueError(f"kind must be one of {tuple(PREFERENCE_KINDS)}")
    if ref_logp is not None:
        _require("ref_logp", ref_logp, torch.float32, logp.shape, dev)
    pairs = n_seqs // 2
    with _use_stream(dev, stream):
        keep, at, nbytes = _workspace(ws, lib.kd_preference_loss_workspace_size(pairs, n), logp)
        loss = logp.new_empty(())
        rewards = logp.new_empty(n_seqs)
        dlogp = torch.empty_like(logp) if grad else None
        _check(lib.kd_preference_loss(logp.data_ptr(), _ptr(ref_logp), _ptr(mask), _ptr(cu_seqlens),
                                      pairs, n, PREFERENCE_KINDS[kind], beta, margin,
                                      label_smoothing, bool(length_normalize),
                                      pairs if pairs_total is None else pairs_total,
                                      loss.data_ptr(), rewards.data_ptr(), _ptr(dlogp), at, nbytes,
                                      _current_stream(dev)),
               "kd_preference_loss")
    _used_on(stream, (logp, ref_logp, mask, cu_seqlens, ws))
    return loss, rewards, dlogp


class PreferenceLoss(torch.autograd.Function):
    """``loss, rewards = PreferenceLoss.apply(logp, options)``: the loss of
    ``preference_loss`` with a gradient to ``logp``; ``options`` is a dict of its
    keyword arguments."""

    @staticmethod
    def forward(ctx, logp, options=None):
        loss, rewards, dlogp = preference_loss(logp, **{**(options or {}), "grad": ctx.needs_input_grad[0]})
        ctx.save_for_backward(dlogp)
        ctx.mark_non_differentiable(rewards)
        return loss, rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        (dlogp,) = ctx.saved_tensors
        return dlogp * g, None


# ------------------------------------------------- the gradients of the whole step

_GRAD_CODES = {torch.float32: KD_DTYPE_F32, torch.bfloat16: KD_DTYPE_BF16}
_dtype_of = operator.attrgetter("dtype")


def _grad_arrays(name: str, tensors):
    """Checks a list of gradients; (count, device, addresses, sizes, type codes).
    A list may hold hundreds of small tensors: every pass over it is a `map`."""
    n = len(tensors)
    if n == 0:
        raise ValueError(f"{name}: at least one tensor is needed")
    Tensor = torch.Tensor
    try:
        codes = array.array("i", map(_GRAD_CODES.__getitem__, map(_dtype_of, tensors)))
        places = set(map(Tensor.get_device, tensors))
    except (KeyError, AttributeError, TypeError):
        raise TypeError(f"{name}: float32 or bfloat16 tensors are needed") from None
    if len(places) != 1 or not tensors[0].is_cuda:
        raise ValueError(f"{name}: all tensors must be on one CUDA device")
    if not all(map(Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name}: must be contiguous")
    return (n, tensors[0].device, array.array("Q", map(Tensor.data_ptr, tensors)),
            array.array("q", map(Tensor.numel, tensors)), codes)


def grad_sumsq(grads, stream=None):
    """Sum of squares of a list of gradients, fp64 [] (its root is their norm)."""
    grads = list(grads)
    n, dev, ptrs, sizes, codes = _grad_arrays("grads", grads)
    lib = load()
    with _use_stream(dev, stream):
        keep, at, nbytes = _workspace(None, lib.kd_grad_clip_workspace_size(n), grads[0])
        out = torch.empty((), dtype=torch.float64, device=dev)
        _check(lib.kd_grad_sumsq(ptrs.buffer_info()[0], sizes.buffer_info()[0], codes.buffer_info()[0], n,
                             out.data_ptr(), at, nbytes, _current_stream(dev)),
               "kd_grad_sumsq")
    _used_on(stream, grads)
    return out


def clip_grad_norm(grads, max_norm: float, out=None, sumsq=None, stream=None):
    """Scales a list of gradients by min(1, max_norm / (norm + 1e-6)), in place or
    into the tensors of ``out`` (same sizes and types); returns the norm before
    it, f32 [].  ``grads``: float32 and bfloat16 CUDA tensors of any shapes, each
    contiguous.  ``sumsq`` fp64 []: the sum of squares to use, where the list is
    a part of what the norm is taken over (``dp.clip_grad_norm``)."""
    lib = load()
    grads, out = list(grads), None if out is None else list(out)
    if stream is None and _native is not None:
        done = _native.clip_grad_norm(grads, out, max_norm, sumsq)
        if done is not None:
            return _native_result(done, "kd_grad_clip")[0]
    n, dev, ptrs, sizes, codes = _grad_arrays("grads", grads)
    outs = ptrs
    if out is not None:
        m, out_dev, outs, out_sizes, out_codes = _grad_arrays("out", out)
        if m != n or out_dev != dev or out_sizes != sizes or out_codes != codes:
            raise ValueError("out: the sizes, types and device of grads are needed")
    if sumsq is not None:
        _require("sumsq", sumsq, torch.float64, (), dev)
    with _use_stream(dev, stream):
        keep, at, nbytes = _workspace(None, lib.kd_grad_clip_workspace_size(n), grads[0])
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _check(lib.kd_grad_clip(ptrs.buffer_info()[0], outs.buffer_info()[0], sizes.buffer_info()[0],
                            codes.buffer_info()[0], n, max_norm, _ptr(sumsq), norm.data_ptr(), at,
                            nbytes, _current_stream(dev)),
               "kd_grad_clip")
    _used_on(stream, grads + (out or []) + [sumsq])
    return norm
