"""Whether a forward through the head keeps its exponentials for the backward is the
caller's choice in the autograd form and in the steps: kept, they take memory from
forward to backward and one rounding more; recomputed, nothing is held."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd, posttrain
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


def _held():
    """Bytes that tensors have asked for (the allocator's own blocks are up to 1 MiB larger)."""
    return torch.cuda.memory_stats()["requested_bytes.all.current"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_autograd_form(dtype):
    require_gpu()
    T, d, V, chunk = 400, 64, 30000, 256
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=51, ignored=0.0)
    x, w = h.clone().requires_grad_(), W.clone().requires_grad_()
    logp, lse, _ = kd.head_logprobs(h, W, tgt, chunk)
    recomputed = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, dW_dtype=dtype)[:2]
    klogp, klse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
    kept = kd.head_logprobs_bwd(h, W, tgt, klse, g, chunk, ws=ws, kept_logp=klogp, dW_dtype=dtype)[:2]
    held = kd.kd_head_logprob_workspace_size(T, d, V, chunk, kd._dtype_code(h), kd.KD_HEAD_KEEP)
    del ws
    for keep, want in ((False, recomputed), (True, kept), (None, kept)):
        before = _held()
        out = kd.HeadLogprobs.apply(x, w, tgt, chunk, 1.0, keep)
        grown = _held() - before
        assert torch.equal(out, logp)
        # logp and lse, and a workspace with the slack of its alignment
        assert grown == 8 * T + (0 if keep is False else held + 1024)
        got = torch.autograd.grad(out, (x, w), g)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del out, got
        assert _held() <= before


def test_too_many_positions_to_keep():
    require_gpu()
    h, W, tgt, g = _inputs(600, 64, 300, torch.bfloat16, seed=52)
    x = h.clone().requires_grad_()
    with pytest.raises(kd.KDError):
        kd.HeadLogprobs.apply(x, W, tgt, 256, 1.0, True)
    adv = torch.ones(4, device="cuda")
    with pytest.raises(kd.KDError):
        posttrain.policy_step(h, W, tgt.view(4, 150), None, adv, chunk=256, keep=True)
    with torch.no_grad():                              # nothing is kept without a backward
        assert torch.equal(kd.HeadLogprobs.apply(x, W, tgt, 256, 1.0, True), kd.head_logprobs(h, W, tgt, 256)[0])


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_steps(kind):
    require_gpu()
    S, L, d, V, chunk = 4, 100, 64, 900, 256
    h, W, tgt, _ = _inputs(S * L, d, V, torch.bfloat16, seed=53)
    tgt = tgt.view(S, L)
    adv = torch.linspace(-1, 1, S, device="cuda")
    size = [kd.kd_head_logprob_workspace_size(S * L, d, V, chunk, kd.KD_DTYPE_BF16, use)
            for use in (kd.KD_HEAD_BOTH, kd.KD_HEAD_KEEP)]

    def step(**kw):
        if kind == "policy":
            return posttrain.policy_step(h, W, tgt, torch.full((S, L), -6.5, device="cuda"), adv, chunk=chunk, **kw)
        return posttrain.preference_step(h, W, tgt, chunk=chunk, **kw)

    def parts(s):
        return s.loss, s.extra, s.logp, s.dH, s.dW

    kept, without = step(keep=True), step(keep=False)
    assert without.ws.numel() == size[0] and kept.ws.numel() == size[1]
    assert all(torch.equal(a, b) for a, b in zip(parts(kept)[:3], parts(without)[:3]))
    assert not torch.equal(kept.dW, without.dW)
    for s, want in ((step(), kept), (step(keep=None), kept),
                    (step(ws=kd.alloc_workspace(size[0], "cuda")), without),
                    (step(ws=kd.alloc_workspace(size[1], "cuda")), kept),
                    (step(ws=kd.alloc_workspace(size[1], "cuda"), keep=False), without)):
        assert kd.read_device_status(s.ws) == kd.KD_OK
        assert all(torch.equal(a, b) for a, b in zip(parts(s), parts(want)))
    with pytest.raises(kd.KDError):
        step(ws=kd.alloc_workspace(size[0], "cuda"), keep=True)
