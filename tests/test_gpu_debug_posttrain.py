"""The post-training operators in the debug build (libkd_debug.so), whose device-side
invariant checks record KD_ERR_INTERNAL: every status word must read KD_OK, and the
results must be those of the release build, bit for bit."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import build, kd, posttrain
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture
def both():
    """A function that runs another one in both builds and compares what it returns."""
    require_gpu()
    path = build.build(debug=True)

    def compare(run):
        want = run()
        prev = kd.use_library(path)
        try:
            assert kd.LIB_PATH == path
            got = run()
            torch.cuda.synchronize()
        finally:
            kd.use_library(prev)
        assert len(want) == len(got)
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, got))

    return compare


def _ok(ws):
    assert kd.read_device_status(ws) == kd.KD_OK


@pytest.mark.parametrize("T,d,V,chunk,dtype", [
    (300, 200, 5000, 100, torch.bfloat16),
    (77, 72, 1003, 33, torch.float32),
    (64, 72, 60000, 64, torch.bfloat16),          # odd boxes, several dW tiles a cluster
    (5000, 72, 72, 2500, torch.bfloat16),         # two launches, many row tiles of odd boxes
    (1024, 256, 32768, 1024, torch.bfloat16),     # several work units a cluster everywhere
])
def test_head(both, T, d, V, chunk, dtype):
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=71)

    def run():
        logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, backward=True)
        _ok(ws)
        out = [logp, lse, *kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws)[:2]]
        _ok(ws)
        if T <= 2 * max(chunk, 256):
            logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
            _ok(ws)
            out += kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp, dW_dtype=dtype)[:2]
            _ok(ws)
        return out

    both(run)


@pytest.mark.parametrize("S,L", [(8, 20), (64, 700)])
def test_objectives(both, S, L):
    gen = torch.Generator("cuda").manual_seed(5)
    logp, old, ref = (-torch.rand((S, L), generator=gen, device="cuda") for _ in range(3))
    mask = torch.rand((S, L), generator=gen, device="cuda") < 0.7
    adv = torch.randn((S,), generator=gen, device="cuda")
    cu = (torch.arange(S + 1, device="cuda") * L).to(torch.int32)

    def run():
        out = []
        for reduction in ("token", "sequence"):
            ws = kd.alloc_workspace(kd.kd_policy_loss_workspace_size(S, S * L), "cuda")
            out += kd.policy_loss(logp, old, adv, mask=mask, ref_logp=ref, kl_coef=0.1, reduction=reduction, ws=ws)
            _ok(ws)
        ws = kd.alloc_workspace(kd.kd_preference_loss_workspace_size(S // 2, S * L), "cuda")
        out += kd.preference_loss(logp.view(-1), ref_logp=ref.view(-1), mask=mask.view(-1), cu_seqlens=cu, ws=ws)
        _ok(ws)
        return out

    both(run)


def test_step_and_clipping(both):
    S, L, d, V = 8, 40, 64, 900
    h, W, tgt, _ = _inputs(S * L, d, V, torch.bfloat16, seed=72)
    adv = torch.linspace(-1, 1, S, device="cuda")
    old = torch.full((S, L), -6.5, device="cuda")

    def run():
        s = posttrain.policy_step(h, W, tgt.view(S, L), old, adv, chunk=64)
        _ok(s.ws)
        norm = kd.clip_grad_norm([s.dW, s.dH.clone()], 0.01)
        return s.loss, s.extra, s.logp, s.dH, s.dW, norm

    both(run)
