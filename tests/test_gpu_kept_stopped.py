"""What a forward kept that was stopped (a wait ran out) is not used: the backward records
KD_ERR_WORKSPACE and gives NaN, and a step that keeps says so."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd, posttrain
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [60, 5000])             # one block of targets, and several
@pytest.mark.parametrize("code", [kd.KD_ERR_TIMEOUT, kd.KD_ERR_INTERNAL, kd.KD_ERR_BAD_INDEX])
def test_backward(T, code):
    require_gpu()
    h, W, tgt, g = _inputs(T, 64, 300, torch.bfloat16, seed=85, ignored=0.0)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, T, keep=True)
    want = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, T, keep=True, ws=ws)
    ws[:4].view(torch.int32).fill_(code)               # as if the forward had recorded it
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    if code == kd.KD_ERR_BAD_INDEX:                    # an error of a row alone
        assert kd.read_device_status(ws) == kd.KD_OK
        assert torch.equal(dH, want[0]) and torch.equal(dW, want[1])
    else:
        assert kd.read_device_status(ws) == kd.KD_ERR_WORKSPACE
        assert bool(torch.isnan(dH).all()) and bool(torch.isnan(dW).all())


@pytest.mark.parametrize("keep,want", [(True, kd.KD_ERR_WORKSPACE), (False, kd.KD_ERR_TIMEOUT)])
def test_step(monkeypatch, keep, want):
    require_gpu()
    h, W, tgt, _ = _inputs(120, 64, 300, torch.bfloat16, seed=86)
    forward = kd.head_logprobs

    def stopped(*args, **kw):
        logp, lse, ws = forward(*args, **kw)
        ws[:4].view(torch.int32).fill_(kd.KD_ERR_TIMEOUT)
        return logp, lse, ws

    monkeypatch.setattr(kd, "head_logprobs", stopped)
    step = posttrain.preference_step(h, W, tgt.view(4, 30), chunk=64, keep=keep)
    assert kd.read_device_status(step.ws) == want
