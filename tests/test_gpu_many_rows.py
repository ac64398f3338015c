"""One chunk of more than 2^27 positions, whose combination has more than 2^32 threads: a
pattern of positions repeated, so that every row has a known result."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu

BASE, TIMES = 4096, (1 << 15) + 3         # 2^27 + 12288 positions


def _every_row(got, want):
    assert got.shape[0] == BASE * TIMES
    assert bool((got.view(TIMES, BASE) == want).all())


def test_head():
    require_gpu()
    h, W, tgt, _ = _inputs(BASE, 8, 16, torch.bfloat16, seed=95)
    logp, lse, _ = kd.head_logprobs(h, W, tgt, BASE)
    T = BASE * TIMES
    got = kd.head_logprobs(h.repeat(TIMES, 1), W, tgt.repeat(TIMES), T)
    assert kd.read_device_status(got[2]) == kd.KD_OK
    _every_row(got[0], logp)
    _every_row(got[1], lse)


def test_loss():
    require_gpu()
    h, W, vals, idx = inputs.make_loss_inputs(BASE, 8, 16, 1, dtype=torch.bfloat16, seed=96, device="cuda")
    loss, lse, kl, _ = kd.fused_kl_fwd(h, W, vals, idx, BASE, kl_rows=True)
    T = BASE * TIMES
    got = kd.fused_kl_fwd(h.repeat(TIMES, 1), W, vals.repeat(TIMES, 1), idx.repeat(TIMES, 1), T, kl_rows=True)
    assert kd.read_device_status(got[3]) == kd.KD_OK
    _every_row(got[1], lse)
    _every_row(got[2], kl)
    # the same sum over fp64, divided by the larger count and rounded once
    assert abs(got[0].item() - kl.double().mean().item()) <= 2 ** -23 * abs(loss.item())
