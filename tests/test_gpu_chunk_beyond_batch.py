"""A chunk of any size is allowed and means the batch where it is larger, also where two
of them pass 64 bits."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu

HUGE = [1 << 40, (1 << 62) - 1, 1 << 62, (1 << 63) - 1]


@pytest.mark.parametrize("chunk", HUGE)
def test_head(chunk):
    require_gpu()
    T, d, V = 300, 64, 700
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=91)
    logp, lse, _ = kd.head_logprobs(h, W, tgt, T)
    want = kd.head_logprobs_bwd(h, W, tgt, lse, g, T)
    assert all(torch.equal(a, b) for a, b in zip(kd.head_logprobs(h, W, tgt, chunk)[:2], (logp, lse)))
    for need in ((True, True), (True, False), (False, True)):
        got = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, need=need)
        assert kd.read_device_status(got[2]) == kd.KD_OK
        assert all(b is None if not n else torch.equal(a, b) for n, a, b in zip(need, want, got))
    klogp, klse, ws = kd.head_logprobs(h, W, tgt, T, keep=True)
    kept = kd.head_logprobs_bwd(h, W, tgt, klse, g, T, ws=ws, kept_logp=klogp)
    klogp, klse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
    got = kd.head_logprobs_bwd(h, W, tgt, klse, g, chunk, ws=ws, kept_logp=klogp)
    assert kd.read_device_status(ws) == kd.KD_OK
    assert torch.equal(kept[0], got[0]) and torch.equal(kept[1], got[1])


@pytest.mark.parametrize("chunk", HUGE)
def test_loss(chunk):
    require_gpu()
    T, d, V, K = 300, 64, 700, 5
    h, W, vals, idx = inputs.make_loss_inputs(T, d, V, K, dtype=torch.bfloat16, seed=92, device="cuda")
    loss, lse, _, _ = kd.fused_kl_fwd(h, W, vals, idx, T)
    want = kd.fused_kl_bwd(h, W, vals, idx, lse, T)
    got = kd.fused_kl_fwd(h, W, vals, idx, chunk)
    assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
    got = kd.fused_kl_bwd(h, W, vals, idx, lse, chunk)
    assert kd.read_device_status(got[2]) == kd.KD_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
