"""A workspace's status word may hold anything when a call starts (an earlier call's
error, a fresh allocation's bytes): the call must neither report it nor stop for it."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu

WORDS = (kd.KD_ERR_TIMEOUT, kd.KD_ERR_INTERNAL, kd.KD_ERR_BAD_INDEX, -1, 0x7FC00000)


@pytest.mark.parametrize("T", [40, 4096, 4097])       # the targets in one block, and in several
@pytest.mark.parametrize("keep", [False, True])
def test_head(T, keep):
    require_gpu()
    d, V = 256, 2000
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=T, ignored=0.0)
    ws = kd.alloc_workspace(kd.kd_head_logprob_workspace_size(T, d, V, T, kd.KD_DTYPE_BF16, kd.KD_HEAD_KEEP), "cuda")
    word = ws[:4].view(torch.int32)

    def run(code):
        word.fill_(code)
        logp, lse, _ = kd.head_logprobs(h, W, tgt, T, keep=keep, ws=ws)
        assert kd.read_device_status(ws) == kd.KD_OK
        # (between a keeping forward and its backward the word is the forward's)
        word.fill_(kd.KD_OK if keep and code in (kd.KD_ERR_TIMEOUT, kd.KD_ERR_INTERNAL) else code)
        dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp if keep else None)
        assert kd.read_device_status(ws) == kd.KD_OK
        return logp, lse, dH, dW

    want = run(0)
    for code in WORDS:
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(run(code), want))


def test_loss_and_objectives():
    require_gpu()
    T, d, V, K = 300, 64, 700, 5
    h, W, vals, idx = inputs.make_loss_inputs(T, d, V, K, dtype=torch.bfloat16, seed=3, device="cuda")
    ws = kd.alloc_workspace(16 << 20, "cuda")
    word = ws[:4].view(torch.int32)
    long = torch.full((4, 5000), -1.0, device="cuda")
    mask = torch.ones((4, 5000), dtype=torch.bool, device="cuda")
    adv = torch.ones(4, device="cuda")
    lse = kd.fused_kl_fwd(h, W, vals, idx, 100)[1]
    calls = [lambda: kd.fused_kl_fwd(h, W, vals, idx, 100, ws=ws)[:2],
             lambda: kd.fused_kl_bwd(h, W, vals, idx, lse, 100, ws=ws)[:2],
             lambda: kd.policy_loss(long, long, adv, ws=ws),
             lambda: kd.policy_loss(long, long, adv, mask=mask, ws=ws),
             lambda: kd.policy_loss(long, long, adv, mask=mask, reduction="sequence", ws=ws),
             lambda: kd.policy_loss(long[:, :9].contiguous(), None, adv, ws=ws),
             lambda: kd.preference_loss(long, ws=ws),
             lambda: kd.preference_loss(long[:, :9].contiguous(), ws=ws)]
    for call in calls:
        word.zero_()
        want = [x.clone() for x in call()]
        for code in WORDS:
            word.fill_(code)
            got = call()
            assert kd.read_device_status(ws) == kd.KD_OK
            assert all(torch.equal(a, b) for a, b in zip(got, want))
