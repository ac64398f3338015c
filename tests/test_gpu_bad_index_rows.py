"""A bad index is an error of its row alone: the call records it and works on the
other rows to the end, with the bits of a call without the bad one."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [50, 5000])             # one block of targets, and several
@pytest.mark.parametrize("keep", [False, True])
def test_other_rows_of_a_bad_target(T, keep):
    require_gpu()
    h, W, tgt, g = _inputs(T, 64, 300, torch.bfloat16, seed=4)
    g = torch.where(tgt >= 0, g, 0.0)
    where = torch.tensor([0, 17, T - 1], device="cuda")
    bad, skip = tgt.clone(), tgt.clone()
    bad[where] = torch.tensor([-1, 300, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    skip[where] = kd.KD_TARGET_IGNORE
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[where] = False
    kw = dict(keep=True) if keep else dict(backward=True)
    want, wlse, wws = kd.head_logprobs(h, W, skip, T, **kw)
    ref = kd.head_logprobs_bwd(h, W, skip, wlse, g, T, ws=wws, kept_logp=want if keep else None)
    assert kd.read_device_status(wws) == kd.KD_OK
    for _ in range(5):
        logp, lse, ws = kd.head_logprobs(h, W, bad, T, **kw)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
        assert torch.equal(logp[rest], want[rest]) and torch.equal(lse, wlse)
        got = kd.head_logprobs_bwd(h, W, bad, lse, g, T, ws=ws, kept_logp=logp if keep else None)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_other_rows_of_a_bad_cache_entry():
    require_gpu()
    T, d, V, K, chunk = 3000, 64, 700, 7, 1000
    h, W, vals, idx = inputs.make_loss_inputs(T, d, V, K, dtype=torch.bfloat16, seed=6, device="cuda")
    bad = idx.clone()
    bad[11, 2], bad[2999, 0] = V, bad[2999, 1]
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[11] = rest[2999] = False
    _, wlse, wkl, _ = kd.fused_kl_fwd(h, W, vals, idx, chunk, kl_rows=True)
    wH = kd.fused_kl_bwd(h, W, vals, idx, wlse, chunk)[0]
    for _ in range(5):
        _, lse, kl, ws = kd.fused_kl_fwd(h, W, vals, bad, chunk, kl_rows=True)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
        assert torch.equal(lse, wlse) and torch.equal(kl[rest], wkl[rest])
        dH = kd.fused_kl_bwd(h, W, vals, bad, lse, chunk, ws=ws)[0]
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
        assert torch.equal(dH[rest], wH[rest])
