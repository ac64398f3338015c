"""A workspace that another keeping forward of the very same sizes has used since: its label
is the same, the rows' log-probabilities are not.  The backward of the first forward
records KD_ERR_WORKSPACE and gives NaN."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [60, 5000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_forwards_and_the_first_one_s_backward(T, dtype):
    require_gpu()
    d, V = 64, 300
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=81)
    h2, _, tgt2, g2 = _inputs(T, d, V, dtype, seed=82)
    ws = kd.alloc_workspace(kd.kd_head_logprob_workspace_size(T, d, V, T, kd._dtype_code(h), kd.KD_HEAD_KEEP), "cuda")
    logp, lse, _ = kd.head_logprobs(h, W, tgt, T, keep=True, ws=ws)
    want = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    for need in ((True, True), (True, False), (False, True)):
        logp, lse, _ = kd.head_logprobs(h, W, tgt, T, keep=True, ws=ws)
        kd.head_logprobs(h2, W, tgt2, T, keep=True, ws=ws)
        dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp, need=need)
        assert kd.read_device_status(ws) == kd.KD_ERR_WORKSPACE
        assert dH is None or bool(torch.isnan(dH[tgt >= 0]).all())
        assert dW is None or bool(torch.isnan(dW).all())
    # the same forward twice is the same forward
    logp, lse, _ = kd.head_logprobs(h, W, tgt, T, keep=True, ws=ws)
    kd.head_logprobs(h, W, tgt, T, keep=True, ws=ws)
    got = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    assert kd.read_device_status(ws) == kd.KD_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_log_probability_that_is_nan():
    """NaN compares as what it is: a row of NaN does not make the workspace a wrong one."""
    require_gpu()
    T, d, V = 60, 64, 300
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=83, ignored=0.0)
    h[4] = float("nan")
    tgt[9] = V
    logp, lse, ws = kd.head_logprobs(h, W, tgt, T, keep=True)
    dH, _, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX            # of the target
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[4] = False
    assert bool(torch.isfinite(dH[rest]).all()) and bool((dH[9] == 0).all())
