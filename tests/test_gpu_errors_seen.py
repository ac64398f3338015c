"""Errors in device data (a target that is no token, a layout that is none) show in
the outputs too, for callers that do not read a workspace's status."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [50, 5000])             # one block of targets, and several
@pytest.mark.parametrize("keep", [False, True])
def test_a_bad_target_gives_nan(T, keep):
    require_gpu()
    h, W, tgt, _ = _inputs(T, 64, 300, torch.bfloat16, seed=4)
    where = torch.tensor([0, 17, T - 1], device="cuda")
    tgt[where] = torch.tensor([-1, 300, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    logp, _, ws = kd.head_logprobs(h, W, tgt, T, keep=keep)
    assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
    nan = torch.zeros(T, dtype=torch.bool, device="cuda")
    nan[where] = True
    assert torch.equal(torch.isnan(logp), nan) and bool((logp[tgt == kd.KD_TARGET_IGNORE] == 0).all())


def test_a_bad_target_in_the_autograd_form():
    require_gpu()
    h, W, tgt, _ = _inputs(40, 64, 300, torch.bfloat16, seed=5)
    tgt[3] = -1                                        # a padding label of another program
    out = kd.HeadLogprobs.apply(h.requires_grad_(), W, tgt, 40)
    assert bool(torch.isnan(out[3])) and not bool(torch.isnan(out[tgt != -1]).any())
