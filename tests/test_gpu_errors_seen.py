"""Errors in device data (a target that is no token, a layout that is none) show in
the outputs too, for callers that do not read a workspace's status."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd, posttrain
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


BAD_CU = {
    "negative": lambda cu, n: cu.__setitem__(0, -1),
    "past the tokens": lambda cu, n: cu.__setitem__(-1, n + 1),
    "far past them": lambda cu, n: cu.__setitem__(3, 2 ** 31 - 1),
    "descending": lambda cu, n: cu.__setitem__(2, cu[3].item() + 1),
    "last": lambda cu, n: cu.__setitem__(-1, cu[-2].item() - 1),
}


@pytest.mark.parametrize("length", [7, 900])          # in one block, and in several
@pytest.mark.parametrize("bad", BAD_CU)
def test_a_bad_layout_makes_the_loss_nan(length, bad):
    require_gpu()
    S = 8
    n = S * length + 5
    cu = (torch.arange(S + 1, dtype=torch.int32) * length + 2).cuda()
    logp = torch.full((n,), -1.0, device="cuda")
    adv = torch.ones(S, device="cuda")
    wrong = cu.clone()
    BAD_CU[bad](wrong, n)
    for mask in (None, torch.ones(n, dtype=torch.bool, device="cuda")):
        for reduction in ("token", "sequence"):
            for grad in (True, False):
                kw = dict(mask=mask, reduction=reduction, grad=grad)
                assert kd.policy_loss(logp, logp, adv, cu_seqlens=cu, **kw)[0].item() == -1.0
                assert torch.isnan(kd.policy_loss(logp, logp, adv, cu_seqlens=wrong, **kw)[0])
        for grad in (True, False):
            good = kd.preference_loss(logp, mask=mask, cu_seqlens=cu, grad=grad)[0]
            assert good.item() == pytest.approx(0.6931472, rel=1e-6)
            assert torch.isnan(kd.preference_loss(logp, mask=mask, cu_seqlens=wrong, grad=grad)[0])
    # a call without a bad layout on the same workspace is a call as ever
    ws = kd.alloc_workspace(kd.kd_policy_loss_workspace_size(S, n), "cuda")
    assert torch.isnan(kd.policy_loss(logp, logp, adv, cu_seqlens=wrong, ws=ws)[0])
    assert kd.policy_loss(logp, logp, adv, cu_seqlens=cu, ws=ws)[0].item() == -1.0


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_a_step_reports_what_its_stages_found(kind, given):
    require_gpu()
    T, d, V, chunk, S = 300, 64, 700, 64, 4
    h, W, tgt, _ = _inputs(T, d, V, torch.bfloat16, seed=8)
    adv = torch.ones(S, device="cuda")
    cu = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device="cuda")
    far = torch.tensor([0, 100, 90, 250, 301], dtype=torch.int32, device="cuda")
    lost = tgt.clone()
    lost[5] = V
    ws = None
    if given:
        ws = kd.alloc_workspace(kd.kd_head_logprob_workspace_size(T, d, V, chunk, kd.KD_DTYPE_BF16, kd.KD_HEAD_KEEP),
                                "cuda")

    def step(targets, layout):
        if kind == "policy":
            old = torch.full_like(targets, -6, dtype=torch.float32)
            return posttrain.policy_step(h, W, targets, old, adv, chunk=chunk, cu_seqlens=layout, ws=ws)
        return posttrain.preference_step(h, W, targets, chunk=chunk, cu_seqlens=layout, ws=ws)

    for targets, layout in ((tgt, cu), (tgt, far), (lost, cu), (lost, far), (tgt, cu)):
        out = step(targets, layout)
        fine = targets is tgt and layout is cu
        assert kd.read_device_status(out.ws) == (kd.KD_OK if fine else kd.KD_ERR_BAD_INDEX)
        assert bool(torch.isnan(out.loss)) != fine
        assert not given or out.ws.data_ptr() == ws.data_ptr()
