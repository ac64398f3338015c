"""A post-training step's workspace tells what any of its stages recorded: each pass
through the head clears the status when it starts, so the step has to carry the first
one's over.  (On the CPU: the calls are stood in for, and plant the status.)"""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd, posttrain

OK, BAD, LATE = kd.KD_OK, kd.KD_ERR_BAD_INDEX, kd.KD_ERR_TIMEOUT


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind", ["policy", "preference"])
@pytest.mark.parametrize("first,objective,second,want", [
    (OK, OK, OK, OK), (LATE, OK, OK, LATE), (BAD, OK, BAD, BAD), (OK, OK, LATE, LATE), (LATE, OK, BAD, LATE),
    (BAD, OK, LATE, LATE), (OK, BAD, OK, BAD), (LATE, BAD, OK, LATE)])
def test_every_stage_is_heard(monkeypatch, packed, kind, first, objective, second, want):
    if objective and not packed:
        pytest.skip("only packed sequences can be wrong in the objective's device data")
    T, d, V = 8, 8, 16

    def record(ws, code):
        ws[:4].view(torch.int32).fill_(code)

    def head_logprobs(h, W, targets, chunk, temperature=1.0, ws=None, **kw):
        ws = torch.zeros(1024, dtype=torch.uint8)
        record(ws, first)
        return torch.zeros(T), torch.zeros(T), ws

    def head_logprobs_bwd(h, W, targets, lse, grad, chunk, temperature=1.0, ws=None, **kw):
        record(ws, second)
        return torch.zeros(T, d), torch.zeros(V, d), ws

    def loss(logp, *args, ws=None, **kw):
        if ws is not None:
            record(ws, objective)
        return torch.zeros(()), torch.zeros(4), torch.zeros_like(logp)

    monkeypatch.setattr(kd, "head_logprobs", head_logprobs)
    monkeypatch.setattr(kd, "head_logprobs_bwd", head_logprobs_bwd)
    monkeypatch.setattr(kd, f"{kind}_loss", loss)
    h, W = torch.zeros(T, d), torch.zeros(V, d)
    targets, kw = torch.zeros((2, 4), dtype=torch.int32), dict(chunk=4)
    if packed:
        targets, kw["cu_seqlens"] = targets.view(-1), torch.tensor([0, 4, 8], dtype=torch.int32)
    kw["keep"] = False
    if kind == "policy":
        step = posttrain.policy_step(h, W, targets, torch.zeros(targets.shape), torch.zeros(2), **kw)
    else:
        step = posttrain.preference_step(h, W, targets, **kw)
    assert step.ws[:4].view(torch.int32).item() == want
