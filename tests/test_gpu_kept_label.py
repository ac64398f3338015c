"""What a keeping forward leaves in a workspace is labelled: a backward that asks for
something else (other sizes, chunk, temperature or type, a workspace that another call
has used since, a second use) records KD_ERR_WORKSPACE and gives NaN, not wrong gradients."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu


def _big(device="cuda"):
    return kd.alloc_workspace(64 << 20, device)


def _refused(ws, dH, dW):
    assert kd.read_device_status(ws) == kd.KD_ERR_WORKSPACE
    assert dH is None or bool(torch.isnan(dH).all())
    assert dW is None or bool(torch.isnan(dW).any())


@pytest.mark.parametrize("T", [50, 5000])             # one block of targets, and several
def test_right_use_and_second_use(T):
    require_gpu()
    h, W, tgt, g = _inputs(T, 64, 300, torch.bfloat16, seed=41, ignored=0.0)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, T, keep=True)
    want = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    assert kd.read_device_status(ws) == kd.KD_OK and bool(torch.isfinite(want[0]).all())
    again = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    _refused(ws, again[0], again[1])
    # and the workspace is as good as new
    logp, lse, ws = kd.head_logprobs(h, W, tgt, T, keep=True, ws=ws)
    got = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp)
    assert kd.read_device_status(ws) == kd.KD_OK and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


OTHER = {
    "temperature": dict(tau=0.9),
    "chunk": dict(chunk=300),
    "rows": dict(T=499),
    "width": dict(d=56),
    "vocabulary": dict(V=296),
}


@pytest.mark.parametrize("other", OTHER)
def test_another_call_of_the_head(other):
    require_gpu()
    base = dict(T=500, d=64, V=300, chunk=260, tau=1.0)
    use = {**base, **OTHER[other]}
    h, W, tgt, g = _inputs(500, 64, 300, torch.bfloat16, seed=42, ignored=0.0)
    tgt = tgt % 296
    logp, lse, ws = kd.head_logprobs(h, W, tgt, base["chunk"], base["tau"], keep=True, ws=_big())
    T, d, V = use["T"], use["d"], use["V"]
    cut = (h[:T, :d].contiguous(), W[:V, :d].contiguous(), tgt[:T].contiguous(), lse[:T].contiguous(), g[:T].contiguous())
    dH, dW, _ = kd.head_logprobs_bwd(*cut, use["chunk"], use["tau"], ws=ws, kept_logp=logp[:T].contiguous())
    _refused(ws, dH, dW)
    for need in ((True, False), (False, True)):
        logp, lse, ws = kd.head_logprobs(h, W, tgt, base["chunk"], base["tau"], keep=True, ws=ws)
        dH, dW, _ = kd.head_logprobs_bwd(*cut, use["chunk"], use["tau"], ws=ws, kept_logp=logp[:T].contiguous(), need=need)
        _refused(ws, dH, dW)


def test_a_workspace_that_another_call_has_used():
    require_gpu()
    T, d, V, chunk = 200, 64, 300, 200
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=43, ignored=0.0)
    ws = _big()
    _, _, vals, idx = inputs.make_loss_inputs(T, d, V, 4, dtype=torch.bfloat16, seed=43, device="cuda")
    x = inputs.make_teacher_logits(16, 3000, seed=7, device="cuda")
    rows = torch.full((4, 50), -1.0, device="cuda")
    adv = torch.ones(4, device="cuda")
    long = torch.full((4, 5000), -1.0, device="cuda")
    mask = torch.ones((4, 5000), dtype=torch.bool, device="cuda")
    lse0 = torch.full((T,), 6.0, device="cuda")
    calls = {
        "scoring": lambda: kd.head_logprobs(h, W, tgt, chunk, ws=ws),
        "recomputing backward": lambda: kd.head_logprobs_bwd(h, W, tgt, lse0, g, chunk, ws=ws),
        "loss": lambda: kd.fused_kl_fwd(h, W, vals, idx, chunk, ws=ws),
        "loss backward": lambda: kd.fused_kl_bwd(h, W, vals, idx, lse0, chunk, ws=ws),
        "top-K": lambda: kd.topk_build(x, 20, ws=ws),
        "policy, one block": lambda: kd.policy_loss(rows, rows, adv, ws=ws),
        "policy": lambda: kd.policy_loss(long, long, adv, ws=ws),
        "policy, counts": lambda: kd.policy_loss(long, long, adv, mask=mask, ws=ws),
        "policy, counts of sequences": lambda: kd.policy_loss(long, long, adv, mask=mask, reduction="sequence", ws=ws),
        "preference, one block": lambda: kd.preference_loss(rows, ws=ws),
        "preference": lambda: kd.preference_loss(long, ws=ws),
    }
    for name, call in calls.items():
        logp, lse, _ = kd.head_logprobs(h, W, tgt, chunk, keep=True, ws=ws)
        call()
        dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)
        assert kd.read_device_status(ws) == kd.KD_ERR_WORKSPACE, name
        _refused(ws, dH, dW)


def test_a_fresh_workspace():
    require_gpu()
    T, d, V, chunk = 200, 64, 300, 200
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=44, ignored=0.0)
    logp, lse, _ = kd.head_logprobs(h, W, tgt, chunk)
    for byte in (0, 0xFF):
        ws = _big()
        ws.fill_(byte)
        dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)
        _refused(ws, dH, dW)


def test_a_bad_target_beside_a_wrong_use():
    """One of the two errors is recorded, and the gradients are NaN."""
    require_gpu()
    T, d, V = 5000, 64, 300
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=45, ignored=0.0)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, T, keep=True)
    tgt[9] = V
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, 0.5, ws=ws, kept_logp=logp)
    assert kd.read_device_status(ws) in (kd.KD_ERR_WORKSPACE, kd.KD_ERR_BAD_INDEX)
    assert bool(torch.isnan(dH[10:]).all())


def test_captured_and_replayed():
    require_gpu()
    T, d, V, chunk = 300, 64, 500, 256
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=46, ignored=0.2)
    g = torch.nan_to_num(g)
    ws = _big()

    def run():
        logp, lse, _ = kd.head_logprobs(h, W, tgt, chunk, keep=True, ws=ws)
        return (logp, *kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)[:2])

    want = [x.clone() for x in run()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        graph.replay()
        assert kd.read_device_status(ws) == kd.KD_OK
        assert all(torch.equal(a, b) for a, b in zip(out, want))
