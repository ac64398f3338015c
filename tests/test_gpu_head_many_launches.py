"""The head's log-probabilities over more positions than one launch of the forward takes
(2048, or a chunk): second and later launches, targets prepared by several blocks (more
than 4096), and many groups of the backward, against the plain fp64 form with the
tolerances of the head's parity tests."""

import pytest
import torch

import objective_plain as plain
from chunked_kl_loss_chunk_b200 import kd, posttrain
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs, _plain

pytestmark = pytest.mark.gpu

EPS = 2 ** -8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,V,chunk", [
    (5000, 72, 1003, 300),      # three launches, nine groups
    (2049, 136, 700, 64),       # one row left for the second launch
    (4097, 64, 515, 1024),      # and for the third; the targets in several blocks
    (9000, 64, 300, 4000),      # launches of a chunk
])
def test_recomputing(T, d, V, chunk, dtype):
    require_gpu()
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=61)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, backward=True)
    assert kd.read_device_status(ws) == kd.KD_OK
    one = kd.head_logprobs(h, W, tgt, T)
    assert torch.equal(one[0], logp) and torch.equal(one[1], lse)
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws)
    assert kd.read_device_status(ws) == kd.KD_OK
    rl, rlse, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt, 1.0, torch.where(tgt >= 0, g, 0.0))
    tol = 5e-3 if dtype == torch.float32 else 1e-3
    assert (lse.double() - rlse).abs().max() <= tol and (logp.double() - rl).abs().max() <= 2 * tol
    assert bool(((dH.double() - rH).abs() <= 2 * EPS * aH + 2 * tol * pH + 1e-30).all())
    assert bool(((dW.double() - rW).abs() <= EPS * aW + 2 * tol * pW + 1e-30).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,V,chunk", [(5000, 72, 1003, 2500), (4500, 136, 700, 2300), (4098, 64, 515, 2049)])
def test_keeping(T, d, V, chunk, dtype):
    """Two launches of a chunk each, whose exponentials and references lie side by side."""
    require_gpu()
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=62)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
    assert kd.read_device_status(ws) == kd.KD_OK
    one = kd.head_logprobs(h, W, tgt, T)
    assert torch.equal(one[0], logp) and torch.equal(one[1], lse)
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)
    assert kd.read_device_status(ws) == kd.KD_OK
    _, _, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt, 1.0, torch.where(tgt >= 0, g, 0.0))
    delta = 1e-2 if dtype == torch.float32 else 2e-3
    assert bool(((dH.double() - rH).abs() <= 3 * EPS * aH + delta * pH + 1e-30).all())
    assert bool(((dW.double() - rW).abs() <= 2 * EPS * aW + delta * pW + 1e-30).all())


@pytest.mark.parametrize("chunk,roundings", [(512, 1), (2600, 2)])      # recomputing, and keeping
def test_policy_step(chunk, roundings):
    require_gpu()
    S, L, d, V = 20, 255, 64, 900
    h, W, tgt, _ = _inputs(S * L, d, V, torch.bfloat16, seed=63)
    tgt = tgt.view(S, L)
    old = kd.head_logprobs(h, W, tgt.view(-1), chunk)[0].view(S, L) \
        + 0.2 * torch.randn((S, L), generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    adv = torch.linspace(-1, 1, S, device="cuda")
    step = posttrain.policy_step(h, W, tgt, old, adv, chunk=chunk)
    assert kd.read_device_status(step.ws) == kd.KD_OK
    want = plain.policy(step.logp.cpu().numpy(), old.cpu().numpy(), adv.cpu().numpy(), plain.layout(S, (S, L), None),
                        mask=(tgt != kd.KD_TARGET_IGNORE).cpu().numpy())
    assert abs(step.loss.item() - want["loss"]) <= 2 ** -19 * want["scale_loss"]
    rl, _, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt.view(-1), 1.0, torch.from_numpy(want["grad"]).cuda().view(-1))
    assert (step.logp.view(-1).double() - rl).abs().max() <= 2e-3
    assert bool(((step.dH.double() - rH).abs() <= (1 + roundings) * EPS * aH + 2e-3 * pH + 1e-30).all())
    assert bool(((step.dW.double() - rW).abs() <= roundings * EPS * aW + 2e-3 * pW + 1e-30).all())


def test_captured_and_replayed():
    """Several launches, the targets in several blocks, kept in one workspace, in a graph."""
    require_gpu()
    T, d, V, chunk = 5000, 64, 700, 2500
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=64)
    ws = kd.alloc_workspace(kd.kd_head_logprob_workspace_size(T, d, V, chunk, kd.KD_DTYPE_BF16, kd.KD_HEAD_KEEP), "cuda")

    def run():
        logp, lse, _ = kd.head_logprobs(h, W, tgt, chunk, keep=True, ws=ws)
        return (logp, *kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)[:2])

    want = [x.clone() for x in run()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for x in out:
            x.zero_()
        graph.replay()
        assert kd.read_device_status(ws) == kd.KD_OK
        assert all(torch.equal(a, b) for a, b in zip(out, want))
