"""Post-training steps: log-probabilities, objective, gradients and clipping run
one after the other, as a training program calls them.

Each stage is compared with its plain fp64 form on what the stage before it gave
(a logp off by a rounding may otherwise move a token across a clipping border).
Tolerances: those of the stages' own tests (dH: up to three roundings to bf16,
2^-8 of sum|dz w| each, where the forward keeps its exponentials, and the logits'
error, 2e-3 of the part that scales with p; dW: up to two).
"""

import numpy as np
import pytest
import torch

import objective_plain as plain
from chunked_kl_loss_chunk_b200 import inputs, kd, posttrain
from gpu_util import require_gpu
from test_gpu_head_logprob import _plain

pytestmark = pytest.mark.gpu


def _batch(layout, d, V, seed):
    """Hidden states, head, targets with ignored prompts, old and reference log-probabilities."""
    gen = torch.Generator("cuda").manual_seed(seed)
    if layout == "rows":
        shape, cu = (6, 37), None
    else:
        cu = torch.tensor([0, 40, 40, 41, 170, 290, 300], dtype=torch.int32, device="cuda")
        shape = (310,)
    T = int(np.prod(shape))
    h, W, _, _ = inputs.make_loss_inputs(T, d, V, 1, dtype=torch.bfloat16, seed=seed, device="cuda")
    tgt = torch.randint(0, V, shape, generator=gen, device="cuda", dtype=torch.int32)
    tgt[torch.rand(shape, generator=gen, device="cuda") < 0.3] = kd.KD_TARGET_IGNORE
    base = kd.head_logprobs(h, W, tgt.reshape(-1), 64)[0].view(shape)
    noise = lambda s: base + s * torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    return h, W, tgt, cu, noise(0.2), noise(0.3), torch.randn((6,), generator=gen, device="cuda")


def _check_head(step, h, W, tgt, tau, dlogp):
    rl, _, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt.reshape(-1), tau, dlogp.reshape(-1))
    delta = 2e-3 / tau
    assert (step.logp.reshape(-1).double() - rl).abs().max() <= delta
    assert bool(((step.dH.double() - rH).abs() <= 3 * 2 ** -8 * aH + delta * pH + 1e-30).all())
    assert bool(((step.dW.double() - rW).abs() <= 2 * 2 ** -8 * aW + delta * pW + 1e-30).all())


@pytest.mark.parametrize("tau", [1.0, 0.8])
@pytest.mark.parametrize("layout", ["rows", "packed"])
def test_policy_step(layout, tau):
    require_gpu()
    h, W, tgt, cu, old, ref, adv = _batch(layout, 96, 1500, 3)
    step = posttrain.policy_step(h, W, tgt, old, adv, chunk=128, temperature=tau, ref_logp=ref, cu_seqlens=cu,
                                 kl_coef=0.05, reduction="sequence")
    assert kd.read_device_status(step.ws) == kd.KD_OK
    want = plain.policy(step.logp.cpu().numpy(), old.cpu().numpy(), adv.cpu().numpy(),
                        plain.layout(6, tgt.shape, None if cu is None else cu.cpu().numpy()),
                        mask=(tgt != kd.KD_TARGET_IGNORE).cpu().numpy(), ref=ref.cpu().numpy(), beta=0.05,
                        reduction="sequence")
    assert abs(step.loss.item() - want["loss"]) <= 2 ** -19 * want["scale_loss"]
    assert step.extra[0].item() == want["stats"][0]
    dlogp = torch.from_numpy(want["grad"]).cuda()
    _check_head(step, h, W, tgt, tau, dlogp)
    # and the clipping that ends the step
    before = [step.dH.clone(), step.dW.clone()]
    size = sum(float(g.double().square().sum()) for g in before) ** 0.5
    norm = kd.clip_grad_norm([step.dH, step.dW], size / 3)
    assert abs(norm.item() - size) <= 2 ** -22 * size
    assert bool(((step.dW - before[1] / 3).abs() <= 1e-5 * before[1].abs() + 1e-30).all())


@pytest.mark.parametrize("layout", ["rows", "packed"])
def test_preference_step(layout):
    require_gpu()
    h, W, tgt, cu, _, ref, _ = _batch(layout, 64, 900, 5)
    step = posttrain.preference_step(h, W, tgt, chunk=100, ref_logp=ref, cu_seqlens=cu, beta=0.2, label_smoothing=0.1)
    want = plain.preference(step.logp.cpu().numpy(),
                            plain.layout(6, tgt.shape, None if cu is None else cu.cpu().numpy()), ref=ref.cpu().numpy(),
                            mask=(tgt != kd.KD_TARGET_IGNORE).cpu().numpy(), beta=0.2, smoothing=0.1)
    assert abs(step.loss.item() - want["loss"]) <= 2 ** -22 * want["loss"] + 1e-12
    _check_head(step, h, W, tgt, 1.0, torch.from_numpy(want["grad"]).cuda())


def test_micro_batches_add_up():
    """Two micro-batches with the batch's token count and one dW give the batch's
    gradient (to the fp32 additions: 2^-20 of sum|dz h|)."""
    require_gpu()
    h, W, tgt, _, old, _, adv = _batch("rows", 64, 700, 7)
    n = float((tgt != kd.KD_TARGET_IGNORE).sum())
    whole = posttrain.policy_step(h, W, tgt, old, adv, chunk=32)
    dW, loss = None, 0.0
    for k in (0, 3):
        rows = slice(37 * k, 37 * (k + 3))
        part = posttrain.policy_step(h[rows], W, tgt[k:k + 3], old[k:k + 3], adv[k:k + 3], chunk=32,
                                     reduction="fixed", denom=n, dW=dW, accumulate_dW=dW is not None)
        dW, loss = part.dW, loss + part.loss.item()
        # the weights 1 / n differ by a rounding, which may move dz across one of bf16's
        assert bool(((part.dH.double() - whole.dH[rows].double()).abs()
                     <= 2 ** -7 * (whole.dH[rows].double().abs() + 1e-3)).all())
    assert loss == pytest.approx(whole.loss.item(), rel=1e-5)
    keep = tgt.reshape(-1) >= 0
    _, _, _, _, _, aW, _, _ = _plain(h, W, tgt.reshape(-1), 1.0, keep * adv.abs().repeat_interleave(37) * 2 / n)
    assert bool(((dW.double() - whole.dW.double()).abs() <= 2 ** -8 * aW + 1e-30).all())


def test_step_captured_in_a_graph():
    require_gpu()
    h, W, tgt, cu, old, ref, adv = _batch("packed", 64, 700, 9)
    # of the size that keeps nothing: the step then recomputes
    ws = kd.alloc_workspace(kd.kd_head_logprob_workspace_size(tgt.numel(), 64, 700, 64, kd.KD_DTYPE_BF16, 1), h.device)

    def run():
        s = posttrain.policy_step(h, W, tgt, old, adv, chunk=64, ref_logp=ref, cu_seqlens=cu, kl_coef=0.1, ws=ws)
        return s.loss, s.extra, s.logp, s.dH, s.dW, kd.clip_grad_norm([s.dH, s.dW], 0.01)

    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for _ in range(2):
        for x in out:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
