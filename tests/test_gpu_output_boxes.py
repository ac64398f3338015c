"""Outputs of GEMMs whose tiles have an odd number of 32-column boxes while a
cluster works on several tiles: the boxes of consecutive tiles must not be
overwritten while they are still read.

Each form is compared with a plain fp64 form, with the tolerances of the head's
parity tests (every dz entry rounded once to the operands' type, twice where the
forward keeps its exponentials; the logits' error times the probabilities), and is
run five times for the same bits.
"""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs, _plain

pytestmark = pytest.mark.gpu


def _same_bits(run, times=5):
    first = [x.clone() for x in run()]
    for _ in range(times - 1):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
    return first


def _near(got, want, mass, prob, roundings, delta):
    assert bool(((got.double() - want).abs() <= roundings * 2 ** -8 * mass + delta * prob + 1e-30).all())


@pytest.mark.parametrize("d", [72, 200])
def test_head_gradient_of_a_tall_head(d):
    """dW [60000, d]: 235 tiles of 3 or 7 boxes over 74 clusters."""
    require_gpu()
    T, V, chunk = 64, 60000, 64
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=21)
    _, lse, _ = kd.head_logprobs(h, W, tgt, chunk)
    rl, rlse, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt, 1.0, torch.where(tgt >= 0, g, 0.0))
    delta = 2e-3

    def run(**kw):
        return kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, **kw)[:2]

    dH, dW = _same_bits(run)
    _near(dH, rH, aH, pH, 2, delta)
    _near(dW, rW, aW, pW, 1, delta)
    _, w16 = _same_bits(lambda: run(dW_dtype=torch.bfloat16))
    assert torch.equal(w16, dW.to(torch.bfloat16))
    twice = _same_bits(lambda: run(dW=dW.clone(), accumulate_dW=True))[1]
    assert torch.equal(twice, 2 * dW)                  # a sum of two equal values is exact


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_positions_over_a_narrow_head(dtype):
    """20000 x 72 x 72: 79 row tiles of 3 boxes in the kept forward, dz and dH."""
    require_gpu()
    T, d, V, chunk = 20000, 72, 72, 20000
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=22)
    g = torch.where(tgt >= 0, g, 0.0)
    rl, rlse, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt, 1.0, g)
    delta = 1e-2 if dtype is torch.float32 else 2e-3

    def recomputed():
        logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, backward=True)
        return (logp, *kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws)[:2])

    def kept():
        logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
        return (logp, *kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)[:2])

    for run, more in ((recomputed, 0), (kept, 1)):
        logp, dH, dW = _same_bits(run)
        assert (logp.double() - rl).abs().max() <= delta
        _near(dH, rH, aH, pH, 2 + more, delta)
        _near(dW, rW, aW, pW, 1 + more, delta)


@pytest.mark.parametrize("T,d,V", [(64, 72, 60000), (20000, 72, 72)])
def test_distillation_loss_gradients(T, d, V):
    """The same shapes through the KL loss; plain fp64 form of its gradient."""
    require_gpu()
    K = 5
    h, W, vals, idx = inputs.make_loss_inputs(T, d, V, K, dtype=torch.bfloat16, seed=23, device="cuda")
    loss, lse, _, ws = kd.fused_kl_fwd(h, W, vals, idx, T)
    dH, dW = _same_bits(lambda: kd.fused_kl_bwd(h, W, vals, idx, lse, T, ws=ws)[:2])
    assert kd.read_device_status(ws) == kd.KD_OK
    hd, Wd = h.double(), W.double()
    a = hd @ Wd.t()
    p = torch.softmax(vals.double(), dim=1)
    dz = torch.softmax(a, dim=1)
    soft = dz / T
    dz = (dz.scatter_add(1, idx.long(), -p)) / T
    _near(dH, dz @ Wd, dz.abs() @ Wd.abs(), soft @ Wd.abs(), 2, 2e-3)
    _near(dW, dz.t() @ hd, dz.abs().t() @ hd.abs(), soft.t() @ hd.abs(), 1, 2e-3)
