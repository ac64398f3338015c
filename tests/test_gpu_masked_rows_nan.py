"""Rows without a target hold whatever a trunk left there (NaN of attention over
nothing, infinities): their hidden states must not reach a gradient.

The expected values are those of the same call with zeros in these rows, bit for bit: the
rows add nothing to dW, and their rows of dH are 0.
"""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd, posttrain
from gpu_util import require_gpu
from test_gpu_head_logprob import _inputs

pytestmark = pytest.mark.gpu

JUNK = (float("nan"), float("inf"), float("-inf"), 3e38)


def _dirty(h, rows):
    """h with junk in these rows: whole rows of one value, and single places."""
    out = h.clone()
    for i, r in enumerate(rows.nonzero()[:, 0].tolist()):
        if i % 3 == 2:
            out[r, i % h.shape[1]] = JUNK[i % 4]
        else:
            out[r] = JUNK[i % 4]
    return out


# one row, less than a tile, several groups of chunks, and more tiles than clusters
SHAPES = [(2, 8, 40, 1), (300, 200, 5000, 100), (1100, 72, 1003, 300), (5000, 72, 72, 5000)]


@pytest.mark.parametrize("T,d,V,chunk", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients(T, d, V, chunk, dtype):
    require_gpu()
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=31, ignored=0.4)
    tgt[0], tgt[1] = kd.KD_TARGET_IGNORE, V - 1
    g[1] = 0.5
    rows = tgt == kd.KD_TARGET_IGNORE
    clean, dirty = torch.where(rows[:, None], torch.zeros_like(h), h), _dirty(h, rows)
    one_group = T <= 2 * max(chunk, 256)

    def run(x, keep, **kw):
        logp, lse, ws = kd.head_logprobs(x, W, tgt, chunk, 0.8, backward=True, keep=keep)
        dH, dW, _ = kd.head_logprobs_bwd(x, W, tgt, lse, g, chunk, 0.8, ws=ws, kept_logp=logp if keep else None, **kw)
        assert kd.read_device_status(ws) == kd.KD_OK
        return logp, dH, dW

    forms = [dict(keep=False), dict(keep=False, need=(True, False)), dict(keep=False, need=(False, True)),
             dict(keep=False, grad_loss=torch.tensor(-2.0, device="cuda"))]
    if one_group:
        forms.append(dict(keep=True))
        if dtype is torch.bfloat16:
            forms += [dict(keep=True, dW_dtype=torch.bfloat16), dict(keep=False, dW_dtype=torch.bfloat16)]
    for form in forms:
        want, got = run(clean, **form), run(dirty, **form)
        for a, b in zip(want, got):
            assert (a is None and b is None) or torch.equal(a, b)
        assert got[1] is None or bool((got[1][rows] == 0).all())
    base = torch.ones((V, d), device="cuda")
    a = run(clean, keep=False, dW=base.clone(), accumulate_dW=True)[2]
    assert torch.equal(a, run(dirty, keep=False, dW=base.clone(), accumulate_dW=True)[2])


def test_bad_targets_add_nothing_either():
    require_gpu()
    T, d, V = 300, 64, 700
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=32, ignored=0.0)
    tgt[7], tgt[90] = -1, V
    rows = (tgt < 0) | (tgt >= V)
    dirty = _dirty(h, rows)
    for keep in (False, True):
        logp, lse, ws = kd.head_logprobs(dirty, W, tgt, T, backward=True, keep=keep)
        dH, dW, _ = kd.head_logprobs_bwd(dirty, W, tgt, lse, g, T, ws=ws, kept_logp=logp if keep else None)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
        assert bool(torch.isfinite(dW).all()) and bool((dH[rows] == 0).all())


@pytest.mark.parametrize("chunk", [64, 512])          # recomputing, and keeping
def test_a_step_over_padded_rows(chunk):
    require_gpu()
    S, L, d, V = 8, 100, 64, 900
    h, W, tgt, _ = _inputs(S * L, d, V, torch.bfloat16, seed=33, ignored=0.5)
    rows = tgt == kd.KD_TARGET_IGNORE
    clean, dirty = torch.where(rows[:, None], torch.zeros_like(h), h), _dirty(h, rows)
    adv = torch.linspace(-1, 1, S, device="cuda")
    tgt = tgt.view(S, L)
    old = torch.full((S, L), -6.5, device="cuda")

    def policy(x):
        s = posttrain.policy_step(x, W, tgt, old, adv, chunk=chunk)
        return s.loss, s.extra, s.logp, s.dH, s.dW, kd.clip_grad_norm([s.dW], 0.01)

    def preference(x):
        s = posttrain.preference_step(x, W, tgt, chunk=chunk)
        return s.loss, s.extra, s.logp, s.dH, s.dW

    for run in (policy, preference):
        want, got = run(clean), run(dirty)
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and bool(torch.isfinite(got[4]).all())
    # captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = policy(dirty)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(policy(clean), out))


def test_autograd_form():
    require_gpu()
    T, d, V = 600, 64, 700
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=34, ignored=0.3)
    rows = tgt == kd.KD_TARGET_IGNORE
    clean, dirty = torch.where(rows[:, None], torch.zeros_like(h), h), _dirty(h, rows)
    for chunk in (64, 300):
        got = []
        for x in (clean, dirty):
            x, w = x.clone().requires_grad_(), W.clone().requires_grad_()
            out = kd.HeadLogprobs.apply(x, w, tgt, chunk)
            got.append((out, *torch.autograd.grad(out, (x, w), torch.nan_to_num(g))))
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_a_row_that_counts_keeps_its_nan():
    """A NaN where a target is stays visible: in its log-probability and in the gradients."""
    require_gpu()
    T, d, V = 70, 64, 300
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=35, ignored=0.0)
    h[5, 3] = float("nan")
    for keep in (False, True):
        logp, lse, ws = kd.head_logprobs(h, W, tgt, T, backward=True, keep=keep)
        assert bool(torch.isnan(logp[5])) and bool(torch.isfinite(logp[6:]).all())
        dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, T, ws=ws, kept_logp=logp if keep else None)
        assert bool(torch.isnan(dH[5]).any()) and bool(torch.isfinite(dH[6:]).all()) and bool(torch.isnan(dW).any())
