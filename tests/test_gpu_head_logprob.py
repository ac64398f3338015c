"""GPU parity of the head's log-probabilities (kd_head_logprob_fwd / _bwd)
against a plain fp64 form.

Tolerances:
  * logp and lse, bf16 operands: the products are exact in fp32 and the d terms
    are added in fp32, so |z| errs by at most d 2^-24 sum|h w| <= about 1e-4
    for d <= 4096 and unit-variance logits; 1e-3 is the bar of the KL loss's lse.
    fp32 operands are read as tf32 (2^-11 relative each): 5e-3, the same bar.
  * dH, dW: each dz entry is rounded once to bf16 (2^-9 relative; tf32 2^-11)
    and a bf16 gradient once more (2^-9): every entry errs by at most
    2^-9 sum|dz w| + 2^-9 |dH|, held here to 2^-8 of the row's sum|dz w|
    (dH) or the column's sum|dz h| (dW).  The logits' own error delta adds
    |g| p (e^delta - 1) to a dz entry g ([v == y] - p): it scales with p alone,
    also where p and [v == y] cancel (p near 1, V == 1), so that term is held
    to 2 delta of the sum over |g| p |w|, not over |dz| |w|.
"""

import numpy as np
import pytest
import torch

from chunked_kl_loss_chunk_b200 import inputs, kd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _plain(h, W, targets, tau, g=None):
    """fp64: logp, lse and, with g, dH, dW and the four sums that the
    tolerances are relative to: |dz||W|, |dz||h|, |g|p|W|, |g|p|h|."""
    h, W = h.detach().double(), W.detach().double()
    a = h @ W.t() / tau
    lse = torch.logsumexp(a, dim=1)
    keep = (targets >= 0) & (targets < W.shape[0])
    y = torch.where(keep, targets, 0).long()
    logp = torch.where(keep, a.gather(1, y[:, None])[:, 0] - lse, 0.0)
    if g is None:
        return logp, lse
    g = torch.where(keep, g.double(), 0.0)[:, None] / tau
    dz = -g * torch.exp(a - lse[:, None])
    gp = dz.abs()
    dz.scatter_add_(1, y[:, None], g)
    return (logp, lse, dz @ W, dz.t() @ h, dz.abs() @ W.abs(), dz.abs().t() @ h.abs(),
            gp @ W.abs(), gp.t() @ h.abs())


def _inputs(T, d, V, dtype, seed, ignored=0.25):
    h, W, _, _ = inputs.make_loss_inputs(T, d, V, 1, dtype=dtype, seed=seed, device="cuda")
    gen = torch.Generator("cuda").manual_seed(seed + 77)
    tgt = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    skip = torch.rand((T,), generator=gen, device="cuda") < ignored
    tgt = torch.where(skip, torch.full_like(tgt, kd.KD_TARGET_IGNORE), tgt)
    g = torch.randn((T,), generator=gen, device="cuda")
    return h, W, tgt, torch.where(skip, torch.full_like(g, float("nan")), g)


SHAPES = [
    (1, 8, 40, 1, torch.bfloat16),
    (300, 200, 5000, 100, torch.bfloat16),
    (77, 72, 1003, 33, torch.float32),
    (129, 64, 257, 4096, torch.bfloat16),
    (5, 4104, 513, 2, torch.bfloat16),
    (600, 128, 2304, 256, torch.float32),
    (1100, 72, 1003, 300, torch.bfloat16),
    (40, 64, 1, 16, torch.bfloat16),
]


@pytest.mark.parametrize("T,d,V,chunk,dtype", SHAPES)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_forward_and_gradients(T, d, V, chunk, dtype, tau):
    require_gpu()
    h, W, tgt, g = _inputs(T, d, V, dtype, seed=T + d)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, tau, backward=True)
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, tau, ws=ws)
    torch.cuda.synchronize()
    assert kd.read_device_status(ws) == kd.KD_OK
    rl, rlse, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt, tau, torch.where(tgt >= 0, g, 0.0))
    tol = 5e-3 if dtype == torch.float32 else 1e-3
    assert (lse.double() - rlse).abs().max() <= tol / tau
    assert (logp.double() - rl).abs().max() <= 2 * tol / tau
    assert bool((logp[tgt < 0] == 0).all())
    eps, delta = 2 ** -8, 2 * tol / tau
    assert bool(((dH.double() - rH).abs() <= 2 * eps * aH + delta * pH + 1e-30).all())
    assert bool(((dW.double() - rW).abs() <= eps * aW + delta * pW + 1e-30).all())
    assert bool((dH[tgt < 0] == 0).all())
    if T <= 2 * max(chunk, 256):
        # the forward keeps its exponentials: the same logp, one rounding more in dz
        kl, klse, kws = kd.head_logprobs(h, W, tgt, chunk, tau, keep=True)
        assert torch.equal(kl, logp) and torch.equal(klse, lse)
        kH, kW, _ = kd.head_logprobs_bwd(h, W, tgt, klse, g, chunk, tau, ws=kws, kept_logp=kl)
        assert kd.read_device_status(kws) == kd.KD_OK
        assert bool(((kH.double() - rH).abs() <= 3 * eps * aH + delta * pH + 1e-30).all())
        assert bool(((kW.double() - rW).abs() <= 2 * eps * aW + delta * pW + 1e-30).all())
        assert bool((kH[tgt < 0] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_kept_exponentials_of_confident_rows(dtype):
    """Rows that give their target nearly all the mass, or none, logits that are far
    apart, and a head with a ragged last block: the target's entry keeps its digits."""
    require_gpu()
    T, d, V, chunk = 96, 64, 1003, 64
    gen = torch.Generator("cuda").manual_seed(4)
    W = torch.randn((V, d), generator=gen, device="cuda").to(dtype)
    tgt = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    tgt[:4] = torch.tensor([0, V - 1, 31, 32], device="cuda")
    h = W[tgt.long()].float()
    h[1::2] *= 0.15
    h[2::4] *= -1.0
    h = h.to(dtype)
    g = torch.randn((T,), generator=gen, device="cuda")
    logp, lse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
    assert logp.max().item() > -1e-3 and logp.min().item() < -50
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, ws=ws, kept_logp=logp)
    rl, rlse, rH, rW, aH, aW, pH, pW = _plain(h, W, tgt, 1.0, g)
    # logits up to about 100: d 2^-24 sum|h w| of them, below 4e-4 (tf32: 2^-10 of sum|h w|, 0.2)
    delta = 4e-4 if dtype is torch.bfloat16 else 0.3
    assert bool(((dH.double() - rH).abs() <= 3 * 2 ** -8 * aH + 2 * delta * pH + 1e-30).all())
    assert bool(((dW.double() - rW).abs() <= 2 * 2 ** -8 * aW + 2 * delta * pW + 1e-30).all())


def test_every_row_ignored():
    require_gpu()
    h, W, tgt, g = _inputs(50, 64, 300, torch.bfloat16, seed=3)
    tgt.fill_(kd.KD_TARGET_IGNORE)
    logp, lse, ws = kd.head_logprobs(h, W, tgt, 32, backward=True)
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, 32, ws=ws)
    assert kd.read_device_status(ws) == kd.KD_OK
    for x in (logp, dH, dW):
        assert bool((x == 0).all())


def test_chunk_invariance_and_forward_workspace():
    """logp and lse are bit-identical for every chunk; the forward alone fits a
    workspace without the backward's dz."""
    require_gpu()
    T, d, V = 333, 128, 4000
    h, W, tgt, _ = _inputs(T, d, V, torch.bfloat16, seed=5)
    a = kd.head_logprobs(h, W, tgt, 64)
    b = kd.head_logprobs(h, W, tgt, 333, backward=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert a[2].numel() < b[2].numel()


def test_bad_target_is_reported():
    require_gpu()
    for bad in (300, -1, -2 ** 31, 2 ** 31 - 1):
        h, W, tgt, g = _inputs(50, 64, 300, torch.bfloat16, seed=4)
        tgt[17] = bad
        _, lse, ws = kd.head_logprobs(h, W, tgt, 32, backward=True)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
        kd.head_logprobs_bwd(h, W, tgt, lse, g, 32, ws=ws)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX


def test_gradient_against_differences():
    """grad_logp . logp along a direction of h, by central differences of the
    fp64 form, against the kernel's dH."""
    require_gpu()
    T, d, V = 64, 96, 700
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=9, ignored=0.0)
    _, lse, _ = kd.head_logprobs(h, W, tgt, 64)
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, 64)
    gen = torch.Generator("cuda").manual_seed(1)
    u = torch.randn((T, d), generator=gen, device="cuda", dtype=torch.float64)
    v = torch.randn((V, d), generator=gen, device="cuda", dtype=torch.float64)
    f = lambda e: (g.double() * _plain(h.double() + e * u, W.double() + e * v, tgt, 1.0)[0]).sum()  # noqa: E731
    diff = ((f(1e-4) - f(-1e-4)) / 2e-4).item()
    _, _, _, _, aH, aW, _, _ = _plain(h, W, tgt, 1.0, g)
    got = ((dH.double() * u).sum() + (dW.double() * v).sum()).item()
    # independent rounding errors of at most 2^-7 of each entry's terms add up as a random walk
    scale = (((aH * u).square().sum() + (aW * v).square().sum()).sqrt() * 2 ** -7).item()
    assert abs(got - diff) <= 4 * scale


def test_autograd_frozen_head_and_accumulation():
    require_gpu()
    T, d, V = 530, 64, 900
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=11, ignored=0.0)
    _, lse, _ = kd.head_logprobs(h, W, tgt, 48)
    dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, 48)
    hl, Wl = h.clone().requires_grad_(), W.clone().requires_grad_()
    # (530 positions in chunks of 48, taken as 256, are more than two chunks: recomputed)
    gh, gw = torch.autograd.grad(kd.HeadLogprobs.apply(hl, Wl, tgt, 48, 1.0), (hl, Wl), g)
    assert torch.equal(gh, dH) and torch.equal(gw, dW.to(torch.bfloat16))
    # formed in one go, dW leaves the kernel in bf16: the rounding of the fp32 one
    for chunk in (265, 530, 1000):
        _, w32, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk)
        _, w16, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk, dW_dtype=torch.bfloat16)
        assert w16.dtype is torch.bfloat16 and torch.equal(w16, w32.to(torch.bfloat16))
        kept, klse, ws = kd.head_logprobs(h, W, tgt, chunk, keep=True)
        kH, kW, _ = kd.head_logprobs_bwd(h, W, tgt, klse, g, chunk, ws=ws, kept_logp=kept, dW_dtype=torch.bfloat16)
        out = kd.HeadLogprobs.apply(hl, Wl, tgt, chunk, 1.0)
        gh, gw = torch.autograd.grad(out, (hl, Wl), g, retain_graph=True)
        assert torch.equal(gh, kH) and torch.equal(gw, kW)
        # what was kept is used up: a second backward recomputes
        gh, gw = torch.autograd.grad(out, (hl, Wl), g)
        assert torch.equal(gh, kd.head_logprobs_bwd(h, W, tgt, lse, g, chunk)[0])
        assert torch.equal(gw, w16)
    with pytest.raises(kd.KDError):
        kd.head_logprobs_bwd(h, W, tgt, lse, g, 64, dW_dtype=torch.bfloat16)
    with torch.no_grad():
        plain = kd.HeadLogprobs.apply(hl, Wl, tgt, 530)
    assert not plain.requires_grad and torch.equal(plain, kd.head_logprobs(h, W, tgt, 530)[0])
    hf = h.clone().requires_grad_()
    (only,) = torch.autograd.grad(kd.HeadLogprobs.apply(hf, W, tgt, 48, 1.0), (hf,), g)
    assert torch.equal(only, dH)
    none, w2, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, 48, need=(False, True))
    assert none is None and torch.equal(w2, dW)
    two = torch.tensor(2.0, device="cuda")
    acc = dW.clone()
    kd.head_logprobs_bwd(h, W, tgt, lse, g, 48, grad_loss=two, dW=acc, accumulate_dW=True)
    # two groups of chunks are added in fp32, in both calls: at most four roundings of 2^-24 of
    # partial sums that are at most 3 sum|dz h| (they may cancel in the result)
    aW = _plain(h, W, tgt, 1.0, g)[5]
    assert bool(((acc.double() - 3 * dW.double()).abs() <= 12 * 2 ** -24 * aW + 1e-30).all())


def test_other_stream_and_captured_replay():
    require_gpu()
    T, d, V = 200, 64, 1500
    h, W, tgt, g = _inputs(T, d, V, torch.bfloat16, seed=13, ignored=0.1)
    want = kd.head_logprobs(h, W, tgt, 64)
    wH, wW, _ = kd.head_logprobs_bwd(h, W, tgt, want[1], g, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kd.head_logprobs(h, W, tgt, 64, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logp, lse, _ = kd.head_logprobs(h, W, tgt, 64)
        dH, dW, _ = kd.head_logprobs_bwd(h, W, tgt, lse, g, 64)
    for _ in range(2):
        logp.zero_(), dH.zero_(), dW.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logp, want[0]) and torch.equal(dH, wH) and torch.equal(dW, wW)


def test_refusals():
    require_gpu()
    h, W, tgt, g = _inputs(16, 64, 100, torch.bfloat16, seed=1)
    lse = torch.zeros(16, device="cuda")
    with pytest.raises(TypeError):
        kd.head_logprobs(h, W, tgt.long(), 8)
    with pytest.raises(TypeError):
        kd.head_logprobs(h, W.float(), tgt, 8)
    with pytest.raises(TypeError):
        kd.head_logprobs(h.half(), W.half(), tgt, 8)
    with pytest.raises(ValueError):
        kd.head_logprobs(h[:, ::2], W[:, ::2], tgt, 8)
    with pytest.raises(ValueError):
        kd.head_logprobs(h, W, tgt[:15], 8)
    with pytest.raises(ValueError):
        kd.head_logprobs(h, W, tgt.cpu(), 8)
    with pytest.raises(kd.KDError):
        kd.head_logprobs(h, W, tgt, 0)
    with pytest.raises(kd.KDError):
        kd.head_logprobs(h, W, tgt, 8, temperature=0.0)
    with pytest.raises(kd.KDError):
        kd.head_logprobs(h, W, tgt, 8, ws=kd.alloc_workspace(1024, h.device))
    with pytest.raises(ValueError):
        kd.head_logprobs_bwd(h, W, tgt, lse, g, 8, accumulate_dW=True)
    with pytest.raises(ValueError):
        kd.head_logprobs_bwd(h, W, tgt, lse, g, 8, need=(False, False))
    with pytest.raises(ValueError):
        kd.head_logprobs_bwd(h, W, tgt, lse, g, 8, kept_logp=lse)
    h2, W2, tgt2, _ = _inputs(513, 64, 100, torch.bfloat16, seed=1)
    with pytest.raises(kd.KDError):
        kd.head_logprobs(h2, W2, tgt2, 256, keep=True)                   # more than two chunks
    with pytest.raises(kd.KDError):
        kd.head_logprobs(h, W, tgt, 8, keep=True, ws=kd.head_logprobs(h, W, tgt, 8, backward=True)[2])
    with pytest.raises(TypeError):
        kd.head_logprobs_bwd(h, W, tgt, lse, g.double(), 8)
