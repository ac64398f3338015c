"""GPU parity of the global gradient norm and clipping against fp64.

Tolerances: at most 8 squares are added in fp32, with as many roundings of
2^-24 of a sum of positive terms, and the rest in fp64: 2^-21 of the sum of
squares, half of it of the norm, which is rounded to fp32 once (2^-24); together
below 2^-21 (NORM).  The factor has the norm's error and a rounding, a product one
more: below 2^-20 of an fp32 value; a bf16 one is rounded to half a step, 2^-8,
besides.
"""

import math

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NORM = 2.0 ** -21


def _values(n, dtype, gen, scale=1.0):
    return torch.randn((n,), generator=gen, device="cuda").mul_(scale).to(dtype)


def _check(got, src, c):
    want = src.double() * c
    tol = 2.0 ** -20 + (2.0 ** -8 if src.dtype is BF16 else 0.0)
    assert got.dtype == src.dtype and got.shape == src.shape
    assert bool(((got.double() - want).abs() <= tol * want.abs() + 1e-40).all())


def _norm(tensors):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in tensors))


LISTS = {
    "one-value": [(1, F32)],
    "with-empties": [(0, F32), (5, BF16), (0, BF16), (33, F32)],
    "around-a-unit": [(8191, F32), (8192, F32), (8193, F32), (16384, BF16), (16383, BF16), (40000, BF16)],
    "mixed": [(7, BF16), (100003, F32), (1, BF16), (65537, BF16), (3, F32), (2 << 20, F32)],
    "many": [(1 + (k * 37) % 300, F32 if k % 3 else BF16) for k in range(2500)],
    "exactly-100": [(k + 1, F32) for k in range(100)],
    "exactly-1001": [(2, BF16) for k in range(1001)],
    "many-blocks": [(30 << 20, BF16), (11 << 20, F32)],
}


@pytest.mark.parametrize("where", ["in-place", "out", "out-at-odd-places"])
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clipping(name, where):
    """Tensors that are views into one buffer per type, one after the other with
    gaps of one element: nothing between them is written."""
    require_gpu()
    gen = torch.Generator("cuda").manual_seed(len(name))
    spec = LISTS[name]
    flat, at, grads, marks = {}, {F32: 3, BF16: 5}, [], {}
    for dt in (F32, BF16):
        flat[dt] = _values(sum(n + 1 for n, d in spec if d == dt) + 16, dt, gen)
        marks[dt] = torch.ones_like(flat[dt], dtype=torch.bool)
    for n, dt in spec:
        grads.append(flat[dt][at[dt]:at[dt] + n])
        marks[dt][at[dt]:at[dt] + n] = False
        at[dt] += n + 1
    src = [t.clone() for t in grads]
    before = {dt: flat[dt].clone() for dt in flat}
    want = _norm(src)
    for max_norm in (0.25 * want, 4.0 * want, math.inf, 0.0):
        for dt in flat:
            flat[dt].copy_(before[dt])
        c = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (want + 1e-6))
        if where == "in-place":
            norm, outs = kd.clip_grad_norm(grads, max_norm), grads
        else:
            shift = 0 if where == "out" else 1
            pads = [torch.full((t.numel() + 3,), 7.0, dtype=t.dtype, device="cuda") for t in grads]
            outs = [p[shift:shift + t.numel()] for p, t in zip(pads, grads)]
            norm = kd.clip_grad_norm(grads, max_norm, out=outs)
            for p, t in zip(pads, grads):
                assert bool((p[:shift] == 7).all()) and bool((p[shift + t.numel():] == 7).all())
        assert abs(norm.item() - want) <= NORM * want
        for g, s in zip(outs[:300], src[:300]):
            _check(g, s, c)
            if c == 1.0:
                assert torch.equal(g, s)
        for dt in flat:
            keep = marks[dt] if where == "in-place" else torch.ones_like(marks[dt])
            assert torch.equal(flat[dt][keep], before[dt][keep])
    total = kd.grad_sumsq([s for s in src])
    assert abs(total.item() - want * want) <= 2.0 ** -21 * want * want


def test_values_whose_squares_leave_fp32():
    require_gpu()
    for scale in (1e30, 1e-30, 3e18, 3e-16, 1e-22):
        g = [torch.full((1000,), scale, device="cuda"), torch.full((5,), 2 * scale, device="cuda", dtype=BF16)]
        want = _norm(g)
        assert 0 < want < 1e33
        mixed = [torch.tensor([scale, 1.0, 0.0, -scale, 0.0, 0.0, 0.0, 0.0, 1e-38], device="cuda")]
        assert abs(kd.clip_grad_norm(mixed, math.inf).item() - _norm(mixed)) <= NORM * _norm(mixed)
        norm = kd.clip_grad_norm(g, 1.0)
        assert abs(norm.item() - want) <= NORM * want
        assert abs(g[0][3].item() - scale * min(1.0, 1.0 / (want + 1e-6))) <= 2.0 ** -19 * abs(g[0][3].item())


def test_infinities_and_nan_follow_the_formula():
    require_gpu()
    g = [torch.tensor([1.0, math.inf, -2.0], device="cuda"), torch.ones(4, device="cuda", dtype=BF16)]
    assert kd.clip_grad_norm(g, 1.0).item() == math.inf
    assert g[0].tolist()[0] == 0 and math.isnan(g[0].tolist()[1]) and bool((g[1] == 0).all())
    g = [torch.tensor([1.0, math.nan], device="cuda"), torch.ones(4, device="cuda")]
    assert math.isnan(kd.clip_grad_norm(g, 1.0).item()) and bool(g[1].isnan().all())
    g = [torch.zeros(9, device="cuda")]
    assert kd.clip_grad_norm(g, 1.0).item() == 0 and bool((g[0] == 0).all())


def test_offsets_past_32_bits():
    require_gpu()
    n = (1 << 31) + 77
    g = torch.full((n,), 0.5, dtype=BF16, device="cuda")
    g[-1] = 2.0
    want = math.sqrt((n - 1) * 0.25 + 4.0)
    norm = kd.clip_grad_norm([g], want / 2)
    assert abs(norm.item() - want) <= NORM * want
    assert g[-1].item() == 1.0 and g[-2].item() == 0.25 and g[0].item() == 0.25
    assert g.sum(dtype=torch.float64).item() == (n - 1) * 0.25 + 1.0


def test_same_bits_every_time_and_given_sum():
    require_gpu()
    gen = torch.Generator("cuda").manual_seed(2)
    src = [_values(n, F32, gen) for n in (100000, 3, 7 << 20)]
    outs = [[torch.empty_like(t) for t in src] for _ in range(2)]
    norms = [kd.clip_grad_norm(src, 1.0, out=o) for o in outs]
    assert torch.equal(norms[0], norms[1])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    # a list in two parts, each scaled by the norm of both
    total = kd.grad_sumsq(src[:1]) + kd.grad_sumsq(src[1:])
    part = [t.clone() for t in src]
    kd.clip_grad_norm(part[:1], 1.0, sumsq=total)
    norm = kd.clip_grad_norm(part[1:], 1.0, sumsq=total)
    assert abs(norm.item() - norms[0].item()) <= 2 * NORM * norm.item()
    for a, b in zip(part, outs[0]):
        assert bool(((a - b).abs() <= 2.0 ** -19 * b.abs()).all())


def test_captured_replay_and_another_stream():
    require_gpu()
    gen = torch.Generator("cuda").manual_seed(3)
    g = [_values(n, dt, gen) for n, dt in ((50000, F32), (123, BF16), (1 << 20, F32))]
    graph = torch.cuda.CUDAGraph()
    kd.clip_grad_norm([t.clone() for t in g], 1.0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = kd.clip_grad_norm(g, 1.0)
    for seed in (4, 5):
        gen = torch.Generator("cuda").manual_seed(seed)
        new = [_values(t.numel(), t.dtype, gen, 3.0) for t in g]
        for a, b in zip(g, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        want = kd.clip_grad_norm(new, 1.0, stream=side)
        side.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(g, new))


def test_refusals():
    require_gpu()
    a, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    for bad in ([], [a.half()], [None], [a, b.cpu()], [torch.ones(8, 8, device="cuda").t()[:3]]):
        with pytest.raises((TypeError, ValueError)):
            kd.clip_grad_norm(bad, 1.0)
    with pytest.raises(kd.KDError):
        kd.clip_grad_norm([a, b], -1.0)
    with pytest.raises(kd.KDError):
        kd.clip_grad_norm([a, b], math.nan)
    for clash in ([a, a], [a, a[10:20]], [a[:33], a[32:]]):              # written twice
        with pytest.raises(kd.KDError):
            kd.clip_grad_norm(clash, 1.0)
    with pytest.raises(kd.KDError):
        kd.clip_grad_norm([a, b], 1.0, out=[b, a])                       # written while read
    for out in ([a], [a, b[:63]], [a, b.bfloat16()]):
        with pytest.raises((TypeError, ValueError)):
            kd.clip_grad_norm([a, b], 1.0, out=out)
    with pytest.raises(TypeError):
        kd.clip_grad_norm([a], 1.0, sumsq=torch.zeros((), device="cuda"))
    c = torch.empty_like(a)
    assert kd.clip_grad_norm([a, a], math.inf, out=[b, c]).item() == pytest.approx(math.sqrt(128))   # read twice is fine
    assert bool((a == 1).all())
