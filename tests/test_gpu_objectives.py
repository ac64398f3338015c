"""GPU parity of the policy and preference losses against plain fp64 forms.

Tolerances.  Policy loss: a token's terms A r, beta k and beta (1 - e^q) are
computed in fp32 from d and q, which are rounded once (2^-24 |d|, so a factor
1 + |d| of relative error 2^-24 in r), with expf (2 ulp, 2^-23), at most four
roundings in products and sums, and the weight (two roundings): below 16
half-steps of 2^-24 of the sum of the magnitudes, held to 2^-19.  The loss adds
four terms at a time in fp32 (within the same 2^-19) and the rest in fp64.
Preference loss: the sums are exact to fp64 (2^-45 of the magnitudes' sum is
allowed for sums of up to 2^8 roundings), each output is rounded to fp32 once
or twice: 2^-22 of the value; the sums' error reaches rewards times beta, and
loss and gradient through the forms' slopes (at most 1 for beta D, 2 beta-free
for the squared form times the distance).
"""

import numpy as np
import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd
from gpu_util import require_gpu
import objective_plain as plain

pytestmark = pytest.mark.gpu

# name: (lengths of packed sequences, tokens before the first and behind the last) or (S, L)
LAYOUTS = {
    "one-token": (1, 1),
    "rows-of-1": (6, 1),
    "rows-of-3": (10, 3),
    "rows-of-129": (4, 129),
    "rows-of-1000": (40, 1000),             # more than one block
    "rows-of-1-many": (20000, 1),
    "row-of-50001": (2, 50001),
    "packed-small": ([3, 0, 1, 128, 0, 0, 77, 5], 0, 0),
    "packed-empty-ends": ([0, 0, 9, 300, 0, 0], 5, 11),
    "packed-all-empty": ([0, 0], 7, 3),
    "packed-long": ([1, 20000, 0, 3, 2, 1, 9000, 64, 0, 130], 3, 4097),
    "packed-many-short": (list(range(9)) * 700, 0, 2),
    "rows-of-1-2048": (2048, 1),
    "rows-of-7": (900, 7),
    "packed-short": ([(k * 7) % 4 for k in range(1501)] + [2], 1, 1),
    "packed-short-among-long": ([1, 2, 0, 3, 500, 1, 1, 1, 0, 0, 2, 700] * 30, 2, 3),
    "packed-many-empty": ([0] * 700 + [5] + [0] * 2000 + [9000, 0, 0, 1] * 2, 0, 0),
    "packed-128s": ([128, 256, 0, 128, 384, 128] * 30, 128, 0),
}


def _make(name, seed, masked):
    spec = LAYOUTS[name]
    rng = np.random.default_rng(seed)
    if len(spec) == 2:
        S, L = spec
        shape, cu = (S, L), None
    else:
        lens, before, behind = spec
        S = len(lens)
        cu = (before + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        shape = (int(cu[-1]) + behind,)
    N = int(np.prod(shape))
    logp = -rng.exponential(1.0, N).astype(np.float32)
    old = (logp + rng.normal(0, 0.2, N)).astype(np.float32)
    ref = (logp + rng.normal(0, 0.3, N) * (rng.random(N) < 0.9)).astype(np.float32)
    mask = None
    ranges = plain.layout(S, shape, cu)
    outside = np.ones(N, bool)
    for a, b in ranges:
        outside[a:b] = False
    if masked:
        mask = rng.random(N) < 0.6
        for b in (0, S - 1):
            if S > 2:
                mask[ranges[b][0]:ranges[b][1]] = False       # sequences that the mask leaves empty
        outside |= ~mask
    for k, x in enumerate((logp, old, ref)):                  # never used there
        x[outside] = rng.choice([np.nan, np.inf, -np.inf, np.finfo(np.float32).min], outside.sum())
    t = lambda x: torch.from_numpy(x.reshape(shape)).cuda()  # noqa: E731
    return dict(S=S, N=N, shape=shape, ranges=ranges, logp=t(logp), old=t(old), ref=t(ref),
                mask=None if mask is None else t(mask),
                cu=None if cu is None else torch.from_numpy(cu).cuda(),
                adv=torch.from_numpy(rng.normal(0, 1, S).astype(np.float32)).cuda(),
                adv_tok=t(np.where(outside, np.nan, rng.normal(0, 1, N)).astype(np.float32)),
                np=dict(logp=logp, old=old, ref=ref, mask=mask))


def _odd_pairs(name):
    spec = LAYOUTS[name]
    return (spec[0] if len(spec) == 2 else len(spec[0])) % 2 == 1


VARIANTS = [
    dict(reduction="token"),
    dict(reduction="token", use_ref=True, kl_coef=0.05, clip_low=0.1, clip_high=0.28),
    dict(reduction="sequence", use_ref=True, kl_coef=0.2),
    dict(reduction="sequence", per_token=True, no_old=True),
    dict(reduction="fixed", denom=123.5, per_token=True, use_ref=True),
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("name", LAYOUTS)
def test_policy_loss(name, masked):
    require_gpu()
    x = _make(name, 5, masked)
    for v in VARIANTS:
        v = dict(v)
        use_ref, per_token, no_old = v.pop("use_ref", 0), v.pop("per_token", 0), v.pop("no_old", 0)
        adv = x["adv_tok"] if per_token else x["adv"]
        ws = kd.alloc_workspace(kd.kd_policy_loss_workspace_size(x["S"], x["N"]), "cuda")
        kw = dict(mask=x["mask"], ref_logp=x["ref"] if use_ref else None, cu_seqlens=x["cu"],
                  advantages_per="token" if per_token else "sequence", ws=ws, **v)
        old = None if no_old else x["old"]
        loss, stats, g = kd.policy_loss(x["logp"], old, adv, **kw)
        assert kd.read_device_status(ws) == kd.KD_OK
        want = plain.policy(x["np"]["logp"], None if no_old else x["np"]["old"], adv.cpu().numpy(), x["ranges"],
                            mask=x["np"]["mask"], ref=x["np"]["ref"] if use_ref else None, per_token=per_token,
                            lo=v.get("clip_low", 0.2), hi=v.get("clip_high", 0.2), beta=v.get("kl_coef", 0.0),
                            reduction=v["reduction"], denom=v.get("denom"))
        tol = 2.0 ** -19
        gn = g.double().cpu().numpy().reshape(-1)
        assert np.all(np.abs(gn - want["grad"]) <= tol * want["scale"] + 1e-37), (v, np.abs(gn - want["grad"]).max())
        assert abs(loss.item() - want["loss"]) <= tol * want["scale_loss"] + 1e-37, (v, loss.item(), want["loss"])
        st = stats.double().cpu().numpy()
        assert st[0] == want["stats"][0]
        assert abs(st[2] - want["stats"][2]) <= 2.0 ** -23 * want["stats"][2]
        assert abs(st[1] - want["stats"][1]) <= tol * 4 * want["stats"][1]     # 1 + |d| below 4 here
        if use_ref:
            assert abs(st[3] - want["stats"][3]) <= tol * 4 * want["stats"][3] + 1e-37
        else:
            assert st[3] == 0
        # the loss alone, and the same call again: the same bits
        loss2, stats2, none = kd.policy_loss(x["logp"], old, adv, **{**kw, "grad": False})
        assert none is None and torch.equal(loss2, loss) and torch.equal(stats2, stats)
        assert torch.equal(kd.policy_loss(x["logp"], old, adv, **kw)[2], g)


@pytest.mark.parametrize("n", [5, 5000])
def test_a_reference_that_holds_tokens_impossible(n):
    """ref_logp very low or -inf: the KL term grows without bound, its gradient is beta (1 - e^q)
    all the same, here w beta to one rounding each of beta, 1 - e^q and the product
    (e^q < 2^-24), and of the weight: 2^-22."""
    require_gpu()
    low = [-np.inf, float(np.finfo(np.float32).min), -1e9, -1e5, -3000.0, -200.0, -40.0]
    logp = torch.full((n, 1), -0.5, device="cuda")
    ref = torch.tensor([low[i % len(low)] for i in range(n)], device="cuda").reshape(n, 1)
    loss, stats, g = kd.policy_loss(logp, None, torch.zeros(n, device="cuda"), ref_logp=ref, kl_coef=0.25,
                                    reduction="fixed", denom=8.0)
    assert loss.item() == np.inf and stats[3].item() == np.inf
    assert torch.all((g.double() - 0.25 / 8).abs() <= 2.0 ** -22 * 0.25 / 8)


@pytest.mark.parametrize("n", [4, 4000])
def test_a_nan_advantage_is_not_clipped(n):
    """The clamp belongs to advantages above and below 0: a NaN reaches loss and gradient, as the
    formula says, and only its own token's."""
    require_gpu()
    logp = torch.full((n, 1), -1.0, device="cuda")
    old = logp + 2.0 * (1 - 2 * (torch.arange(n, device="cuda") % 2)).reshape(n, 1)      # r = e^-2, e^2
    adv = torch.where(torch.arange(n, device="cuda") < n // 2, torch.nan, 0.0)
    loss, stats, g = kd.policy_loss(logp, old, adv)
    assert torch.isnan(loss) and stats[2].item() == 0
    assert torch.equal(torch.isnan(g).flatten(), torch.isnan(adv)) and torch.all(g[n // 2:] == 0)


@pytest.mark.parametrize("pairs", [1, 700])
def test_an_impossible_rejected_answer(pairs):
    """z = +inf: -log sigmoid(z) is 0, and so are the slope and, without label smoothing, the loss;
    with it the loss is infinite."""
    require_gpu()
    logp = torch.full((2 * pairs, 2), -1.0, device="cuda")
    logp[pairs:, 1] = -torch.inf
    loss, rewards, g = kd.preference_loss(logp)
    assert loss.item() == 0 and torch.all(g == 0) and torch.all(rewards[pairs:] == -torch.inf)
    loss, _, g = kd.preference_loss(logp, label_smoothing=0.25, beta=0.5)
    assert loss.item() == np.inf
    assert torch.all(((g[:pairs].double() * pairs) - 0.125).abs() <= 2.0 ** -22)


def test_clipping_is_decided_as_in_exact_arithmetic():
    """Ratios within a few roundings of the borders, both signs of the advantage."""
    require_gpu()
    rng = np.random.default_rng(3)
    lo, hi = 0.2, 0.28
    old = np.concatenate([-rng.exponential(2.0, 20000), np.zeros(8)]).astype(np.float32)
    theta = np.where(np.arange(old.size) % 2 == 0, np.log1p(hi), np.log1p(-lo))
    logp = (old + theta).astype(np.float32)
    for _ in range(3):
        step = rng.integers(-1, 2, old.size)
        logp = np.where(step > 0, np.nextafter(logp, np.float32(np.inf)),
                        np.where(step < 0, np.nextafter(logp, np.float32(-np.inf)), logp)).astype(np.float32)
        d = logp.astype(np.float64) - old.astype(np.float64)
        # the rounded difference cannot tell: the case is there
        tie = (logp - old) == theta.astype(np.float32)
        assert tie.sum() > 100
        adv = np.where(theta > 0, 1.0, -1.0).astype(np.float32)
        clipped = np.where(theta > 0, d > np.log1p(hi), d < np.log1p(-lo))
        t = lambda x: torch.from_numpy(x).cuda()[None]  # noqa: E731
        _, stats, g = kd.policy_loss(t(logp), t(old), t(adv), advantages_per="token", clip_low=lo, clip_high=hi)
        assert np.array_equal(g[0].cpu().numpy() == 0, clipped)
        assert stats[2].item() == pytest.approx(clipped.mean(), rel=2 ** -23)


def test_infinite_log_probabilities_that_count():
    """-inf in the new policy: ratio 0, gradient 0; in the old one: an infinite
    ratio, clipped for a positive advantage; the other tokens are unaffected."""
    require_gpu()
    inf = float("inf")
    logp = torch.tensor([[-1.0, -inf, -1.0, -2.0]], device="cuda")
    old = torch.tensor([[-1.0, -1.0, -inf, -2.0]], device="cuda")
    adv = torch.tensor([2.0], device="cuda")
    loss, stats, g = kd.policy_loss(logp, old, adv)
    assert g[0].tolist() == [-0.5, 0.0, 0.0, -0.5]
    assert loss.item() == pytest.approx(-(2 + 0 + 2 * 1.2 + 2) / 4, rel=1e-6)


PREF_VARIANTS = [
    dict(kind="sigmoid", beta=0.1),
    dict(kind="sigmoid", beta=2.0, margin=0.5, smoothing=0.1, normalize=True, no_ref=True),
    dict(kind="hinge", beta=0.5, margin=-0.25),
    dict(kind="ipo", beta=0.1, normalize=True),
    dict(kind="ipo", beta=0.3, pairs_total=12345),
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("name", [n for n in LAYOUTS if not _odd_pairs(n)])
def test_preference_loss(name, masked):
    require_gpu()
    x = _make(name, 6, masked)
    B = x["S"] // 2
    for v in PREF_VARIANTS:
        v = dict(v)
        no_ref, total = v.pop("no_ref", False), v.pop("pairs_total", None)
        if total is not None:
            total = max(total, B)
        ws = kd.alloc_workspace(kd.kd_preference_loss_workspace_size(B, x["N"]), "cuda")
        kw = dict(ref_logp=None if no_ref else x["ref"], mask=x["mask"], cu_seqlens=x["cu"], kind=v["kind"],
                  beta=v["beta"], margin=v.get("margin", 0.0), label_smoothing=v.get("smoothing", 0.0),
                  length_normalize=v.get("normalize", False), pairs_total=total, ws=ws)
        loss, rewards, g = kd.preference_loss(x["logp"], **kw)
        assert kd.read_device_status(ws) == kd.KD_OK
        want = plain.preference(x["np"]["logp"], x["ranges"], ref=None if no_ref else x["np"]["ref"],
                                mask=x["np"]["mask"], pairs_total=total, **v)
        err_s = 2.0 ** -45 * want["size"] + 1e-300
        top = max(np.abs(want["rewards"] / v["beta"]).max() * 2 + 0.5 / v["beta"], 1.0)
        slope = {"sigmoid": v["beta"], "hinge": v["beta"], "ipo": 2 * top}[v["kind"]]
        curve = {"sigmoid": v["beta"] ** 2, "hinge": 0.0, "ipo": 2.0}[v["kind"]]
        near = 2.0 ** -22
        rn = rewards.double().cpu().numpy()
        assert np.all(np.abs(rn - want["rewards"]) <= near * np.abs(want["rewards"]) + v["beta"] * err_s)
        assert abs(loss.item() - want["loss"]) <= near * abs(want["loss"]) + 2 * slope * err_s
        gn = g.double().cpu().numpy().reshape(-1)
        share = 1.0 / (B if total is None else total)
        assert np.all(np.abs(gn - want["grad"]) <= near * np.abs(want["grad"]) + 2 * curve * err_s * share)
        loss2, rewards2, none = kd.preference_loss(x["logp"], **{**kw, "grad": False})
        assert none is None and torch.equal(loss2, loss) and torch.equal(rewards2, rewards)
        assert torch.equal(kd.preference_loss(x["logp"], **kw)[2], g)


@pytest.mark.parametrize("name", ["rows-of-129", "rows-of-1000", "packed-small", "packed-long"])
def test_gradients_against_differences(name):
    """Central differences of the fp64 forms along a random direction."""
    require_gpu()
    x = _make(name, 8, True)
    rng = np.random.default_rng(4)
    on = x["np"]["mask"].copy()
    inside = np.zeros(x["N"], bool)
    for a, b in x["ranges"]:
        inside[a:b] = True
    u = np.where(on & inside, rng.normal(0, 1, x["N"]), 0.0)
    lp = np.where(on & inside, x["np"]["logp"], 0.0).astype(np.float64)
    eps = 1e-6
    _, _, g = kd.policy_loss(x["logp"], x["old"], x["adv"], mask=x["mask"], ref_logp=x["ref"], kl_coef=0.1,
                             cu_seqlens=x["cu"], reduction="sequence")
    f = lambda e: plain.policy(lp + e * u, x["np"]["old"], x["adv"].cpu().numpy(), x["ranges"],  # noqa: E731
                               mask=on, ref=x["np"]["ref"], beta=0.1, reduction="sequence")["loss"]
    diff = (f(eps) - f(-eps)) / (2 * eps)
    got = float((g.double().cpu().numpy().reshape(-1) * u).sum())
    # fp32 gradients (2^-19 of about the loss's size) and differences of fp64 values (1e-16 / eps, eps^2)
    assert abs(got - diff) <= 1e-6 * max(1.0, abs(diff))
    _, _, g = kd.preference_loss(x["logp"], ref_logp=x["ref"], mask=x["mask"], cu_seqlens=x["cu"], beta=0.05)
    f = lambda e: plain.preference(lp + e * u, x["ranges"], ref=x["np"]["ref"], mask=on, beta=0.05)["loss"]  # noqa: E731
    diff = (f(eps) - f(-eps)) / (2 * eps)
    got = float((g.double().cpu().numpy().reshape(-1) * u).sum())
    assert abs(got - diff) <= 1e-6 * max(1.0, abs(diff))


@pytest.mark.parametrize("name", ["packed-small", "packed-long"])
@pytest.mark.parametrize("bad", [[-1], [10 ** 9], "swap", [-2 ** 31], [2 ** 31 - 1]])
def test_bad_cu_seqlens_are_reported(name, bad):
    require_gpu()
    x = _make(name, 9, True)
    cu = x["cu"].clone()
    if bad == "swap":
        cu[3], cu[4] = x["cu"][4] + 1, x["cu"][3]
    else:
        cu[4] = bad[0]
    ws = kd.alloc_workspace(kd.kd_policy_loss_workspace_size(x["S"], x["N"]), "cuda")
    for reduction in ("token", "sequence"):
        kd.policy_loss(x["logp"], x["old"], x["adv"], mask=x["mask"], cu_seqlens=cu, reduction=reduction, ws=ws)
        assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
    ws = kd.alloc_workspace(kd.kd_preference_loss_workspace_size(x["S"] // 2, x["N"]), "cuda")
    kd.preference_loss(x["logp"], mask=x["mask"], cu_seqlens=cu, ws=ws)
    assert kd.read_device_status(ws) == kd.KD_ERR_BAD_INDEX
    # the status word is cleared by the next call on the same workspace
    kd.preference_loss(x["logp"], mask=x["mask"], cu_seqlens=x["cu"], ws=ws)
    assert kd.read_device_status(ws) == kd.KD_OK


def test_any_byte_but_0_counts():
    require_gpu()
    x = _make("rows-of-1000", 10, True)
    gen = torch.Generator("cuda").manual_seed(1)
    byte = torch.randint(1, 256, x["mask"].shape, generator=gen, device="cuda", dtype=torch.uint8)
    byte = torch.where(x["mask"], byte, torch.zeros_like(byte))
    for reduction in ("token", "sequence"):
        a, b = (kd.policy_loss(x["logp"], x["old"], x["adv"], mask=m, reduction=reduction) for m in (x["mask"], byte))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = (kd.preference_loss(x["logp"], mask=m, length_normalize=True) for m in (x["mask"], byte))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_autograd():
    require_gpu()
    x = _make("rows-of-129", 10, True)
    leaf = x["logp"].clone().requires_grad_()
    opts = dict(mask=x["mask"], ref_logp=x["ref"], kl_coef=0.1, reduction="sequence")
    loss, stats = kd.PolicyLoss.apply(leaf, x["old"], x["adv"], opts)
    (g,) = torch.autograd.grad(3.0 * loss, leaf)
    want = kd.policy_loss(x["logp"], x["old"], x["adv"], **opts)
    assert torch.equal(loss, want[0]) and torch.equal(stats, want[1]) and torch.equal(g, want[2] * 3.0)
    opts = dict(ref_logp=x["ref"], mask=x["mask"], beta=0.3)
    loss, rewards = kd.PreferenceLoss.apply(leaf, opts)
    (g,) = torch.autograd.grad(loss * 2.0, leaf)
    want = kd.preference_loss(x["logp"], **opts)
    assert torch.equal(loss, want[0]) and torch.equal(rewards, want[1]) and torch.equal(g, want[2] * 2.0)
    with torch.no_grad():
        loss, _ = kd.PolicyLoss.apply(x["logp"], x["old"], x["adv"], dict(mask=x["mask"]))
    assert not loss.requires_grad


@pytest.mark.parametrize("name", ["packed-small", "packed-long"])
def test_two_captured_graphs_and_another_stream(name):
    """Two graphs captured on the same inputs replay one after the other with new
    contents in the inputs; a call on another stream gives the same."""
    require_gpu()
    x, y = _make(name, 11, True), _make(name, 12, True)
    logp, old = x["logp"].clone(), x["old"].clone()
    calls = [lambda s=None: kd.policy_loss(logp, old, x["adv"], mask=x["mask"], cu_seqlens=x["cu"],
                                           reduction="sequence", stream=s),
             lambda s=None: kd.preference_loss(logp, ref_logp=old, mask=x["mask"], cu_seqlens=x["cu"], stream=s)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c()
        graphs.append((g, out))
    for src in (x, y):
        keep = x["mask"] & (src["logp"].isfinite())
        logp.copy_(torch.where(keep, src["logp"], x["logp"]))
        old.copy_(torch.where(keep & src["old"].isfinite(), src["old"], x["old"]))
        for g, _ in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for (g, out), c in zip(graphs, calls):
            want = c()
            for a, b in zip(out, want):
                assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
            again = c(side)
            side.synchronize()
            for a, b in zip(again, want):
                assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("name", ["rows-of-129", "rows-of-1000", "packed-small", "packed-long"])
def test_slices_of_a_batch(name, shift):
    """Arrays that begin at any element of a buffer: the same bits as aligned ones,
    and nothing around the gradient is written."""
    require_gpu()
    x = _make(name, 14, True)

    def moved(t):
        buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        view = buf[shift:shift + t.numel()].view(t.shape)
        return view.copy_(t)

    y = {k: moved(x[k]) for k in ("logp", "old", "ref", "mask", "adv", "adv_tok")}
    cu = None if x["cu"] is None else moved(x["cu"])
    for per in ("sequence", "token"):
        a, b = (z["adv"] if per == "sequence" else z["adv_tok"] for z in (x, y))
        kw = dict(kl_coef=0.1, reduction="sequence", advantages_per=per)
        want = kd.policy_loss(x["logp"], x["old"], a, mask=x["mask"], ref_logp=x["ref"], cu_seqlens=x["cu"], **kw)
        got = kd.policy_loss(y["logp"], y["old"], b, mask=y["mask"], ref_logp=y["ref"], cu_seqlens=cu, **kw)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    want = kd.preference_loss(x["logp"], ref_logp=x["ref"], mask=x["mask"], cu_seqlens=x["cu"])
    got = kd.preference_loss(y["logp"], ref_logp=y["ref"], mask=y["mask"], cu_seqlens=cu)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    # the gradient into a place of the caller's, by the raw call
    n, S = x["N"], x["S"]
    out = torch.full((n + 16,), 7.0, device="cuda")
    ws = kd.alloc_workspace(kd.kd_preference_loss_workspace_size(S // 2, n), "cuda")
    small = torch.empty(S + 1, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    assert kd.kd_preference_loss(p(x["logp"]), p(x["ref"]), p(x["mask"]), p(x["cu"]), S // 2, n, 0, 0.1, 0.0, 0.0, 0,
                                 S // 2, small.data_ptr(), small.data_ptr() + 4, out.data_ptr() + 4 * (shift + 4),
                                 ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == kd.KD_OK
    assert torch.equal(out[shift + 4:shift + 4 + n], want[2].reshape(-1))
    assert bool((out[:shift + 4] == 7).all()) and bool((out[shift + 4 + n:] == 7).all())


def test_offsets_past_32_bits():
    """2^30 + 640 tokens: byte offsets pass 2^32."""
    require_gpu()
    S, L = 4, (1 << 28) + 160
    n = S * L
    logp = torch.full((S, L), -1.0, device="cuda")
    logp[3, -1] = -0.75
    old = torch.full((S, L), -1.0, device="cuda")
    adv = torch.tensor([1.0, 1.0, 1.0, 2.0], device="cuda")
    loss, stats, g = kd.policy_loss(logp, old, adv, clip_high=0.5)
    assert stats[0].item() == float(np.float32(n))
    assert loss.item() == pytest.approx(-1.25, rel=1e-6)
    assert g[0, 0].item() == pytest.approx(-1 / n, rel=1e-6) and g[2, -1].item() == pytest.approx(-1 / n, rel=1e-6)
    assert g[3, -1].item() == pytest.approx(-2 * np.exp(0.25) / n, rel=1e-6)
    del old
    loss, rewards, g = kd.preference_loss(logp, beta=1e-6)
    assert rewards[2].item() == pytest.approx(-L * 1e-6, rel=1e-6)
    assert rewards[3].item() == pytest.approx((-L + 0.25) * 1e-6, rel=1e-6)
    # pairs (0, 2) with D = 0 and (1, 3) with D = -1/4: beta sigmoid(-beta D) / 2 for each rejected token
    assert g[2, 0].item() == pytest.approx(1e-6 * 0.5 / 2, rel=1e-6)
    assert g[3, -1].item() == g[3, 0].item() == pytest.approx(1e-6 / (1 + np.exp(-0.25e-6)) / 2, rel=1e-6)


@pytest.mark.parametrize("S,L", [(2, 3), (2, 5000), (2048, 9)])
def test_a_batch_that_the_mask_leaves_empty(S, L):
    require_gpu()
    x = torch.full((S, L), float("nan"), device="cuda")
    mask = torch.zeros((S, L), dtype=torch.uint8, device="cuda")
    adv = torch.full((S,), float("nan"), device="cuda")
    for reduction in ("token", "sequence"):
        loss, stats, g = kd.policy_loss(x, x, adv, mask=mask, ref_logp=x, kl_coef=0.1, reduction=reduction)
        assert loss.item() == 0 and stats.tolist() == [0, 0, 0, 0] and bool((g == 0).all())
    loss, rewards, g = kd.preference_loss(x, mask=mask, length_normalize=True)
    assert loss.item() == pytest.approx(np.log(2), rel=1e-6) and bool((rewards == 0).all()) and bool((g == 0).all())
