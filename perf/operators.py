"""The post-training operators that are measured: cases, inputs, plain forms and 64-bit values.

Four operators, used one after the other by a training step on sampled or compared answers:

* ``head``: log-probabilities of given tokens through the output head (``kd.head_logprobs``), forward
  only ("score") or with the gradients of h and W ("train");
* ``policy``: the clipped policy loss with a KL term and its gradient for each token (``kd.policy_loss``);
* ``preference``: the paired preference loss and its gradient for each token (``kd.preference_loss``);
* ``clip``: the global norm of a list of gradients, and the clipped gradients (``kd.clip_grad_norm``).

``run`` computes an operator from elementary torch operations, or with ``own`` set through the
framework's entry points; both return the same outputs.
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # Scoring a handful of sampled tokens with a small head; nothing divides a tile.
        dict(name="score-300", op="head", train=False, T=300, d=200, V=5000, chunk=100, tau=1.0, ignored=0.2),
        # Reference log-probabilities of 2048 positions under the 131072-token head.
        dict(name="score-head-2k", op="head", train=False, T=2048, d=4096, V=131072, chunk=2048, tau=1.0, ignored=0.0),
        # A ragged micro-batch of answers (prompt positions ignored) through the 201088-token head.
        dict(name="train-vocab-201k", op="head", train=True, T=777, d=2880, V=201088, chunk=512, tau=0.7, ignored=0.4),
        # One chunk of the 131072-token head, log-probabilities and both gradients.
        dict(name="train-head-2k", op="head", train=True, T=2048, d=4096, V=131072, chunk=2048, tau=1.0, ignored=0.1),
        # A micro-batch of eight short padded answers: latency counts.
        dict(name="policy-8x64", op="policy", S=8, L=64, packed=False, masked=True, ref=False, per_token=False,
             low=0.2, high=0.2, kl=0.0, reduction="token", denom=0.0),
        # A step's packed answers, one token to 8192 each, mean of the sequences' means, KL to a reference.
        dict(name="policy-packed-256", op="policy", S=256, L=8192, packed=True, masked=True, ref=True, per_token=False,
             low=0.2, high=0.28, kl=0.04, reduction="sequence", denom=0.0),
        # A large batch of long padded answers with advantages for each token (a critic's).
        dict(name="policy-256x32k", op="policy", S=256, L=32768, packed=False, masked=True, ref=True, per_token=True,
             low=0.2, high=0.2, kl=0.001, reduction="token", denom=0.0),
        # Four padded pairs of short answers: latency counts.
        dict(name="preference-4x100", op="preference", B=4, L=100, packed=False, masked=True, ref=True, kind="sigmoid",
             beta=0.1, margin=0.0, smoothing=0.0, normalize=False),
        # Packed pairs of very different lengths, length-normalised, without a reference.
        dict(name="preference-packed-96", op="preference", B=96, L=8192, packed=True, masked=True, ref=False,
             kind="sigmoid", beta=2.0, margin=0.5, smoothing=0.1, normalize=True),
        # A large batch of padded pairs against a reference, squared form.
        dict(name="preference-512x4k", op="preference", B=512, L=4096, packed=False, masked=True, ref=True, kind="ipo",
             beta=0.1, margin=0.0, smoothing=0.0, normalize=True),
        # The small tensors of a model whose gradients are views into one flat buffer, at odd offsets.
        dict(name="clip-flat-290", op="clip", n=290, most=1 << 17, flat=True, types="mixed", max_norm=1.0, big=0),
        # The gradients of the 131072-token head (fp32 dW, bf16 dH) beside those of a few blocks.
        dict(name="clip-head-32k", op="clip", n=12, most=1 << 24, flat=False, types="mixed", max_norm=0.5, big=131072 * 4096),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(("head", "policy", "preference", "clip"))
    if op == "head":
        train = rng.random() < 0.5
        d = 8 * _log(rng, 8, 512)
        V = _log(rng, 257, 201088)
        most = 2048 * 4096 * 131072 // (d * V)
        T = _log(rng, 1, max(1, min(2048, most)))
        return dict(op=op, train=train, T=T, d=d, V=V, chunk=_log(rng, 64, 2048), tau=rng.choice((1.0, 0.7, 1.3)),
                    ignored=rng.choice((0.0, 0.1, 0.5)))
    if op == "policy":
        S = _log(rng, 1, 1024)
        return dict(op=op, S=S, L=_log(rng, 1, min(32768, (256 * 32768) // S)), packed=rng.random() < 0.5,
                    masked=rng.random() < 0.8, ref=rng.random() < 0.6, per_token=rng.random() < 0.4,
                    low=rng.choice((0.1, 0.2)), high=rng.choice((0.2, 0.28)), kl=rng.choice((0.001, 0.04, 0.1)),
                    reduction=rng.choice(("token", "sequence", "fixed")), denom=float(rng.randint(100, 100000)))
    if op == "preference":
        B = _log(rng, 1, 1024)
        return dict(op=op, B=B, L=_log(rng, 1, min(32768, (512 * 4096) // B)), packed=rng.random() < 0.5,
                    masked=rng.random() < 0.8, ref=rng.random() < 0.7, kind=rng.choice(("sigmoid", "hinge", "ipo")),
                    beta=rng.choice((0.05, 0.1, 0.5)), margin=0.0, smoothing=0.0, normalize=rng.random() < 0.5)
    n = _log(rng, 1, 400)
    return dict(op=op, n=n, most=_log(rng, 64, min(1 << 24, (1 << 29) // n)), flat=rng.random() < 0.5,
                types=rng.choice(("f32", "bf16", "mixed")), max_norm=rng.choice((0.1, 1.0, 1e6)), big=0)


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    return g


def _lengths(S, L):
    """Answer lengths between one token and L, most of them far below it; a case's lengths are its own, so that its
    outputs have one shape."""
    rng = random.Random(S * 100003 + L)
    return [max(1, min(L, int(L * math.exp(-rng.expovariate(0.7))))) for _ in range(S)]


def _sequences(case, S, seed):
    """Layout and mask of S answers: the first tokens of each belong to the prompt and are masked out, the rest of a
    padded row lies behind its end; an answer now and then is masked out altogether."""
    rng = random.Random(int(seed) * 7 + 1)
    L = case["L"]
    lens = _lengths(S, L)
    prompts = [n if k and rng.random() < 0.03 else int(n * rng.uniform(0.0, 0.6)) for k, n in enumerate(lens)]
    lens_t = torch.tensor(lens, dtype=torch.int64, device=_DEV)
    prompts_t = torch.tensor(prompts, dtype=torch.int64, device=_DEV)
    if case["packed"]:
        cu = torch.zeros(S + 1, dtype=torch.int64, device=_DEV)
        cu[1:] = torch.cumsum(lens_t, 0)
        N = sum(lens)
        seq = torch.repeat_interleave(torch.arange(S, device=_DEV), lens_t, output_size=N)
        pos = torch.arange(N, device=_DEV) - cu[seq]
        mask = pos >= prompts_t[seq]
        return (N,), cu.to(torch.int32), (mask if case["masked"] else None), torch.zeros(N, dtype=torch.bool, device=_DEV)
    pos = torch.arange(L, device=_DEV)[None, :]
    mask = (pos >= prompts_t[:, None]) & (pos < lens_t[:, None])
    behind = (pos >= lens_t[:, None]) if case["masked"] else torch.zeros((S, L), dtype=torch.bool, device=_DEV)
    return (S, L), None, (mask if case["masked"] else None), behind


def _tensors(case):
    """Sizes and types of a case's gradients."""
    rng = random.Random(case["n"] * 100003 + case["most"])
    sizes = [_log(rng, 1, case["most"]) for _ in range(case["n"])]
    kinds = [_DT[case["types"]] if case["types"] != "mixed" else rng.choice((torch.float32, torch.bfloat16)) for _ in sizes]
    return (sizes + [case["big"]], kinds + [torch.float32]) if case["big"] else (sizes, kinds)


def _token_logps(shape, behind, g):
    """Log-probabilities as sampled answers have them: most near 0, a long tail; -inf in the padding."""
    x = -torch.empty(shape, device=_DEV).exponential_(1.5, generator=g)
    return torch.where(behind, torch.full_like(x, -math.inf), x)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op == "head":
        T, d, V = case["T"], case["d"], case["V"]
        st["h"] = torch.randn((T, d), generator=g, device=_DEV).to(torch.bfloat16)
        st["W"] = (torch.randn((V, d), generator=g, device=_DEV) / math.sqrt(d)).to(torch.bfloat16)
        tgt = torch.randint(0, V, (T,), generator=g, device=_DEV, dtype=torch.int32)
        skip = torch.rand((T,), generator=g, device=_DEV) < case["ignored"]
        skip[0] = False
        st["targets"] = torch.where(skip, torch.full_like(tgt, -100), tgt)
        if case["train"]:
            st["grad"] = torch.randn((T,), generator=g, device=_DEV) / T
            st["h"].requires_grad_()
            st["W"].requires_grad_()
        return st
    if op == "policy":
        S = case["S"]
        shape, st["cu"], st["mask"], behind = _sequences(case, S, seed)
        st["old"] = _token_logps(shape, behind, g)
        st["logp"] = torch.where(behind, st["old"], (st["old"] + 0.15 * torch.randn(shape, generator=g, device=_DEV)))
        st["ref_logp"] = st["old"] + 0.1 * torch.randn(shape, generator=g, device=_DEV) if case["ref"] else None
        st["adv"] = torch.randn(shape if case["per_token"] else (S,), generator=g, device=_DEV)
        return st
    if op == "preference":
        shape, st["cu"], st["mask"], behind = _sequences(case, 2 * case["B"], seed)
        st["logp"] = _token_logps(shape, behind, g)
        st["ref_logp"] = None
        if case["ref"]:
            st["ref_logp"] = torch.where(behind, st["logp"], st["logp"] + 0.05 * torch.randn(shape, generator=g, device=_DEV))
        return st
    sizes, kinds = _tensors(case)
    types = [dt for dt in (torch.float32, torch.bfloat16) if dt in kinds]
    # views into one buffer for each type: back to back, at whatever offset comes, or each on a boundary of its own
    width = [n if case["flat"] else -(-n // 64) * 64 for n in sizes]
    total = {dt: sum(w for w, k in zip(width, kinds) if k == dt) for dt in types}
    flat = {dt: torch.randn((total[dt],), generator=g, device=_DEV).mul_(1e-2).to(dt) for dt in types}
    st["flat"] = {str(dt): torch.zeros_like(flat[dt]) for dt in types}
    at, st["grads"], st["out"] = {dt: 0 for dt in types}, [], []
    for n, w, k in zip(sizes, width, kinds):
        st["grads"].append(flat[k][at[k]:at[k] + n])
        st["out"].append(st["flat"][str(k)][at[k]:at[k] + n])
        at[k] += w
    return st


# ----------------------------------------------------------------------------------- the operators

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _own_head(st):
    from chunked_kl_loss_chunk_b200 import kd
    if not st["train"]:
        logp, lse, _ = kd.head_logprobs(st["h"], st["W"], st["targets"], st["chunk"], st["tau"])
        return {"logp": logp, "lse": lse}
    logp = kd.HeadLogprobs.apply(st["h"], st["W"], st["targets"], st["chunk"], st["tau"])
    dH, dW = torch.autograd.grad(logp, (st["h"], st["W"]), st["grad"])
    return {"logp": logp.detach(), "dH": dH, "dW": dW}


def _own_policy(st):
    from chunked_kl_loss_chunk_b200 import kd
    loss, stats, dlogp = kd.policy_loss(
        st["logp"], st["old"], st["adv"], mask=st["mask"], ref_logp=st["ref_logp"], cu_seqlens=st["cu"],
        advantages_per="token" if st["per_token"] else "sequence", clip_low=st["low"], clip_high=st["high"],
        kl_coef=st["kl"] if st["ref"] else 0.0, reduction=st["reduction"], denom=st["denom"] if st["reduction"] == "fixed" else None)
    return {"loss": loss, "stats": stats, "dlogp": dlogp}


def _own_preference(st):
    from chunked_kl_loss_chunk_b200 import kd
    loss, rewards, dlogp = kd.preference_loss(
        st["logp"], ref_logp=st["ref_logp"], mask=st["mask"], cu_seqlens=st["cu"], kind=st["kind"], beta=st["beta"],
        margin=st["margin"], label_smoothing=st["smoothing"], length_normalize=st["normalize"])
    return {"loss": loss, "rewards": rewards, "dlogp": dlogp}


def _own_clip(st):
    from chunked_kl_loss_chunk_b200 import kd
    norm = kd.clip_grad_norm(st["grads"], st["max_norm"], out=st["out"])
    return {"norm": norm, "out": st["flat"]}


def _plain_head(st):
    h, W = st["h"].detach().float(), st["W"].detach().float()
    keep = st["targets"] >= 0
    y = torch.where(keep, st["targets"], 0).long()[:, None]
    a = (h @ W.t()) / st["tau"]
    top = a.max(dim=1, keepdim=True).values
    lse = top + (a - top).exp().sum(dim=1, keepdim=True).log()
    logp = torch.where(keep, (a.gather(1, y) - lse)[:, 0], 0.0)
    if not st["train"]:
        return {"logp": logp, "lse": lse[:, 0]}
    g = torch.where(keep, st["grad"], 0.0)[:, None] / st["tau"]
    dz = -g * (a - lse).exp()
    dz.scatter_add_(1, y, g)
    return {"logp": logp, "dH": (dz @ W).to(st["h"].dtype), "dW": (dz.t() @ h).to(st["W"].dtype)}


def _ids(st, S):
    """For each token its sequence, and the first token of each sequence and the end of the last."""
    x = st["logp"]
    N = x.numel()
    cu = st["cu"].long() if st["cu"] is not None else torch.arange(S + 1, device=x.device) * (N // S)
    seq = torch.bucketize(torch.arange(N, device=x.device), cu[1:], right=True)
    keep = st["mask"].reshape(-1) if st["mask"] is not None else torch.ones(N, dtype=torch.bool, device=x.device)
    return seq, cu, keep


def _per_sequence(v, cu):
    """Sums of v over each sequence, in 64 bits."""
    run_sum = torch.cat([torch.zeros(1, dtype=torch.float64, device=v.device), v.double().cumsum(0)])
    return run_sum[cu[1:]] - run_sum[cu[:-1]]


def _plain_policy(st):
    S, shape = st["S"], st["logp"].shape
    seq, cu, keep = _ids(st, S)
    logp, old = st["logp"].reshape(-1), st["old"].reshape(-1)
    adv = st["adv"].reshape(-1) if st["per_token"] else st["adv"][seq]
    zero = torch.zeros((), device=logp.device)
    d = torch.where(keep, logp.double() - old.double(), 0.0)
    clipped = ((adv > 0) & (d > math.log1p(st["high"]))) | ((adv < 0) & (d < math.log1p(-st["low"])))
    clipped = clipped & keep
    ratio = d.float().exp()
    bound = torch.where(adv > 0, 1 + st["high"], 1 - st["low"])
    term = -torch.where(clipped, adv * bound, adv * ratio)
    grad = -torch.where(clipped, zero, adv * ratio)
    kl = torch.zeros_like(logp)
    if st["ref_logp"] is not None:
        q = torch.where(keep, st["ref_logp"].reshape(-1).double() - logp.double(), 0.0)
        kl = (q.expm1() - q).float()
        term = term + st["kl"] * kl
        grad = grad - st["kl"] * q.expm1().float()
    n = keep.double().sum()
    if st["reduction"] == "token":
        w = (1 / n.clamp(min=1)).float().expand_as(logp)
    elif st["reduction"] == "sequence":
        w = (1 / (S * _per_sequence(keep, cu).clamp(min=1))).float()[seq]
    else:
        w = torch.full_like(logp, 1 / st["denom"])
    total = torch.where(keep, w * term, zero).double().sum().float()
    some = n.clamp(min=1)
    stats = torch.stack([n, torch.where(keep, ratio, zero).double().sum() / some, clipped.double().sum() / some,
                         torch.where(keep, kl, zero).double().sum() / some]).float()
    return {"loss": total, "stats": stats, "dlogp": torch.where(keep, w * grad, zero).reshape(shape)}


def _plain_preference(st):
    B, shape, beta = st["B"], st["logp"].shape, st["beta"]
    seq, cu, keep = _ids(st, 2 * B)
    x = st["logp"].reshape(-1).double()
    if st["ref_logp"] is not None:
        x = x - st["ref_logp"].reshape(-1).double()
    s = _per_sequence(torch.where(keep, x, 0.0), cu)
    n = _per_sequence(keep, cu).clamp(min=1)
    per = 1 / n if st["normalize"] else torch.ones_like(n)
    s = s * per
    delta = s[:B] - s[B:]
    if st["kind"] == "ipo":
        loss, slope = (delta - 1 / (2 * beta)).square(), 2 * (delta - 1 / (2 * beta))
    elif st["kind"] == "hinge":
        z = beta * delta - st["margin"]
        loss, slope = (1 - z).clamp(min=0), -beta * (z < 1).double()
    else:
        z, e = beta * delta - st["margin"], st["smoothing"]
        up, down = z.clamp(min=0) + (-z.abs()).exp().log1p(), (-z).clamp(min=0) + (-z.abs()).exp().log1p()
        loss = (1 - e) * down + e * up
        slope = beta * (e - 1 / (1 + z.exp()))
    coef = (torch.cat([slope, -slope]) * per / B).float()
    return {"loss": loss.mean().float(), "rewards": (beta * s).float(),
            "dlogp": torch.where(keep, coef[seq], 0.0).reshape(shape)}


def _plain_clip(st):
    norm = torch.stack([x.float().square().sum(dtype=torch.float64) for x in st["grads"]]).sum().sqrt()
    coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    [o.copy_(x.float() * coef) for o, x in zip(st["out"], st["grads"])]
    return {"norm": norm.float(), "out": st["flat"]}


_OWN = {"head": _own_head, "policy": _own_policy, "preference": _own_preference, "clip": _own_clip}
_PLAIN = {"head": _plain_head, "policy": _plain_policy, "preference": _plain_preference, "clip": _plain_clip}


# --------------------------------------------------------------------------------- work and 64 bits

def _tokens(case, S):
    return sum(_lengths(S, case["L"])) if case["packed"] else S * case["L"]


def work(case):
    op = case["op"]
    if op == "head":
        T, d, V = case["T"], case["d"], case["V"]
        read = 2 * T * d + 2 * V * d + 4 * T
        if not case["train"]:
            return {"bytes": read + 8 * T, "flops": 2 * T * d * V}
        # without keeping the logits the backward projects again: 2 products forward and back, 2 for the gradients
        return {"bytes": read + 4 * T + 4 * T + 2 * T * d + 2 * V * d, "flops": 8 * T * d * V}
    if op == "policy":
        N, S = _tokens(case, case["S"]), case["S"]
        each = 4 * (2 + case["ref"] + case["per_token"]) + case["masked"] + 4
        return {"bytes": N * each + (0 if case["per_token"] else 4 * S) + 20, "flops": 20 * N}
    if op == "preference":
        N, S = _tokens(case, 2 * case["B"]), 2 * case["B"]
        return {"bytes": N * (4 * (1 + case["ref"]) + case["masked"] + 4) + 4 * S + 4, "flops": 4 * N}
    sizes, kinds = _tensors(case)
    each = sum(n * k.itemsize for n, k in zip(sizes, kinds))
    return {"bytes": 2 * each + 4, "flops": 3 * sum(sizes)}


def exact(case, seed):
    """The operator's definition in 64 bits; gradients by automatic differentiation of it."""
    st = prepare(case, seed)
    return {"head": _exact_head, "policy": _exact_policy, "preference": _exact_preference, "clip": _exact_clip}[case["op"]](st)


def _exact_head(st):
    with torch.set_grad_enabled(st["train"]):
        h = st["h"].detach().double().requires_grad_(st["train"])
        W = st["W"].detach().double().requires_grad_(st["train"])
        rows = torch.nonzero(st["targets"] >= 0)[:, 0]
        z = torch.nn.functional.linear(h, W) / st["tau"]
        picked = torch.log_softmax(z, dim=-1)[rows, st["targets"][rows].long()]
        logp = torch.zeros(st["T"], dtype=torch.float64, device=_DEV).index_put((rows,), picked)
        if not st["train"]:
            return {"logp": logp, "lse": torch.logsumexp(z, dim=-1)}
        dH, dW = torch.autograd.grad((logp * st["grad"].double()).sum(), (h, W))
    return {"logp": logp.detach(), "dH": dH, "dW": dW}


def _parts(st, S):
    """For each sequence the places of its tokens that count."""
    N = st["logp"].numel()
    ends = st["cu"].tolist() if st["cu"] is not None else [k * (N // S) for k in range(S + 1)]
    keep = st["mask"].reshape(-1) if st["mask"] is not None else torch.ones(N, dtype=torch.bool, device=_DEV)
    on = torch.nonzero(keep)[:, 0]
    cuts = torch.searchsorted(on, torch.tensor(ends, device=_DEV)).tolist()
    return [on[a:b] for a, b in zip(cuts, cuts[1:])]


def _exact_policy(st):
    S = st["S"]
    leaf = st["logp"].reshape(-1).double().requires_grad_()
    old = st["old"].reshape(-1).double()
    loss = torch.zeros((), dtype=torch.float64, device=_DEV)
    parts = _parts(st, S)
    n = sum(p.numel() for p in parts)
    sums = [0.0, 0.0, 0.0]
    for b, p in enumerate(parts):
        if p.numel() == 0:
            continue
        adv = (st["adv"].reshape(-1)[p] if st["per_token"] else st["adv"][b]).double()
        ratio = torch.exp(leaf[p] - old[p])
        held = ratio.clamp(1 - st["low"], 1 + st["high"])
        part = -torch.minimum(ratio * adv, held * adv)
        with torch.no_grad():
            sums[0] = sums[0] + ratio.sum()
            sums[1] = sums[1] + (held * adv < ratio * adv).sum().double()
        if st["ref_logp"] is not None:
            q = st["ref_logp"].reshape(-1)[p].double() - leaf[p]
            k = torch.special.expm1(q) - q
            part = part + st["kl"] * k
            sums[2] = sums[2] + k.detach().sum()
        share = {"token": 1 / max(n, 1), "sequence": 1 / (S * p.numel()), "fixed": 1 / st["denom"] if st["denom"] else 0.0}
        loss = loss + share[st["reduction"]] * part.sum()
    grad = torch.autograd.grad(loss, leaf)[0] if n else torch.zeros_like(leaf)
    stats = torch.stack([torch.as_tensor(float(v) / max(n, 1), dtype=torch.float64) for v in sums])
    return {"loss": loss.detach(), "stats": torch.cat([torch.tensor([float(n)], dtype=torch.float64), stats]),
            "dlogp": grad.reshape(st["logp"].shape)}


def _exact_preference(st):
    B, beta = st["B"], st["beta"]
    leaf = st["logp"].reshape(-1).double().requires_grad_()
    scores = []
    for p in _parts(st, 2 * B):
        v = leaf[p] if st["ref_logp"] is None else leaf[p] - st["ref_logp"].reshape(-1)[p].double()
        scores.append(v.sum() / (max(p.numel(), 1) if st["normalize"] else 1))
    s = torch.stack(scores)
    delta = s[:B] - s[B:]
    if st["kind"] == "ipo":
        each = (delta - 0.5 / beta) ** 2
    elif st["kind"] == "hinge":
        each = torch.relu(1 - (beta * delta - st["margin"]))
    else:
        z = beta * delta - st["margin"]
        each = -(1 - st["smoothing"]) * torch.nn.functional.logsigmoid(z) - st["smoothing"] * torch.nn.functional.logsigmoid(-z)
    loss = each.mean()
    grad = torch.autograd.grad(loss, leaf)[0]
    return {"loss": loss.detach(), "rewards": (beta * s).detach(), "dlogp": grad.reshape(st["logp"].shape)}


def _exact_clip(st):
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(x, dtype=torch.float64)) ** 2 for x in st["grads"]))
    factor = min(1.0, st["max_norm"] / (norm + 1e-6))
    out = {k: torch.zeros(v.shape, dtype=torch.float64, device=_DEV) for k, v in st["flat"].items()}
    for x, o in zip(st["grads"], st["out"]):
        at = o.storage_offset()
        out[str(x.dtype)][at:at + x.numel()] = x.double() * factor
    return {"norm": norm, "out": out}
