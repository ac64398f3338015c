"""Plain fp64 forms of the policy and preference losses, sequence by sequence,
for the tests (NumPy, no framework code)."""

import numpy as np


def layout(S, shape, cu):
    """Token ranges of S sequences of an array of this shape."""
    if cu is None:
        L = shape[1]
        return [(b * L, (b + 1) * L) for b in range(S)]
    return [(int(cu[b]), int(cu[b + 1])) for b in range(S)]


def policy(logp, old, adv, ranges, mask=None, ref=None, per_token=False, lo=0.2, hi=0.2, beta=0.0,
           reduction="token", denom=None):
    """dict: loss, stats, grad, and `scale` (for each token the sum of its terms'
    magnitudes times its weight) with `scale_loss`, the same for the loss."""
    logp = np.asarray(logp, np.float64).reshape(-1)
    N = logp.size
    grad, scale = np.zeros(N), np.zeros(N)
    keep = np.ones(N, bool) if mask is None else np.asarray(mask, bool).reshape(-1)
    tokens = [np.array([t for t in range(a, b) if keep[t]], np.int64) for a, b in ranges]
    n = sum(len(t) for t in tokens)
    loss = scale_loss = ratios = clips = kls = 0.0
    for b, t in enumerate(tokens):
        if len(t) == 0:
            continue
        A = np.asarray(adv, np.float64).reshape(-1)[t] if per_token else np.full(len(t), float(adv[b]))
        d = np.zeros(len(t)) if old is None else logp[t] - np.asarray(old, np.float64).reshape(-1)[t]
        r = np.exp(d)
        clip = ((A > 0) & (d > np.log1p(hi))) | ((A < 0) & (d < np.log1p(-lo)))
        term = -np.where(clip, A * np.where(A > 0, 1 + hi, 1 - lo), A * r)
        g = -np.where(clip, 0.0, A * r)
        s = np.where(clip, 0.0, np.abs(A) * r * (1 + np.abs(d)))
        sl = np.abs(term) * (1 + np.abs(d))
        if ref is not None:
            q = np.asarray(ref, np.float64).reshape(-1)[t] - logp[t]
            k = np.expm1(q) - q
            kls += k.sum()
            term, g = term + beta * k, g - beta * np.expm1(q)
            s = s + beta * (np.exp(q) + 1) * (1 + np.abs(q))
            sl = sl + beta * (np.exp(q) + 1) * (1 + np.abs(q))
        w = {"token": 1 / n, "sequence": 1 / (len(ranges) * len(t)), "fixed": 1 / denom if denom else 0}[reduction]
        loss += w * term.sum()
        scale_loss += w * sl.sum()
        ratios += r.sum()
        clips += clip.sum()
        grad[t], scale[t] = w * g, w * s
    m = max(n, 1)
    return dict(loss=loss, stats=np.array([n, ratios / m, clips / m, kls / m]), grad=grad, scale=scale,
                scale_loss=scale_loss)


def preference(logp, ranges, ref=None, mask=None, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0,
               normalize=False, pairs_total=None):
    """dict: loss, rewards, grad, and `size`, the largest sum of magnitudes of a sequence."""
    logp = np.asarray(logp, np.float64).reshape(-1)
    keep = np.ones(logp.size, bool) if mask is None else np.asarray(mask, bool).reshape(-1)
    B = len(ranges) // 2
    tokens = [np.array([t for t in range(a, b) if keep[t]], np.int64) for a, b in ranges]
    s, per, size = np.zeros(2 * B), np.ones(2 * B), 0.0
    for b, t in enumerate(tokens):
        if len(t):
            x = logp[t] - (0 if ref is None else np.asarray(ref, np.float64).reshape(-1)[t])
            if normalize:
                per[b] = 1 / len(t)
            s[b] = x.sum() * per[b]
            size = max(size, np.abs(x).sum() * per[b])
    total = B if pairs_total is None else pairs_total
    loss, grad = 0.0, np.zeros(logp.size)
    for i in range(B):
        D = s[i] - s[i + B]
        z = beta * D - margin
        if kind == "ipo":
            l, slope = (D - 0.5 / beta) ** 2, 2 * (D - 0.5 / beta)
        elif kind == "hinge":
            l, slope = max(0.0, 1 - z), -beta if z < 1 else 0.0
        else:
            l = (1 - smoothing) * np.logaddexp(0, -z) + smoothing * np.logaddexp(0, z)
            slope = beta * (smoothing - 1 / (1 + np.exp(z)))
        loss += l / total
        grad[tokens[i]] = slope * per[i] / total
        grad[tokens[i + B]] = -slope * per[i + B] / total
    return dict(loss=loss, rewards=beta * s, grad=grad, size=size)
