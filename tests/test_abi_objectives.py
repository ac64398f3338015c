"""Refusals of the post-training entry points (no GPU needed: every call fails
its argument checks, which come before any CUDA call)."""

import math

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd

FAKE = 0x7F0000000000  # 1024-aligned fake device address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    from chunked_kl_loss_chunk_b200 import build
    build.build()
    return kd.load()


def _head(call, **kw):
    a = dict(h=FAKE, W=FAKE, dtype=kd.KD_DTYPE_BF16, T=256, d=256, V=4096, targets=FAKE, chunk=64, tau=1.0, keep=0,
             logp=FAKE, lse=FAKE, g=FAKE, gl=None, dH=FAKE, dW=FAKE, dWt=0, acc=0, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    head = (a["h"], a["W"], a["dtype"], a["T"], a["d"], a["V"], a["targets"], a["chunk"], a["tau"])
    if call == "fwd":
        return kd.kd_head_logprob_fwd(*head, a["keep"], a["logp"], a["lse"], a["ws"], a["ws_bytes"], None)
    return kd.kd_head_logprob_bwd(*head, a["lse"], FAKE if a["keep"] else None, a["g"], a["gl"], a["dH"], a["dW"], a["dWt"], a["acc"], a["ws"],
                                  a["ws_bytes"], None)


@pytest.mark.parametrize("call", ["fwd", "bwd"])
def test_head_logprob_refusals(call):
    for kw in (dict(h=None), dict(W=None), dict(targets=None), dict(T=0), dict(chunk=0), dict(tau=0.0), dict(V=0),
               dict(tau=math.nan), dict(h=FAKE + 8), dict(targets=FAKE + 2), dict(ws=None), dict(ws=FAKE + 256),
               dict(lse=None), dict(lse=FAKE + 2)):
        assert _head(call, **kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(dtype=7), dict(d=12), dict(V=2 ** 31), dict(T=1 << 40), dict(T=1 << 31, chunk=1 << 31)):
        assert _head(call, **kw) == kd.KD_ERR_UNSUPPORTED, kw
    assert _head(call, ws_bytes=1024) == kd.KD_ERR_WORKSPACE
    # what the forward keeps has to fit one group of two chunks, and its workspace
    assert _head(call, keep=1, T=513) == _head(call, keep=1, T=600, chunk=299) == kd.KD_ERR_UNSUPPORTED
    assert _head(call, keep=1, chunk=128, ws_bytes=kd.kd_head_logprob_workspace_size(256, 256, 4096, 128, 1, 1)) \
        == kd.KD_ERR_WORKSPACE
    if call == "fwd":
        assert _head(call, logp=None) == kd.KD_ERR_INVALID_ARG
    else:
        assert _head(call, g=None) == kd.KD_ERR_INVALID_ARG
        assert _head(call, dH=None, dW=None) == kd.KD_ERR_INVALID_ARG
        assert _head(call, gl=FAKE + 2) == kd.KD_ERR_INVALID_ARG
        # a bf16 dW: of bf16 operands, formed in one go, not added to
        for kw in (dict(dWt=2), dict(dWt=1, T=513), dict(dWt=1, T=600, chunk=299), dict(dWt=1, chunk=256, acc=1),
                   dict(dWt=1, chunk=256, dtype=kd.KD_DTYPE_F32)):
            assert _head(call, **kw) == kd.KD_ERR_UNSUPPORTED, kw


def test_policy_factors_beyond_fp32():
    """kl_coef and 1 / denom are used in fp32: an infinite one would turn zeros into NaN."""
    for kw in (dict(kl=1e39), dict(kl=-1e39), dict(red=2, denom=1e-39), dict(red=2, denom=5e-324)):
        assert _policy(**kw) == kd.KD_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("name", ["grad", "stream"])
def test_step_options(name):
    """A step needs the objective's gradient, and the objective on the step's stream."""
    from chunked_kl_loss_chunk_b200 import posttrain
    h, W, targets = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(TypeError, match=name):
        posttrain.policy_step(h, W, targets, None, torch.zeros(2), chunk=4, **{name: None})
    with pytest.raises(TypeError, match=name):
        posttrain.preference_step(h, W, targets, chunk=4, **{name: None})


def test_head_workspace_sizes():
    size = kd.kd_head_logprob_workspace_size
    fwd, both = (size(2048, 4096, 131072, 2048, kd.KD_DTYPE_BF16, b) for b in (0, 1))
    assert 0 < fwd < 20 << 20 and both >= 2 * 2048 * 131072 * 2
    assert both == kd.kd_fused_kl_workspace_size(2048, 4096, 131072, 1, 2048, kd.KD_DTYPE_BF16)
    assert size(0, 8, 8, 1, 1, 0) == 0
    kept = size(2048, 4096, 131072, 2048, kd.KD_DTYPE_BF16, kd.KD_HEAD_KEEP)
    assert both < kept <= both + 2048 * 131072 // 4 and size(600, 64, 500, 299, 1, kd.KD_HEAD_KEEP) == 0
    # chunks of less than a tile's rows are taken as 256
    assert size(512, 64, 500, 1, 1, kd.KD_HEAD_KEEP) == size(512, 64, 500, 256, 1, kd.KD_HEAD_KEEP) > 0
    # the forward's need is refused by the backward, and accepted by the forward's own check
    assert _head("bwd", ws_bytes=kd.kd_head_logprob_workspace_size(256, 256, 4096, 64, 1, 0)) == kd.KD_ERR_WORKSPACE


def _policy(**kw):
    a = dict(logp=FAKE, old=FAKE, ref=FAKE, adv=FAKE, per=0, mask=FAKE, cu=None, S=8, N=64, lo=0.2, hi=0.2, kl=0.1,
             red=0, denom=0.0, loss=FAKE, stats=FAKE, g=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return kd.kd_policy_loss(a["logp"], a["old"], a["ref"], a["adv"], a["per"], a["mask"], a["cu"], a["S"], a["N"],
                             a["lo"], a["hi"], a["kl"], a["red"], a["denom"], a["loss"], a["stats"], a["g"], a["ws"],
                             a["ws_bytes"], None)


def test_policy_refusals():
    for kw in (dict(logp=None), dict(adv=None), dict(loss=None), dict(stats=None), dict(ws=None),
               dict(logp=FAKE + 2), dict(old=FAKE + 1), dict(ref=FAKE + 2), dict(g=FAKE + 3),
               dict(per=1, adv=FAKE + 2), dict(adv=FAKE + 2), dict(ws=FAKE + 512), dict(cu=FAKE + 2),
               dict(S=0), dict(N=0), dict(S=-1), dict(N=65), dict(lo=-0.1), dict(lo=1.5), dict(lo=math.nan),
               dict(hi=-0.1), dict(hi=math.nan), dict(kl=math.nan), dict(kl=math.inf), dict(kl=0.1, ref=None),
               dict(red=3), dict(red=-1), dict(red=2), dict(red=2, denom=-1.0), dict(red=2, denom=math.inf)):
        assert _policy(**kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(N=2 ** 31), dict(N=2 ** 31 - 1023, cu=FAKE), dict(S=2 ** 31, cu=FAKE)):
        assert _policy(**kw) == kd.KD_ERR_UNSUPPORTED, kw
    assert _policy(ws_bytes=1024) == kd.KD_ERR_WORKSPACE
    # slices of a batch: the elements' alignment is enough
    assert _policy(ws_bytes=1024, logp=FAKE + 4, old=FAKE + 8, mask=FAKE + 1, adv=FAKE + 4, g=FAKE + 12) == kd.KD_ERR_WORKSPACE
    assert kd.kd_policy_loss_workspace_size(0, 5) == 0 == kd.kd_policy_loss_workspace_size(5, 2 ** 31)


def _pref(**kw):
    a = dict(logp=FAKE, ref=FAKE, mask=FAKE, cu=None, B=4, N=64, kind=0, beta=0.1, margin=0.0, eps=0.0, norm=0,
             total=4, loss=FAKE, rew=FAKE, g=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return kd.kd_preference_loss(a["logp"], a["ref"], a["mask"], a["cu"], a["B"], a["N"], a["kind"], a["beta"],
                                 a["margin"], a["eps"], a["norm"], a["total"], a["loss"], a["rew"], a["g"], a["ws"],
                                 a["ws_bytes"], None)


def test_preference_refusals():
    for kw in (dict(logp=None), dict(loss=None), dict(rew=None), dict(ws=None), dict(logp=FAKE + 2),
               dict(ref=FAKE + 1), dict(g=FAKE + 2), dict(cu=FAKE + 1), dict(B=0), dict(N=0),
               dict(N=65), dict(kind=3), dict(kind=-1), dict(beta=0.0), dict(beta=-1.0), dict(beta=math.inf),
               dict(margin=math.nan), dict(eps=0.5), dict(eps=-0.1), dict(kind=2, margin=0.5), dict(kind=1, eps=0.1),
               dict(kind=2, eps=0.1), dict(total=3)):
        assert _pref(**kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(N=2 ** 31), dict(B=2 ** 30, total=2 ** 30, cu=FAKE)):
        assert _pref(**kw) == kd.KD_ERR_UNSUPPORTED, kw
    assert _pref(ws_bytes=1024) == kd.KD_ERR_WORKSPACE
    assert _pref(ws_bytes=1024, logp=FAKE + 4, ref=FAKE + 8, mask=FAKE + 3, g=FAKE + 4) == kd.KD_ERR_WORKSPACE
    assert kd.kd_preference_loss_workspace_size(0, 5) == 0 == kd.kd_preference_loss_workspace_size(2 ** 30, 5)


def test_python_refusals_without_a_gpu():
    x, a = torch.zeros(4, 8), torch.zeros(4)
    with pytest.raises(TypeError):
        kd.policy_loss(x.double(), x, a) if torch.cuda.is_available() else kd.policy_loss([1.0], x, a)
    for call in (lambda: kd.policy_loss(x, x, a), lambda: kd.preference_loss(x)):
        with pytest.raises(ValueError, match="CUDA device"):      # there is no CPU fallback
            call()


def _clip(n=2, grads=(FAKE, FAKE + 4096), outs=(FAKE, FAKE + 4096), sizes=(100, 7), types=(0, 1), max_norm=1.0,
          sumsq=None, norm=FAKE, ws=FAKE, ws_bytes=1 << 40, what="clip"):
    import ctypes
    arr = lambda t, v: None if v is None else (t * max(len(v), 1))(*v)  # noqa: E731
    g, o = arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs)
    s, t = arr(ctypes.c_int64, sizes), arr(ctypes.c_int, types)
    if what == "sumsq":
        return kd.kd_grad_sumsq(g, s, t, n, norm, ws, ws_bytes, None)
    return kd.kd_grad_clip(g, o, s, t, n, max_norm, sumsq, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("what", ["clip", "sumsq"])
def test_grad_refusals(what):
    for kw in (dict(n=0), dict(n=-1), dict(grads=None), dict(sizes=None), dict(types=None), dict(norm=None),
               dict(norm=FAKE + 2), dict(ws=None), dict(ws=FAKE + 512), dict(sizes=(100, -1)),
               dict(grads=(None, FAKE), outs=(FAKE + 64, FAKE)), dict(grads=(FAKE + 2, FAKE + 4096)),
               dict(grads=(FAKE, FAKE + 4097))):
        assert _clip(what=what, **kw) == kd.KD_ERR_INVALID_ARG, kw
    assert _clip(what=what, types=(0, 2)) == kd.KD_ERR_UNSUPPORTED
    assert _clip(what=what, sizes=(1 << 40, 7), outs=(FAKE, FAKE)) == kd.KD_ERR_UNSUPPORTED
    assert _clip(what=what, ws_bytes=1024) == kd.KD_ERR_WORKSPACE
    assert kd.kd_grad_clip_workspace_size(0) == 0
    assert kd.kd_grad_clip_workspace_size(5000) > kd.kd_grad_clip_workspace_size(999)


def test_grad_clip_refuses_shared_memory():
    bad = kd.KD_ERR_INVALID_ARG
    far = FAKE + (1 << 20)
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(outs=None), dict(outs=(None, FAKE)),
               dict(sumsq=FAKE + 4), dict(outs=(FAKE + 2, FAKE + 4096)),
               dict(grads=(FAKE, FAKE), outs=(FAKE, FAKE)),                         # the same one twice
               dict(grads=(FAKE, FAKE + 396), outs=(FAKE, FAKE + 396)),             # the last 4 bytes
               dict(grads=(FAKE, far), outs=(far, FAKE)),                           # exchanged
               dict(grads=(FAKE, far), outs=(far + 12, far + 64)),                  # an output on a gradient
               dict(grads=(FAKE, far), outs=(FAKE + 4, far)),                       # on its own, shifted
               dict(grads=(FAKE, far), outs=(far + 4096, far + 4096 + 398))):       # two outputs
        assert _clip(**kw) == bad, kw
    # what only touches, and gradients that share memory but are only read, pass on to the next check
    for kw in (dict(grads=(FAKE, FAKE + 400), outs=(FAKE, FAKE + 400)),
               dict(grads=(FAKE, FAKE + 4), outs=(far, far + 400)),
               dict(grads=(FAKE, FAKE), outs=(FAKE, FAKE), sizes=(100, 0))):
        assert _clip(ws_bytes=16, **kw) == kd.KD_ERR_WORKSPACE, kw
