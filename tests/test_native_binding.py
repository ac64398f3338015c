"""The C++ half of the Python binding (_kd_native), on the CPU: it takes the usual
case only and leaves everything else, by None, to kd.py's own checks."""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd


@pytest.fixture(scope="module", autouse=True)
def lib():
    from chunked_kl_loss_chunk_b200 import build
    build.build()
    return kd.load()


def test_none_for_what_is_not_on_a_gpu():
    x, a = torch.zeros(4, 8), torch.zeros(4)
    n = kd._native
    assert n.policy_loss(x, x, None, a, False, None, None, 0.2, 0.2, 0.0, 0, 0.0, True, None) is None
    assert n.preference_loss(x, None, None, None, 0, 0.1, 0.0, 0.0, False, None, True, None) is None
    assert n.head_logprobs(x, x, a.int(), 4, 1.0, 0, None) is None
    assert n.head_logprobs_bwd(x, x, a.int(), a, None, a, None, 4, 1.0, True, True, False, None) is None
    assert n.clip_grad_norm([x, a], None, 1.0, None) is None
    assert n.clip_grad_norm([], None, 1.0, None) is None


@pytest.mark.parametrize("bad", [None, 3, "x", [1.0], object()])
def test_none_for_what_is_no_tensor(bad):
    n = kd._native
    x = torch.zeros(4, 8)
    assert n.policy_loss(bad, x, None, x, False, None, None, 0.2, 0.2, 0.0, 0, 0.0, True, None) is None
    assert n.preference_loss(bad, None, None, None, 0, 0.1, 0.0, 0.0, False, None, True, None) is None
    assert n.head_logprobs(bad, x, x, 4, 1.0, 0, None) is None
    assert n.clip_grad_norm([bad], None, 1.0, None) is None
    assert n.clip_grad_norm(bad, None, 1.0, None) is None
    with pytest.raises((TypeError, ValueError)):
        kd.policy_loss(bad, x, x)
    with pytest.raises((TypeError, ValueError)):
        kd.clip_grad_norm([bad], 1.0)


def test_wrong_number_of_arguments():
    n = kd._native
    for f in (n.policy_loss, n.preference_loss, n.head_logprobs, n.head_logprobs_bwd, n.clip_grad_norm):
        with pytest.raises(TypeError):
            f(1, 2)
    with pytest.raises(TypeError):
        kd._native.bind(1)
