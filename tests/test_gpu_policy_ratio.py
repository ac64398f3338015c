"""The mean ratio that the policy loss reports, where the ratios are far below one
and most tokens do not count.

Tolerance: the sum of a lane's ratios is of at most 64 positive terms in fp32, each
off by the 2^-22 of the hardware's 2^x and |x| 2^-24 of its argument (|x| < 32); the
rest is in fp64 and rounded once: (63 + 2 + 32 + 4 + 1) 2^-24 is below 2^-17.
"""

import pytest
import torch

from chunked_kl_loss_chunk_b200 import kd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [64, 2000])        # in one block, and in several
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shift", [-20.0, -12.0, 0.0, 8.0])
def test_mean_ratio_of_a_masked_batch(length, packed, shift):
    require_gpu()
    S = 16
    gen = torch.Generator("cuda").manual_seed(3)
    logp = -torch.rand((S, length), generator=gen, device="cuda") - 1.0
    old = logp - shift
    mask = torch.arange(S * length, device="cuda").view(S, length) % 4 == 1
    mask[3] = False
    adv = torch.ones(S, device="cuda")
    kw = {}
    if packed:
        logp, old, mask = logp.view(-1), old.view(-1), mask.view(-1)
        kw["cu_seqlens"] = torch.arange(S + 1, dtype=torch.int32, device="cuda") * length
    stats = kd.policy_loss(logp, old, adv, mask=mask, **kw)[1]
    want = torch.exp(logp.double() - old.double())[mask].mean().item()
    assert stats[0].item() == mask.sum().item()
    assert abs(stats[1].item() - want) <= 2 ** -17 * want
    everything = kd.policy_loss(logp, old, adv, **kw)[1]
    want = torch.exp(logp.double() - old.double()).mean().item()
    assert abs(everything[1].item() - want) <= 2 ** -17 * want
