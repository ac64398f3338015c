"""Clipping of a data-parallel step's gradients to the norm over the whole batch
(host logic, on CPU with two gloo ranks; the kernels are stood in for)."""

import math

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from test_multirank import _free_port


def _compute(grads, max_norm, sumsq=None):
    """Plain fp64 in the place of libkd's kernels."""
    if max_norm is None:
        return sum(t.double().square().sum() for t in grads)
    norm = sumsq.sqrt()
    for t in grads:
        t.mul_(min(1.0, max_norm / (norm.item() + 1e-6)))
    return norm.float()


def _batch(rows):
    gen = torch.Generator().manual_seed(7)
    return (torch.randn((5, 4), generator=gen, dtype=torch.float64),
            torch.randn((rows, 4), generator=gen, dtype=torch.float64))


def _rank(rank, world, port, out):
    import datetime
    import os
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from chunked_kl_loss_chunk_b200 import dp
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=60))
    try:
        res = []
        for rows in (7, 1):                       # rank 1 holds three rows, then none
            dW, dH = _batch(rows)
            sh = dp.shard_rows(rows, world, rank)
            mine = dH[sh.row0:sh.row0 + sh.rows].clone()
            norm = dp.clip_grad_norm([dW], [mine], 0.5, compute=_compute)
            res.append((float(norm), dW.tolist(), mine.tolist()))
        only = torch.full((3,), 2.0, dtype=torch.float64) if rank == 0 else torch.zeros(0, dtype=torch.float64)
        res.append(float(dp.clip_grad_norm([], [only], 100.0, compute=_compute, device="cpu")))
        out[rank] = res
    finally:
        dist.destroy_process_group()


def test_two_ranks_clip_to_the_batch_norm():
    with mp.get_context("spawn").Manager() as mgr:
        out = mgr.dict()
        mp.start_processes(_rank, args=(2, _free_port(), out), nprocs=2, join=True, start_method="spawn")
        res = dict(out)
    for k, rows in enumerate((7, 1)):
        dW, dH = _batch(rows)
        norm = math.sqrt(float(dW.square().sum() + dH.square().sum()))
        c = min(1.0, 0.5 / (norm + 1e-6))
        got_rows = []
        for rank in (0, 1):
            n, w, h = res[rank][k]
            assert n == pytest.approx(norm, rel=1e-6)
            assert torch.allclose(torch.tensor(w, dtype=torch.float64), c * dW, rtol=1e-12)
            got_rows += h
        assert torch.allclose(torch.tensor(got_rows, dtype=torch.float64), c * dH, rtol=1e-12)
    assert res[0][2] == res[1][2] == pytest.approx(math.sqrt(12.0), rel=1e-6)


def test_one_process_and_nothing_to_clip():
    from chunked_kl_loss_chunk_b200 import dp
    w = torch.full((4,), 3.0, dtype=torch.float64)
    assert float(dp.clip_grad_norm([w], [], 1.0, compute=_compute)) == pytest.approx(6.0)
    assert torch.allclose(w, torch.full((4,), 0.5, dtype=torch.float64), rtol=1e-6)
    assert float(dp.clip_grad_norm([], [], 1.0, compute=_compute)) == 0.0
