"""Clipping of a data-parallel step's gradients where a rank holds none of the
replicated tensors (host logic, on CPU with gloo ranks; the kernels are stood in for):
every rank must get the batch's norm and clip with it."""

import math

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from test_dp_clip import _compute
from test_multirank import _free_port


def _tensors():
    gen = torch.Generator().manual_seed(11)
    return (torch.randn((6, 4), generator=gen, dtype=torch.float64),
            [torch.randn((3, 4), generator=gen, dtype=torch.float64) for _ in range(3)])


# which of the three ranks hold the replicated tensor, and which a part of the sharded one
HOLDERS = [((0, 1, 2), (0, 1, 2)), ((0,), (0, 1, 2)), ((1, 2), (0, 2)), ((2,), ()), ((), (1,)), ((), ())]


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
        for rep, sha in HOLDERS:
            W, parts = _tensors()
            replicated = [W] if rank in rep else []
            sharded = [parts[rank]] if rank in sha else []
            norm = dp.clip_grad_norm(replicated, sharded, 0.5, compute=_compute, device="cpu")
            res.append((float(norm), W.tolist(), parts[rank].tolist()))
        out[rank] = res
    finally:
        dist.destroy_process_group()


def test_a_rank_without_replicated_tensors_clips_alike():
    with mp.get_context("spawn").Manager() as mgr:
        out = mgr.dict()
        mp.start_processes(_rank, args=(3, _free_port(), out), nprocs=3, join=True, start_method="spawn")
        res = dict(out)
    for k, (rep, sha) in enumerate(HOLDERS):
        W, parts = _tensors()
        total = (float(W.square().sum()) if rep else 0.0) + sum(float(parts[r].square().sum()) for r in sha)
        norm = math.sqrt(total)
        c = min(1.0, 0.5 / (norm + 1e-6))
        for rank in range(3):
            n, w, part = res[rank][k]
            assert n == pytest.approx(norm, rel=1e-6), (k, rank)
            assert torch.allclose(torch.tensor(w, dtype=torch.float64), (c if rank in rep else 1.0) * W, rtol=1e-12)
            assert torch.allclose(torch.tensor(part, dtype=torch.float64), (c if rank in sha else 1.0) * parts[rank],
                                  rtol=1e-12)
