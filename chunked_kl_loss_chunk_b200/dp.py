"""Data-parallel sharding of the fused chunked KL loss along the positions.

The loss is a mean over the T_total positions of a batch and every position's
terms (its logsumexp, its KL, its row of dz and of dH) depend on that position
alone; only dW = dz^T h sums over positions.  So a batch splits along T over
ranks with no exchange inside the loss: each rank runs the fused forward and
backward on its own contiguous block of rows, normalised by the batch's
T_total (``kd_fused_kl_fwd_shard`` / ``kd_fused_kl_bwd_shard``), and then one
all-reduce (sum) of the scalar loss and of dW [V, d] fp32 over the ranks gives
the batch's loss and dW.  dH needs no exchange: each rank holds exactly the
batch gradient's rows of its shard.

The pages run the method on a single GPU; they describe the multi-node
sharding it made unnecessary (goaixin.org, "Breaking the Memory Barrier ...",
section "Detailed Chronology and Technical Evolution"; andresseo.expert,
section "What a Single H200 GPU Can Now Do That Once Required Four Nodes").
This module is the plain data-parallel form of the same loss.

Host logic only: the per-shard work runs in libkd's kernels, the exchange in
``torch.distributed`` (NCCL on GPUs, gloo on CPU).  ``shard_step`` takes the
per-shard computation as an argument so that the partitioning, the
normalisation and the reduction can be exercised on CPU ranks.
"""

from __future__ import annotations

from typing import Callable, NamedTuple

import torch
import torch.distributed as dist


class Shard(NamedTuple):
    row0: int      # first position of this rank's block
    rows: int      # positions in the block (0 when T_total < world)


def shard_rows(T_total: int, world: int, rank: int) -> Shard:
    """Contiguous, balanced split of T_total positions over `world` ranks: the
    first T_total % world ranks get one position more.  Blocks tile
    [0, T_total) in rank order."""
    if T_total < 0 or world < 1 or not (0 <= rank < world):
        raise ValueError("need T_total >= 0, world >= 1 and 0 <= rank < world")
    base, extra = divmod(T_total, world)
    rows = base + (1 if rank < extra else 0)
    row0 = rank * base + min(rank, extra)
    return Shard(row0, rows)


def kd_shard_compute(h, W, t_vals, t_idx, T_total: int, chunk: int, temperature: float = 1.0,
                     cache: str = "logits", tau_squared: bool = False, grad_loss=None):
    """One rank's shard on the GPU: (loss part [] f32, dH [rows, d], dW part
    [V, d] f32), all from libkd's kernels."""
    from chunked_kl_loss_chunk_b200 import kd
    loss, lse, _, ws = kd.fused_kl_fwd(h, W, t_vals, t_idx, chunk, temperature, cache=cache,
                                       tau_squared=tau_squared, T_total=T_total)
    dH, dW, _ = kd.fused_kl_bwd(h, W, t_vals, t_idx, lse, chunk, temperature, grad_loss=grad_loss,
                                ws=ws, cache=cache, tau_squared=tau_squared, T_total=T_total)
    return loss, dH, dW


def shard_step(h, W, t_vals, t_idx, T_total: int, chunk: int, temperature: float = 1.0, *,
               compute: Callable = kd_shard_compute, group=None, dtype=torch.float32, **kw):
    """Loss and gradients of a batch of T_total positions of which this rank
    holds the rows in `h`, `t_vals`, `t_idx` (its ``shard_rows`` block).

    Returns (loss, dH, dW): the batch's loss and dW, identical on every rank
    after the all-reduce, and dH for this rank's rows.  A rank with no rows
    contributes zeros and still joins both collectives, so every rank takes the
    same collective steps in the same order.  `dtype` is the type of the loss
    and dW that `compute` returns (fp32 for libkd)."""
    rows = h.shape[0]
    V, d = W.shape
    if rows > 0:
        loss, dH, dW = compute(h, W, t_vals, t_idx, T_total, chunk, temperature, **kw)
        loss = loss.reshape(1)
    else:
        loss = torch.zeros(1, dtype=dtype, device=W.device)
        dH = torch.empty((0, d), dtype=h.dtype, device=W.device)
        dW = torch.zeros((V, d), dtype=dtype, device=W.device)
    world = dist.get_world_size(group) if dist.is_available() and dist.is_initialized() else 1
    if world > 1:
        dist.all_reduce(dW, op=dist.ReduceOp.SUM, group=group)
        dist.all_reduce(loss, op=dist.ReduceOp.SUM, group=group)
    return loss.reshape(()), dH, dW


def kd_clip_compute(grads, max_norm, sumsq=None):
    """The sum of squares of `grads` (max_norm None), or their clipping in place
    with a given one, in libkd's kernels."""
    from chunked_kl_loss_chunk_b200 import kd
    if max_norm is None:
        return kd.grad_sumsq(grads)
    return kd.clip_grad_norm(grads, max_norm, sumsq=sumsq)


def clip_grad_norm(replicated, sharded, max_norm: float, *, compute: Callable = kd_clip_compute,
                   group=None, device=None):
    """Clips the parameters' gradients of a data-parallel step in place to their norm
    over the whole batch, and returns that norm (the same on every rank).  (dH is the
    gradient of an activation; what the trunk makes of it belongs here, dH does not.)

    `replicated`: tensors that every rank holds alike (dW after ``shard_step``), counted
    once whichever ranks hold them, but a rank holds all of them or none; `sharded`: each
    rank's own part of gradients that are split over the ranks (optimiser shards, rows of
    an embedding), whose sums of squares are added.
    Either may be empty, also on some ranks only: every rank joins the one all-reduce
    (of three fp64 values on `device`, by default the tensors')."""
    replicated = [t for t in replicated if t.numel()]
    sharded = [t for t in sharded if t.numel()]
    both = replicated + sharded
    if device is None:
        device = both[0].device if both else torch.device("cpu")
    zero = torch.zeros((), dtype=torch.float64, device=device)
    # sums of squares of the two lists, and whether this rank holds the first: the mean over
    # the ranks that do counts the replicated tensors once, and is the same on every rank
    parts = torch.stack([compute(sharded, None) if sharded else zero,
                         compute(replicated, None) if replicated else zero,
                         zero + float(bool(replicated))])
    world = dist.get_world_size(group) if dist.is_available() and dist.is_initialized() else 1
    if world > 1:
        dist.all_reduce(parts, op=dist.ReduceOp.SUM, group=group)
    total = parts[0] + parts[1] / parts[2].clamp(min=1.0)
    if both:
        return compute(both, max_norm, total)
    return total.sqrt().to(torch.float32)
