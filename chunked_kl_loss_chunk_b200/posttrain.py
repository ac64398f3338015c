"""Post-training steps through the output head: tokens in, gradients of h and W out.

What follows distillation trains the same head on sampled or compared answers.
A step is three calls of ``kd``: the log-probabilities of the answers' tokens
(``head_logprobs``), an objective over them with its gradient for each token
(``policy_loss`` or ``preference_loss``), and the way of that gradient back into
h and W (``head_logprobs_bwd``); the [T, V] logits are never materialised, and
one workspace serves both passes through the head.  dH goes back into the trunk
behind the head; ``kd.clip_grad_norm`` (or ``dp.clip_grad_norm`` over ranks) then clips
dW together with the trunk's parameter gradients.  (dH itself is no parameter's gradient
and has no part in that norm.)

Positions without a target may hold anything, NaN included, in h as in the arrays of the
objectives.

Nothing synchronises, so a step can be captured in a CUDA graph.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from chunked_kl_loss_chunk_b200 import kd


class Step(NamedTuple):
    loss: torch.Tensor        # f32 []
    extra: torch.Tensor       # policy_step: stats f32 [4]; preference_step: rewards f32 [2 pairs]
    logp: torch.Tensor        # f32, like targets
    dH: torch.Tensor          # [T, d], dtype of h
    dW: torch.Tensor          # [V, d] f32
    ws: torch.Tensor          # the head's workspace, for the next step, with the step's errors in device data
                              # (a bad target or cu_seqlens) or its waits for kd.read_device_status


def _through_head(h, W, targets, objective, objective_bytes, cu_seqlens, options, chunk, temperature, ws, dW,
                  accumulate_dW, keep):
    for name in ("grad", "stream"):        # the step needs the gradient, and all of it on one stream
        if name in options:
            raise TypeError(f"{name}: not an option of a step")
    flat = targets.reshape(-1)
    # up to two chunks the forward keeps what the backward needs of the logits (a given workspace
    # decides by its size), unless the caller has decided
    decided = keep is not None
    keep = keep if decided else kd._one_group(h.shape[0], chunk)
    if keep and not decided and ws is not None:
        keep = ws.numel() >= kd.kd_head_logprob_workspace_size(*h.shape, W.shape[0], chunk, kd._dtype_code(h),
                                                               kd.KD_HEAD_KEEP)
    logp, lse, ws = kd.head_logprobs(h, W, flat, chunk, temperature, ws=ws, backward=True, keep=keep)
    status = ws[:4].view(torch.int32)
    # the backward clears the forward's; one that uses what a forward kept has seen it
    found = [] if keep else [status.clone()]
    shaped = logp.view(targets.shape)
    # only packed sequences can be wrong in the objective's device data
    own = None
    if cu_seqlens is not None:
        own = kd.alloc_workspace(objective_bytes(max(cu_seqlens.numel() - 1, 1), flat.numel()), h.device)
    loss, extra, dlogp = objective(shaped, targets != kd.KD_TARGET_IGNORE, own)
    if own is not None:
        found.append(own[:4].view(torch.int32))
    dH, dW, _ = kd.head_logprobs_bwd(h, W, flat, lse, dlogp.view(-1), chunk, temperature, ws=ws, dW=dW,
                                     accumulate_dW=accumulate_dW, kept_logp=logp if keep else None)
    for code in found:                 # of several errors the one that stopped more work
        torch.maximum(status, code, out=status)
    return Step(loss, extra, shaped, dH, dW, ws)


def policy_step(h, W, targets, old_logp, advantages, *, chunk: int, temperature: float = 1.0, ref_logp=None,
                cu_seqlens=None, ws=None, dW=None, accumulate_dW: bool = False, keep: bool | None = None,
                **options) -> Step:
    """Clipped policy loss of sampled answers and its gradients.

    h [T, d], W [V, d]; ``targets`` int32 [sequences, tokens], or [T] with
    ``cu_seqlens``: the sampled token at each position, KD_TARGET_IGNORE where
    there is none (prompts, padding), which is also the loss's mask.
    ``old_logp``, ``ref_logp`` like ``targets``; ``options`` go to
    ``kd.policy_loss`` (clip_low, clip_high, kl_coef, reduction, denom,
    advantages_per).  For micro-batches, ``reduction="fixed"`` with the batch's
    token count and ``accumulate_dW=True`` add up to the batch's gradient.
    ``keep``: whether the forward through the head keeps its exponentials for the
    backward, as in ``kd.head_logprobs``; None: where T is at most two chunks and a
    given ``ws`` is large enough."""
    return _through_head(h, W, targets, lambda logp, mask, own: kd.policy_loss(
        logp, old_logp, advantages, mask=mask, ref_logp=ref_logp, cu_seqlens=cu_seqlens, ws=own, **options),
        kd.kd_policy_loss_workspace_size, cu_seqlens, options, chunk, temperature, ws, dW, accumulate_dW, keep)


def preference_step(h, W, targets, *, chunk: int, temperature: float = 1.0, ref_logp=None, cu_seqlens=None,
                    ws=None, dW=None, accumulate_dW: bool = False, keep: bool | None = None, **options) -> Step:
    """Paired preference loss of compared answers and its gradients.

    ``targets`` as for ``policy_step``, over 2 pairs sequences: the chosen
    answers, then the rejected ones.  ``keep`` as there.  ``options`` go to ``kd.preference_loss``
    (kind, beta, margin, label_smoothing, length_normalize, pairs_total)."""
    return _through_head(h, W, targets, lambda logp, mask, own: kd.preference_loss(
        logp, ref_logp=ref_logp, mask=mask, cu_seqlens=cu_seqlens, ws=own, **options),
        lambda n_seqs, n: kd.kd_preference_loss_workspace_size(max(n_seqs // 2, 1), n), cu_seqlens, options, chunk,
        temperature, ws, dW, accumulate_dW, keep)
