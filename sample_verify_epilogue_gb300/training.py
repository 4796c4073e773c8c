"""Training on decoded tokens as differentiable torch functions, and gradient clipping.

``token_logprobs``, ``policy_loss`` and ``preference_loss`` run the library's call of that name in their forward pass and
its backward call in their backward pass, each on torch's current stream at that time; the gradient reaches the logits
alone: old and reference log-probabilities, advantages and weights are constants.  A training loop that knows its
weights beforehand gets loss and gradient together from ``binding.dspark_policy_loss(..., grad=...)`` and
``binding.dspark_preference_loss(..., grad=...)`` instead.

Rows have to be evenly spaced: for logits [B, T, V] whose position t predicts token t + 1, pass all of them with the tokens
moved up by one and -1 at the last position, rather than ``logits[:, :-1]``.  A step is captured into a CUDA graph with
``torch.autograd.grad``, or ``backward`` while no eager graph of the same leaves is alive.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding


def _like(t, *shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=t.device)


def _saved(ctx, logits, rows):
    return _like(logits, *rows, binding.DSPARK_SAVED_FLOATS) if ctx.needs_input_grad[0] else None


def _grad(logits):
    return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)


def _contiguous(t):
    return None if t is None else t.contiguous()


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature):
        rows = logits.shape[:-1]
        logprobs, entropy, status = _like(logits, *rows), _like(logits, *rows), _like(logits, *rows, dtype=torch.int32)
        saved = _saved(ctx, logits, rows)
        binding.dspark_token_logprobs(logits, tokens, logprobs=logprobs, entropy=entropy, row_status=status, saved=saved,
                                      temperature=temperature)
        ctx.save_for_backward(logits, tokens, saved)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(status)
        return logprobs, entropy, status

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logprobs, grad_entropy, _):
        logits, tokens, saved = ctx.saved_tensors
        if grad_logprobs is None and grad_entropy is None:
            return None, None, None
        grad = _grad(logits)
        binding.dspark_token_logprobs_backward(logits, tokens, saved=saved, grad=grad, grad_logprobs=_contiguous(grad_logprobs),
                                               grad_entropy=_contiguous(grad_entropy), temperature=ctx.temperature)
        return grad, None, None


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, old, advantages, ref, weights, options):
        rows = logits.shape[:-1]
        loss, logprobs, status = _like(logits, *rows), _like(logits, *rows), _like(logits, *rows, dtype=torch.int32)
        saved = _saved(ctx, logits, rows)
        binding.dspark_policy_loss(logits, tokens, old, advantages, loss=loss, row_status=status, logprobs=logprobs, saved=saved,
                                   ref_logprobs=ref, weights=weights, **options)
        ctx.save_for_backward(logits, tokens, old, advantages, ref, weights, saved)
        ctx.options = options
        ctx.mark_non_differentiable(logprobs, status)
        return loss, logprobs, status

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, *_):
        logits, tokens, old, advantages, ref, weights, saved = ctx.saved_tensors
        grad = _grad(logits)
        binding.dspark_policy_loss_backward(logits, tokens, old, advantages, saved=saved, grad=grad, grad_loss=grad_loss.contiguous(),
                                            ref_logprobs=ref, weights=weights, **ctx.options)
        return grad, None, None, None, None, None, None


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, row_offsets, ref, weights, options):
        rows, pairs = logits.shape[:-1], (row_offsets.numel() - 1) // 2
        loss, rewards, pair_status = _like(logits, pairs), _like(logits, pairs, 2), _like(logits, pairs, dtype=torch.int32)
        saved = _like(logits, *rows, binding.DSPARK_SAVED_FLOATS)
        binding.dspark_preference_loss(logits, tokens, row_offsets, loss=loss, saved=saved,
                                       row_status=_like(logits, *rows, dtype=torch.int32), pair_status=pair_status, rewards=rewards,
                                       ref_logprobs=ref, weights=weights, **options)
        ctx.save_for_backward(logits, tokens, saved)
        ctx.temperature = options["temperature"]
        ctx.mark_non_differentiable(rewards, pair_status)
        return loss, rewards, pair_status

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, *_):
        logits, tokens, saved = ctx.saved_tensors
        grad = _grad(logits)
        binding.dspark_preference_loss_backward(logits, tokens, saved=saved, grad=grad, grad_loss=grad_loss.contiguous(),
                                                temperature=ctx.temperature)
        return grad, None, None, None, None, None


def token_logprobs(logits, tokens, *, temperature=1.0):
    """(log-probability, entropy, status) of every row of logits [..., V] at its token [...] int32 (-1: none): see
    dspark_token_logprobs.  Log-probability and entropy are differentiable."""
    return _TokenLogprobs.apply(logits, tokens, temperature)


def policy_loss(logits, tokens, old_logprobs, advantages, *, ref_logprobs=None, weights=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, entropy_coef=0.0, temperature=1.0):
    """(loss, log-probability, status) of every row of logits [..., V]: see dspark_policy_loss.  The loss is differentiable."""
    return _PolicyLoss.apply(logits, tokens, old_logprobs, advantages, ref_logprobs, weights,
                             dict(clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef, entropy_coef=entropy_coef,
                                  temperature=temperature))


def preference_loss(logits, tokens, row_offsets, *, ref_logprobs=None, weights=None, beta=0.1, margin=0.0, label_smoothing=0.0,
                    mean=False, temperature=1.0):
    """(loss [P], rewards [P, 2], status [P]) of the pairs of sequences that row_offsets [2P + 1] cuts logits [..., V] into:
    see dspark_preference_loss.  The loss is differentiable."""
    return _PreferenceLoss.apply(logits, tokens, row_offsets, ref_logprobs, weights,
                                 dict(beta=beta, margin=margin, label_smoothing=label_smoothing, mean=mean, temperature=temperature))


def clip_grads_(parameters, max_norm):
    """Scale the gradients of ``parameters`` (or of one) in place so that their norm taken together is at most max_norm; (norm
    before, status) on the GPU, each [1]: see dspark_clip_grads.  Parameters without a gradient are left out; where none has one
    the norm is 0.  A loop whose gradients stay where they are makes a ``binding.GradTable`` and its buffers once and calls
    ``binding.dspark_clip_grads``."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = [p.grad for p in parameters]
    if parameters and all(g is None for g in grads):
        return torch.zeros(1, device=parameters[0].device), torch.zeros(1, dtype=torch.int32, device=parameters[0].device)
    table = binding.GradTable(grads)
    first = table.tensors[0][0]
    norm, status = _like(first, 1), _like(first, 1, dtype=torch.int32)
    workspace = _like(first, binding.dspark_clip_workspace_bytes(table), dtype=torch.uint8)
    binding.dspark_clip_grads(table, max_norm, norm=norm, status=status, workspace=workspace)
    return norm, status
