"""The distillation loss as a differentiable torch function.

``distill_loss`` runs dspark_distill in its forward pass and dspark_distill_backward in its backward
pass, each on torch's current stream at that time; the gradient reaches the student's logits
alone.  A training loop that knows its row weights beforehand gets loss and gradient from one
launch with ``dspark_distill(..., grad=...)`` instead.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, student, teacher_ids, teacher_logits, teacher_lse, t2d, weights, temperature):
        rows = student.shape[:-1]
        loss = torch.empty(rows, dtype=torch.float32, device=student.device)
        status = torch.empty(rows, dtype=torch.int32, device=student.device)
        saved = torch.empty(*rows, 4, dtype=torch.float32, device=student.device)
        binding.dspark_distill(student, teacher_ids, teacher_logits, loss=loss, row_status=status, saved=saved,
                               teacher_lse=teacher_lse, t2d=t2d, weights=weights, temperature=temperature)
        ctx.save_for_backward(student, teacher_ids, teacher_logits, teacher_lse, t2d, weights, saved)
        ctx.temperature, ctx.status = temperature, status
        ctx.mark_non_differentiable(status)
        return loss, status

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, _):
        student, ids, logits, lse, t2d, weights, saved = ctx.saved_tensors
        grad = torch.empty(student.shape, dtype=student.dtype, device=student.device)
        binding.dspark_distill_backward(student, ids, logits, saved=saved, grad=grad, grad_loss=grad_loss.contiguous(),
                                        teacher_lse=lse, t2d=t2d, weights=weights, temperature=ctx.temperature,
                                        row_status=ctx.status)
        return grad, None, None, None, None, None, None


def distill_loss(student, teacher_ids, teacher_logits, teacher_lse=None, *, t2d=None, weights=None, temperature=1.0):
    """(loss, status) of every row of student [..., V]: see dspark_distill for the arguments.

    The teacher's record, ``teacher_lse`` and ``weights`` are constants: no gradient reaches them.  The
    backward pass adds to status, where a row's copies did not come in time (DSPARK_ROW_INTERNAL).
    """
    return _DistillLoss.apply(student, teacher_ids, teacher_logits, teacher_lse, t2d, weights, temperature)
