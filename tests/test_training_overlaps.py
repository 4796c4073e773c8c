"""Gradients that share memory with the logits other than as a whole are refused, before any CUDA call (CPU only)."""
import pytest

from tests.test_rows_refusals import bd  # noqa: F401
from tests.test_training_refusals import call

CALLS = ("logprobs_backward", "policy", "policy_backward", "preference", "preference_backward")
AT = 1 << 20


@pytest.mark.parametrize("what", CALLS)
@pytest.mark.parametrize("kw", [
    dict(grad=AT + 2), dict(grad=AT - 2), dict(grad=AT + 18), dict(grad=AT + 38), dict(grad=AT - 38), dict(grad=AT + 20), dict(grad=AT - 20),
    dict(logits_dtype=1, grad=AT + 4), dict(logits_stride=32, grad_stride=32, grad=AT + 18), dict(logits_stride=32, grad_stride=32, grad=AT + 64),
    dict(logits_stride=32, grad_stride=32, grad=AT + 46), dict(logits_stride=32, grad_stride=32, grad=AT - 46), dict(grad_stride=32, grad=AT + 22),
    dict(logits_stride=32, grad=AT + 24), dict(n_rows=1, grad=AT - 18), dict(n_rows=1, logits_stride=1 << 40, grad_stride=1 << 40, grad=AT + 18),
    dict(logits_dtype=1, logits_stride=32, grad_stride=32, grad=AT + 40 * 3 - 4)])
def test_partial_overlaps_are_refused(bd, what, kw):  # noqa: F811
    """Two rows of ten logits (bf16 where nothing else is said): elements that belong to both, or rows of different strides that lie
    among each other."""
    assert call(bd, what, dict(logits=AT, **kw)) == 1


N = 1 << 24                                                  # rows, and logits of each: more than one launch takes, which is an error of its own


@pytest.mark.parametrize("what", [w for w in CALLS if w.endswith("backward")])
@pytest.mark.parametrize("stride,grad_stride,offset", [
    (N, N, N * N), (N, N, -N * N), (2 * N, 2 * N, N), (2 * N, 2 * N, -N), (2 * N, 2 * N, 7 * N), (2 * N + 9, 2 * N + 9, N + 9), (N, N, 0),
    (N, 2 * N, N * N), (2 * N, N, -N * N), (2 * N, N, 2 * N * N - N)])
def test_neighbours_are_taken(bd, what, stride, grad_stride, offset):  # noqa: F811
    """In place, behind or before each other, or row between row: refused for their size alone."""
    at = 1 << 56
    kw = dict(n_rows=N, V=N, logits=at, grad=at + 2 * offset, logits_stride=stride, grad_stride=grad_stride)
    assert call(bd, what, kw) == 2
    for one in (-2, 2):
        assert call(bd, what, kw | dict(grad=at + 2 * offset + one)) == (1 if overlap(stride, grad_stride, 2 * offset + one) else 2)


def overlap(stride, grad_stride, by):
    """Whether N rows of N 2-byte elements, and N others ``by`` bytes on, share any (or the rows of other strides lie among each other)."""
    if by >= 2 * ((N - 1) * stride + N) or -by >= 2 * ((N - 1) * grad_stride + N):
        return False
    return stride != grad_stride or by // 2 % stride < N or -(by // 2) % stride < N
