"""Calls of the operators around the epilogue that a server or a trainer makes beside the plain ones: empty
lists and masks, several host threads, explicit streams, records with masked entries."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _rows as R  # noqa: E402
from tests.test_rows_gpu import bd, check_distill, check_process, distill_batch, distill_call, process_batch  # noqa: E402,F401


@pytest.mark.parametrize("lowest", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.3, 0.7, 1.0, 2.0])
@pytest.mark.parametrize("form", ["fused", "two_call"])
def test_teacher_logit_of_the_lowest_value(bd, form, T, lowest):
    """A record entry that a mask set to its type's lowest value has p = 0, also where that over T leaves
    fp32's range."""
    c = distill_batch(np.random.default_rng(21), 6, 3001, 20, "fp32", T, True)
    c["w"] = None
    c["logits"][[0, 1, 4], 7] = float(torch.finfo(R.TORCH[lowest]).min)
    c["logits"][1, 10:] = float(torch.finfo(R.TORCH[lowest]).min)
    check_distill(c, distill_call(bd, c, "fp32", form), "fp32")
