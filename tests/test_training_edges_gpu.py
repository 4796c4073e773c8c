"""Where the calls that train on decoded tokens could go wrong at an edge: upstream gradients that are not finite, ratios next to
where clipping begins, losses next to fp32's largest number, tokens with nearly all the mass, factors below the smallest normal
number, every launch shape's loops."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import training as O  # noqa: E402
from tests import _rows as R  # noqa: E402
from tests import _training as T_  # noqa: E402
from tests.test_clip_gpu import clip_call  # noqa: E402
from tests.test_rows_gpu import bd  # noqa: E402,F401
from tests.test_training_gpu import (  # noqa: E402
    HIGH, LOW, check_logprobs, check_policy, check_preference, full, logprobs_call, policy_batch, policy_call, preference_batch,
    preference_call)

U = R.U


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("up", [np.nan, np.inf, -np.inf])
def test_upstream_of_pairs_without_a_gradient(bd, up, dtype):  # noqa: F811
    """A loss that is NaN usually comes back as an upstream gradient that is NaN: rows of a pair with a status have a gradient of 0 all
    the same, and so have those of a pair of weight 0; the other pairs' is right."""
    c = preference_batch(np.random.default_rng(14), (3, 2, 4, 3, 2, 2, 3, 3), 1003, dtype, tail=1)
    off = c["off"]
    c["y"][:] = 5
    c["w"][0] = 0.0
    c["x"][off[2], 7] = np.nan                               # pair 1: one of its rows
    c["ref"][off[5]] = np.nan                                # pair 2: its difference
    ups = np.array([up, up, up, 0.7])
    got = preference_call(bd, c, dtype, "two_call", up=ups)
    assert not got["grad"][:off[6]].any()
    assert list(got["pair_status"]) == [0, bd.ROW_NONFINITE, bd.ROW_NONFINITE, 0]
    plain = preference_call(bd, c, dtype, "two_call", up=np.array([1.0, 1.0, 1.0, 0.7]))
    assert np.array_equal(got["grad"], plain["grad"]) and got["grad"][off[6]:off[8]].any(1).all()
    # pairs whose offsets are bad
    c["off"] = off.copy()
    c["off"][4] = 0
    got = preference_call(bd, c, dtype, "two_call", up=np.full(4, up))
    assert list(got["pair_status"][1:]) == [bd.ROW_BAD_PARAMS] * 3 and not got["grad"].any()
