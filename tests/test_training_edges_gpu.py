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


def own_logprobs(bd, x, y, dtype, T=1.0):  # noqa: F811
    return logprobs_call(bd, x, y, dtype, T, entropy=False)[0]


def clipped_call(bd, x, y, dtype, old, adv, form, low, high, w=None, T=1.0, ref=None, kl=0.0):  # noqa: F811
    """(loss, status, gradient) of a policy loss with these borders."""
    logits, tokens, rows = R.on_gpu(x, dtype), R.i32(y), len(x)
    loss, st, saved = full(rows, 9.0), full(rows, -1, torch.int32), torch.full((rows, 8), 9.0, device="cuda")
    grad = torch.full_like(logits, 77.0)
    given = dict(clip_low=low, clip_high=high, weights=None if w is None else R.f32(w), ref_logprobs=None if ref is None else R.f32(ref),
                 kl_coef=kl, temperature=T)
    bd.dspark_policy_loss(logits, tokens, R.f32(old), R.f32(adv), loss=loss, row_status=st, saved=saved,
                          grad=grad if form == "fused" else None, **given)
    if form == "two_call":
        bd.dspark_policy_loss_backward(logits, tokens, R.f32(old), R.f32(adv), saved=saved, grad=grad, **given)
    return loss.double().cpu().numpy(), st.cpu().numpy(), grad.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["fused", "two_call"])
def test_ratio_at_a_border_has_its_gradient(bd, form, dtype):  # noqa: F811
    """A row's own log-probability as its old one, clip 0 on both sides: rho is 1 to the rounding of two log-probabilities and counts
    as not clipped, so every row has the gradient of rho A.  The same where the border is elsewhere, and none a little beyond it."""
    rng = np.random.default_rng(15)
    rows, V = 200, 1003
    x, y = T_.token_rows(rng, rows, V, dtype, special=False)
    lp = own_logprobs(bd, x, y, dtype)
    adv = (rng.uniform(0.5, 2, rows) * rng.choice([-1, 1], rows)).astype(np.float32)
    for low, high in ((0.0, 0.0), (0.25, 0.5)):
        edge = np.where(adv > 0, np.log1p(high), np.log1p(-low))
        for beyond in (False, True):
            # (beyond: by 1e-4, where the largest log-probability's rounding is 2^-20 of it)
            old = (lp - edge - (np.sign(adv) * 1e-4 if beyond else 0)).astype(np.float32)
            loss, st, grad = clipped_call(bd, x, y, dtype, old, adv, form, low, high)
            assert not st.any()
            for r in range(rows):
                if beyond:
                    assert not grad[r].any(), r
                    continue
                row = O.token_row(x[r], y[r], 1.0)
                rho = np.exp(row["logp"][y[r]] - float(old[r]))
                slack = 2.0 ** -20 + 2.0 ** -22 * abs(row["logp"][y[r]]) + T_.row_errors(row, V)[2]
                want = O.token_grad(row, -float(adv[r]) * rho, 0.0, 1.0)
                tol = T_.grad_bound(row, float(adv[r]) * rho, 0.0, V, 1.0, dtype, want, abs(float(adv[r])) * rho * slack)
                assert (np.abs(grad[r] - want) <= tol).all(), (r, np.abs(grad[r] - want).max())
                assert abs(loss[r] + float(adv[r]) * rho) <= abs(float(adv[r])) * rho * 2 * slack, r


@pytest.mark.parametrize("high", [0.0, 0.25])
def test_both_forms_clip_the_same_rows(bd, high):  # noqa: F811
    """Ratios within some 1e-6 of where clipping begins: the gradient in one call and the one from what that call has saved are of the
    same rows, all or nothing."""
    rng = np.random.default_rng(16)
    rows, V = 2000, 67
    x, y = T_.token_rows(rng, rows, V, "fp32", special=False)
    lp = own_logprobs(bd, x, y, "fp32")
    adv = np.ones(rows, np.float32)
    seen = set()
    for at in (0.0, 2.0 ** -20):                             # of the border itself, and of what counts as at it
        slack = at + (2.0 ** -22 * np.abs(lp) if at else 0)
        old = (lp - np.log1p(high) - slack + rng.uniform(-1e-6, 1e-6, rows)).astype(np.float32)
        logits, tokens = R.on_gpu(x, "fp32"), R.i32(y)
        loss, st, saved = full(rows, 9.0), full(rows, -1, torch.int32), torch.zeros(rows, 8, device="cuda")
        fused, then = torch.full_like(logits, 77.0), torch.full_like(logits, 77.0)
        args = (logits, tokens, R.f32(old), R.f32(adv))
        bd.dspark_policy_loss(*args, loss=loss, row_status=st, saved=saved, grad=fused, clip_low=0.0, clip_high=high)
        bd.dspark_policy_loss_backward(*args, saved=saved, grad=then, clip_low=0.0, clip_high=high)
        a, b = (t.ne(0).any(1).cpu().numpy() for t in (fused, then))
        assert np.array_equal(a, b), (at, int((a != b).sum()))
        seen |= set(a.tolist())
    assert seen == {True, False}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_losses_next_to_the_largest_number(bd, dtype):  # noqa: F811
    """Advantages of fp32's largest number: a row whose loss is not finite has a status, a NaN loss and a gradient of 0, the others
    have none of these."""
    rng = np.random.default_rng(17)
    rows, V = 2000, 67
    x, y = T_.token_rows(rng, rows, V, dtype, special=False)
    lp = own_logprobs(bd, x, y, dtype)
    old = (lp + rng.uniform(-1e-6, 1e-6, rows)).astype(np.float32)
    for adv, w in ((np.float32(3.4028235e38), None), (np.float32(2.0 ** 127), np.full(rows, 2, np.float32))):
        loss, st, grad = clipped_call(bd, x, y, dtype, old, np.full(rows, -adv, np.float32), "fused", 0.2, 0.2, w=w)
        bad = st != 0
        assert bad.any() and not bad.all() and set(st[bad].tolist()) == {bd.ROW_NONFINITE}
        assert np.isnan(loss[bad]).all() and np.isfinite(loss[~bad]).all()
        assert not grad[bad].any() and (grad[~bad] != 0).any(1).all()


def test_one_cta_waits_in_vain(bd, monkeypatch):  # noqa: F811
    """A test build in which the second CTA of every row that is split waits, 50 ms long, for what nobody sends: its part of the
    gradient is 0, and though the first CTA has all it needs, the row reports DSPARK_ROW_INTERNAL and a NaN loss.  Rows of one CTA,
    rows that are not read, and the calls after it are as ever."""
    from sample_verify_epilogue_gb300 import binding as b_
    from sample_verify_epilogue_gb300.build import build_variant
    lib = b_.open_library(build_variant("expired_token_peers", ["-DDSPARK_TEST_EXPIRED_PEERS"], ["token_rows.cu"]))
    expired = b_._Calls(lib)
    rng = np.random.default_rng(24)
    c = policy_batch(rng, 5, 140001, "bf16", 1.0, special=False)
    c["y"][1], c["y"][3] = -1, 140001
    one = policy_batch(rng, 6, 1003, "bf16", 1.0, special=False)
    with monkeypatch.context() as m:
        m.setattr(b_, "_calls_of", expired)
        got = policy_call(bd, c, "bf16", 1.0, 0.1, 0.01, "fused", pad=1, shift=1)
        check_policy(one, policy_call(bd, one, "bf16", 1.0, 0.1, 0.01, "fused"), "bf16", 1.0, 0.1, 0.01)
    read = [0, 4]                                            # (2 has weight 0)
    assert (got["status"][read] == b_.ROW_INTERNAL).all() and np.isnan(got["loss"][read]).all()
    assert (got["grad"][read] == 0).any(1).all()
    assert got["status"][1] == 0 and got["status"][2] == 0 and got["status"][3] == b_.ROW_BAD_TOKEN
    good = policy_call(bd, c, "bf16", 1.0, 0.1, 0.01, "fused", pad=1, shift=1)
    check_policy(c, good, "bf16", 1.0, 0.1, 0.01, bad={3: b_.ROW_BAD_TOKEN})


LOG2E = float(np.float32(np.log2(np.e)))                     # a temperature by which logits are their own exponents of two


def sure_rows(rng, rows, T):
    """Two logits a row, 0 and the token's, whose odds are e^-23 to e^-24: the sum over the others is a power of two, without
    rounding, so that what is off comes of the row's end."""
    y = rng.integers(0, 2, rows)
    x = np.zeros((rows, 2))
    x[np.arange(rows), y] = R.rounded(rng.uniform(23, 24, rows) * T, "fp32")
    return x, y, x[np.arange(rows), y] / T


@pytest.mark.parametrize("T", [1.0, LOG2E])
@pytest.mark.parametrize("form", ["logprobs", "fused", "two_call"])
def test_gradients_of_sure_tokens(bd, form, T):  # noqa: F811
    """The gradient of a token with nearly all the mass is q = 1 - p to fp32's last bits.  Roundings: the logarithm of the
    sum and the unit's mean error in it u each, the exponential 4 u (ex2 too), its correction, 1 + t, the division and the product u each,
    1 / T and two products by it u each, and rho for the policy (exp of next to nothing) 2 u: 14 u.  d in one float would add up to
    16 u at odds of e^-23."""
    rng = np.random.default_rng(18)
    rows = 1000
    x, y, d = sure_rows(rng, rows, T)
    want = 1 / (1 + np.exp(d)) / T
    if form == "logprobs":
        grad = logprobs_call(bd, x, y, "fp32", T, entropy=False, up=(np.ones(rows), None))[3]
    else:
        grad = clipped_call(bd, x, y, "fp32", np.zeros(rows), np.full(rows, -1.0), form, 0.2, 0.2, T=T)[2]
        want = want * np.exp(-1 / (1 + np.exp(d)))
    at = grad[np.arange(rows), y]
    assert (np.abs(at - want) <= 14 * U * want).all(), np.abs(at / want - 1).max() / U


def test_slopes_of_settled_pairs(bd):  # noqa: F811
    """A pair whose answers are far apart: the slope sigma(-z) keeps fp32's bits where z is no float.  Both rows have the same log p,
    so z is beta times the references' difference, in pairs of floats: sigma(-z) 8 u with its correction, two products by beta and 1 / n u
    each; the token's q, a half, 4 u, its product u: 15 u."""
    rng = np.random.default_rng(20)
    P = 300
    x = np.zeros((2 * P, 2))
    y = np.zeros(2 * P, np.int64)
    ref = np.zeros(2 * P)
    beta = float(np.float32(0.1))
    ref[0::2] = R.rounded(rng.uniform(-240, -170, P), "fp32")
    ref[1::2] = R.rounded(rng.uniform(-1, 1, P), "fp32")
    c = dict(x=x, y=y, off=np.arange(2 * P + 1), ref=ref.astype(np.float32), w=None)
    got = preference_call(bd, c, "fp32", "fused", beta=beta)
    z = beta * (-ref[0::2] + ref[1::2])
    want = -beta * np.exp(-np.logaddexp(0, z)) * 0.5         # at the chosen token
    at = got["grad"][0::2, 0]
    assert (np.abs(at - want) <= 15 * U * np.abs(want)).all(), np.abs(at / want - 1).max() / U


@pytest.mark.parametrize("form", ["fused", "two_call"])
def test_gradients_of_a_small_kl_term(bd, form):  # noqa: F811
    """Rows whose gradient is the KL term's alone (A = 0): e^D - 1 for log-ratios that are small but not next to nothing, at tokens
    whose log-probability is next to 0, so that D is the reference's.  expm1 2 u more than above, D's own rounding u |D e^D / (e^D - 1)|
    < 2 u, the product u: 19 u."""
    rng = np.random.default_rng(19)
    rows = 2000
    x, y, d = sure_rows(rng, rows, LOG2E)
    ref = (rng.uniform(0.01, 0.3, rows) * rng.choice([-1, 1], rows)).astype(np.float32)
    grad = clipped_call(bd, x, y, "fp32", np.zeros(rows), np.zeros(rows), form, 0.2, 0.2, T=LOG2E, ref=ref, kl=1.0)[2]
    q = 1 / (1 + np.exp(d))
    want = -np.expm1(ref.astype(np.float64) + np.log1p(np.exp(-d))) * q / LOG2E
    at = grad[np.arange(rows), y]
    assert (np.abs(at - want) <= 19 * U * np.abs(want)).all(), np.abs(at / want - 1).max() / U


def test_clip_factor_to_the_last_bit(bd):  # noqa: F811
    """n ones, whose sum of squares has no rounding: each comes out as max_norm / sqrt(n), rounded once.  (u, and 2^-40 for the
    root in a pair of floats; from a norm rounded to a float it is 2 u.)"""
    worst = 0.0
    for n in range(2, 300, 7):
        for max_norm in (1.0, float(np.float32(0.7))):
            g = torch.ones(n, device="cuda")
            norm, status = clip_call(bd, [g], max_norm)
            want = max_norm / n ** 0.5
            assert status == 0 and abs(norm - n ** 0.5) <= U * n ** 0.5 * (1 + 2.0 ** -20)
            worst = max(worst, float((g.double() / want - 1).abs().max()))
    assert worst <= U * (1 + 2.0 ** -12), worst / U


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size,max_norm", [(1e38, 1e-3), (3e38, 1e-8), (1e38, 1e-30), (2e37, 1.2e-38), (1e30, 1e-20), (1.5, 2e-38), (1e20, 1e-40), (3e38, 1e-44)])
def test_clip_factors_below_the_smallest_number(bd, size, max_norm, dtype, out):  # noqa: F811
    """Gradients near fp32's largest number, clipped to small norms: the factor lies below fp32's numbers, what it makes does not."""
    rng = np.random.default_rng(21)
    v = np.concatenate([rng.uniform(-0.2, 0.2, 30) * size, rng.normal(0, 1e-3, 4000) * size, rng.normal(0, 1e-9, 40) * size])
    g = torch.from_numpy(v.astype(np.float32)).to(R.TORCH[dtype]).cuda()
    held = g.double().cpu().numpy()
    m = float(np.float32(max_norm))
    outs = [torch.full(v.shape, 7.0, device="cuda")] if out else None
    norm, status = clip_call(bd, [g], m, outs)
    want_norm, want = O.clip([held], m)
    assert status == 0 and abs(norm - want_norm) <= 14 * U * want_norm
    got = (outs[0] if out else g).double().cpu().numpy()
    kind = "fp32" if out else dtype
    # the norm's sum 12 u (squares of a chunk), the factor and the products u each; a step of the smallest numbers
    tol = (16 * U + R.HALF[kind]) * np.abs(want[0]) + (2.0 ** -133 if kind == "bf16" else 2.0 ** -149)
    assert (np.abs(got - want[0]) <= tol).all(), (np.abs(got - want[0]) - tol).max()


@pytest.mark.parametrize("size,max_norm", [(2.0 ** -100, 2.0 ** -101), (2.0 ** -60, 3e-38), (2.0 ** -130, 1e-40), (2.0 ** -128, 3e-41), (2.0 ** -140, 1e-43)])
def test_clip_small_gradients_to_smaller_norms(bd, size, max_norm):  # noqa: F811
    """The factor to its last bit where max_norm, its quotient's remainder or the gradients lie near or below the smallest normal
    number: u of what comes out, and half a step of the smallest numbers (once more where the norm's is one)."""
    m = float(np.float32(max_norm))
    for n in range(2, 300, 7):
        g = torch.full((n,), size, device="cuda")
        norm, status = clip_call(bd, [g], m)
        want = min(m / n ** 0.5, size)
        assert status == 0 and abs(norm - n ** 0.5 * size) <= U * n ** 0.5 * size * (1 + 2.0 ** -12) + 2.0 ** -150
        assert float((g.double() - want).abs().max()) <= 2 * U * want + 2.0 ** -150, n


@pytest.mark.parametrize("rows,V,dtype", [(500, 16411, "bf16"), (600, 5003, "fp32"), (913, 16411, "bf16"), (1000, 8209, "fp32"),
                                          (1216, 16400, "bf16"), (1217, 16411, "bf16"), (1300, 8203, "fp32"), (300, 8209, "fp32")])
def test_loops_of_every_launch_shape(bd, rows, V, dtype):  # noqa: F811
    """Rows by 256, 128 and 512 threads, by four and by six vectors at a time, long enough for the loop over whole batches, the last
    vectors and both ragged ends, with tokens in each of them."""
    rng = np.random.default_rng(rows)
    x, y = T_.token_rows(rng, rows, V, dtype)
    for r in range(20, 60):                                  # the first and the last vectors' logits
        y[r] = r - 20 if r < 40 else V - 60 + r
    x = R.rounded(x, dtype)
    up = rng.normal(0, 1, (2, rows)).astype(np.float32)
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, pad=2, shift=3, up=up), up)
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, entropy=False, up=(up[0], None)), (up[0], None))


@pytest.mark.parametrize("rows,V,dtype", [(450, 5003, "fp32"), (900, 8003, "bf16"), (450, 8209, "fp32"), (201, 16411, "bf16")])
def test_loops_of_kept_rows(bd, rows, V, dtype):  # noqa: F811
    """Policy losses whose rows are one CTA's, of 128 threads and of 256."""
    rng = np.random.default_rng(rows)
    c = policy_batch(rng, rows, V, dtype, 1.0, special=False)
    for ent in (0.0, 0.02):
        got = policy_call(bd, c, dtype, 1.0, 0.05, ent, "fused", pad=2, shift=3)
        check_policy(c, got, dtype, 1.0, 0.05, ent)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_clip_dense_gradients_of_other_orders(bd, dtype):  # noqa: F811
    """Gradients of transposed and channels-last parameters, whose elements fill their memory in another order; into outputs of the
    same order too.  What has gaps or shares memory is refused."""
    rng = np.random.default_rng(22)

    def make():
        a = torch.from_numpy(rng.normal(0, 1, (33, 70)).astype(np.float32)).to(R.TORCH[dtype]).cuda().t()
        b = torch.from_numpy(rng.normal(0, 1, (2, 3, 5, 7)).astype(np.float32)).to(R.TORCH[dtype]).cuda().to(memory_format=torch.channels_last)
        return [a, b, torch.ones(1, 9, device="cuda").t()]

    for out in (None, "same", "fp32"):
        g = make()
        held = [t.double().cpu().numpy() for t in g]
        outs = None if out is None else [torch.empty_like(t, dtype=torch.float32 if out == "fp32" else t.dtype) for t in g]
        assert outs is None or all(o.stride() == t.stride() for o, t in zip(outs, g))
        norm, status = clip_call(bd, g, 2.0, outs)
        want, scaled = O.clip(held, 2.0)
        assert status == 0 and abs(norm - want) <= 14 * U * want
        for t, w in zip(g if out is None else outs, scaled):
            half = R.HALF["bf16" if t.dtype is torch.bfloat16 else "fp32"]
            assert (np.abs(t.double().cpu().numpy() - w) <= (16 * U + half) * np.abs(w) + 2.0 ** -133).all()
    a = torch.ones(4, 6, device="cuda")
    for grads, outs in (([a[:, ::2]], None), ([a[:, :3]], None), ([a[0].expand(4, 6)], None), ([a.t()], [torch.ones(6, 4, device="cuda")]),
                        ([a], [torch.ones(6, 4, device="cuda").t()]), ([a, a.t()], None)):
        with pytest.raises(ValueError):
            bd.GradTable(grads, outs)


def test_clip_grads_of_a_parameter_and_of_none(bd):  # noqa: F811
    """A single parameter in place of a list; parameters of which none has a gradient: the norm of nothing is 0."""
    from sample_verify_epilogue_gb300.training import clip_grads_
    p = torch.nn.Parameter(torch.zeros(4, 4, device="cuda"))
    q = torch.nn.Parameter(torch.zeros(3, device="cuda"))
    norm, status = clip_grads_(iter([p, q]), 1.0)
    assert norm.shape == (1,) and float(norm) == 0.0 and int(status) == 0 and norm.is_cuda
    p.grad = torch.full((4, 4), 2.0, device="cuda")
    norm, status = clip_grads_(p, 4.0)
    assert float(norm) == 8.0 and int(status) == 0 and bool((p.grad == 1.0).all())
    with pytest.raises(ValueError):
        clip_grads_([], 1.0)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("rows", [4, 1000])
def test_logits_next_to_the_last_whole_exponent(bd, rows, entropy):  # noqa: F811
    """Logits of some 2.9 million, where one thread's reference has a whole exponent and another's has none (they begin at 2^22):
    their sums join without a jump.  Exponents by whole references lose 2^-24 of some 64 powers of two, a batch of them as often as not
    the same way, others 2^-24 of their own: 64 u log 2 < 3e-6, and as much again for the token's; 2e-5 with margin."""
    rng = np.random.default_rng(23)
    V = 9001
    x = R.rounded(2.0 ** 22 * np.log(2) + rng.integers(-60, 20, (rows, 1)) * 0.25 + rng.integers(-12, 13, (rows, V)) * 0.25, "fp32")
    x[1::2] *= -1
    y = rng.integers(0, V, rows)
    lp, H, st, grad = logprobs_call(bd, x, y, "fp32", entropy=entropy, up=(np.ones(rows), np.ones(rows) if entropy else None))
    assert not st.any()
    for r in range(rows):
        row = O.token_row(x[r], y[r], 1.0)
        assert abs(lp[r] - row["logp"][y[r]]) < 2e-5, r
        assert H is None or abs(H[r] - row["entropy"]) < 4e-5, r
        want = O.token_grad(row, 1.0, 1.0 if entropy else 0.0, 1.0)
        assert (np.abs(grad[r] - want) <= 2e-5 * row["p"] * (1 + 10 * entropy) + 1e-6 * np.abs(want) + (4e-5 if entropy else 2e-5) * (np.arange(V) == y[r])).all(), r


@pytest.mark.parametrize("mean", [False, True])
def test_rewards_beyond_the_largest_number(bd, mean):  # noqa: F811
    """beta times a log ratio that fp32 does not hold: rewards are infinite, not NaN, and so is the loss of the pair that has
    the smaller one chosen."""
    x = np.zeros((4, 8))
    c = dict(x=x, y=np.zeros(4, np.int64), off=np.arange(5), ref=np.array([5, -5, -5, 5], np.float32), w=None)
    got = preference_call(bd, c, "fp32", "fused", beta=2e38, mean=mean)
    assert not got["pair_status"].any()
    assert got["rewards"][0, 0] == -np.inf and got["rewards"][1, 1] == -np.inf
    assert got["rewards"][0, 1] == np.inf and got["rewards"][1, 0] == np.inf
    assert list(got["loss"]) == [np.inf, 0.0]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_old_logprobs_are_of_the_losses_temperature(bd, dtype):  # noqa: F811
    """Tokens drawn at a temperature of 0.7 from a truncated distribution: the verify call's log-probabilities are those of the whole
    distribution at 1, and the ratios of a loss at temperature 1 are 1; dspark_token_logprobs at 0.7 goes with a loss at 0.7."""
    from sample_verify_epilogue_gb300.runner import EpilogueCall
    from workloads.generate import make_batch, row_params
    B, K, V = 5, 3, 5001
    batch = make_batch(B=B, K_max=K, V=V, logits_dtype=dtype, rows=[row_params(0.7, 0, 0.9, 0.0, 0.0, K)] * B, seed=5, philox_seed=5,
                       history_len=0, want_logprobs=True)
    call = EpilogueCall(batch)
    call.run()
    tokens, raw, n = call.out["tokens"], call.out["logprobs"], B * (K + 1)
    live = (tokens >= 0).view(-1)
    assert int(live.sum()) >= B
    lp, st, loss = full(n, 9.0), full(n, -1, torch.int32), full(n, 9.0)
    adv = torch.ones(n, device="cuda")
    for T, old in ((1.0, raw.contiguous().view(-1)), (0.7, lp)):
        if T != 1.0:
            bd.dspark_token_logprobs(call.x, tokens, logprobs=lp, row_status=st, temperature=T)
        bd.dspark_policy_loss(call.x, tokens, old, adv, loss=loss, row_status=st, temperature=T)
        # the verify call's log-probabilities are within 1e-4
        assert not st.any() and float((loss[live] + 1).abs().max()) < 2e-4 and not loss[~live].any()
