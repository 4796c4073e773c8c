"""What trains on decoded tokens on the GPU against its float64 oracle: token log-probabilities with their gradient,
the policy and the preference loss."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import training as O  # noqa: E402
from tests import _rows as R  # noqa: E402
from tests import _training as T_  # noqa: E402
from tests.test_rows_gpu import bd  # noqa: E402,F401

U = R.U
SIZES = [(1, 1), (1, 2), (3, 7), (4, 17), (9, 1003), (9, 8193), (9, 32003), (700, 501), (9, 151936)]


def full(rows, value, dtype=torch.float32):
    return torch.full((rows,), value, dtype=dtype, device="cuda")


def close(got, want, tol, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


def fin(v):
    """|v|, 0 for an infinity (which has to come out as it is)."""
    return abs(v) if np.isfinite(v) else 0.0


# ---------------------------------------------------------------- token log-probabilities
def logprobs_call(bd, x, y, dtype, T=1.0, pad=0, shift=0, entropy=True, up=None, in_place=False, out_shift=None):  # noqa: F811
    """(log-probabilities, entropies, status, gradient)"""
    rows = len(x)
    logits, tokens = R.on_gpu(x, dtype, pad, shift), R.i32(y)
    lp, st, saved = full(rows, 9.0), full(rows, -1, torch.int32), torch.full((rows, 8), 9.0, device="cuda")
    H = full(rows, 9.0) if entropy else None
    bd.dspark_token_logprobs(logits, tokens, logprobs=lp, entropy=H, row_status=st, saved=saved if up is not None else None,
                             temperature=T)
    grad = None
    if up is not None:
        grad = logits if in_place else R.on_gpu(np.full(x.shape, 77.0), dtype, pad, shift if out_shift is None else out_shift)
        bd.dspark_token_logprobs_backward(logits, tokens, saved=saved, grad=grad, temperature=T,
                                          grad_logprobs=None if up[0] is None else R.f32(up[0]),
                                          grad_entropy=None if up[1] is None else R.f32(up[1]))
        grad = grad.double().cpu().numpy()
    return lp.cpu().numpy(), None if H is None else H.cpu().numpy(), st.cpu().numpy(), grad


def check_logprobs(x, y, dtype, T, got, up=None, bad={}):
    lp, H, st, grad = got
    V = x.shape[1]
    for r in range(len(x)):
        if r in bad or y[r] < 0:
            want = np.nan if r in bad else 0.0
            assert st[r] == bad.get(r, 0)
            close(lp[r], want, 0)
            if H is not None:
                close(H[r], want, 0)
            assert grad is None or not grad[r].any()
            continue
        row = O.token_row(x[r], y[r], T)
        es, ed, elp, eH = T_.row_errors(row, V)
        assert st[r] == 0
        close(lp[r], row["logp"][y[r]], elp, ("logp", r))
        if H is not None:
            close(H[r], row["entropy"], eH, ("entropy", r))
        if grad is not None:
            a, h = (0.0 if u is None else float(np.float32(u[r])) for u in up)
            want = O.token_grad(row, a, h, T)
            close(grad[r], want, T_.grad_bound(row, a, h, V, T, dtype, want), ("grad", r))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V", SIZES)
def test_token_logprobs(bd, rows, V, dtype):  # noqa: F811
    rng = np.random.default_rng(V + rows)
    for T in (1.0, 0.7, 2.5):
        x, y = T_.token_rows(rng, rows, V, dtype)
        up = rng.normal(0, 1, (2, rows))
        check_logprobs(x, y, dtype, T, logprobs_call(bd, x, y, dtype, T, up=up), up)
        if T == 1.0:
            check_logprobs(x, y, dtype, T, logprobs_call(bd, x, y, dtype, T, entropy=False, up=(up[0], None)), (up[0], None))
            check_logprobs(x, y, dtype, T, logprobs_call(bd, x, y, dtype, T, up=(None, up[1])), (None, up[1]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift,out_shift", [(1, 0, 0), (3, 5, 5), (8, 1, 0), (0, 3, 6), (5, 2, 1)])
def test_token_logprobs_strides_and_alignment(bd, pad, shift, out_shift, dtype):  # noqa: F811
    rng = np.random.default_rng(pad + shift)
    for rows, V in ((11, 5001), (9, 40)):
        x, y = T_.token_rows(rng, rows, V, dtype)
        y[0], y[1] = 0, V - 1                                # the ragged ends
        up = rng.normal(0, 1, (2, rows))
        for r in (0, 1):
            x[r, y[r]] = 3.0
        for in_place in (False, True):
            got = logprobs_call(bd, x, y, dtype, 1.3, pad, shift, up=up, in_place=in_place, out_shift=out_shift)
            check_logprobs(x, y, dtype, 1.3, got, up)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_between_rows_is_left_alone(bd, dtype):  # noqa: F811
    rng = np.random.default_rng(1)
    x, y = T_.token_rows(rng, 6, 1001, dtype)
    logits, grad = R.on_gpu(x, dtype), torch.full((6, 1013), 5.0, dtype=R.TORCH[dtype], device="cuda")
    lp, st, saved = full(6, 0.0), full(6, 0, torch.int32), torch.empty(6, 8, device="cuda")
    bd.dspark_token_logprobs(logits, R.i32(y), logprobs=lp, row_status=st, saved=saved)
    bd.dspark_token_logprobs_backward(logits, R.i32(y), saved=saved, grad=grad[:, :1001], grad_logprobs=full(6, 1.0))
    assert (grad[:, 1001:] == 5).all() and not (grad[:, :1001] == 5).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [5, 1003, 40001])
def test_row_status(bd, V, dtype):  # noqa: F811
    rng = np.random.default_rng(V)
    rows = 12
    x, y = T_.token_rows(rng, rows, V, dtype, special=False)
    x[0, (y[0] + 1) % V] = np.nan
    x[1, y[1]] = np.nan
    x[2, (y[2] + 2) % V] = np.inf
    x[3, y[3]] = np.inf
    x[4] = -np.inf
    x[5, :] = np.nan
    y[6], y[7], y[8] = V, -2, -1
    x[8] = np.nan                                            # not read
    bad = {r: bd.ROW_NONFINITE for r in range(6)} | {6: bd.ROW_BAD_TOKEN, 7: bd.ROW_BAD_TOKEN}
    up = rng.normal(0, 1, (2, rows))
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, up=up), up, bad)
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, entropy=False), bad=bad)


def test_entropy_gradient_needs_the_entropy(bd):  # noqa: F811
    x, y = T_.token_rows(np.random.default_rng(2), 3, 100, "fp32", special=False)
    up = np.ones((2, 3))
    assert np.isnan(logprobs_call(bd, x, y, "fp32", entropy=False, up=up)[3]).any(1).all()


# ---------------------------------------------------------------- policy loss
LOW, HIGH = 0.2, 0.3


def policy_batch(rng, rows, V, dtype, T, special=True):
    x, y = T_.token_rows(rng, rows, V, dtype, special)
    lp = np.zeros(rows)
    for r in range(rows):
        if y[r] >= 0:
            lp[r] = O.token_row(x[r], y[r], T)["logp"][y[r]]
    lp = np.where(np.isfinite(lp), lp, -5.0)
    move = rng.normal(0, 0.3, rows)
    for border in (np.log(1 - LOW), np.log(1 + HIGH)):       # a ratio at a border is decided by the last bit
        move = np.where(np.abs(move - border) < 1e-3, border + 3e-3, move)
    w = rng.uniform(0.5, 2, rows)
    if rows > 4:
        w[2] = 0.0
    adv = rng.normal(0, 1, rows)
    if rows > 3:
        adv[3] = 0.0
    return dict(x=x, y=y, old=(lp - move).astype(np.float32), ref=(lp + rng.normal(0, 0.4, rows)).astype(np.float32),
                adv=adv.astype(np.float32), w=w.astype(np.float32))


def policy_call(bd, c, dtype, T, kl_coef, entropy_coef, form, use_ref=True, up=None, pad=0, shift=0, in_place=False):  # noqa: F811
    rows = len(c["x"])
    logits = R.on_gpu(c["x"], dtype, pad, shift)
    tokens, old, adv = R.i32(c["y"]), R.f32(c["old"]), R.f32(c["adv"])
    given = dict(ref_logprobs=R.f32(c["ref"]) if use_ref else None, weights=None if c["w"] is None else R.f32(c["w"]),
                 clip_low=LOW, clip_high=HIGH, kl_coef=kl_coef, entropy_coef=entropy_coef, temperature=T)
    out = {k: full(rows, 9.0) for k in ("loss", "logprobs", "entropy")} | ({"kl": full(rows, 9.0)} if use_ref else {})
    st, saved = full(rows, -1, torch.int32), torch.full((rows, 8), 9.0, device="cuda")
    grad = None
    if form != "forward":
        grad = logits if in_place else R.on_gpu(np.full(c["x"].shape, 77.0), dtype, pad, shift)
    bd.dspark_policy_loss(logits, tokens, old, adv, row_status=st, saved=saved if form != "forward" else None,
                          grad=grad if form == "fused" else None, **out, **given)
    if form == "two_call":
        bd.dspark_policy_loss_backward(logits, tokens, old, adv, saved=saved, grad=grad,
                                       grad_loss=None if up is None else R.f32(up), **given)
    return {k: v.cpu().numpy() for k, v in out.items()} | {"status": st.cpu().numpy(),
                                                          "grad": None if grad is None else grad.double().cpu().numpy()}


def check_policy(c, got, dtype, T, kl_coef, entropy_coef, use_ref=True, up=None, bad={}):
    x, y, V = c["x"], c["y"], c["x"].shape[1]
    for r in range(len(x)):
        w = 1.0 if c["w"] is None else float(c["w"][r])
        assert got["status"][r] == bad.get(r, 0), r
        if r in bad or y[r] < 0 or w == 0:
            close(got["loss"][r], np.nan if r in bad else 0.0, 0)
            assert got["grad"] is None or not got["grad"][r].any()
            continue
        row = O.token_row(x[r], y[r], T)
        es, ed, elp, eH = T_.row_errors(row, V)
        lp, old, adv, ref = row["logp"][y[r]], float(c["old"][r]), float(c["adv"][r]), float(c["ref"][r]) if use_ref else None
        loss, a, h, kl = O.policy_row(lp, row["entropy"], old, adv, ref, w, LOW, HIGH, kl_coef, entropy_coef)
        el = elp + 2 * U * (abs(lp) + abs(old) if np.isfinite(lp) else 0)
        rho = np.exp(lp - old)
        erho = rho * (1.01 * el + 8 * U)
        ea = abs(adv) * erho + 4 * U * abs(adv) * (rho + 1)
        eloss = ea + entropy_coef * eH
        if use_ref:
            D = ref - lp
            eD = el + 2 * U * abs(D) if np.isfinite(lp) else 0.0
            ekl = abs(np.expm1(D)) * eD * 1.01 + np.exp(D) * eD ** 2 + 24 * U * kl if np.isfinite(lp) else 0.0
            close(got["kl"][r], kl, ekl + T_.FLUSH, ("kl", r))
            if kl_coef:
                ea += kl_coef * (np.exp(D) * eD * 1.01 + 8 * U * abs(np.expm1(D)))
                eloss += kl_coef * ekl
        ea, eloss = w * ea + 8 * U * abs(a), w * eloss + 16 * U * (abs(loss) + w * abs(adv) * (rho + 1.5) + w * abs(entropy_coef * row["entropy"]))
        close(got["loss"][r], loss, eloss, ("loss", r))
        close(got["logprobs"][r], lp, elp, ("logp", r))
        close(got["entropy"][r], row["entropy"], eH, ("entropy", r))
        if got["grad"] is not None:
            u = 1.0 if up is None else float(np.float32(up[r]))
            want = O.token_grad(row, a * u, h * u, T)
            close(got["grad"][r], want, T_.grad_bound(row, a * u, h * u, V, T, dtype, want, abs(u) * ea * 1.01), ("grad", r))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V", SIZES)
def test_policy_loss(bd, rows, V, dtype):  # noqa: F811
    rng = np.random.default_rng(V + 7 * rows)
    up = rng.uniform(-1, 2, rows).astype(np.float32)
    for T, kl, ent in ((1.0, 0.0, 0.0), (1.3, 0.1, 0.0), (0.8, 0.05, 0.02)):
        c = policy_batch(rng, rows, V, dtype, T, special=False)
        for form in ("forward", "fused", "two_call"):
            got = policy_call(bd, c, dtype, T, kl, ent, form, up=up)
            check_policy(c, got, dtype, T, kl, ent, up=up if form == "two_call" else None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V", [(9, 33), (12, 5003), (11, 40001)])
def test_policy_loss_special_rows(bd, rows, V, dtype):  # noqa: F811
    """Masked tokens, sure and impossible ones, rows of one value; no reference, so that a masked token's loss is finite."""
    rng = np.random.default_rng(V)
    for ent in (0.0, 0.05):
        c = policy_batch(rng, rows, V, dtype, 1.0)
        for form in ("fused", "two_call"):
            check_policy(c, policy_call(bd, c, dtype, 1.0, 0.0, ent, form, use_ref=False), dtype, 1.0, 0.0, ent, use_ref=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift,in_place", [(3, 1, False), (0, 5, True), (8, 0, True), (1, 0, False)])
def test_policy_loss_strides_and_in_place(bd, pad, shift, in_place, dtype):  # noqa: F811
    rng = np.random.default_rng(shift)
    for rows, V in ((10, 5001), (6, 70001)):
        c = policy_batch(rng, rows, V, dtype, 1.0, special=False)
        c["w"] = None
        for form in ("fused", "two_call"):
            got = policy_call(bd, c, dtype, 1.0, 0.1, 0.01, form, pad=pad, shift=shift, in_place=in_place)
            check_policy(c, got, dtype, 1.0, 0.1, 0.01)


@pytest.mark.parametrize("form", ["forward", "fused", "two_call"])
def test_policy_loss_status(bd, form):  # noqa: F811
    rng = np.random.default_rng(3)
    rows, V = 12, 2003
    c = policy_batch(rng, rows, V, "fp32", 1.0, special=False)
    c["x"][0, 5] = np.nan
    c["x"][1] = -np.inf
    c["y"][4] = V
    c["old"][5] = np.nan
    c["ref"][6] = np.inf
    c["x"][7, c["y"][7]] = -np.inf                           # a masked token under a KL term
    c["old"][8], c["adv"][8] = -500.0, -1.0                  # the ratio overflows where nothing clips it
    c["old"][9], c["adv"][9] = -500.0, 1.0                   # ... and where clipping binds
    c["adv"][10], c["old"][10] = 0.0, -500.0                 # ... and where it counts for nothing
    c["x"][2] = np.nan                                       # weight 0: not read
    bad = {r: bd.ROW_NONFINITE for r in (0, 1, 5, 6, 7, 8)} | {4: bd.ROW_BAD_TOKEN}
    got = policy_call(bd, c, "fp32", 1.0, 0.1, 0.0, form)
    # (the three rows' ratios are out of fp32's range: their bounds are not made)
    for r in (9, 10):
        assert got["status"][r] == 0 and np.isfinite(got["loss"][r])
    part = [r for r in range(rows) if r not in (9, 10)]
    keep = {k: v[part] for k, v in c.items()}
    check_policy(keep, {k: None if v is None else v[part] for k, v in got.items()}, "fp32", 1.0, 0.1, 0.0,
                 bad={part.index(r): s for r, s in bad.items()})


@pytest.mark.parametrize("form", ["fused", "two_call"])
def test_policy_reference_without_a_term(bd, form):  # noqa: F811
    """A reference that is asked about but has no weight in the loss: what it holds changes nothing but the KL."""
    c = policy_batch(np.random.default_rng(4), 6, 2003, "fp32", 1.0, special=False)
    plain = policy_call(bd, c, "fp32", 1.0, 0.0, 0.0, form)
    c["ref"][:3] = np.inf, -np.inf, np.nan
    got = policy_call(bd, c, "fp32", 1.0, 0.0, 0.0, form)
    assert not got["status"].any()
    for k in ("loss", "logprobs", "grad"):
        assert np.array_equal(got[k], plain[k])
    assert np.isposinf(got["kl"][:2]).all() and np.array_equal(got["kl"][3:], plain["kl"][3:])


def test_policy_ratio_at_a_border_is_not_clipped(bd):  # noqa: F811
    """rho = 1 with clip 0 on both sides: the gradient of rho A, as at the first step on a rollout."""
    x = np.zeros((2, 4))
    lp = np.float32(np.log(0.25))
    c = dict(x=x, y=np.array([1, 2]), old=None, adv=np.array([1.0, -2.0], np.float32), ref=np.zeros(2, np.float32), w=None)
    logits, tokens = R.on_gpu(x, "fp32"), R.i32(c["y"])
    got_lp, st = full(2, 0.0), full(2, -1, torch.int32)
    bd.dspark_token_logprobs(logits, tokens, logprobs=got_lp, row_status=st)
    assert abs(float(got_lp[0]) - lp) < 1e-6
    loss, grad, saved = full(2, 0.0), torch.empty_like(logits), torch.empty(2, 8, device="cuda")
    bd.dspark_policy_loss(logits, tokens, got_lp, R.f32(c["adv"]), loss=loss, row_status=st, saved=saved, grad=grad, clip_low=0.0,
                          clip_high=0.0)
    rho = np.exp(-1.3862943611198906 - got_lp.double().cpu().numpy())   # 1 to a bit of the log-probability
    want = -c["adv"] * np.minimum(rho, 1) if (rho >= 1).all() else -c["adv"]
    assert np.abs(loss.cpu().numpy() - want).max() < 1e-6


# ---------------------------------------------------------------- preference loss
def preference_batch(rng, lengths, V, dtype, T=1.0, tail=2, first=0):
    rows = first + sum(lengths) + tail
    x, y = T_.token_rows(rng, rows, V, dtype, special=False)
    y[rng.random(rows) < 0.2] = -1
    off = first + np.concatenate([[0], np.cumsum(lengths)])
    lp = np.array([O.token_row(x[r], y[r], T)["logp"][y[r]] if y[r] >= 0 else 0.0 for r in range(rows)])
    return dict(x=x, y=y, off=off, ref=(lp + rng.normal(0, 0.5, rows)).astype(np.float32),
                w=rng.uniform(0.5, 2, len(lengths) // 2).astype(np.float32))


def preference_call(bd, c, dtype, form, T=1.0, beta=0.1, margin=0.0, smoothing=0.0, mean=False, use_ref=True, up=None, pad=0,  # noqa: F811
                    shift=0, in_place=False):
    rows, P = len(c["x"]), len(c["off"]) // 2
    logits, tokens = R.on_gpu(c["x"], dtype, pad, shift), R.i32(c["y"])
    loss, rewards, lp = full(P, 9.0), torch.full((P, 2), 9.0, device="cuda"), full(rows, 9.0)
    st, pst, saved = full(rows, -1, torch.int32), full(P, -1, torch.int32), torch.full((rows, 8), 9.0, device="cuda")
    grad = None
    if form != "forward":
        grad = logits if in_place else R.on_gpu(np.full(c["x"].shape, 77.0), dtype, pad, shift)
    bd.dspark_preference_loss(logits, tokens, R.i32(c["off"]), loss=loss, saved=saved, row_status=st, pair_status=pst,
                              rewards=rewards, logprobs=lp, ref_logprobs=R.f32(c["ref"]) if use_ref else None,
                              weights=None if c["w"] is None else R.f32(c["w"]), grad=grad if form == "fused" else None, beta=beta,
                              margin=margin, label_smoothing=smoothing, mean=mean, temperature=T)
    if form == "two_call":
        bd.dspark_preference_loss_backward(logits, tokens, saved=saved, grad=grad, grad_loss=R.f32(np.ones(P) if up is None else up),
                                           temperature=T)
    return dict(loss=loss.cpu().numpy(), rewards=rewards.cpu().numpy(), logprobs=lp.cpu().numpy(), status=st.cpu().numpy(),
                pair_status=pst.cpu().numpy(), grad=None if grad is None else grad.double().cpu().numpy())


def check_preference(c, got, dtype, T=1.0, beta=0.1, margin=0.0, smoothing=0.0, mean=False, use_ref=True, up=None, bad_rows={},
                     bad_pairs={}):
    x, y, V, off = c["x"], c["y"], c["x"].shape[1], c["off"]
    rows, P = len(x), len(off) // 2
    info = [O.token_row(x[r], y[r], T) if y[r] >= 0 and r not in bad_rows else None for r in range(rows)]
    errs = [None if i is None else T_.row_errors(i, V) for i in info]
    for r in range(rows):
        assert got["status"][r] == bad_rows.get(r, 0), r
        close(got["logprobs"][r], np.nan if r in bad_rows else 0.0 if info[r] is None else info[r]["logp"][y[r]],
              0 if info[r] is None else errs[r][2], ("logp", r))
    a, ea = np.zeros(rows), np.zeros(rows)
    for p in range(P):
        assert got["pair_status"][p] == bad_pairs.get(p, 0), p
        if p in bad_pairs:
            assert np.isnan(got["loss"][p]) and np.isnan(got["rewards"][p]).all()
            continue
        sums, counts, es = [], [], []
        for k in (2 * p, 2 * p + 1):
            live = [r for r in range(off[k], off[k + 1]) if info[r] is not None]
            sums.append(sum(info[r]["logp"][y[r]] - (float(c["ref"][r]) if use_ref else 0.0) for r in live))
            counts.append(len(live))
            # pairs of floats: the log-probabilities' own errors before their rounding, 2^-40 for the sums
            n = max(len(live), 1) if mean else 1
            es.append(beta / n * sum(errs[r][2] + 2.0 ** -40 * fin(info[r]["logp"][y[r]]) for r in live))
        w = 1.0 if c["w"] is None else float(c["w"][p])
        loss, rewards, slopes = O.preference_pair(sums, counts, beta, margin, smoothing, mean, w)
        for k in (0, 1):
            close(got["rewards"][p, k], rewards[k], es[k] + 8 * U * fin(rewards[k]), ("reward", p))
        ez = es[0] + es[1] + 8 * U * (fin(rewards[0]) + fin(rewards[1]) + abs(margin))
        close(got["loss"][p], loss, 1.01 * w * ez + 16 * U * fin(loss) + T_.FLUSH, ("loss", p))
        u = 1.0 if up is None else float(np.float32(up[p]))
        for k in (0, 1):
            a[off[2 * p + k]:off[2 * p + k + 1]] = slopes[k] * u
            n = max(counts[k], 1) if mean else 1
            ea[off[2 * p + k]:off[2 * p + k + 1]] = abs(u) * (w * beta / n * (0.25 * ez * 1.01 + 16 * U) + 8 * U * abs(slopes[k]))
    if got["grad"] is None:
        return
    for r in range(rows):
        if info[r] is None or a[r] == 0:
            assert not got["grad"][r].any(), r
        else:
            want = O.token_grad(info[r], a[r], 0.0, T)
            close(got["grad"][r], want, T_.grad_bound(info[r], a[r], 0.0, V, T, dtype, want, ea[r]), ("grad", r))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["forward", "fused", "two_call"])
@pytest.mark.parametrize("lengths,V", [((1, 1), 1), ((1, 2), 7), ((3, 5, 0, 4), 1003), ((40, 33, 1, 300, 0, 0), 257), ((5, 7), 40001)])
def test_preference_loss(bd, lengths, V, form, dtype):  # noqa: F811
    rng = np.random.default_rng(V + len(lengths))
    up = rng.uniform(-1, 2, len(lengths) // 2).astype(np.float32)
    for how in (dict(), dict(mean=True, smoothing=0.1, margin=0.5, use_ref=False, beta=0.7), dict(T=1.4, smoothing=0.3, beta=0.02)):
        c = preference_batch(rng, lengths, V, dtype, how.get("T", 1.0), first=3 if V > 7 else 0)
        got = preference_call(bd, c, dtype, form, up=up, **how)
        check_preference(c, got, dtype, up=up if form == "two_call" else None, **how)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_preference_loss_long_sequences(bd, dtype):  # noqa: F811
    """Sums of thousands of log ratios that cancel; every row behind the last sequence has a gradient of 0."""
    c = preference_batch(np.random.default_rng(8), (3001, 2500), 65, dtype, tail=70)
    for form in ("fused", "two_call"):
        check_preference(c, preference_call(bd, c, dtype, form), dtype)


@pytest.mark.parametrize("pad,shift,in_place", [(3, 1, False), (0, 5, True), (8, 0, True)])
def test_preference_loss_strides_and_in_place(bd, pad, shift, in_place):  # noqa: F811
    c = preference_batch(np.random.default_rng(9), (6, 3, 4, 9), 5001, "bf16")
    c["w"] = None
    for form in ("fused", "two_call"):
        check_preference(c, preference_call(bd, c, "bf16", form, pad=pad, shift=shift, in_place=in_place), "bf16")


def test_preference_loss_many_pairs(bd):  # noqa: F811
    c = preference_batch(np.random.default_rng(10), tuple(i % 3 for i in range(1400)), 19, "fp32")
    check_preference(c, preference_call(bd, c, "fp32", "fused"), "fp32")


@pytest.mark.parametrize("at", [None, 1, 2900, 2901, 5999, 6000])
def test_preference_loss_runs_of_pairs(bd, at):  # noqa: F811
    """More pairs than CTAs, which take them in runs; an offset that descends ends a run's good pairs and all later ones."""
    P = 3000
    c = preference_batch(np.random.default_rng(13), tuple(i % 3 for i in range(2 * P)), 11, "fp32")
    bad = {}
    if at is not None:
        c["off"][at] = -1 if at < 2 else c["off"][at - 1] - 1
        bad = {p: bd.ROW_BAD_PARAMS for p in range(P) if (np.diff(c["off"][:2 * p + 3]) < 0).any()}
        assert len(bad) == P - (at - 1) // 2
    check_preference(c, preference_call(bd, c, "fp32", "fused"), "fp32", bad_pairs=bad)


def test_preference_loss_status(bd):  # noqa: F811
    """Bad rows spoil their own pair; a margin that is no number too."""
    c = preference_batch(np.random.default_rng(11), (4,) * 12, 1003, "fp32", tail=3)
    off, V = c["off"], 1003
    c["y"][:] = 5
    c["x"][off[1], 7] = np.nan
    c["y"][off[2]] = V
    c["ref"][off[5]] = np.nan
    c["x"][off[6], 5] = c["x"][off[7], 5] = -np.inf          # masked tokens in both: their difference is no number
    c["x"][off[8], 5] = -np.inf                              # in the chosen one alone: the loss is infinite, its gradient is not
    bad_rows = {int(off[1]): bd.ROW_NONFINITE, int(off[2]): bd.ROW_BAD_TOKEN}
    bad_pairs = {0: bd.ROW_NONFINITE, 1: bd.ROW_BAD_TOKEN, 2: bd.ROW_NONFINITE, 3: bd.ROW_NONFINITE}
    for form in ("forward", "fused", "two_call"):
        check_preference(c, preference_call(bd, c, "fp32", form), "fp32", bad_rows=bad_rows, bad_pairs=bad_pairs)


@pytest.mark.parametrize("at,value", [(0, -1), (3, 2), (4, 1000), (8, 41), (2, 4), (8, -5)])
def test_preference_loss_bad_offsets(bd, at, value):  # noqa: F811
    """Offsets that descend or leave the rows: the pairs from there on are errors, those before are right."""
    c = preference_batch(np.random.default_rng(12), (5,) * 8, 101, "fp32", tail=0)
    off = c["off"].copy()
    off[at] = value
    c["off"] = off
    bad = {}
    for p in range(4):
        upto = off[:2 * p + 3]
        if (np.diff(upto) < 0).any() or upto[0] < 0 or upto[-1] > 40:
            bad[p] = bd.ROW_BAD_PARAMS
    assert bad
    for form in ("fused", "two_call"):
        check_preference(c, preference_call(bd, c, "fp32", form), "fp32", bad_pairs=bad)


@pytest.mark.parametrize("rows,V,dtype", [(1825, 4003, "fp32"), (3649, 301, "bf16"), (1900, 16411, "bf16")])
def test_token_logprobs_of_many_rows(bd, rows, V, dtype):  # noqa: F811
    """Rows that CTAs of 64 threads take."""
    rng = np.random.default_rng(rows)
    x, y = T_.token_rows(rng, rows, V, dtype)
    up = rng.normal(0, 1, (2, rows)).astype(np.float32)
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, up=up), up)
