"""Distillation where the student's largest logit lies far above everything outside the record: what
the record leaves of the teacher's mass (one class, p_r) is still pulled towards, however small the
student's q_r.  Compared with the formulas in log space, 64 bits: q_r itself may be e^-3000."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def bd():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from sample_verify_epilogue_gb300 import binding
    binding.load_library()
    return binding


from tests import _rows as R  # noqa: E402


def log_sum(x):
    m = x.max()
    return m + np.log(np.exp(x - m).sum())


def row_reference(s, ids, logits, lse, T, w, V, dtype):
    """(loss, its bound, gradient, its bound) of a row with p_r > 0 and something outside the record.

    The bounds count roundings as those of _rows do, with every part relative to itself: ep of a p, dz of a sum
    of exponentials (or its logarithm), u per operation; the tail's logarithm is made of the gap between
    two exponents, u of it each for the product by ln 2, the addition and the product by p_r, and for c, which
    stands for log2(e)/T.  The gradient outside is the difference of two parts, and exponentials below 2^-126
    of the largest outside are flushed."""
    members = ids[ids >= 0]
    z = logits[ids >= 0].astype(np.float64) / T
    logp = z - float(lse)
    p = np.exp(logp)
    p_r = 1.0 - p.sum()
    y = s / T
    outside = np.ones(V, bool)
    outside[members] = False
    log_z, log_r = log_sum(y), log_sum(y[outside])
    logq = y - log_z
    log_qr = log_r - log_z
    loss = (p * (logp - logq[members])).sum() + p_r * (np.log(p_r) - log_qr)
    q, soft_out = np.exp(logq), np.where(outside, np.exp(np.minimum(y - log_r, 0.0)), 0.0)
    grad = q - p_r * soft_out
    grad[members] -= p

    u, dz = R.U, R.sum_bound(V)
    big = np.abs(logp).max() + abs(float(lse)) + 1
    ep = 4 * u * big + 4 * u
    dr = ep / p_r
    ratio = np.abs(logp - logq[members])
    tail = np.abs(np.log(p_r) - log_qr)
    loss_tol = (p * (ep * ratio + ep)).sum() + p.sum() * dz + ep + p_r * (dr * (tail + 1) + 2 * dz + 8 * u + 4 * u * tail)
    with np.errstate(invalid="ignore"):
        arg = np.where(np.isfinite(s), np.abs(y - y.max()), 0.0)
        arg_out = np.where(outside & np.isfinite(s), np.abs(y - y[outside].max()), 0.0)
    parts = q * (dz + R.EX2 + 3 * u * arg + 8 * u) + p_r * soft_out * (dz + R.EX2 + 3 * u * arg_out + 8 * u + dr)
    parts[members] += p * (ep + 8 * u)
    flush = 2.0 ** -126 * (1 + 2 * p_r)                      # (the outside sum is at least a half)
    g_tol = abs(w) / T * (parts + flush) + R.HALF[dtype] * np.abs(w / T * grad) + 2.0 ** -133
    return w * loss, abs(w) * loss_tol + u * abs(w * loss), w / T * grad, g_tol


def batch(rng, V, n, gaps, T, p_r, on_top, dtype, outside=None):
    """A row per gap: the record's mass is 1 - p_r, ``on_top`` of its members lie gap * T above the largest logit
    outside; ``outside``: what else than the members is finite (the rest is -inf)."""
    rows = len(gaps)
    s = rng.normal(0, 3, (rows, V)) * T
    ids = np.full((rows, n + 1), -1, np.int32)
    logits = np.zeros((rows, n + 1), np.float32)
    lse = np.float32(rng.uniform(1, 4, rows))
    for r, gap in enumerate(gaps):
        members = rng.choice(V, n, replace=False).astype(np.int32)
        ids[r, :n] = members
        logits[r, :n] = T * (np.log(rng.dirichlet(np.ones(n)) * (1 - p_r)) + lse[r])
        free = np.setdiff1d(np.arange(V), members)
        if outside is not None:
            keep = free[outside(free)]
            s[r, np.setdiff1d(free, keep)] = -np.inf
            free = keep
        s[r, members[:on_top]] = s[r, free].max() + gap * T + rng.uniform(0, 1, on_top) * T
    return dict(s=R.rounded(s, dtype), ids=ids, logits=logits, lse=lse, T=T)


def check(bd, c, dtype, form, w, up=None, pad=0):
    up = up if form == "two_call" else None                  # the one form that takes an upstream gradient
    s = R.on_gpu(c["s"], dtype, pad)
    rows, V = c["s"].shape
    given = dict(temperature=c["T"], teacher_lse=R.f32(c["lse"]), weights=R.f32(w))
    loss = torch.full((rows,), 5.0, device="cuda")
    st = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    grad = None if form == "forward" else R.on_gpu(np.full(c["s"].shape, 9.0), dtype, pad)
    ids, logits = R.i32(c["ids"]), R.f32(c["logits"])
    if form == "two_call":
        saved = torch.empty(rows, 4, device="cuda")
        bd.dspark_distill(s, ids, logits, loss=loss, row_status=st, saved=saved, **given)
        bd.dspark_distill_backward(s, ids, logits, saved=saved, grad=grad, grad_loss=R.f32(up), **given)
    else:
        bd.dspark_distill(s, ids, logits, loss=loss, row_status=st, grad=grad, **given)
    torch.cuda.synchronize()
    assert not st.any()
    loss, grad = loss.double().cpu().numpy(), None if grad is None else grad.double().cpu().numpy()
    for r in range(rows):
        args = (c["s"][r], c["ids"][r], c["logits"][r], c["lse"][r], c["T"])
        want, tol = row_reference(*args, float(w[r]), V, dtype)[:2]
        assert abs(loss[r] - want) <= tol, (r, loss[r], want, tol)
        if grad is not None:
            g, g_tol = row_reference(*args, float(w[r]) * (1.0 if up is None else float(up[r])), V, dtype)[2:]
            assert np.isfinite(grad[r]).all(), r
            assert (np.abs(grad[r] - g) <= g_tol).all(), (r, np.abs(grad[r] - g).max())


FORMS = ["forward", "fused", "two_call"]
GAPS = [20, 60, 66, 70, 80, 86, 88, 95, 120, 300, 700, 3000]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1.0, 0.1, 2.0])
@pytest.mark.parametrize("p_r,on_top", [(0.65, 1), (0.1, 3), (0.9, 8)])
def test_gap(bd, p_r, on_top, T, form, dtype):
    rng = np.random.default_rng(int(100 * p_r) + on_top)
    V = 5001
    c = batch(rng, V, 12, GAPS, T, p_r, on_top, dtype)
    w = rng.uniform(0.5, 60.0, len(GAPS)).astype(np.float32)
    up = rng.uniform(-30, 30, len(GAPS)).astype(np.float32)
    check(bd, c, dtype, form, w, up, pad=1)


@pytest.mark.parametrize("form", FORMS)
def test_gap_one_outside(bd, form):
    """A vocabulary of nine, eight of them members at the top."""
    rng = np.random.default_rng(2)
    c = batch(rng, 9, 8, GAPS, 1.0, 0.9, 8, "fp32")
    check(bd, c, "fp32", form, np.full(len(GAPS), 50.0, np.float32), np.full(len(GAPS), 7.0, np.float32))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("part", ["last", "first", "few"])
def test_gap_outside_in_one_place(bd, part, form):
    """All but one part of the row is masked: most of its CTAs have nothing outside the record."""
    V = 40001
    rng = np.random.default_rng(3)
    outside = {"last": lambda t: t >= V - 11, "first": lambda t: t < 9, "few": lambda t: t % 9001 == 5}[part]
    c = batch(rng, V, 20, GAPS, 0.5, 0.4, 2, "fp32", outside)
    w = rng.uniform(0.5, 2, len(GAPS)).astype(np.float32)
    check(bd, c, "fp32", form, w, w)


@pytest.mark.parametrize("form", FORMS)
def test_gap_between_parts(bd, form):
    """What lies outside differs by hundreds from one part of the row to the next; in 4 rows the members lie
    above all of it, in 4 above the lower parts alone."""
    V = 33001
    rng = np.random.default_rng(4)
    c = batch(rng, V, 30, [5, 90, 130, 400] * 2, 1.0, 0.5, 4, "fp32")
    c["s"] = R.rounded(c["s"] + 0.02 * np.arange(V), "fp32")
    members = c["ids"][:, :30]
    top = np.take_along_axis(c["s"], members[:, :4], 1)
    np.put_along_axis(c["s"], members[:, :4], R.rounded(np.where(np.arange(8)[:, None] < 4, top + 700, top - 300), "fp32"), 1)
    w = rng.uniform(0.5, 2, 8).astype(np.float32)
    check(bd, c, "fp32", form, w, w)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("V,dtype", [(151936, "fp32"), (300001, "bf16")])
def test_gap_long_rows(bd, V, dtype, form):
    """Rows that stream through the buffers, twice for both results."""
    rng = np.random.default_rng(5)
    gaps = [30, 87, 100, 500]
    c = batch(rng, V, 64, gaps, 1.0, 0.3, 2, dtype)
    w = rng.uniform(0.5, 2, len(gaps)).astype(np.float32)
    check(bd, c, dtype, form, w, w)
