"""The operators around the epilogue on the GPU against their float64 oracle: logit processing,
top-logit records, drafter distillation."""
import math

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


from oracle import rows as O  # noqa: E402
from tests import _rows as R  # noqa: E402

LOWEST = {"bf16": float(torch.finfo(torch.bfloat16).min), "fp32": float(torch.finfo(torch.float32).min)}


# ---------------------------------------------------------------- logit processing
def process_batch(rng, B, K, V, dtype, history=20, bias=6, masks=True, special=True):
    W = K + 1
    x = R.rounded(rng.normal(0, 3, (B, W, V)), dtype)
    if special and V > 20:
        x[0, 0, 3], x[0, 0, 5], x[-1, -1, 7] = -np.inf, LOWEST[dtype], -0.0
    hist, bias_rows = [], []
    hot = rng.permutation(V)[:max(1, V // 4)]
    for b in range(B):
        ids = np.unique(rng.choice(hot, min(history, V)))
        hist.append([(int(t), int(rng.integers(0, 5))) for t in ids] if b % 3 != 2 else [])
        ids = np.unique(np.concatenate([rng.choice(hot, min(bias, V)), rng.integers(0, V, 3)]))
        bias_rows.append([(int(t), -np.inf if rng.random() < 0.2 else float(np.float32(rng.normal(0, 4)))) for t in ids]
                         if b % 4 != 1 else [])
    drafts = rng.choice(hot, (B, max(K, 1)))
    if K > 2:
        drafts[:, 2] = drafts[:, 0]
    rows = np.zeros(B, [("r", "f4"), ("p", "f4"), ("f", "f4"), ("k", "i4")])
    rows["r"], rows["p"], rows["f"] = rng.choice([1, 1.3, 0.8], B), rng.choice([0, 0.5, -0.25], B), rng.choice([0, 0.3], B)
    rows["k"] = [K - b % (K + 1) if b else K for b in range(B)]
    mask_rows = allowed = None
    if masks:
        share = rng.choice([0.0, 0.01, 0.5, 0.99, 1.0], B * W)
        allowed = rng.random((B * W, V)) < share[:, None]
        mask_rows = np.where(rng.random((B, W)) < 0.3, -1, rng.permutation(B * W).reshape(B, W))
    return dict(x=x, hist=hist, bias=bias_rows, drafts=drafts, rows=rows, mask_rows=mask_rows, allowed=allowed)


def process_call(bd, c, dtype, pad=0, shift=0, in_place=False, out_shift=None, stream=None):
    B, W, V = c["x"].shape
    x = R.on_gpu(c["x"], dtype, pad, shift)
    out = x if in_place else R.on_gpu(np.full(c["x"].shape, 77.0), dtype, pad, shift if out_shift is None else out_shift)
    status = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    bd.dspark_process_logits(
        x, torch.from_numpy(c["rows"].view(np.uint8).copy()).cuda(), out=out, row_status=status,
        draft_ids=R.i32(c["drafts"]) if W > 1 else None,
        history=R.csr(c["hist"], np.int32, np.int32) if c["hist"] is not None else None,
        bias=R.csr(c["bias"], np.int32, np.float32) if c["bias"] is not None else None,
        mask=R.pack_mask(c["allowed"]) if c["allowed"] is not None else None,
        mask_rows=R.i32(c["mask_rows"]) if c["mask_rows"] is not None else None, stream=stream)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), status.cpu().numpy()


def check_process(c, got, status, dtype, untouched):
    B, W, V = c["x"].shape
    assert (status == 0).all()
    for b in range(B):
        r = c["rows"][b]
        r_, p_, f_ = float(r["r"]), float(r["p"]), float(r["f"])
        counts, bias = dict(c["hist"][b]) if c["hist"] else {}, dict(c["bias"][b]) if c["bias"] else {}
        for j in range(W):
            if j > r["k"]:
                assert np.array_equal(got[b, j], untouched[b, j], equal_nan=True)
                continue
            allowed = None
            if c["allowed"] is not None:
                k = c["mask_rows"][b, j] if c["mask_rows"] is not None else b * W + j
                allowed = c["allowed"][k] if k >= 0 else None
            want = O.process_row(c["x"][b, j], r_, p_, f_, counts, c["drafts"][b, :j], bias, allowed)
            # what the type cannot hold is -inf: a repetition penalty on its lowest value
            want[want < LOWEST[dtype] * (1 + R.HALF[dtype] / 2)] = -np.inf
            # five fp32 operations, each half a step of the largest value on the way, then the type's
            with np.errstate(invalid="ignore"):
                way = np.abs(c["x"][b, j]) * max(r_, 1 / r_, 1)
            way[~np.isfinite(way)] = 0
            worst = max([0] + [abs(v) for v in bias.values() if np.isfinite(v)]) + abs(p_) + abs(f_) * (5 + W)
            with np.errstate(invalid="ignore"):
                tol = 6 * R.U * (way + worst) + R.HALF[dtype] * np.abs(want)
                same = np.isfinite(want)
                assert (np.abs(got[b, j] - want)[same] <= tol[same]).all(), (b, j)
            assert np.array_equal(got[b, j][~same], want[~same], equal_nan=True), (b, j)
            if dtype == "fp32":        # tokens that no rule names keep their bits
                named = set(counts) | set(bias) | set(c["drafts"][b, :j].tolist())
                rest = np.setdiff1d(np.nonzero(same)[0], list(named))
                assert np.array_equal(got[b, j][rest], c["x"][b, j][rest])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (1, 0, 7), (2, 1, 17), (3, 3, 1003), (5, 4, 8193), (2, 2, 32003), (2, 8, 151936)])
def test_process(bd, B, K, V, dtype):
    c = process_batch(np.random.default_rng(V + B), B, K, V, dtype, history=300 if V > 1000 else 5)
    got, status = process_call(bd, c, dtype)
    check_process(c, got, status, dtype, np.full(c["x"].shape, 77.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift,out_shift", [(1, 0, 0), (3, 5, 5), (8, 1, 0), (0, 3, 6)])
def test_process_strides_and_alignment(bd, pad, shift, out_shift, dtype):
    c = process_batch(np.random.default_rng(pad + shift), 3, 2, 5001, dtype)
    got, status = process_call(bd, c, dtype, pad, shift, out_shift=out_shift)
    check_process(c, got, status, dtype, np.full(c["x"].shape, 77.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,pad,shift", [(9, 0, 0), (5001, 0, 0), (40000, 3, 1)])
def test_process_in_place(bd, V, pad, shift, dtype):
    c = process_batch(np.random.default_rng(V), 4, 3, V, dtype, history=400 if V > 1000 else 4)
    got, status = process_call(bd, c, dtype, pad, shift, in_place=True)
    check_process(c, got, status, dtype, c["x"])


@pytest.mark.parametrize("part", ["history", "bias", "mask", "drafts", "nothing"])
def test_process_parts(bd, part):
    c = process_batch(np.random.default_rng(3), 3, 2, 3001, "bf16", masks=part == "mask")
    if part != "history":
        c["hist"] = None
    if part != "bias":
        c["bias"] = None
    if part in ("bias", "mask", "nothing"):
        c["rows"]["r"], c["rows"]["p"], c["rows"]["f"] = 1, 0, 0
    if part == "mask":                                    # mask rows of their own position
        c["mask_rows"] = None
    got, status = process_call(bd, c, "bf16")
    check_process(c, got, status, "bf16", np.full(c["x"].shape, 77.0))


def test_process_nan_in_masked_places(bd):
    c = process_batch(np.random.default_rng(9), 2, 1, 2003, "bf16", masks=True, special=False)
    c["mask_rows"] = np.arange(4).reshape(2, 2)
    c["allowed"][:] = np.random.default_rng(1).random((4, 2003)) < 0.5
    c["allowed"][3] = False
    c["x"][:, :, ::7] = np.nan
    c["x"][:, :, 1::7] = np.inf
    got, status = process_call(bd, c, "bf16")
    assert (status == 0).all()
    for b in range(2):
        for j in range(c["rows"]["k"][b] + 1):
            off = ~c["allowed"][2 * b + j]
            assert np.isneginf(got[b, j][off]).all()
            assert np.isnan(got[b, j][::7][~off[::7]]).all()


def test_process_every_token_listed(bd):
    """Lists as long as the vocabulary: many listed tokens per span."""
    rng = np.random.default_rng(4)
    c = process_batch(rng, 2, 2, 20001, "fp32", masks=False)
    c["hist"] = [[(t, t % 3) for t in range(20001)], [(t, 1) for t in range(0, 20001, 2)]]
    c["bias"] = [[(t, float(np.float32(0.25 * (t % 9)))) for t in range(20001)], [(t, -1.5) for t in range(1, 20001, 3)]]
    for in_place in (False, True):
        got, status = process_call(bd, c, "fp32", in_place=in_place)
        check_process(c, got, status, "fp32", c["x"] if in_place else np.full(c["x"].shape, 77.0))


def test_process_status(bd):
    """Each bad request is reported; its neighbours are right."""
    from sample_verify_epilogue_gb300 import binding as b_
    B, K, V = 9, 2, 1003
    c = process_batch(np.random.default_rng(5), B, K, V, "fp32")
    c["rows"]["k"] = K
    c["mask_rows"][:] = 0
    want = np.zeros(B, int)
    c["rows"]["r"][0], want[0] = 0.0, b_.ROW_BAD_PARAMS
    c["rows"]["p"][1], want[1] = np.nan, b_.ROW_BAD_PARAMS
    c["rows"]["k"][2], want[2] = K + 1, b_.ROW_BAD_PARAMS
    c["hist"][3], want[3] = [(5, 1), (5, 1)], b_.ROW_BAD_HISTORY
    c["hist"][4], want[4] = [(3, 1), (V, 2)], b_.ROW_BAD_HISTORY
    c["bias"][5], want[5] = [(2, 1.0), (9, np.nan)], b_.ROW_BAD_BIAS
    c["drafts"][6, 1], want[6] = -1, b_.ROW_BAD_DRAFT
    c["mask_rows"][7, 1], want[7] = len(c["allowed"]), b_.ROW_BAD_MASK
    got, status = process_call(bd, c, "fp32")
    assert np.array_equal(status, want)
    good = {k: (v[8:] if k != "allowed" else v) for k, v in c.items()}
    check_process(good, got[8:], status[8:], "fp32", np.full(good["x"].shape, 77.0))


# ---------------------------------------------------------------- top logits
def top_call(bd, x, dtype, n, temperature=1.0, pad=0, shift=0, want_lse=True):
    t = R.on_gpu(x, dtype, pad, shift)
    rows = x.shape[:-1]
    v = torch.full((*rows, n), 5.0, device="cuda")
    i = torch.full((*rows, n), 5, dtype=torch.int32, device="cuda")
    lse = torch.full(rows, 5.0, device="cuda") if want_lse else None
    st = torch.full(rows, -1, dtype=torch.int32, device="cuda")
    bd.dspark_top_logits(t, values=v, ids=i, lse=lse, row_status=st, temperature=temperature)
    torch.cuda.synchronize()
    return [None if a is None else a.cpu().numpy().reshape(-1, *a.shape[len(rows):]) for a in (v, i, lse, st)]


def check_top(x, n, temperature, got):
    V = x.shape[-1]
    v, i, lse, st = got
    for r, row in enumerate(x.reshape(-1, V)):
        wv, wi, wl, ok = O.top_row(row, n, temperature)
        assert st[r] == (0 if ok else 4)
        assert np.array_equal(i[r], wi), r
        assert np.array_equal(v[r].astype(np.float64), wv), r
        if lse is not None:
            if ok:
                assert abs(lse[r] - wl) <= R.sum_bound(V) + 2 * R.U * abs(wl) + 2 * R.U * abs(row.max() / temperature)
            else:
                assert np.isnan(lse[r])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V,n,T", [(1, 1, 1, 1.0), (3, 5, 8, 1.0), (2, 256, 256, 0.5), (4, 1003, 20, 2.0),
                                        (3, 8200, 64, 1.0), (2, 33001, 256, 0.7), (9, 151936, 20, 1.0), (2, 262144, 128, 1.5)])
def test_top(bd, rows, V, n, T, dtype):
    x = R.rounded(np.random.default_rng(V + n).normal(0, 3, (rows, V)), dtype)
    check_top(x, n, T, top_call(bd, x, dtype, n, T))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [7, 301])
@pytest.mark.parametrize("V", [255, 1024, 1030, 2049, 4096, 8185, 8193, 24600])
def test_top_short_rows(bd, V, rows, dtype):
    """Records that take much of a row, where a row has few vectors to a thread: few rows (spread over CTAs,
    looked at again in shared memory) and many; grammars that leave less than the record wants; ties."""
    rng = np.random.default_rng(V)
    x = rng.normal(0, 3, (rows, V))
    x[1, rng.permutation(V)[:V - 100]] = -np.inf
    x[2] = np.round(x[2])
    x[3, : V // 2] = -np.inf
    x[4] = np.sort(x[4])
    for n in (1, 200, 256):
        y = R.rounded(x, dtype)
        check_top(y, n, 1.3, top_call(bd, y, dtype, n, 1.3, 1, 3 if n == 200 else 0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two_values", "zeros", "mostly_masked", "lowest", "negative"])
@pytest.mark.parametrize("n", [1, 50, 256])
def test_top_hard_rows(bd, kind, n, dtype):
    """Rows that fill the key buffer, ties across the whole row, masked rows."""
    V = 40001
    rng = np.random.default_rng(n)
    x = np.zeros((2, V))
    if kind == "equal":
        x[:] = 1.25
    elif kind == "ascending":
        x[:] = np.linspace(-20, 20, V)
    elif kind == "descending":
        x[:] = np.linspace(20, -20, V)
    elif kind == "two_values":
        x[:] = np.where(rng.random((2, V)) < 0.9, 2.0, 3.0)
    elif kind == "zeros":
        x[:] = np.where(rng.random((2, V)) < 0.5, 0.0, -0.0)
    elif kind == "mostly_masked":
        x[:] = -np.inf
        x[0, ::3001], x[1, 39999] = rng.normal(0, 1, 14), 0.5
    elif kind == "lowest":
        x[:] = LOWEST[dtype]
        x[1, 7::5003] = rng.normal(0, 1, len(x[1, 7::5003]))
    elif kind == "negative":
        x[:] = -rng.gamma(2.0, 5.0, (2, V))
    x = R.rounded(x, dtype)
    check_top(x, n, 1.0, top_call(bd, x, dtype, n))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (8, 1)])
def test_top_strides(bd, pad, shift, dtype):
    x = R.rounded(np.random.default_rng(pad).normal(0, 3, (2, 3, 9001)), dtype)
    check_top(x, 33, 1.0, top_call(bd, x, dtype, 33, pad=pad, shift=shift, want_lse=shift != 1))


def test_top_nonfinite(bd):
    x = np.random.default_rng(1).normal(0, 3, (5, 20001)).astype(np.float32).astype(np.float64)
    x[0, 19000], x[1, 3], x[2] = np.nan, np.inf, -np.inf
    x[4, :5000] = -np.inf
    check_top(x, 7, 1.0, top_call(bd, x, "fp32", 7))


def test_rows_past_32_bit_offsets(bd):
    """A row more than 2^31 elements into its buffer."""
    V, stride, n = 1003, (1 << 31) + 24, 9
    buf = torch.empty(stride + V, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((2, V), (stride, 1))
    x = R.rounded(np.random.default_rng(2).normal(0, 3, (2, V)), "bf16")
    t.copy_(torch.from_numpy(x).to(torch.bfloat16))
    v, i = torch.empty(2, n, device="cuda"), torch.empty(2, n, dtype=torch.int32, device="cuda")
    lse, st = torch.empty(2, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    bd.dspark_top_logits(t, values=v, ids=i, lse=lse, row_status=st)
    check_top(x, n, 1.0, [a.cpu().numpy() for a in (v, i, lse, st)])
    loss = torch.empty(2, device="cuda")
    bd.dspark_distill(t, i, v, loss=loss, row_status=st, grad=t, teacher_lse=lse)
    want = O.distill_row(x[1], i[1].cpu().numpy(), v[1].cpu().numpy(), float(lse[1]), 1.0, 1.0)
    assert np.abs(t[1].double().cpu().numpy() - want[1]).max() <= 1e-5
    t.copy_(torch.from_numpy(x).to(torch.bfloat16))
    rows = torch.from_numpy(np.array([(2.0, 0, 0, 1)], "f4,f4,f4,i4").view(np.uint8).copy()).cuda()
    h = (R.i32([0, 1]), R.i32([5]), R.i32([0]))
    bd.dspark_process_logits(t.view(1, 2, V) if t.is_contiguous() else t[None], rows, out=t[None], row_status=st[:1], history=h,
                             draft_ids=R.i32([[9]]))
    want = O.process_row(x[1], 2.0, 0.0, 0.0, {5: 0}, [9], {}, None)
    assert np.array_equal(t[1].double().cpu().numpy(), R.rounded(want, "bf16"))


# ---------------------------------------------------------------- distillation
def distill_batch(rng, rows, V, n, dtype, T, tail, reduced=False):
    target_V = 2 * V + 3 if reduced else V
    t2d = None
    teacher = rng.normal(0, 3, (rows, target_V))
    if reduced:
        subset = np.sort(rng.choice(target_V, V, replace=False))
        t2d = np.full(target_V, -1, np.int32)
        t2d[subset] = np.arange(V)
        s = teacher[:, subset] + rng.normal(0, 1, (rows, V))
    else:
        s = teacher + rng.normal(0, 1, (rows, V))
    m = min(n, target_V)
    ids = np.full((rows, n), -1, np.int32)
    logits = np.full((rows, n), -np.inf, np.float32)
    order = np.argsort(-teacher, axis=1, kind="stable")[:, :m]
    ids[:, :m] = order
    logits[:, :m] = np.take_along_axis(teacher, order, 1)
    if m > 3:
        ids[::2, 2] = -1
    z = teacher / T
    lse = (z.max(1) + np.log(np.exp(z - z.max(1, keepdims=True)).sum(1))).astype(np.float32)
    w = rng.uniform(0.5, 2.0, rows).astype(np.float32)
    if rows > 3:
        w[3] = 0.0
        ids[2] = -1
    return dict(s=R.rounded(s, dtype), ids=ids, logits=logits, lse=lse if tail else None, t2d=t2d, w=w, T=T)


def distill_call(bd, c, dtype, form, pad=0, shift=0, gshift=None, up=None, in_place=False):
    s = R.on_gpu(c["s"], dtype, pad, shift)
    rows = c["s"].shape[:-1]
    given = dict(temperature=c["T"], teacher_lse=None if c["lse"] is None else R.f32(c["lse"]),
                 t2d=None if c["t2d"] is None else R.i32(c["t2d"]), weights=None if c["w"] is None else R.f32(c["w"]))
    loss = torch.full(rows, 5.0, device="cuda")
    st = torch.full(rows, -1, dtype=torch.int32, device="cuda")
    grad = None
    if form != "forward":
        grad = s if in_place else R.on_gpu(np.full(c["s"].shape, 9.0), dtype, pad, shift if gshift is None else gshift)
    ids, logits = R.i32(c["ids"]), R.f32(c["logits"])
    if form == "two_call":
        saved = torch.empty(*rows, 4, device="cuda")
        bd.dspark_distill(s, ids, logits, loss=loss, row_status=st, saved=saved, **given)
        bd.dspark_distill_backward(s, ids, logits, saved=saved, grad=grad, grad_loss=None if up is None else R.f32(up), **given)
    else:
        bd.dspark_distill(s, ids, logits, loss=loss, row_status=st, grad=grad, **given)
    torch.cuda.synchronize()
    return loss.cpu().numpy().reshape(-1), None if grad is None else grad.double().cpu().numpy(), st.cpu().numpy().reshape(-1)


def check_distill(c, got, dtype, up=None, bad=()):
    loss, grad, st = got
    V = c["s"].shape[-1]
    for r in range(len(loss)):
        if r in bad:
            continue
        ids = c["ids"][r]
        if c["t2d"] is not None:
            ids = np.where(ids < 0, -1, c["t2d"][np.maximum(ids, 0)])
        w = 1.0 if c["w"] is None else float(c["w"][r])
        lse = None if c["lse"] is None else float(c["lse"][r])
        want, wgrad, d = O.distill_row(c["s"][r], ids, c["logits"][r], lse, c["T"], w)
        assert st[r] == (4 if np.isnan(want) else 0), r
        with np.errstate(over="ignore"):
            out = np.float32(want)                           # a loss past fp32's range is infinite
        if np.isfinite(out):
            assert abs(loss[r] - want) <= R.loss_bound(d, V, w, lse, c["T"]) + R.U * abs(want), (r, loss[r], want)
        else:
            assert np.array_equal(loss[r], out, equal_nan=True), (r, loss[r], want)
        if grad is not None:
            g = 1.0 if up is None else float(up[r])
            tol = R.grad_bound(d, V, w * g, c["T"], lse, c["s"][r], dtype, wgrad * g)
            assert (np.abs(grad[r] - wgrad * g) <= tol).all(), (r, np.abs(grad[r] - wgrad * g).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["forward", "fused", "two_call"])
@pytest.mark.parametrize("rows,V,n,T,tail", [(1, 1, 1, 1.0, True), (5, 7, 8, 1.0, False), (4, 19, 3, 2.0, True),
                                             (6, 1003, 20, 1.5, True), (5, 8200, 256, 1.0, False),
                                             (4, 33001, 64, 1.0, True), (4, 151936, 100, 2.0, False)])
def test_distill(bd, rows, V, n, T, tail, form, dtype):
    rng = np.random.default_rng(V + n)
    c = distill_batch(rng, rows, V, n, dtype, T, tail)
    up = rng.uniform(-1, 2, rows).astype(np.float32) if form == "two_call" else None
    check_distill(c, distill_call(bd, c, dtype, form, up=up), dtype, up=up)


@pytest.mark.parametrize("V,dtype,shift", [(32003, "fp32", 1), (50001, "fp32", 3), (75968, "fp32", 0), (74530, "fp32", 1),
                                           (100003, "bf16", 5)])
def test_distill_rows_enough_to_fill(bd, V, dtype, shift):
    """More rows than the GPU has SMs: a row goes to 3, 5, 6, 7 and 5 CTAs."""
    rng = np.random.default_rng(V)
    c = distill_batch(rng, 161, V, 50, dtype, 1.0, True)
    c["w"][rng.permutation(161)[:140]] = 0
    check_distill(c, distill_call(bd, c, dtype, "fused", 1, shift), dtype)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("form", ["fused", "two_call"])
def test_distill_reduced_vocabulary(bd, form, tail):
    c = distill_batch(np.random.default_rng(8), 6, 5003, 40, "bf16", 1.0, tail, reduced=True)
    check_distill(c, distill_call(bd, c, "bf16", form), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["fused", "two_call"])
@pytest.mark.parametrize("pad,shift,gshift,in_place", [(1, 0, 0, False), (3, 5, 5, False), (8, 1, 0, False), (1, 1, 1, True), (0, 0, 0, True)])
def test_distill_strides_and_in_place(bd, pad, shift, gshift, in_place, form, dtype):
    c = distill_batch(np.random.default_rng(pad), 5, 9001, 30, dtype, 1.0, True)
    check_distill(c, distill_call(bd, c, dtype, form, pad, shift, gshift, in_place=in_place), dtype)


@pytest.mark.parametrize("form", ["fused", "two_call"])
@pytest.mark.parametrize("tail", [True, False])
def test_distill_edge_rows(bd, form, tail):
    """Masked student logits (members among them), the type's lowest value, records that carry all
    of the mass or next to none of it, a -inf entry, an unweighted batch."""
    V, n = 5001, 16
    c = distill_batch(np.random.default_rng(6), 8, V, n, "fp32", 1.0, tail)
    c["w"] = None
    c["ids"][2] = c["ids"][1]
    c["logits"][2] = c["logits"][1]
    c["s"][0, 1000:4000] = -np.inf
    members = c["ids"][0][c["ids"][0] >= 0]
    c["s"][0, members] = 1.0                                 # stay finite: the loss is finite
    c["s"][1, :] = LOWEST["fp32"]
    c["s"][1, c["ids"][1][0]] = 2.0
    c["s"][4, c["ids"][4][0]] += 60.0                        # the student puts all mass on one member
    c["logits"][5] -= 40.0                                   # (tail) a record with no mass
    c["logits"][6, 1] = -np.inf
    c["s"][7, c["ids"][7][0]] = -np.inf                      # q = 0 where p > 0: an infinite loss
    got = distill_call(bd, c, "fp32", form)
    assert np.isposinf(got[0][7])
    # row 1: the other members lie 3e38 below: an infinite loss too, as in the oracle's float64 up to its size
    check_distill(c, got, "fp32", bad=(1, 7))
    assert got[2][1] == 0 and got[0][1] > 1e37
    d = O.distill_row(c["s"][7], c["ids"][7], c["logits"][7], None if not tail else float(c["lse"][7]), 1.0, 1.0)
    assert np.isfinite(got[1][7]).all() and np.abs(got[1][7] - d[1]).max() < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("tail", [True, False])
def test_distill_rows_of_the_lowest_value(bd, tail, T, dtype):
    """Masks that write the type's lowest value: a row that is nothing else, one with all but its members at
    it, one with all but a single other logit at it."""
    V, n = 9001, 12
    c = distill_batch(np.random.default_rng(16), 4, V, n, dtype, T, tail)
    c["w"] = None
    c["ids"][2:] = c["ids"][0]
    c["logits"][2:] = c["logits"][0]
    c["s"][0, :] = LOWEST[dtype]
    members = c["ids"][1][c["ids"][1] >= 0]
    kept = c["s"][1, members]
    c["s"][1, :] = LOWEST[dtype]
    c["s"][1, members] = kept
    c["s"][2, :] = LOWEST[dtype]
    c["s"][2, 77] = LOWEST[dtype] * 0.5
    got = distill_call(bd, c, dtype, "fused")
    check_distill(c, got, dtype)                             # row 1 with a tail: q_r = 0; row 2: a loss of some 1e37


def test_distill_status(bd):
    from sample_verify_epilogue_gb300 import binding as b_
    V, n = 5001, 16
    c = distill_batch(np.random.default_rng(7), 10, V, n, "bf16", 1.0, True)
    c["w"][:] = 1
    c["w"][9] = 0
    c["ids"][0, 1] = V
    c["ids"][1, 1] = c["ids"][1, 0]
    c["logits"][2, 3], c["ids"][2] = np.nan, c["ids"][3]
    c["lse"][4] = np.inf
    c["ids"][5, 0] = -2
    c["s"][6, 17], c["s"][7, 4000], c["s"][8] = np.nan, np.inf, -np.inf
    c["s"][9, 3] = np.nan                                    # weight 0: not read
    for form in ("fused", "two_call"):
        loss, grad, st = distill_call(bd, c, "bf16", form)
        want = np.array([b_.ROW_BAD_TEACHER] * 3 + [0] + [b_.ROW_BAD_TEACHER] * 2 + [b_.ROW_NONFINITE] * 3 + [0])
        assert np.array_equal(st, want)
        assert np.array_equal(np.isnan(loss), want != 0) and loss[9] == 0
        assert (grad[want != 0] == 0).all() and (grad[9] == 0).all() and np.abs(grad[3]).max() > 0
        check_distill(c, (loss, grad, st), "bf16", bad=set(np.nonzero(want)[0]) | {9})


def test_distill_gradient_by_differences(bd):
    """The fused gradient against central differences of the float64 loss at the kernel's own inputs."""
    V, n = 257, 12
    c = distill_batch(np.random.default_rng(11), 3, V, n, "fp32", 1.5, True)
    _, grad, _ = distill_call(bd, c, "fp32", "fused")
    h = 1e-5
    for r in range(2):
        for v in list(range(0, V, 16)) + list(c["ids"][r][c["ids"][r] >= 0][:4]):
            two = []
            for e in (h, -h):
                s = c["s"][r].copy()
                s[v] += e
                two.append(O.distill_row(s, c["ids"][r], c["logits"][r], float(c["lse"][r]), 1.5, float(c["w"][r]))[0])
            # differences: third derivative h^2 and float64 roundings over h
            assert abs((two[0] - two[1]) / (2 * h) - grad[r, v]) < 1e-8 + 2e-5 * abs(grad[r, v]) + 1e-7


def test_distill_autograd(bd):
    from sample_verify_epilogue_gb300.distill import distill_loss
    rng = np.random.default_rng(12)
    c = distill_batch(rng, 6, 3001, 10, "fp32", 1.0, True)
    c["w"][:] = 1
    student = R.f32(c["s"]).view(2, 3, 3001).requires_grad_()
    loss, status = distill_loss(student, R.i32(c["ids"]), R.f32(c["logits"]), teacher_lse=R.f32(c["lse"]), weights=R.f32(c["w"]))
    up = rng.uniform(0, 2, 6).astype(np.float32)
    (loss * R.f32(up).view(2, 3)).sum().backward()
    got = loss.detach().cpu().numpy().reshape(-1), student.grad.double().cpu().numpy().reshape(6, -1), status.cpu().numpy().reshape(-1)
    check_distill(c, got, "fp32", up=up)


# ---------------------------------------------------------------- streams, graphs, repeatability
def test_streams_and_graph(bd):
    """On another stream than the current one, and captured into a graph: the same bits each time."""
    x = torch.randn(12, 40001, device="cuda").to(torch.bfloat16)
    n = 40
    v, i = torch.empty(12, n, device="cuda"), torch.empty(12, n, dtype=torch.int32, device="cuda")
    lse, st, loss = torch.empty(12, device="cuda"), torch.empty(12, dtype=torch.int32, device="cuda"), torch.empty(12, device="cuda")
    y, g = torch.empty_like(x), torch.empty_like(x)
    rows = torch.from_numpy(np.array([(1.2, 0.1, 0.2, 2)] * 4, "f4,f4,f4,i4").view(np.uint8).copy()).cuda()
    d = torch.randint(0, 40001, (4, 2), device="cuda", dtype=torch.int32)
    status = torch.empty(4, dtype=torch.int32, device="cuda")

    def step():
        bd.dspark_process_logits(x.view(4, 3, -1), rows, out=y.view(4, 3, -1), row_status=status, draft_ids=d)
        bd.dspark_top_logits(y, values=v, ids=i, lse=lse, row_status=st)
        bd.dspark_distill(x, i, v, loss=loss, row_status=st, grad=g, teacher_lse=lse)

    step()
    torch.cuda.synchronize()
    first = [a.clone() for a in (y, v, i, lse, loss, g)]
    side = torch.cuda.Stream()
    for a in (y, v, lse, loss, g):
        a.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, v, i, lse, loss, g)))
    for a in (y, v, lse, loss, g):
        a.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (y, v, i, lse, loss, g)))


def test_between_copies_and_fills(bd):
    """A launch waits for whatever its stream holds before it, and what follows waits for it: copies from and
    to the host, fills, a fork to another stream and back; eagerly and in a graph."""
    R_, V, n = 24, 30011, 16
    host = (torch.randn(3, R_, V) * 3).pin_memory()
    x, y, g = (torch.zeros(R_, V, device="cuda") for _ in range(3))
    v, i = torch.empty(R_, n, device="cuda"), torch.empty(R_, n, dtype=torch.int32, device="cuda")
    st, status = torch.empty(R_, dtype=torch.int32, device="cuda"), torch.empty(R_, dtype=torch.int32, device="cuda")
    lse, loss, loss2 = (torch.empty(R_, device="cuda") for _ in range(3))
    back = torch.empty(R_, V).pin_memory()
    rows = torch.from_numpy(np.array([(1.2, 0.1, 0.2, 0)] * R_, "f4,f4,f4,i4").view(np.uint8).copy()).cuda()
    bias = (torch.arange(R_ + 1, dtype=torch.int32).cuda(), torch.arange(R_, dtype=torch.int32).cuda() * 7,
            torch.full((R_,), -math.inf, device="cuda"))
    side = torch.cuda.Stream()

    def step():
        x.copy_(host[0], non_blocking=True)
        bd.dspark_process_logits(x.view(R_, 1, V), rows, out=y.view(R_, 1, V), row_status=status, bias=bias)
        x.zero_()
        bd.dspark_top_logits(y, values=v, ids=i, lse=lse, row_status=st)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            bd.dspark_distill(y, i, v, loss=loss2, row_status=status, teacher_lse=lse)
        x.copy_(host[1], non_blocking=True)
        bd.dspark_distill(x, i, v, loss=loss, row_status=st, grad=g, teacher_lse=lse)
        back.copy_(g, non_blocking=True)
        torch.cuda.current_stream().wait_stream(side)
        y.zero_()
        g.zero_()

    def check():
        torch.cuda.synchronize()
        want = host[0].clone()
        want[torch.arange(R_), torch.arange(R_) * 7] = -math.inf
        top = torch.topk(want, n)
        assert torch.equal(v.cpu(), top.values) and torch.equal(i.cpu().long(), top.indices)
        # the record of y against y itself has no divergence, against x some
        assert loss2.abs().max() < 1e-5 and loss.min() > 0.1
        q = torch.softmax(host[1].double(), -1)
        p = torch.exp(top.values.double() - torch.logsumexp(want.double(), -1, keepdim=True))
        inside = torch.zeros(R_, V, dtype=torch.bool).scatter_(1, top.indices, True)
        left, q_left = 1 - p.sum(-1, keepdim=True), torch.where(inside, 0.0, q).sum(-1, keepdim=True)
        grad = (q * (1 - left / q_left)).scatter(1, top.indices, q.gather(1, top.indices) - p)
        assert (back.double() - grad).abs().max() < 2e-6   # a dozen roundings of values below 1, 2^-24 each
        assert not y.any() and not g.any()

    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for a in (v, lse, loss, back):
            a.zero_()
        graph.replay()
        check()


def test_chain_with_the_epilogue(bd):
    """Processed logits go through dspark_verify_sample, greedily: with the same penalties the
    epilogue's own path gives the same tokens, and a mask keeps every token inside it."""
    from sample_verify_epilogue_gb300.runner import EpilogueCall
    from workloads.generate import make_batch, row_params
    B, K, V = 3, 3, 5001
    batch = make_batch(B=B, K_max=K, V=V, logits_dtype="fp32", rows=[row_params(0.0, 0, 1.0, 0.4, 0.3, K)] * B, seed=3,
                       philox_seed=3, history_len=64, draft_mode="argmax")
    call = EpilogueCall(batch)
    call.run()
    own = call.results()
    rows = torch.from_numpy(np.array([(1.0, 0.4, 0.3, K)] * B, "f4,f4,f4,i4").view(np.uint8).copy()).cuda()
    status = torch.empty(B, dtype=torch.int32, device="cuda")
    raw = call.x.clone()
    call.rows = torch.from_numpy(np.array([row_params(0.0, 0, 1.0, 0, 0, K)] * B, batch.rows.dtype).view(np.uint8).copy()).cuda()
    bd.dspark_process_logits(raw, rows, out=call.x, row_status=status, draft_ids=call.d, history=call.counts)
    call.run()
    got = call.results()
    assert np.array_equal(got["tokens"], own["tokens"]) and np.array_equal(got["accept_len"], own["accept_len"])
    allowed = np.zeros((1, V), bool)
    allowed[0, 100:200] = True
    bd.dspark_process_logits(raw, rows, out=call.x, row_status=status, draft_ids=call.d, history=call.counts,
                             mask=R.pack_mask(allowed), mask_rows=torch.zeros(B, K + 1, dtype=torch.int32, device="cuda"))
    call.run()
    tokens = call.results()["tokens"]
    tokens = tokens[tokens >= 0]
    assert len(tokens) and ((tokens >= 100) & (tokens < 200)).all()
    assert math.isfinite(float(call.x[0, 0, 150]))


def test_example_round_trip(bd):
    """The example's rounds: the drafter's loss falls, and no emitted token breaks its grammar or its ban."""
    from examples.constrained_verify_distill import run
    losses, accepted, legal = run(rounds=20, B=16, K=3, V=5003, draft_V=1201, hidden=16, n=32, say=lambda *_: None)
    # (a round's 48 rows are other rows than the last one's: means over five rounds)
    assert legal and all(np.isfinite(losses)) and np.mean(losses[-5:]) < 0.9 * np.mean(losses[:5])
