"""Calls of the operators around the epilogue that a server or a trainer makes beside the plain ones: empty
lists and masks, several host threads, explicit streams, records with masked entries."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _rows as R  # noqa: E402
from tests.test_rows_gpu import (  # noqa: E402,F401
    bd, check_distill, check_process, check_top, distill_batch, distill_call, process_batch, process_call, top_call)


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


def test_calls_from_two_threads(bd):
    """Loss and gradient of rows of two lengths from two host threads at once, whose CTAs keep spans of 36 and
    of 72 KB: a launch needs its own limit whatever the other thread does at the time."""
    import ctypes
    import threading
    lib, calls = bd.load_library(), []
    for V in (72000, 144000):
        c = distill_batch(np.random.default_rng(V), 2, V, 16, "fp32", 1.0, True)
        t = [R.f32(c["s"]), R.i32(c["ids"]), R.f32(c["logits"]), R.f32(c["lse"]), R.f32(c["w"]), torch.zeros(2, device="cuda"),
             R.i32([-1, -1]), torch.zeros(2, V, device="cuda")]
        s, ids, logits, lse, w, loss, st, grad = (ctypes.c_void_p(a.data_ptr()) for a in t)
        stream = torch.cuda.Stream()
        teacher = bd.dspark_teacher_t(ids, logits, lse, c["ids"].shape[1], None, 0)
        p = bd.dspark_distill_params_t(2, V, bd.DSPARK_FP32, V, V, 1.0, w, ctypes.c_void_p(stream.cuda_stream), st)
        calls.append((c, t, stream, (s, ctypes.byref(teacher), ctypes.byref(p), loss, None, grad)))
    torch.cuda.synchronize()
    failed, barrier = [], threading.Barrier(2)

    def work(args):
        barrier.wait()
        failed.append(sum(lib.dspark_distill(*args) != 0 for _ in range(20000)))

    threads = [threading.Thread(target=work, args=(a[3],)) for a in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for c, t, _, _ in calls:
        check_distill(c, (t[5].cpu().numpy(), t[7].double().cpu().numpy(), t[6].cpu().numpy()), "fp32")


@pytest.mark.parametrize("which", ["history", "bias", "both"])
def test_process_empty_lists(bd, which):
    """Lists without an entry in the whole batch (a first decoding step, no biases): offsets of zeros, columns
    of no elements."""
    B, K, V = 3, 2, 1003
    c = process_batch(np.random.default_rng(31), B, K, V, "fp32")
    if which in ("history", "both"):
        c["hist"] = [[]] * B
    if which in ("bias", "both"):
        c["bias"] = [[]] * B

    def columns(rows, *dtypes):
        full = R.csr(rows, *dtypes)
        return full if any(rows) else (full[0], *(a[:0] for a in full[1:]))

    x, out, status = R.on_gpu(c["x"], "fp32"), R.on_gpu(np.full(c["x"].shape, 77.0), "fp32"), R.i32(np.full(B, -1))
    bd.dspark_process_logits(
        x, torch.from_numpy(c["rows"].view(np.uint8).copy()).cuda(), out=out, row_status=status, draft_ids=R.i32(c["drafts"]),
        history=columns(c["hist"], np.int32, np.int32), bias=columns(c["bias"], np.int32, np.float32),
        mask=R.pack_mask(c["allowed"]), mask_rows=R.i32(c["mask_rows"]))
    check_process(c, out.double().cpu().numpy(), status.cpu().numpy(), "fp32", np.full(c["x"].shape, 77.0))


def test_process_mask_without_rows(bd):
    """No mask row at all: right where no position names one, an error of the request whose position does, and
    refused where every position has its own."""
    from sample_verify_epilogue_gb300 import binding as b_
    B, K, V = 3, 2, 1003
    c = process_batch(np.random.default_rng(32), B, K, V, "fp32", masks=False)
    c["rows"]["k"] = K
    x, rows = R.on_gpu(c["x"], "fp32"), torch.from_numpy(c["rows"].view(np.uint8).copy()).cuda()
    none = torch.empty(0, (V + 31) // 32, dtype=torch.int32, device="cuda")
    c["mask_rows"] = np.full((B, K + 1), -1)
    for bad in (False, True):
        out, status = R.on_gpu(np.full(c["x"].shape, 77.0), "fp32"), R.i32(np.full(B, -1))
        if bad:
            c["mask_rows"][0, 1] = 0
        bd.dspark_process_logits(
            x, rows, out=out, row_status=status, draft_ids=R.i32(c["drafts"]), history=R.csr(c["hist"], np.int32, np.int32),
            bias=R.csr(c["bias"], np.int32, np.float32), mask=none, mask_rows=R.i32(c["mask_rows"]))
        got, st = out.double().cpu().numpy(), status.cpu().numpy()
        assert np.array_equal(st, [b_.ROW_BAD_MASK if bad else 0, 0, 0])
        part = {k: v[int(bad):] for k, v in c.items() if k not in ("allowed", "mask_rows")}
        check_process(part | dict(allowed=None), got[int(bad):], st[int(bad):], "fp32", np.full(c["x"].shape, 77.0)[int(bad):])
    with pytest.raises(ValueError):
        bd.dspark_process_logits(x, rows, out=out, row_status=status, mask=none)


@pytest.mark.parametrize("short", ["history", "bias", "no_history", "no_bias"])
def test_process_offsets_past_the_lists(bd, short):
    """Offsets that pass their columns are an error of their request: nothing past the columns is read, and
    the requests before it are right."""
    from sample_verify_epilogue_gb300 import binding as b_
    B, K, V = 4, 2, 1003
    c = process_batch(np.random.default_rng(33), B, K, V, "fp32")
    c["hist"][B - 1] = c["bias"][B - 1] = [(3, 1.0), (5, 2.0), (900, 1.0)]
    hist, bias = R.csr(c["hist"], np.int32, np.int32), R.csr(c["bias"], np.int32, np.float32)

    def cut(lists, n):
        return (lists[0], *(a[:n].clone() for a in lists[1:]))

    n = 0 if short.startswith("no") else len(hist[1] if short == "history" else bias[1]) - 1
    if short in ("history", "no_history"):
        hist = cut(hist, n)
        want = np.where(hist[0].cpu().numpy()[1:] > n, b_.ROW_BAD_HISTORY, 0)
    else:
        bias = cut(bias, n)
        want = np.where(bias[0].cpu().numpy()[1:] > n, b_.ROW_BAD_BIAS, 0)
    x, out, status = R.on_gpu(c["x"], "fp32"), R.on_gpu(np.full(c["x"].shape, 77.0), "fp32"), R.i32(np.full(B, -1))
    bd.dspark_process_logits(
        x, torch.from_numpy(c["rows"].view(np.uint8).copy()).cuda(), out=out, row_status=status, draft_ids=R.i32(c["drafts"]),
        history=hist, bias=bias, mask=R.pack_mask(c["allowed"]), mask_rows=R.i32(c["mask_rows"]))
    got, st = out.double().cpu().numpy(), status.cpu().numpy()
    assert np.array_equal(st, want)
    for b in np.nonzero(want == 0)[0]:
        one = {k: v[b:b + 1] for k, v in c.items() if k != "allowed"} | dict(allowed=c["allowed"])
        check_process(one, got[b:b + 1], st[b:b + 1], "fp32", np.full((1, K + 1, V), 77.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [1, 3])
def test_rows_that_start_inside_a_vector(bd, shift, dtype):
    """Rows whose first and last vectors are ragged, streamed through buffers that are filled several times:
    what was stored there for a ragged vector never shows in a later piece."""
    rows, V, n = 200, 70001, 40
    rng = np.random.default_rng(shift)
    c = distill_batch(rng, rows, V, n, dtype, 1.0, True)
    c["s"][:, 0] = R.rounded(rng.normal(30, 3, rows), dtype)     # what a stale first or last vector would show most
    c["s"][:, V - 1] = R.rounded(rng.normal(40, 3, rows), dtype)
    live = set(range(0, rows, 9))
    c["w"][[r for r in range(rows) if r not in live]] = 0.0
    up = rng.uniform(0.5, 2, rows).astype(np.float32)
    for form in ("forward", "two_call"):
        check_distill(c, distill_call(bd, c, dtype, form, 3, shift, up=up), dtype, up=up)
    x = R.rounded(np.concatenate([c["s"][:24], c["s"][:24]], 1), dtype)
    for rows_ in (24, 3):
        check_top(x[:rows_], n, 1.0, top_call(bd, x[:rows_], dtype, n, 1.0, 3, shift))
    many = np.repeat(x[:8], 25, 0)                               # a CTA to a row
    check_top(many, n, 1.0, top_call(bd, many, dtype, n, 1.0, 3, shift))


def test_expired_waits(bd, monkeypatch):
    """A test build in which every wait for a copy counts as expired at once (the CTA still waits for what is in
    flight before it ends): rows that were to be read report DSPARK_ROW_INTERNAL and give no result, backward's
    included; rows that are not read are as ever, and so are the calls after it."""
    from sample_verify_epilogue_gb300 import binding as b_
    from sample_verify_epilogue_gb300.build import build_variant
    lib = b_.open_library(build_variant("expired_copies", ["-DDSPARK_TEST_EXPIRED_WAITS"], ["top_logits.cu", "distill.cu"]))
    expired = b_._Calls(lib)
    rng = np.random.default_rng(41)
    # a span in one piece, spans that stream, two CTAs and more to a row, ragged rows, both passes over long rows
    for rows, V, dtype, shift in ((6, 5003, "bf16", 1), (200, 30001, "fp32", 3), (5, 151936, "fp32", 0)):
        c = distill_batch(rng, rows, V, 20, dtype, 1.0, True)
        c["ids"][1, 1] = c["ids"][1, 0]                          # a bad record
        up = np.ones(rows, np.float32)
        read = np.ones(rows, bool)
        read[[1, 2, 3]] = False                                  # bad, empty, weight 0
        normal = distill_call(bd, c, dtype, "two_call", 1, shift, up=up)
        for form in ("forward", "fused"):
            with monkeypatch.context() as m:
                m.setattr(b_, "_calls_of", expired)
                loss, grad, st = distill_call(bd, c, dtype, form, 1, shift)
            assert (st[read] == b_.ROW_INTERNAL).all() and st[1] == b_.ROW_BAD_TEACHER and not st[2:4].any()
            assert np.isnan(loss[read]).all() and not loss[2:4].any()
            assert grad is None or not grad.any()
        # backward alone, from the sums of a good call
        s, ids, logits, w, lse = R.on_gpu(c["s"], dtype, 1, shift), R.i32(c["ids"]), R.f32(c["logits"]), R.f32(c["w"]), R.f32(c["lse"])
        loss, saved, status = torch.empty(rows, device="cuda"), torch.empty(rows, 4, device="cuda"), R.i32(np.full(rows, -1))
        bd.dspark_distill(s, ids, logits, loss=loss, saved=saved, row_status=status, weights=w, teacher_lse=lse)
        grad = R.on_gpu(np.full(c["s"].shape, 9.0), dtype, 1, shift)
        before = status.cpu().numpy()
        with monkeypatch.context() as m:
            m.setattr(b_, "_calls_of", expired)
            bd.dspark_distill_backward(s, ids, logits, saved=saved, grad=grad, row_status=status, weights=w, teacher_lse=lse)
        assert np.array_equal(status.cpu().numpy(), np.where(read, b_.ROW_INTERNAL, before))
        assert not grad.any()
        # records
        n = 30
        v, i, st = torch.zeros(rows, n, device="cuda"), R.i32(np.zeros((rows, n))), R.i32(np.full(rows, -1))
        lse = torch.zeros(rows, device="cuda")
        with monkeypatch.context() as m:
            m.setattr(b_, "_calls_of", expired)
            bd.dspark_top_logits(s, values=v, ids=i, lse=lse, row_status=st)
        assert (st == b_.ROW_INTERNAL).all() and torch.isneginf(v).all() and (i == -1).all() and torch.isnan(lse).all()
        check_top(c["s"], n, 1.0, top_call(bd, c["s"], dtype, n, 1.0, 1, shift))
        again = distill_call(bd, c, dtype, "two_call", 1, shift, up=up)
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(normal, again))
        check_distill(c, again, dtype, bad=(1,))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,K,V", [(3, 9, 2003), (2, 33, 901), (5, 64, 260)])
def test_process_long_prefixes(bd, B, K, V, dtype):
    """Many drafts before a position, among them repeats and tokens of the lists."""
    c = process_batch(np.random.default_rng(K), B, K, V, dtype, history=120, bias=30)
    got, status = process_call(bd, c, dtype, 1, 3)
    check_process(c, got, status, dtype, np.full(c["x"].shape, 77.0))


def test_explicit_streams(bd):
    """Calls on a stream that is not the current one: what the other stream holds before them comes before them."""
    side = torch.cuda.Stream()
    on = side.cuda_stream
    rng = np.random.default_rng(51)
    c = process_batch(rng, 3, 2, 30001, "fp32")
    x, out, late = R.on_gpu(c["x"], "fp32"), R.on_gpu(np.full(c["x"].shape, 77.0), "fp32"), R.on_gpu(np.zeros(c["x"].shape), "fp32")
    status, rows = R.i32(np.full(3, -1)), torch.from_numpy(c["rows"].view(np.uint8).copy()).cuda()
    given = dict(draft_ids=R.i32(c["drafts"]), history=R.csr(c["hist"], np.int32, np.int32), bias=R.csr(c["bias"], np.int32, np.float32),
                 mask=R.pack_mask(c["allowed"]), mask_rows=R.i32(c["mask_rows"]))
    d = distill_batch(rng, 6, 30001, 20, "fp32", 1.0, True)
    s, ids, logits, lse, w = R.f32(d["s"]), R.i32(d["ids"]), R.f32(d["logits"]), R.f32(d["lse"]), R.f32(d["w"])
    student, loss, st = torch.zeros_like(s), torch.full((6,), 5.0, device="cuda"), R.i32(np.full(6, -1))
    saved, grad, up = torch.zeros(6, 4, device="cuda"), torch.zeros_like(s), torch.ones(6, device="cuda")
    n = 20
    v, i, tl, ts = torch.zeros(6, n, device="cuda"), R.i32(np.zeros((6, n))), torch.zeros(6, device="cuda"), R.i32(np.full(6, -1))
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = torch.tanh(busy @ busy)                       # some time before the inputs are there
        late.copy_(x)
        student.copy_(s)
    bd.dspark_process_logits(late, rows, out=out, row_status=status, stream=on, **given)
    bd.dspark_top_logits(student, values=v, ids=i, lse=tl, row_status=ts, stream=on)
    bd.dspark_distill(student, ids, logits, loss=loss, saved=saved, row_status=st, teacher_lse=lse, weights=w, stream=on)
    bd.dspark_distill_backward(student, ids, logits, saved=saved, grad=grad, grad_loss=up, teacher_lse=lse, weights=w, stream=on)
    side.synchronize()
    check_process(c, out.double().cpu().numpy(), status.cpu().numpy(), "fp32", np.full(c["x"].shape, 77.0))
    check_distill(d, (loss.cpu().numpy(), grad.double().cpu().numpy(), st.cpu().numpy()), "fp32")
    check_top(d["s"], n, 1.0, [a.cpu().numpy() for a in (v, i, tl, ts)])


def test_distill_loss_in_a_graph(bd):
    """A training step's loss and its gradient captured together and replayed on new inputs."""
    from sample_verify_epilogue_gb300.distill import distill_loss
    rng = np.random.default_rng(52)
    batches = [distill_batch(rng, 5, 4001, 16, "fp32", 1.0, True) for _ in range(3)]
    student = torch.zeros(5, 4001, device="cuda", requires_grad=True)
    ids, logits, lse, w = (torch.zeros_like(a) for a in (R.i32(batches[0]["ids"]), R.f32(batches[0]["logits"]),
                                                         R.f32(batches[0]["lse"]), R.f32(batches[0]["w"])))

    def load(c):
        with torch.no_grad():
            for a, b in ((student, R.f32(c["s"])), (ids, R.i32(c["ids"])), (logits, R.f32(c["logits"])), (lse, R.f32(c["lse"])),
                         (w, R.f32(c["w"]))):
                a.copy_(b)

    def step():
        loss, status = distill_loss(student, ids, logits, lse, weights=w)
        grad, = torch.autograd.grad(loss.sum(), student)
        return loss.detach(), grad, status

    load(batches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad, status = step()
    for c in batches:
        load(c)
        graph.replay()
        check_distill(c, (loss.cpu().numpy(), grad.double().cpu().numpy(), status.cpu().numpy()), "fp32")
