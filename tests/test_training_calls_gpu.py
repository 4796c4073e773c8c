"""Calls that a trainer makes of the token losses beside the plain ones: through autograd, captured, on other streams, from two
threads, over more rows than 32 bits count elements of, and after a verify call, whose log-probabilities they take."""
import ctypes
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import training as O  # noqa: E402
from tests import _rows as R  # noqa: E402
from tests import _training as T_  # noqa: E402
from tests.test_rows_gpu import bd  # noqa: E402,F401
from tests.test_training_gpu import (  # noqa: E402
    HIGH, LOW, check_logprobs, check_policy, check_preference, full, logprobs_call, policy_batch, policy_call, preference_batch,
    preference_call)

OPTIONS = dict(clip_low=LOW, clip_high=HIGH, kl_coef=0.1, entropy_coef=0.01)


def host(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_of_token_logprobs(bd, dtype):  # noqa: F811
    """Both results, either alone, and neither; upstream gradients that are expanded scalars."""
    from sample_verify_epilogue_gb300.training import token_logprobs
    rng = np.random.default_rng(1)
    x, y = T_.token_rows(rng, 10, 1003, dtype)
    up = rng.normal(0, 1, (2, 10)).astype(np.float32)
    for use in ("both", "logprobs", "entropy", "sums"):
        logits = R.on_gpu(x, dtype).requires_grad_()
        lp, H, st = token_logprobs(logits, R.i32(y), temperature=0.9)
        assert lp.requires_grad and H.requires_grad and not st.requires_grad
        ups = [up[0], up[1]]
        if use == "both":
            ((lp * R.f32(up[0])).sum() + (H * R.f32(up[1])).sum()).backward()
        elif use == "logprobs":
            (lp * R.f32(up[0])).sum().backward()
            ups[1] = None
        elif use == "entropy":
            (H * R.f32(up[1])).sum().backward()
            ups[0] = None
        else:
            (lp.sum() - 2 * H.sum()).backward()
            ups = [np.ones(10, np.float32), np.full(10, -2, np.float32)]
        got = lp.detach().cpu().numpy(), H.detach().cpu().numpy(), st.cpu().numpy(), host(logits.grad)
        # a masked token's -inf times its upstream gradient is the loss's business; the gradient is finite
        check_logprobs(x, y, dtype, float(np.float32(0.9)), got, ups)
    with torch.no_grad():
        lp, H, st = token_logprobs(R.on_gpu(x, dtype), R.i32(y))
    assert not lp.requires_grad


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_of_the_losses(bd, dtype):  # noqa: F811
    from sample_verify_epilogue_gb300.training import policy_loss, preference_loss
    rng = np.random.default_rng(2)
    c = policy_batch(rng, 9, 1003, dtype, 1.0, special=False)
    up = rng.uniform(0.5, 2, 9).astype(np.float32)
    logits = R.on_gpu(c["x"], dtype).view(3, 3, 1003).requires_grad_()
    loss, lp, st = policy_loss(logits, *(a.view(3, 3) for a in (R.i32(c["y"]), R.f32(c["old"]), R.f32(c["adv"]))),
                               ref_logprobs=R.f32(c["ref"]).view(3, 3), weights=R.f32(c["w"]).view(3, 3), **OPTIONS)
    assert loss.shape == (3, 3) and not lp.requires_grad
    (loss * R.f32(up).view(3, 3)).sum().backward()
    want = policy_call(bd, c, dtype, 1.0, 0.1, 0.01, "two_call", up=up)
    assert np.array_equal(want["loss"], loss.detach().view(-1).cpu().numpy())
    assert np.array_equal(want["grad"], host(logits.grad).reshape(9, -1))
    check_policy(c, want, dtype, 1.0, 0.1, 0.01, up=up)

    c = preference_batch(rng, (4, 3, 5, 1), 1003, dtype)
    logits = R.on_gpu(c["x"], dtype).requires_grad_()
    loss, rewards, st = preference_loss(logits, R.i32(c["y"]), R.i32(c["off"]), ref_logprobs=R.f32(c["ref"]),
                                        weights=R.f32(c["w"]), beta=0.2, margin=0.1, label_smoothing=0.1, mean=True)
    loss.mean().backward()
    how = dict(beta=0.2, margin=0.1, smoothing=0.1, mean=True)
    want = preference_call(bd, c, dtype, "two_call", up=np.full(2, 0.5), **how)
    assert np.array_equal(want["loss"], loss.detach().cpu().numpy()) and np.array_equal(want["rewards"], rewards.cpu().numpy())
    assert np.array_equal(want["grad"], host(logits.grad))
    check_preference(c, want, dtype, up=np.full(2, 0.5), **how)


def test_gradients_by_differences(bd):  # noqa: F811
    """The losses' own values at logits moved by h against their gradients: the difference quotient is off by the third
    derivative's h^2 / 6 (bounded by 8 times the largest factor here), and two losses' roundings over 2h."""
    rng = np.random.default_rng(3)
    V, h = 37, 0.02
    c = policy_batch(rng, 6, V, "fp32", 1.0, special=False)
    c["w"][:] = 1.0
    got = policy_call(bd, c, "fp32", 1.0, 0.1, 0.01, "fused")
    p = preference_batch(rng, (3, 3), V, "fp32", tail=0)
    p["y"][:] = rng.integers(0, V, 6)
    pref = preference_call(bd, p, "fp32", "fused")
    for v in range(0, V, 5):
        for r in range(6):
            e = np.zeros((6, V))
            e[r, v] = h
            up, down = (policy_call(bd, c | dict(x=c["x"] + s * e), "fp32", 1.0, 0.1, 0.01, "forward") for s in (1, -1))
            lo, hi = np.exp(c["old"][r] + np.log(1 - LOW)), np.exp(c["old"][r] + np.log(1 + HIGH))
            near = [np.exp(q["logprobs"][r]) for q in (up, down)]
            if (min(near) < lo < max(near)) or (min(near) < hi < max(near)):
                continue                                     # clipping begins between the two
            size = 1 + abs(c["adv"][r]) * np.exp(got["logprobs"][r] - c["old"][r]) * 1.1
            tol = 8 * size * h * h / 6 + 2e-6 * size / h
            assert abs((up["loss"][r] - down["loss"][r]) / (2 * h) - got["grad"][r, v]) < tol, (r, v)
            up, down = (preference_call(bd, p | dict(x=p["x"] + s * e), "fp32", "forward") for s in (1, -1))
            assert abs((up["loss"][0] - down["loss"][0]) / (2 * h) - pref["grad"][r, v]) < 8 * h * h / 6 + 2e-6 / h, (r, v)


def test_captured_steps(bd):  # noqa: F811
    """Loss and gradient of each kind captured together, and replayed on new inputs; two graphs alive at once."""
    from sample_verify_epilogue_gb300.training import policy_loss, preference_loss, token_logprobs
    rng = np.random.default_rng(4)
    V, rows = 4001, 10
    batches = [(policy_batch(rng, rows, V, "fp32", 1.0, special=False), preference_batch(rng, (2, 3, 1, 2), V, "fp32")) for _ in range(3)]
    names = ("x", "y", "old", "ref", "adv", "w")
    c0, p0 = batches[0]
    up = R.f32(rng.normal(0, 1, (2, rows)))

    def tensors(c, keys):
        return {k: (R.i32 if k in ("y", "off") else R.f32)(c[k]) for k in keys}

    pol, prf = tensors(c0, names), tensors(p0, ("x", "y", "off", "ref", "w"))
    pol["x"].requires_grad_()
    prf["x"].requires_grad_()

    def load(c, p):
        with torch.no_grad():
            for held, new in ((pol, tensors(c, names)), (prf, tensors(p, ("x", "y", "off", "ref", "w")))):
                for k in held:
                    held[k].copy_(new[k])

    def first():
        lp, H, st = token_logprobs(pol["x"], pol["y"])
        grad, = torch.autograd.grad((lp * up[0]).sum() + (H * up[1]).sum(), pol["x"])
        return lp.detach(), H.detach(), st, grad

    def second():
        loss, _, st = policy_loss(pol["x"], pol["y"], pol["old"], pol["adv"], ref_logprobs=pol["ref"], weights=pol["w"], **OPTIONS)
        grad, = torch.autograd.grad(loss.sum(), pol["x"])
        loss2, rewards, pst = preference_loss(prf["x"], prf["y"], prf["off"], ref_logprobs=prf["ref"], weights=prf["w"])
        grad2, = torch.autograd.grad(loss2.sum(), prf["x"])
        return loss.detach(), st, grad, loss2.detach(), rewards, pst, grad2

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first()
        second()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for step in (first, second):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for c, p in batches:
        load(c, p)
        for graph, _ in graphs:
            graph.replay()
        lp, H, st, grad = graphs[0][1]
        check_logprobs(c["x"], c["y"], "fp32", 1.0, (lp.cpu().numpy(), H.cpu().numpy(), st.cpu().numpy(), host(grad)), host(up))
        loss, st, grad, loss2, rewards, pst, grad2 = graphs[1][1]
        want = policy_call(bd, c, "fp32", 1.0, 0.1, 0.01, "two_call")
        assert np.array_equal(want["loss"], loss.cpu().numpy()) and np.array_equal(want["grad"], host(grad))
        check_policy(c, want, "fp32", 1.0, 0.1, 0.01)
        want = preference_call(bd, p, "fp32", "two_call")
        assert np.array_equal(want["loss"], loss2.cpu().numpy()) and np.array_equal(want["rewards"], rewards.cpu().numpy())
        assert np.array_equal(want["grad"], host(grad2)) and not pst.any()


def test_explicit_streams(bd):  # noqa: F811
    """Calls on a stream that is not the current one: what the other stream holds before them comes before them."""
    side = torch.cuda.Stream()
    on = side.cuda_stream
    rng = np.random.default_rng(5)
    c, p = policy_batch(rng, 8, 30001, "fp32", 1.0, special=False), preference_batch(rng, (3, 4), 30001, "fp32")
    x, late = R.f32(c["x"]), torch.zeros(8, 30001, device="cuda")
    px, plate = R.f32(p["x"]), torch.zeros(p["x"].shape, device="cuda")
    y, old, adv, ref, w = R.i32(c["y"]), R.f32(c["old"]), R.f32(c["adv"]), R.f32(c["ref"]), R.f32(c["w"])
    py, off, pref, pw = R.i32(p["y"]), R.i32(p["off"]), R.f32(p["ref"]), R.f32(p["w"])
    rows = len(p["x"])
    loss, lp, ent, kl, st = full(8, 9.0), full(8, 9.0), full(8, 9.0), full(8, 9.0), full(8, -1, torch.int32)
    saved, grad = torch.zeros(8, 8, device="cuda"), torch.zeros_like(late)
    lp2, H2, saved2, grad2, st2 = full(8, 9.0), full(8, 9.0), torch.zeros(8, 8, device="cuda"), torch.zeros_like(late), full(8, -1, torch.int32)
    ploss, prew, pst, plp, prs = full(1, 9.0), torch.zeros(1, 2, device="cuda"), full(1, -1, torch.int32), full(rows, 9.0), full(rows, -1, torch.int32)
    psaved, pgrad, one = torch.zeros(rows, 8, device="cuda"), torch.zeros_like(plate), torch.ones(8, device="cuda")
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = torch.tanh(busy @ busy)                   # some time before the inputs are there
        late.copy_(x)
        plate.copy_(px)
    bd.dspark_policy_loss(late, y, old, adv, loss=loss, row_status=st, logprobs=lp, entropy=ent, kl=kl, saved=saved, grad=grad,
                          ref_logprobs=ref, weights=w, stream=on, **OPTIONS)
    bd.dspark_token_logprobs(late, y, logprobs=lp2, entropy=H2, row_status=st2, saved=saved2, stream=on)
    bd.dspark_token_logprobs_backward(late, y, saved=saved2, grad=grad2, grad_logprobs=one, grad_entropy=one, stream=on)
    bd.dspark_preference_loss(plate, py, off, loss=ploss, saved=psaved, row_status=prs, pair_status=pst, rewards=prew, logprobs=plp,
                              ref_logprobs=pref, weights=pw, stream=on)
    bd.dspark_preference_loss_backward(plate, py, saved=psaved, grad=pgrad, grad_loss=one[:1], stream=on)
    side.synchronize()
    check_policy(c, dict(loss=loss.cpu().numpy(), logprobs=lp.cpu().numpy(), entropy=ent.cpu().numpy(), kl=kl.cpu().numpy(),
                         status=st.cpu().numpy(), grad=host(grad)), "fp32", 1.0, 0.1, 0.01)
    check_logprobs(c["x"], c["y"], "fp32", 1.0, (lp2.cpu().numpy(), H2.cpu().numpy(), st2.cpu().numpy(), host(grad2)), np.ones((2, 8)))
    check_preference(p, dict(loss=ploss.cpu().numpy(), rewards=prew.cpu().numpy(), pair_status=pst.cpu().numpy(),
                             logprobs=plp.cpu().numpy(), status=prs.cpu().numpy(), grad=host(pgrad)), "fp32")


def test_calls_from_two_threads(bd):  # noqa: F811
    """Policy losses with gradients of rows of two lengths from two host threads at once, whose CTAs keep spans of 36 and of
    72 KB: a launch needs its own limit whatever the other thread does at the time."""
    lib, calls = bd.load_library(), []
    for V in (72000, 144000):
        c = policy_batch(np.random.default_rng(V), 2, V, "fp32", 1.0, special=False)
        t = [R.f32(c["x"]), R.i32(c["y"]), R.f32(c["old"]), R.f32(c["ref"]), R.f32(c["adv"]), R.f32(c["w"]), full(2, 9.0), full(2, 9.0),
             full(2, 9.0), full(2, 9.0), torch.zeros(2, 8, device="cuda"), torch.zeros(2, V, device="cuda"), full(2, -1, torch.int32)]
        x, y, old, ref, adv, w, loss, lp, ent, kl, saved, grad, st = (ctypes.c_void_p(a.data_ptr()) for a in t)
        stream = torch.cuda.Stream()
        o = bd.dspark_policy_t(old, ref, adv, w, LOW, HIGH, 0.1, 0.01)
        p = bd.dspark_token_params_t(2, V, bd.DSPARK_FP32, V, V, 1.0, y, ctypes.c_void_p(stream.cuda_stream), st)
        calls.append((c, t, (x, ctypes.byref(o), ctypes.byref(p), loss, lp, ent, kl, saved, grad), stream))
    torch.cuda.synchronize()
    failed, barrier = [], threading.Barrier(2)

    def work(args):
        barrier.wait()
        failed.append(sum(lib.dspark_policy_loss(*args) != 0 for _ in range(10000)))

    threads = [threading.Thread(target=work, args=(a[2],)) for a in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for c, t, _, _ in calls:
        check_policy(c, dict(loss=t[6].cpu().numpy(), logprobs=t[7].cpu().numpy(), entropy=t[8].cpu().numpy(), kl=t[9].cpu().numpy(),
                             status=t[12].cpu().numpy(), grad=host(t[11])), "fp32", 1.0, 0.1, 0.01)


@pytest.mark.parametrize("dtype,V", [("bf16", 294912), ("bf16", 300001), ("fp32", 150001), ("bf16", 896000), ("bf16", 900001),
                                     ("fp32", 448000), ("fp32", 450001)])
def test_rows_around_the_longest_kept_ones(bd, dtype, V):  # noqa: F811
    """Rows that eight spans just hold, and rows that they do not, which are read twice; also unaligned."""
    rng = np.random.default_rng(V)
    c = policy_batch(rng, 6, V, dtype, 1.0, special=False)
    for pad, shift in ((0, 0), (3, 1)):
        check_policy(c, policy_call(bd, c, dtype, 1.0, 0.1, 0.01, "fused", pad=pad, shift=shift), dtype, 1.0, 0.1, 0.01)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-np.inf, "lowest"])
def test_rows_that_begin_with_a_mask(bd, value, dtype):  # noqa: F811
    """The first tens of thousands of tokens masked, then some; logits that rise along the row: references that are set late
    and raised often."""
    rng = np.random.default_rng(6)
    V, rows = 90001, 6
    x, y = T_.token_rows(rng, rows, V, dtype, special=False)
    lowest = R.rounded(-3.38e38, dtype)
    x[:3, :60000] = -np.inf if value == -np.inf else lowest
    x[3] = np.linspace(-400, 400, V) + rng.normal(0, 1, V)
    x[4] = np.linspace(0, 3000, V)
    x[5, 1:] = -np.inf if value == -np.inf else lowest
    y[:6] = [70000, 5, 89999, V - 1, V // 2, 0]
    x[0, 70000] = 2.0
    x = R.rounded(x, dtype)
    up = rng.normal(0, 1, (2, rows))
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, up=up), up)
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, entropy=False, up=(up[0], None)), (up[0], None))
    lp = np.array([O.token_row(x[r], y[r], 1.0)["logp"][y[r]] for r in range(rows)])
    lp = np.where(np.isfinite(lp) & (lp > -80), lp, -5.0)
    c = dict(x=x, y=y, old=lp.astype(np.float32), ref=lp.astype(np.float32), adv=rng.normal(0, 1, rows).astype(np.float32), w=None)
    for form in ("fused", "two_call"):
        for ent in (0.0, 0.05):
            check_policy(c, policy_call(bd, c, dtype, 1.0, 0.0, ent, form, use_ref=False), dtype, 1.0, 0.0, ent, use_ref=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [300.0, 3e4, 1e6, 1e8, 1e30])
def test_large_logits(bd, size, dtype):  # noqa: F811
    """Logits whose neighbours in the type are far apart: a few of them have all the mass, or one; at exponents around and
    past four million, where no whole one is taken, too."""
    rng = np.random.default_rng(int(np.log10(size)))
    rows, V = 8, 5003
    x = R.rounded(size * (1 + rng.uniform(-0.01, 0.01, (rows, V))) * rng.choice([-1, 1], rows)[:, None], dtype)
    x[4:, ::7] = x[4:].max(1, keepdims=True)                 # many ties for the largest
    y = rng.integers(0, V, rows)
    y[5] = 7
    y[6:] = np.argmax(x[6:], 1)
    up = rng.normal(0, 1, (2, rows))
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, up=up), up)
    check_logprobs(x, y, dtype, 1.0, logprobs_call(bd, x, y, dtype, entropy=False, up=(up[0], None)), (up[0], None))


@pytest.mark.parametrize("T", [1e-3, 0.05, 30.0, 1e4])
def test_temperatures(bd, T):  # noqa: F811
    rng = np.random.default_rng(7)
    for dtype in ("bf16", "fp32"):
        x, y = T_.token_rows(rng, 9, 5003, dtype)
        up = rng.normal(0, 1, (2, 9))
        t = float(np.float32(T))
        check_logprobs(x, y, dtype, t, logprobs_call(bd, x, y, dtype, T, up=up), up)


def test_more_elements_than_32_bits_count(bd):  # noqa: F811
    """The last rows of 6 GB of logits, the others without a token: results, gradient, and the rows before left at 0."""
    rng = np.random.default_rng(8)
    rows, V, n = 20000, 151936, 6
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("memory")
    logits = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    c = policy_batch(rng, n, V, "bf16", 1.0, special=False)
    logits[-n:] = R.on_gpu(c["x"], "bf16")
    tokens, old, adv, ref, w = (torch.zeros(rows, dtype=t, device="cuda") for t in (torch.int32,) + (torch.float32,) * 4)
    tokens[:] = -1
    for t, k in ((tokens, "y"), (old, "old"), (adv, "adv"), (ref, "ref"), (w, "w")):
        t[-n:] = torch.from_numpy(np.asarray(c[k])).to(t.dtype).cuda()
    out = {k: full(rows, 9.0) for k in ("loss", "logprobs", "entropy", "kl")}
    st, saved, grad = full(rows, -1, torch.int32), torch.empty(rows, 8, device="cuda"), torch.full_like(logits, 5.0)
    given = dict(ref_logprobs=ref, weights=w, **OPTIONS)
    for form in ("fused", "two_call"):
        grad.fill_(5.0)
        bd.dspark_policy_loss(logits, tokens, old, adv, row_status=st, saved=saved, grad=grad if form == "fused" else None, **out, **given)
        if form == "two_call":
            bd.dspark_policy_loss_backward(logits, tokens, old, adv, saved=saved, grad=grad, **given)
        got = {k: v[-n:].cpu().numpy() for k, v in out.items()} | dict(status=st[-n:].cpu().numpy(), grad=host(grad[-n:]))
        check_policy(c, got, "bf16", 1.0, 0.1, 0.01)
        assert not out["loss"][:-n].any() and not st.any() and all(not grad[k:k + 2000].any() for k in range(0, rows - n - 2000, 2000))


def test_expired_waits(bd, monkeypatch):  # noqa: F811
    """A test build in which every wait for a copy counts as expired at once (the CTA still waits for what is in flight before
    it ends): the rows that were to be read report DSPARK_ROW_INTERNAL, give a NaN loss and a gradient of 0; rows that are
    not read are as ever, and so are the calls after it."""
    from sample_verify_epilogue_gb300 import binding as b_
    from sample_verify_epilogue_gb300.build import build_variant
    lib = b_.open_library(build_variant("expired_token_copies", ["-DDSPARK_TEST_EXPIRED_WAITS"], ["token_rows.cu"]))
    expired = b_._Calls(lib)
    rng = np.random.default_rng(9)
    for rows, V, dtype, shift in ((7, 5003, "bf16", 1), (200, 30001, "fp32", 3), (5, 140001, "fp32", 0)):
        c = policy_batch(rng, rows, V, dtype, 1.0, special=False)
        c["y"][1], c["y"][3] = -1, V
        with monkeypatch.context() as m:
            m.setattr(b_, "_calls_of", expired)
            got = policy_call(bd, c, dtype, 1.0, 0.1, 0.01, "fused", pad=1, shift=shift)
        read = np.ones(rows, bool)
        read[[1, 2, 3]] = False                              # no token, weight 0, out of range
        assert (got["status"][read] == b_.ROW_INTERNAL).all() and np.isnan(got["loss"][read]).all() and not got["grad"].any()
        assert got["status"][1] == 0 and got["status"][2] == 0 and got["status"][3] == b_.ROW_BAD_TOKEN
        good = policy_call(bd, c, dtype, 1.0, 0.1, 0.01, "fused", pad=1, shift=shift)
        check_policy(c, good, dtype, 1.0, 0.1, 0.01, bad={3: b_.ROW_BAD_TOKEN})


def test_chain_after_a_verify_call(bd):  # noqa: F811
    """A rollout's step: the verify call's tokens and raw log-probabilities go into the policy loss on the same logits, where
    every ratio is 1; the gradients of all positions are then clipped together."""
    from sample_verify_epilogue_gb300.runner import EpilogueCall
    from workloads.generate import make_batch, row_params
    B, K, V = 5, 3, 5001
    batch = make_batch(B=B, K_max=K, V=V, logits_dtype="fp32", rows=[row_params(1.0, 0, 1.0, 0.0, 0.0, K)] * B, seed=4, philox_seed=4,
                       history_len=0, want_logprobs=True)
    call = EpilogueCall(batch)
    call.run()
    tokens, old = call.out["tokens"], call.out["logprobs"]
    live = tokens >= 0
    assert int(live.sum()) >= B
    g = torch.Generator(device="cuda").manual_seed(1)
    adv = torch.randn(B, K + 1, generator=g, device="cuda")
    loss, lp, st = full(B * (K + 1), 9.0), full(B * (K + 1), 9.0), full(B * (K + 1), -1, torch.int32)
    saved, grad = torch.empty(B * (K + 1), 8, device="cuda"), torch.empty_like(call.x)
    bd.dspark_policy_loss(call.x, tokens, old, adv, loss=loss, row_status=st, logprobs=lp, saved=saved, grad=grad)
    assert not st.any()
    x, t = call.x.double().cpu().numpy(), tokens.cpu().numpy()
    for b in range(B):
        for j in range(K + 1):
            r = b * (K + 1) + j
            if t[b, j] < 0:
                assert float(loss[r]) == 0 and not grad[b, j].any()
                continue
            row = O.token_row(x[b, j], t[b, j], 1.0)
            # the verify call's log-probabilities are within 1e-4, so is the ratio from 1
            assert abs(float(lp[r]) - row["logp"][t[b, j]]) < 1e-5
            assert abs(float(loss[r]) + float(adv[b, j])) < 2e-4 * abs(float(adv[b, j])) + 1e-6
            want = O.token_grad(row, -float(adv[b, j]), 0.0, 1.0)
            assert np.abs(host(grad[b, j]) - want).max() < 3e-4 * abs(float(adv[b, j])) + 1e-7
    held = host(grad)
    table = bd.GradTable(list(grad.view(B * (K + 1), V).unbind()))
    norm, status = full(1, 0.0), full(1, -1, torch.int32)
    ws = torch.empty(bd.dspark_clip_workspace_bytes(table), dtype=torch.uint8, device="cuda")
    bd.dspark_clip_grads(table, 0.5, norm=norm, status=status, workspace=ws)
    want, scaled = O.clip([held], 0.5)
    assert want > 0.5 and abs(float(norm) - want) < 1e-5 * want and int(status) == 0
    assert np.abs(host(grad) - scaled[0]).max() < 1e-6


def test_results_come_again(bd):  # noqa: F811
    """The same call gives the same bits, whatever else the GPU does."""
    rng = np.random.default_rng(10)
    c = policy_batch(rng, 40, 32003, "bf16", 1.0, special=False)
    p = preference_batch(rng, (9, 7, 4, 6), 32003, "bf16")
    first = policy_call(bd, c, "bf16", 1.0, 0.1, 0.01, "fused"), preference_call(bd, p, "bf16", "fused")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(30):
            busy = torch.tanh(busy @ busy)
    for _ in range(3):
        again = policy_call(bd, c, "bf16", 1.0, 0.1, 0.01, "fused"), preference_call(bd, p, "bf16", "fused")
        for a, b in zip(first, again):
            assert all(np.array_equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tokens_that_change_before_the_backward_call(bd, dtype):  # noqa: F811
    """A backward call whose tokens are out of range by then writes nothing beside its rows."""
    V, kind = 1003, torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(6, V, generator=g, device="cuda").to(kind)
    tokens = torch.tensor([5, 1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    saved, ones = torch.empty(6, 8, device="cuda"), full(6, 1.0)
    bd.dspark_token_logprobs(x, tokens, logprobs=full(6, 9.0), entropy=full(6, 9.0), row_status=full(6, -1, torch.int32), saved=saved)
    late = torch.tensor([5, V, -1, V + 3, -7, 5], dtype=torch.int32, device="cuda")

    def run(t):
        held = torch.full((8, V + 9), 77.0, dtype=kind, device="cuda")
        grad = held[1:7, 3:3 + V]                            # another alignment than the logits'
        bd.dspark_token_logprobs_backward(x, t, saved=saved, grad=grad, grad_logprobs=ones, grad_entropy=ones)
        rest = held.clone()
        rest[1:7, 3:3 + V] = 77.0
        assert bool((rest == 77.0).all())
        return grad

    first, then = run(tokens), run(late)
    assert torch.equal(first[0], then[0]) and torch.equal(first[5], then[5]) and bool(torch.isfinite(then).all())
