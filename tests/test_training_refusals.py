"""What the calls that train on decoded tokens refuse, before any CUDA call (CPU only), and their oracle."""
import ctypes

import numpy as np
import pytest

from tests.test_rows_refusals import bd, vp  # noqa: F401


def token_params(bd, kw):  # noqa: F811
    given = dict(n_rows=2, V=10, logits_dtype=0, logits_stride=10, grad_stride=10, temperature=1.0, tokens=64, row_status=512)
    return bd.dspark_token_params_t(**(given | kw))


BAD_ROWS = [dict(n_rows=0), dict(n_rows=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(logits_dtype=3), dict(logits_stride=9),
            dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
            dict(temperature=1e-45), dict(tokens=None), dict(logits=None), dict(logits=4097)]
BAD_FORWARD = BAD_ROWS + [dict(row_status=None)]
BAD_GRAD = [dict(grad=8193), dict(grad_stride=9), dict(grad=4096, grad_stride=12)]


def call(bd, what, kw):  # noqa: F811
    """The status of one of the calls with ``kw`` in place of good arguments (device addresses that are never read)."""
    kw = dict(kw)
    lib = bd.load_library()
    logits, grad, saved = kw.pop("logits", 4096), kw.pop("grad", 8192), kw.pop("saved", 64)
    outs = {k: kw.pop(k) for k in ("out", "up", "up2", "pair_status", "n_pairs", "kl") if k in kw}
    policy = dict(old_logprobs=64, ref_logprobs=64, advantages=64, weights=None, clip_low=0.2, clip_high=0.2, kl_coef=0.1,
                  entropy_coef=0.0)
    policy |= {k: kw.pop(k) for k in list(kw) if k in policy}
    pref = dict(n_pairs=outs.get("n_pairs", 2), row_offsets=64, ref_logprobs=None, weights=None, beta=0.1, margin=0.0,
                label_smoothing=0.0, mean=0)
    pref |= {k: kw.pop(k) for k in list(kw) if k in pref}
    p = ctypes.byref(token_params(bd, kw))
    o, f = ctypes.byref(bd.dspark_policy_t(**policy)), ctypes.byref(bd.dspark_preference_t(**pref))
    out = vp(outs.get("out", 64))
    if what == "logprobs":
        return lib.dspark_token_logprobs(vp(logits), p, out, None, vp(saved))
    if what == "logprobs_backward":
        return lib.dspark_token_logprobs_backward(vp(logits), p, vp(saved), vp(outs.get("up", 64)), vp(outs.get("up2", 64)), vp(grad))
    if what == "policy":
        return lib.dspark_policy_loss(vp(logits), o, p, out, None, None, vp(outs.get("kl")), vp(saved), vp(grad))
    if what == "policy_backward":
        return lib.dspark_policy_loss_backward(vp(logits), o, p, vp(saved), None, vp(grad))
    if what == "preference":
        return lib.dspark_preference_loss(vp(logits), f, p, out, None, vp(outs.get("pair_status", 64)), None, vp(saved), vp(grad))
    return lib.dspark_preference_loss_backward(vp(logits), p, outs.get("n_pairs", 2), vp(saved), vp(64), vp(grad))


@pytest.mark.parametrize("what,kw", [(w, kw) for w in ("logprobs", "policy", "preference") for kw in BAD_FORWARD] +
                         [(w, kw) for w in ("logprobs_backward", "policy_backward", "preference_backward") for kw in BAD_ROWS] +
                         [(w, kw) for w in ("logprobs_backward", "policy", "policy_backward", "preference", "preference_backward")
                          for kw in BAD_GRAD])
def test_rows_are_refused(bd, what, kw):  # noqa: F811
    assert call(bd, what, kw) == 1


@pytest.mark.parametrize("what,kw", [
    ("logprobs", dict(out=None)), ("logprobs", dict(saved=68)), ("logprobs_backward", dict(saved=None)),
    ("logprobs_backward", dict(saved=72)), ("logprobs_backward", dict(grad=None)), ("logprobs_backward", dict(up=None, up2=None)),
    ("policy", dict(out=None)), ("policy", dict(saved=None)), ("policy", dict(saved=65)), ("policy", dict(old_logprobs=None)),
    ("policy", dict(advantages=None)), ("policy", dict(ref_logprobs=None)), ("policy", dict(ref_logprobs=None, kl_coef=0.0, kl=64)),
    ("policy", dict(clip_low=-0.1)), ("policy", dict(clip_low=1.5)), ("policy", dict(clip_low=float("nan"))),
    ("policy", dict(clip_high=-1.0)), ("policy", dict(clip_high=float("inf"))), ("policy", dict(kl_coef=float("nan"))),
    ("policy", dict(entropy_coef=float("inf"))), ("policy_backward", dict(saved=None)), ("policy_backward", dict(grad=None)),
    ("policy_backward", dict(saved=68)), ("policy_backward", dict(clip_high=-1.0)), ("policy_backward", dict(old_logprobs=None)),
    ("preference", dict(out=None)), ("preference", dict(saved=None)), ("preference", dict(saved=72)),
    ("preference", dict(pair_status=None)), ("preference", dict(row_offsets=None)), ("preference", dict(n_pairs=0)),
    ("preference", dict(n_pairs=(1 << 16) + 1)), ("preference", dict(beta=0.0)), ("preference", dict(beta=float("inf"))),
    ("preference", dict(beta=float("nan"))), ("preference", dict(margin=float("nan"))), ("preference", dict(label_smoothing=1.0)),
    ("preference", dict(label_smoothing=-0.1)), ("preference_backward", dict(saved=None)), ("preference_backward", dict(grad=None)),
    ("preference_backward", dict(n_pairs=0)), ("preference_backward", dict(saved=68))])
def test_call_refuses(bd, what, kw):  # noqa: F811
    assert call(bd, what, kw) == 1


def test_null_structures(bd):  # noqa: F811
    lib, p = bd.load_library(), ctypes.byref(token_params(bd, {}))
    assert lib.dspark_token_logprobs(vp(4096), None, vp(64), None, None) == 1
    assert lib.dspark_policy_loss(vp(4096), None, p, vp(64), None, None, None, vp(64), None) == 1
    assert lib.dspark_policy_loss_backward(vp(4096), None, p, vp(64), None, vp(8192)) == 1
    assert lib.dspark_preference_loss(vp(4096), None, p, vp(64), None, vp(64), None, vp(64), None) == 1


# ---------------------------------------------------------------- clipping
def clip_call(bd, entries, n=None, max_norm=1.0, norm=64, status=64, ws=256, ws_bytes=1 << 30):  # noqa: F811
    arr = (bd.dspark_grad_t * max(1, len(entries)))(*(bd.dspark_grad_t(*e) for e in entries))
    n = len(entries) if n is None else n
    return bd._Calls(bd.load_library()).dspark_clip_grads(ctypes.addressof(arr) if entries else None, n, max_norm, norm, status, ws,
                                                          ws_bytes, None)


GOOD = (64, 64, 10, 1, 1)


@pytest.mark.parametrize("entry", [(None, 64, 10, 1, 1), (64, None, 10, 1, 1), (64, 64, -1, 1, 1), (64, 64, 10, 2, 1), (64, 128, 10, 1, 0),
                                   (64, 64, 10, 0, 1), (66, 128, 10, 1, 1), (64, 130, 10, 0, 1), (65, 128, 10, 0, 0)])
def test_clip_refuses_entries(bd, entry):  # noqa: F811
    assert clip_call(bd, [GOOD, entry]) == 1


def test_clip_refuses(bd):  # noqa: F811
    assert clip_call(bd, []) == 1
    assert clip_call(bd, [GOOD], n=0) == 1 and clip_call(bd, [GOOD], n=-3) == 1 and clip_call(bd, [GOOD], n=(1 << 16) + 1) == 1
    for bad in (-1.0, float("nan")):
        assert clip_call(bd, [GOOD], max_norm=bad) == 1
    assert clip_call(bd, [GOOD], norm=None) == 1 and clip_call(bd, [GOOD], status=None) == 1
    assert clip_call(bd, [(64, 64, 1 << 44, 1, 1)]) == 2
    need = bd.load_library().dspark_clip_workspace_bytes(1)
    assert need > 0 and bd.load_library().dspark_clip_workspace_bytes(0) == 0
    assert bd.load_library().dspark_clip_workspace_bytes((1 << 16) + 1) == 0
    assert clip_call(bd, [GOOD], ws=None) == 3 and clip_call(bd, [GOOD], ws=128) == 3 and clip_call(bd, [GOOD], ws_bytes=need - 1) == 3


def test_binding_refuses(bd):  # noqa: F811
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 40)
    for fn, args, kw in ((bd.dspark_token_logprobs, (x, x), dict(logprobs=x, row_status=x)),
                         (bd.dspark_token_logprobs_backward, (x, x), dict(saved=x, grad=x)),
                         (bd.dspark_policy_loss, (x, x, x, x), dict(loss=x, row_status=x)),
                         (bd.dspark_policy_loss_backward, (x, x, x, x), dict(saved=x, grad=x)),
                         (bd.dspark_preference_loss, (x, x, x), dict(loss=x, saved=x, row_status=x, pair_status=x)),
                         (bd.dspark_preference_loss_backward, (x, x), dict(saved=x, grad=x, grad_loss=x))):
        with pytest.raises(ValueError, match="CUDA"):
            fn(*args, **kw)
    with pytest.raises(ValueError, match="grad is missing"):
        bd.dspark_token_logprobs_backward(x, x, saved=x, grad=None)
    with pytest.raises(ValueError, match="grad needs saved"):
        bd.dspark_policy_loss(x, x, x, x, loss=x, row_status=x, grad=x)
    with pytest.raises(ValueError, match="row_status"):
        bd.dspark_policy_loss(x, x, x, x, loss=x, row_status=None)
    with pytest.raises(ValueError, match="CUDA"):
        bd.GradTable([x])
    with pytest.raises(ValueError, match="no gradients"):
        bd.GradTable([None])
    with pytest.raises(ValueError, match="outputs"):
        bd.GradTable([x], [x, x])


# ---------------------------------------------------------------- the oracle
def test_oracle_gradients_by_differences():
    from oracle import training as O
    rng = np.random.default_rng(0)
    V, T, h = 12, 1.7, 1e-6
    for y in (0, 5):
        x = rng.normal(0, 2, V)
        x[y] += 3
        for how in ("logp", "policy", "clipped"):
            old = O.token_row(x, y, T)["logp"][y] - (0.1 if how != "clipped" else 0.9)

            def parts(x):
                r = O.token_row(x, y, T)
                if how == "logp":
                    return 0.7 * r["logp"][y] - 0.4 * r["entropy"], 0.7, -0.4, r
                L, a, b, _ = O.policy_row(r["logp"][y], r["entropy"], old, 1.3, -2.0, 0.8, 0.2, 0.3, 0.05, 0.02)
                return L, a, b, r

            _, a, b, r = parts(x)
            grad = O.token_grad(r, a, b, T)
            for v in range(V):
                e = np.zeros(V)
                e[v] = h
                assert abs((parts(x + e)[0] - parts(x - e)[0]) / (2 * h) - grad[v]) < 1e-8
    for mean in (False, True):
        sums, counts = np.array([-3.0, -4.5]), (4, 3)
        _, _, slopes = O.preference_pair(sums, counts, 0.3, 0.1, 0.2, mean, 1.5)
        for k in (0, 1):
            e = np.eye(2)[k] * h
            d = (O.preference_pair(sums + e, counts, 0.3, 0.1, 0.2, mean, 1.5)[0] -
                 O.preference_pair(sums - e, counts, 0.3, 0.1, 0.2, mean, 1.5)[0]) / (2 * h)
            assert abs(d - slopes[k]) < 1e-8


def test_oracle_known_values():
    """Hand-worked rows and pairs."""
    from oracle import training as O
    r = O.token_row([np.log(1.0), np.log(2.0), np.log(5.0)], 1, 1.0)
    assert np.allclose(r["p"], [1 / 8, 2 / 8, 5 / 8]) and np.isclose(r["logp"][1], np.log(0.25))
    assert np.isclose(r["entropy"], -(np.log(1 / 8) / 8 + np.log(2 / 8) / 4 + 5 * np.log(5 / 8) / 8))
    assert np.allclose(O.token_grad(r, 1.0, 0.0, 2.0), [-1 / 16, 3 / 8, -5 / 16])
    assert np.allclose(O.policy_row(np.log(0.25), 0.0, np.log(0.2), 2.0, None, 1.0, 0.2, 0.2, 0.0, 0.0)[:2], [-2.4, 0.0])
    assert np.allclose(O.policy_row(np.log(0.25), 0.0, np.log(0.2), -2.0, None, 0.5, 0.2, 0.2, 0.0, 0.0)[:2], [1.25, 1.25])
    loss, rewards, slopes = O.preference_pair([1.0, -1.0], (2, 1), 0.5, 0.0, 0.0, False, 1.0)
    assert np.isclose(loss, np.log1p(np.exp(-1.0))) and np.allclose(rewards, [0.5, -0.5])
    assert np.allclose(slopes, [-0.5 / (1 + np.e), 0.5 / (1 + np.e)])
    norm, out = O.clip([[3.0], [4.0, 12.0]], 6.5)
    assert norm == 13.0 and np.allclose(out[1], [2.0, 6.0])
