"""What the operators around the epilogue refuse, before any CUDA call (CPU only), and their oracle."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def bd():
    from sample_verify_epilogue_gb300.build import build
    build()
    from sample_verify_epilogue_gb300 import binding
    binding.load_library()
    return binding


def vp(x):
    return ctypes.c_void_p(x)


def process(bd, logits=4096, out=8192, history=None, bias=None, mask=None, **kw):
    given = dict(B=2, K_max=1, V=100, logits_dtype=0, logits_stride=100, out_stride=100, rows=256, row_status=512)
    p = bd.dspark_process_params_t(**(given | kw))
    by = [None if s is None else ctypes.byref(s) for s in (history, bias, mask)]
    return bd.load_library().dspark_process_logits(vp(logits), vp(out), None, *by, ctypes.byref(p))


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(out=None), dict(rows=None), dict(row_status=None), dict(B=0), dict(B=2049), dict(K_max=-1),
    dict(K_max=65), dict(V=0), dict(V=(1 << 24) + 1), dict(logits_dtype=2), dict(logits_stride=99), dict(out_stride=99),
    dict(logits=4097), dict(out=8193), dict(logits=4096, out=4096, out_stride=104), dict(logits=4098, logits_dtype=1)])
def test_process_refuses(bd, kw):
    assert process(bd, **kw) == 1


def test_process_refuses_lists(bd):
    assert process(bd, history=bd.dspark_counts_t(64, None, 64)) == 1
    assert process(bd, history=bd.dspark_counts_t(64, 64, None)) == 1
    assert process(bd, bias=bd.dspark_bias_t(64, 64, None)) == 1
    assert process(bd, mask=bd.dspark_mask_t(64, 3, 4, None)) == 1          # 100 tokens need 4 words
    assert process(bd, mask=bd.dspark_mask_t(64, 4, 0, 64)) == 1
    assert process(bd, mask=bd.dspark_mask_t(64, 4, 3, None)) == 1          # 4 positions without an index
    assert process(bd, mask=bd.dspark_mask_t(66, 4, 4, None)) == 1


@pytest.mark.parametrize("kw", [
    dict(n_rows=0), dict(n_rows=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(logits_dtype=3), dict(logits_stride=9),
    dict(n=0), dict(n=257), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
    dict(temperature=float("inf")), dict(temperature=1e-45), dict(row_status=None)])
def test_top_refuses(bd, kw):
    given = dict(n_rows=2, V=10, logits_dtype=0, logits_stride=10, n=4, temperature=1.0, row_status=512)
    p = bd.dspark_top_params_t(**(given | kw))
    assert bd.load_library().dspark_top_logits(vp(4096), ctypes.byref(p), vp(64), vp(64), None) == 1


@pytest.mark.parametrize("drop", [0, 2, 3])
def test_top_refuses_null(bd, drop):
    p = bd.dspark_top_params_t(n_rows=2, V=10, logits_stride=10, n=4, temperature=1.0, row_status=512)
    a = [vp(4096), ctypes.byref(p), vp(64), vp(64), None]
    a[drop] = None
    assert bd.load_library().dspark_top_logits(*a) == 1


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw", [
    dict(n_rows=0), dict(V=0), dict(V=(1 << 24) + 1), dict(logits_dtype=7), dict(student_stride=9), dict(grad_stride=9),
    dict(temperature=0.0), dict(temperature=float("nan")), dict(n=0), dict(n=257), dict(ids=None), dict(logits=None),
    dict(t2d=64, target_V=0), dict(student=None), dict(student=4097), dict(grad=4099), dict(student=8192, grad_stride=12)])
def test_distill_refuses(bd, kw, backward):
    kw = dict(kw)
    student, grad = kw.pop("student", 4096), kw.pop("grad", 8192)
    t = bd.dspark_teacher_t(**(dict(ids=64, logits=64, lse=None, n=4, t2d=None, target_V=0) |
                               {k: kw.pop(k) for k in ("ids", "logits", "n", "t2d", "target_V") if k in kw}))
    p = bd.dspark_distill_params_t(**(dict(n_rows=2, V=10, logits_dtype=0, student_stride=10, grad_stride=10, temperature=1.0,
                                           row_status=512) | kw))
    lib = bd.load_library()
    fn = lib.dspark_distill_backward if backward else lib.dspark_distill
    assert fn(vp(student), ctypes.byref(t), ctypes.byref(p), vp(64), vp(64), vp(grad)) == 1


def test_distill_refuses_null_outputs(bd):
    lib = bd.load_library()
    t = bd.dspark_teacher_t(64, 64, None, 4, None, 0)
    p = bd.dspark_distill_params_t(n_rows=2, V=10, student_stride=10, grad_stride=10, temperature=1.0, row_status=512)
    a = vp(4096), ctypes.byref(t), ctypes.byref(p)
    assert lib.dspark_distill(*a, None, None, None) == 1
    assert lib.dspark_distill_backward(*a, None, None, vp(64)) == 1
    assert lib.dspark_distill_backward(*a, vp(64), None, None) == 1
    p.row_status = None
    assert lib.dspark_distill(*a, vp(64), None, None) == 1
    assert lib.dspark_distill(vp(4096), None, ctypes.byref(p), vp(64), None, None) == 1
    assert lib.dspark_distill(vp(4096), ctypes.byref(t), None, vp(64), None, None) == 1


def test_binding_refuses(bd):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 40)
    with pytest.raises(ValueError, match="CUDA"):
        bd.dspark_process_logits(x, None, out=x, row_status=None)
    with pytest.raises(ValueError, match="CUDA"):
        bd.dspark_top_logits(x, values=x, ids=x, row_status=None)
    with pytest.raises(ValueError, match="CUDA"):
        bd.dspark_distill(x, x, x, loss=x, row_status=x)
    assert bd._rows_of("x", x) == (6, 40, 40)
    assert bd._rows_of("x", torch.zeros(2, 3, 48)[..., :40]) == (6, 40, 48)
    assert bd._rows_of("x", torch.zeros(5, 1, 40)[1:2]) == (1, 40, 40)
    for bad in (torch.zeros(40, 6).t(), torch.zeros(2, 3, 80)[..., ::2], torch.zeros(2, 4, 40)[:, :3],
                torch.zeros(1, 40).expand(3, 40), torch.zeros(0, 40)):
        with pytest.raises(ValueError):
            bd._rows_of("x", bad)
    with pytest.raises(TypeError):
        bd._dtype_of(torch.zeros(1, dtype=torch.float16))
    assert bd._flat("t", torch.zeros(4), torch.float32, 4, -1)
    for bad in (None, torch.zeros(5), torch.zeros(4, dtype=torch.int32), torch.zeros(8)[::2]):
        with pytest.raises(ValueError):
            bd._flat("t", bad, torch.float32, 4, -1)
    with pytest.raises(ValueError):
        bd._flat("t", torch.zeros(4), torch.float32, 4, 0)


def test_oracle_gradient_by_differences():
    """The oracle's gradient against central differences of its loss, both forms of the teacher."""
    from oracle import rows as O
    rng = np.random.default_rng(0)
    V, n, T, h = 40, 6, 1.7, 1e-6
    teacher, s = rng.normal(0, 2, V), rng.normal(0, 2, V)
    ids = np.append(np.argsort(-teacher)[:n], -1)
    logits = np.append(teacher[ids[:n]], 0.0)
    for lse in (None, float(np.log(np.exp(teacher / T).sum()))):
        loss, grad, _ = O.distill_row(s, ids, logits, lse, T, 0.8)
        assert loss > 0
        for v in range(V):
            e = np.zeros(V)
            e[v] = h
            d = (O.distill_row(s + e, ids, logits, lse, T, 0.8)[0] - O.distill_row(s - e, ids, logits, lse, T, 0.8)[0]) / (2 * h)
            assert abs(d - grad[v]) < 1e-8


def test_oracle_known_values():
    """Hand-worked rows: penalties and masks; ties to the lowest id; a student equal to its teacher."""
    from oracle import rows as O
    y = O.process_row([2.0, -2.0, 1.0, 4.0, 0.0], 2.0, 0.5, 0.25, {0: 0, 1: 2}, [3, 3], {2: 1.5, 3: -1.0},
                      np.array([1, 1, 1, 1, 0], bool))
    assert np.array_equal(y, [1.0, -5.0, 2.5, 0.0, -np.inf])
    v, i, lse, ok = O.top_row([1.0, 3.0, -np.inf, 3.0], 4, 1.0)
    assert ok and np.array_equal(i, [1, 3, 0, -1]) and np.array_equal(v, [3, 3, 1, -np.inf])
    assert abs(lse - np.log(2 * np.exp(3) + np.exp(1))) < 1e-12
    t = np.array([0.3, 1.0, -0.5, 2.0])
    loss, grad, _ = O.distill_row(t, [3, 1], t[[3, 1]], np.log(np.exp(t).sum()), 1.0, 1.0)
    assert abs(loss) < 1e-12 and np.abs(grad).max() < 1e-12
