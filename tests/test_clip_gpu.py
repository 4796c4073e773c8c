"""The norm of many gradients and their clipping on the GPU, against float64."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import training as O  # noqa: E402
from tests import _rows as R  # noqa: E402
from tests.test_rows_gpu import bd  # noqa: E402,F401

U = R.U
# squares of a chunk: each u, 8 (bf16: 16) of a lane's sum one after the other, 3 joins; then pairs of floats.  The norm is
# the root (half of that), rounded; the factor one division more; the product one
NORM = 0.5 * 24 * U + 2 * U
TINY = 2.0 ** -149


def clip_call(bd, grads, max_norm, out=None, table=None):  # noqa: F811
    t = bd.GradTable(grads, out) if table is None else table
    norm, status = torch.full((1,), 9.0, device="cuda"), torch.full((1,), -1, dtype=torch.int32, device="cuda")
    ws = torch.full((bd.dspark_clip_workspace_bytes(t),), 255, dtype=torch.uint8, device="cuda")
    bd.dspark_clip_grads(t, max_norm, norm=norm, status=status, workspace=ws)
    return float(norm), int(status)


def check(bd, values, dtypes, max_norm, out_dtypes=None, shifts=None, out_shifts=None):  # noqa: F811
    """values: arrays; in place without out_dtypes."""
    grads, outs = [], []
    for k, (v, dt) in enumerate(zip(values, dtypes)):
        s = 0 if shifts is None else shifts[k]
        buf = torch.full((v.size + s + 3,), 7.0, dtype=R.TORCH[dt], device="cuda")
        buf[s:s + v.size] = torch.from_numpy(np.ascontiguousarray(v, np.float32).ravel()).to(R.TORCH[dt])
        grads.append((buf, s, v.size))
        if out_dtypes is not None:
            so = 0 if out_shifts is None else out_shifts[k]
            outs.append((torch.full((v.size + so + 3,), 7.0, dtype=R.TORCH[out_dtypes[k]], device="cuda"), so, v.size))

    def part(b):
        return b[0][b[1]:b[1] + b[2]]

    held = [part(g).double().cpu().numpy() for g in grads]
    want_norm, want = O.clip(held, max_norm)
    norm, status = clip_call(bd, [part(g) for g in grads], max_norm, [part(o) for o in outs] if outs else None)
    assert status == 0
    assert abs(norm - want_norm) <= NORM * want_norm + TINY, (norm, want_norm)
    for k, (w, h) in enumerate(zip(want, held)):
        b = outs[k] if outs else grads[k]
        got = part(b).double().cpu().numpy()
        dt = (out_dtypes or dtypes)[k]
        if want_norm <= max_norm * (1 - 4 * NORM):
            assert np.array_equal(got, h)
        else:
            tol = (NORM + 3 * U) * np.abs(w) + R.HALF[dt] * np.abs(w) + (2.0 ** -133 if dt == "bf16" else TINY)
            assert (np.abs(got - w) <= tol).all(), (k, np.abs(got - w).max())
        rest = torch.cat([b[0][:b[1]], b[0][b[1] + b[2]:]])
        assert (rest == 7).all()                             # what lies around is left as it is
    return norm


@pytest.mark.parametrize("out", [None, "same", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [(1,), (0, 1, 2), (7, 4096, 4097, 8191, 8192, 8193), (1000003, 5, 0, 33333), (100,) * 99])
def test_clip(bd, sizes, dtype, out):  # noqa: F811
    rng = np.random.default_rng(len(sizes))
    values = [rng.normal(0, 0.5, n) for n in sizes]
    out_dtypes = None if out is None else [dtype if out == "same" else "fp32"] * len(sizes)
    for max_norm in (0.25, 1e9):
        check(bd, values, [dtype] * len(sizes), max_norm, out_dtypes)


@pytest.mark.parametrize("out", [False, True])
def test_clip_mixed_types_and_alignment(bd, out):  # noqa: F811
    rng = np.random.default_rng(5)
    sizes = [1, 3, 17, 5000, 12345, 40001, 8, 15, 16, 9999]
    values = [rng.normal(0, 1, n) for n in sizes]
    dtypes = ["bf16", "fp32"] * 5
    for s in range(0, 8, 3):
        shifts = [(s + k) % 8 for k in range(10)]
        outs = ["fp32" if k % 3 else dt for k, dt in enumerate(dtypes)] if out else None
        check(bd, values, dtypes, 0.5, outs, shifts, [(k * 3 + s) % 5 for k in range(10)])
        check(bd, values, dtypes, 0.5, outs, shifts, shifts)


@pytest.mark.parametrize("n", [100, 101, 1000, 1001, 2500])
def test_clip_long_lists(bd, n):  # noqa: F811
    """Lists around the launches' sizes, some tensors empty."""
    rng = np.random.default_rng(n)
    values = [rng.normal(0, 1, int(rng.integers(0, 40))) for _ in range(n)]
    values[n // 2] = rng.normal(0, 1, 50001)
    check(bd, values, ["fp32" if k % 2 else "bf16" for k in range(n)], 1.0)
    check(bd, values, ["bf16"] * n, 1.0, ["fp32"] * n)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 2e-23, 1e-12, 1e12, 1e18, 3e19, 1e30, 1e35])
def test_clip_range(bd, scale, dtype):  # noqa: F811
    """Squares beyond fp32's range on either side."""
    rng = np.random.default_rng(6)
    values = [rng.normal(0, 1, n) * scale for n in (3001, 70000, 5)]
    check(bd, values, [dtype] * 3, float(np.float32(10 * scale)))
    check(bd, values + [np.zeros(9000), rng.normal(0, 1, 4000) * 1e-3], [dtype] * 5, float(np.float32(10 * scale)))


@pytest.mark.parametrize("bits", [1, 0x8000, 0x10000, 0x007FFFFF])
def test_clip_smallest_numbers(bd, bits):  # noqa: F811
    """Numbers below the smallest normal one: their norm is right, and what they are scaled to."""
    v = np.array([bits], np.uint32).view(np.float32)
    g = torch.from_numpy(np.repeat(v, 9)).cuda()
    norm, status = clip_call(bd, [g], float("inf"))
    want = 3 * float(v[0])
    assert status == 0 and abs(norm - want) <= NORM * want + TINY


def test_clip_zero(bd):  # noqa: F811
    for dtype in ("bf16", "fp32"):
        assert check(bd, [np.zeros(5000), np.zeros(3)], [dtype] * 2, 1.0) == 0.0
        assert check(bd, [np.zeros(5000), np.zeros(0)], [dtype] * 2, 0.0, ["fp32"] * 2) == 0.0
        assert check(bd, [np.zeros(0)], [dtype], 1.0) == 0.0
        assert check(bd, [np.ones(4)], [dtype], 0.0) == 2.0


def test_clip_norm_alone(bd):  # noqa: F811
    rng = np.random.default_rng(7)
    check(bd, [rng.normal(0, 100, 30000)], ["bf16"], float("inf"))


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("out", [None, "same", "fp32"])
def test_clip_not_finite(bd, out, value):  # noqa: F811
    """The gradients stay as they are, NaNs with their bits."""
    rng = np.random.default_rng(8)
    for dtype in ("bf16", "fp32"):
        g = [torch.from_numpy(rng.normal(0, 1, n).astype(np.float32)).to(R.TORCH[dtype]).cuda() for n in (9000, 31)]
        g[1][30] = value
        before = [t.clone() for t in g]
        outs = None if out is None else [torch.full_like(t, 7.0, dtype=t.dtype if out == "same" else torch.float32) for t in g]
        norm, status = clip_call(bd, g, 0.5, outs)
        assert status == bd.ROW_NONFINITE and not np.isfinite(norm)
        for b, t in zip(before, outs or g):
            assert torch.equal(b.to(t.dtype).view(torch.uint8), t.view(torch.uint8))
    # a norm that fp32 does not hold, of finite gradients
    g = [torch.full((100,), 3e38, device="cuda")]
    norm, status = clip_call(bd, g, 1.0)
    assert norm == np.inf and status == bd.ROW_NONFINITE and (g[0] == 3e38).all()


def test_clip_same_bits(bd):  # noqa: F811
    """The same list gives the same bits, whatever ran before it."""
    g = torch.Generator(device="cuda").manual_seed(1)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (1 << 20, 77777, 3)]
    outs = [[torch.empty_like(t) for t in grads] for _ in range(5)]
    norms = [clip_call(bd, grads, 1.0, o)[0] for o in outs]
    assert len(set(norms)) == 1
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_clip_shapes_and_missing_gradients(bd):  # noqa: F811
    g = [torch.ones(3, 5, device="cuda"), None, torch.ones((), device="cuda"), torch.ones(2, 3, 4, device="cuda")[1]]
    norm, status = clip_call(bd, g, 1.0)
    assert status == 0 and abs(norm - 28 ** 0.5) < 1e-5
    assert abs(float(g[3][0, 0]) - 28 ** -0.5) < 1e-6


def test_clip_refuses_tables(bd):  # noqa: F811
    a, b = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
    for grads, out in (([a, a], None), ([a, b], [b, a]), ([a], [torch.ones(5, device="cuda")]), ([a], [torch.ones(4)]), ([a], [None]),
                       ([a], [torch.ones(4, device="cuda", dtype=torch.bfloat16)]), ([torch.ones(4, 4, device="cuda").t()[:2]], None),
                       ([torch.ones(8, device="cuda")[::2]], None), ([a, torch.ones(4)], None)):
        with pytest.raises(ValueError):
            bd.GradTable(grads, out)
    with pytest.raises(TypeError):
        bd.GradTable([a.half()])
    t = bd.GradTable([a])
    norm, status = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(bd.dspark_clip_workspace_bytes(t), dtype=torch.uint8, device="cuda")
    for bad in (dict(workspace=ws[1:]), dict(workspace=ws[:-1]), dict(norm=torch.zeros(2, device="cuda")), dict(status=norm), dict(max_norm=-1.0)):
        given = dict(max_norm=1.0, norm=norm, status=status, workspace=ws) | bad
        with pytest.raises((ValueError, RuntimeError)):
            bd.dspark_clip_grads(t, given.pop("max_norm"), **given)


def test_clip_grads_of_parameters(bd):  # noqa: F811
    from sample_verify_epilogue_gb300.training import clip_grads_
    p = [torch.nn.Parameter(torch.zeros(4, 4, device="cuda")) for _ in range(3)]
    p[0].grad, p[2].grad = torch.ones(4, 4, device="cuda"), torch.full((4, 4), 2.0, device="cuda")
    norm, status = clip_grads_(p, 2.0)
    assert abs(float(norm) - 80 ** 0.5) < 1e-5 and int(status) == 0
    assert abs(float(p[2].grad[0, 0]) - 4 / 80 ** 0.5) < 1e-6 and p[1].grad is None


def test_clip_in_graphs(bd):  # noqa: F811
    """Captured and replayed on new gradients; two graphs with a workspace each."""
    grads = [torch.zeros(50001, device="cuda"), torch.zeros(33, device="cuda", dtype=torch.bfloat16)]
    table = bd.GradTable(grads)
    runs = []
    for max_norm in (1.0, 3.0):
        norm, status = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.zeros(bd.dspark_clip_workspace_bytes(table), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            bd.dspark_clip_grads(table, max_norm, norm=norm, status=status, workspace=ws)
        runs.append((graph, norm, max_norm))
    rng = np.random.default_rng(9)
    for _ in range(3):
        for graph, norm, max_norm in runs:
            values = [rng.normal(0, 1, t.numel()) for t in grads]
            for t, v in zip(grads, values):
                t.copy_(torch.from_numpy(v))
            held = [t.double().cpu().numpy() for t in grads]
            graph.replay()
            want_norm, want = O.clip(held, max_norm)
            assert abs(float(norm) - want_norm) <= NORM * want_norm
            assert np.abs(grads[0].double().cpu().numpy() - want[0]).max() < 1e-6


def test_clip_on_another_stream(bd):  # noqa: F811
    side = torch.cuda.Stream()
    g, late = torch.randn(300001, device="cuda"), torch.zeros(300001, device="cuda")
    table = bd.GradTable([late])
    norm, status = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(bd.dspark_clip_workspace_bytes(table), dtype=torch.uint8, device="cuda")
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = torch.tanh(busy @ busy)
        late.copy_(g)
    bd.dspark_clip_grads(table, 1.0, norm=norm, status=status, workspace=ws, stream=side.cuda_stream)
    side.synchronize()
    want = float(g.double().norm())
    assert abs(float(norm) - want) <= NORM * want and abs(float(late.double().norm()) - 1) < 1e-5


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.get_device_properties(0).total_memory < 40 << 30, reason="memory")
def test_clip_beyond_32_bits(bd):  # noqa: F811
    """More elements than 32 bits count: the last ones are in the norm, and scaled."""
    n = (1 << 32) + 5
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[-2], g[0], g[(1 << 31) + 1] = 3.0, 4.0, 12.0, 84.0
    norm, status = clip_call(bd, [g], 8.5)
    assert status == 0 and abs(norm - 85) < 1e-4
    assert [float(g[k]) for k in (-1, -2, 0, (1 << 31) + 1)] == [float(torch.tensor(v / 10).bfloat16()) for v in (3, 4, 12, 84)]


def test_clip_refuses_overlaps(bd):  # noqa: F811
    """Memory that two entries share is refused, whole or in part; neighbours and empty gradients are not."""
    flat, wide = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    half = torch.ones(16, device="cuda", dtype=torch.bfloat16)
    for grads, out in (([flat[:8], flat[7:9]], None), ([flat, flat[63:]], None), ([flat[8:16], flat[:32]], None),
                       ([flat[:8], flat[8:16]], [wide[:8], wide[7:15]]), ([flat[:8], flat[8:16]], [wide[:8], wide[:8]]),
                       ([flat[:8]], [flat[4:12]]), ([half, flat[:8]], [flat[4:20], wide[:8]])):
        with pytest.raises(ValueError, match="overlap"):
            bd.GradTable(grads, out)
    for grads, out in (([flat[8:16], flat[:8], flat[8:8], flat[16:]], None), ([flat[8:8], flat[8:16]], None),
                       ([half, flat[:8]], [wide[:16], wide[16:24]])):
        assert len(bd.GradTable(grads, out)) == len(grads)
    norm, status = clip_call(bd, [flat[8:16], flat[:8], flat[8:8], flat[16:]], 2.0)
    assert status == 0 and norm == 8.0 and bool((flat == 0.25).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scales", [(1e30, 1.0, 1e-30), (1.0, 1e-30), (1e-30, 1e-20, 0.0), (2e-14, 1e-25), (2e17, 2e17), (1e19, 2e17), (1e25, 1e-12),
                                    (3e-41, 1e-38), (1.0, 3e19)])
def test_clip_shares_of_every_size(bd, scales, dtype):  # noqa: F811
    """Tensors of many shares each, whose sums lie on either side of fp32's range, or leave it together."""
    rng = np.random.default_rng(7)
    values = [rng.uniform(0.5, 1, 900001) * s for s in scales]
    held = [torch.from_numpy(v.astype(np.float32)).to(R.TORCH[dtype]).double() for v in values]
    norm = float(sum((h * h).sum() for h in held)) ** 0.5
    for max_norm in (norm / 3, norm * 2):
        check(bd, values, [dtype] * len(values), float(np.float32(max_norm)))
