"""Inputs, float64 results and error bounds for the tests of the operators around the epilogue.

Bounds count roundings.  u = 2^-24 is half a step of fp32; a result rounds once more to its own
type (half a step relative to its value).  A sum of exponentials has, relative to itself:
  - per term, 2^((x-m)c): the difference, c and the product each u relative to the exponent a (in
    natural units), which enters as 3u|a| e^a <= 3u/e of the largest term; the exponential
    itself 2^-22;
  - adding: a thread's terms one after another (at most V/256 + 32, u each), then at most 24 joins
    of two sums, each two scalings (2^-22 + u) and an addition.
"""
import numpy as np
import torch

U = 2.0 ** -24
EX2 = 2.0 ** -22
HALF = {"bf16": 2.0 ** -8, "fp32": U}
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rounded(x, dtype):
    """x as the type holds it, in float64."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(TORCH[dtype]).double().numpy()


def on_gpu(x, dtype, pad=0, shift=0):
    """x [..., V] on the GPU with rows V + pad apart, the first one ``shift`` elements into its buffer."""
    x = np.asarray(x)
    V, rows = x.shape[-1], int(np.prod(x.shape[:-1]))
    buf = torch.zeros(shift + rows * (V + pad), dtype=TORCH[dtype], device="cuda")
    strides = [V + pad] * (x.ndim - 1)
    for d in range(x.ndim - 3, -1, -1):
        strides[d] = strides[d + 1] * x.shape[d + 1]
    t = buf.as_strided(x.shape, (*strides, 1), shift)
    t.copy_(torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TORCH[dtype]))
    return t


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()


def csr(rows, *dtypes):
    """Offsets and columns of per-request lists of tuples."""
    off = np.cumsum([0] + [len(r) for r in rows])
    cols = [np.array([e[k] for r in rows for e in r] or [0], dt) for k, dt in enumerate(dtypes)]
    return (i32(off), *(torch.from_numpy(c).cuda() for c in cols))


def pack_mask(allowed):
    """bool [n, V] -> int32 words [n, ceil(V/32)]."""
    n, V = allowed.shape
    bits = np.zeros((n, (V + 31) // 32 * 32), bool)
    bits[:, :V] = allowed
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def sum_bound(V):
    """Relative error of a row's sum of exponentials."""
    return EX2 + 3 * U + (V // 256 + 32) * U + 24 * (2 * (EX2 + U) + U)


def loss_bound(d, V, weight, lse, temperature):
    """Bound of the loss of one row from its float64 parts: the normaliser's logarithm, each p's
    rounding (its logarithm's terms are u relative each; expf 2u; joining n of them in pairs of floats)
    against the ratio it multiplies, the tail's likewise."""
    if d is None:
        return 0.0
    big = np.abs(d["logp"][d["p"] > 0]).max(initial=0.0) + (abs(lse) if lse is not None else 0.0) + 1
    ep = 4 * U * big + 4 * U                                 # relative error of a p
    dz = sum_bound(V)
    ratio = np.abs(d["logp"] - d["logq"])[d["p"] > 0]
    tot = (d["p"][d["p"] > 0] * (ep * ratio + ep)).sum() + d["p"].sum() * dz + ep
    if d["ratio"]:
        dr = ep / d["p_r"] if d["p_r"] > ep else 1.0
        tot += d["p_r"] * (dr * (abs(np.log(d["ratio"])) + 1) + 2 * dz + 8 * U)
    return abs(weight) * tot


def grad_bound(d, V, weight, temperature, lse, s, dtype, exact):
    """Bound of each gradient entry: the two opposing parts, each relative to itself, and the result's
    rounding."""
    if d is None:
        return np.zeros(V)
    dz = sum_bound(V)
    big = np.abs(d["logp"][d["p"] > 0]).max(initial=0.0) + (abs(lse) if lse is not None else 0.0) + 1
    ep = 4 * U * big + 4 * U
    with np.errstate(invalid="ignore"):
        arg = np.where(np.isfinite(s), np.abs(s - d["m"]) / temperature, 0.0)
    rel = dz + EX2 + 3 * U * arg + 8 * U
    dr = min(1.0, ep / d["p_r"]) if d["p_r"] > 0 else 0.0
    parts = d["q"] * (d["mass"] * rel + d["ratio"] * (2 * rel + dr))
    parts[d["members"]] += d["p"] * (ep + 8 * U)
    # exponentials below 2^-126 flush to zero
    flush = 2.0 ** -126 * (d["mass"] + d["ratio"])
    return abs(weight) / temperature * (parts + flush) + HALF[dtype] * np.abs(exact) + 2.0 ** -133
