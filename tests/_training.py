"""Inputs and error bounds for the tests of what trains on decoded tokens.

Bounds count roundings, first order with a margin for the products of small errors.  u = 2^-24, EX2 = 2^-22 the
exponential's; a row's sum of exponentials R has tests/_rows.sum_bound relative to itself.  expf and log1pf are off by
2 u and 2 u of their result at most (2 ulp and 1 ulp in CUDA's tables, an ulp being up to 2 u), logf by 2 u.
  d = log R - s_y     es = sum_bound, and u of each exponent's product with log2(e)/T rounded to fp32:
                      ed = es + 3 u |s_y - m| + 4 u |d|
  log p_y             q ed + 8 u |log p_y|       (dlog p_y / dd = -q, q = 1 - p_y)
  q, p_y              relative p_y ed + 8 u, q ed + 8 u
  H                   the sum of its terms' errors (see entropy_bound)
  p_v                 relative es + EX2 + 3 u |s_v - m| + q's + 8 u
  flushing            exponentials below 2^-126 are 0.  They are by a whole exponent r = ceil(m c + 5) < m c + 6, m the
                      largest logit: what is below 2^-120 of the largest may be 0
"""
import numpy as np

from tests import _rows as R

U, EX2 = R.U, R.EX2
FLUSH = 2.0 ** -120


def row_errors(r, V):
    """es, ed and the error of log p_y, H of an oracle row."""
    es = R.sum_bound(V)
    if not np.isfinite(r["d"]):
        d, gap = 0.0, 0.0
    else:
        d, gap = abs(r["d"]), abs(r["s"][r["y"]] - r["m"])
    ed = es + 3 * U * gap + 4 * U * d
    lp = abs(r["logp"][r["y"]]) if np.isfinite(r["logp"][r["y"]]) else 0.0
    elp = 1.01 * (r["q"] * ed + 8 * U * lp) + FLUSH
    return es, ed, elp, entropy_bound(r, es, ed)


def entropy_bound(r, es, ed):
    """H = p_y sp + q (sm + H_R), sp = log(1 + e^d), sm = log(1 + e^-d), H_R = log R - W / R: relative errors of p_y and q,
    sp's and sm's by d's and their own, H_R's by the sums' (W's terms e z: es relative, and their exponents' as theirs)."""
    if not np.isfinite(r["d"]):
        q, py, sp, sm = r["q"], 1 - r["q"], 0.0, 0.0
    else:
        q, py = r["q"], 1 / (1 + np.exp(min(r["d"], 700)))
        sp, sm = np.logaddexp(0, r["d"]), np.logaddexp(0, -r["d"])
    others = np.delete(r["s"], r["y"])
    others = others[np.isfinite(others)]
    if len(others):
        z = others - others.max()
        e = np.exp(z)
        lr, wr = np.log(e.sum()), -(e * z).sum() / e.sum()
    else:
        lr = wr = 0.0
    rel_p, rel_q = q * ed + 8 * U, py * ed + 8 * U
    spread = (es + 4 * U * (abs(lr) + 1)) + wr * (3 * es + 8 * U)
    out = py * sp * rel_p + py * (q * ed + 8 * U * sp) + q * (sm + lr + wr) * rel_q + q * (py * ed + 8 * U * sm + spread)
    return 1.02 * out + 4 * U * abs(r["entropy"]) + FLUSH


def grad_bound(r, a, h, V, temperature, dtype, exact, ea=0.0):
    """Of each gradient entry; ea: absolute error of a (h is exact)."""
    es, ed, elp, eH = row_errors(r, V)
    y, p = r["y"], r["p"]
    with np.errstate(invalid="ignore"):
        arg = np.where(np.isfinite(r["s"]), np.abs(r["s"] - (r["m"] if np.isfinite(r["m"]) else 0.0)), 0.0)
    py = p[y]
    rel = es + EX2 + 3 * U * arg + py * ed + 16 * U
    with np.errstate(invalid="ignore"):
        inner = np.where(p > 0, np.abs(r["logp"] + r["entropy"]), 0.0)
        size = np.where(p > 0, np.abs(r["logp"]), 0.0) + r["entropy"]
    ein = eH + es + py * ed + 3 * U * arg + 8 * U * (size + arg)
    part = p * ((abs(a) + ea) * rel + ea + abs(h) * (inner * rel + ein))
    part[y] = (abs(a) + ea) * r["q"] * (py * ed + 8 * U) + ea * r["q"] + \
        abs(h) * py * (inner[y] * (r["q"] * ed + 12 * U) + eH + elp + 8 * U * size[y])
    flush = FLUSH * (abs(a) + ea + abs(h) * (1 + r["entropy"] + 128))
    return 1.02 * (part + flush) / temperature + R.HALF[dtype] * np.abs(exact) + 2.0 ** -133


def token_rows(rng, rows, V, dtype, special=True):
    """Logits and a token of each row, from next to no probability to next to all of it."""
    x = rng.normal(0, 3, (rows, V))
    y = rng.integers(0, V, rows)
    x[np.arange(rows), y] += rng.uniform(0, 24, rows)
    y32 = y.copy()
    if special and V > 16:
        kinds = rng.permutation(rows)
        for k, r in enumerate(kinds[:8]):
            if k == 0:
                y32[r] = -1                                  # no token
            elif k == 1:
                x[r, rng.random(V) < 0.7] = -np.inf          # masked tokens, the token itself not
                x[r, y[r]] = 1.0
            elif k == 2:
                x[r, y[r]] = -np.inf                         # the token itself is masked
                if np.isneginf(x[r]).all():
                    x[r, (y[r] + 1) % V] = 0.0
            elif k == 3:
                x[r, y[r]] = 150.0                           # sure of its token
            elif k == 4:
                x[r, rng.random(V) < 0.5] = R.rounded(-3.38e38, dtype)
                x[r, y[r]] = 2.0
            elif k == 5:
                x[r] = -np.inf                               # nothing else is possible
                x[r, y[r]] = -2.5
            elif k == 6:
                x[r, y[r]] = -60.0                           # next to impossible
            elif k == 7:
                x[r] = x[r, 0]                               # all the same
    return R.rounded(x, dtype), y32
