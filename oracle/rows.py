"""Float64 oracle of the operators around the epilogue: logit processing, top-logit records and
drafter distillation, one row at a time, written from the formulas in include/dspark.h."""
from __future__ import annotations

import numpy as np


def process_row(x, repetition, presence, frequency, counts, prefix, bias, allowed):
    """The processed logits of one verify position.

    x [V]; counts {token: history count}; prefix: drafts before this position; bias {token: bias};
    allowed: bool [V] or None.
    """
    y = np.asarray(x, np.float64).copy()
    c = dict(counts)
    for t in prefix:
        c[int(t)] = c.get(int(t), 0) + 1
    for t, n in c.items():
        y[t] = y[t] / repetition if y[t] > 0 else y[t] * repetition
        if n > 0:
            y[t] -= frequency * n + presence
    for t, v in bias.items():
        y[t] += v
    if allowed is not None:
        y[~allowed] = -np.inf
    return y


def top_row(x, n, temperature):
    """(values [n], ids [n], log-sum-exp, ok) of one row."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or not np.isfinite(x).any():
        return np.full(n, -np.inf), np.full(n, -1), np.nan, False
    order = np.argsort(-x, kind="stable")
    order = order[np.isfinite(x[order])][:n]
    values, ids = np.full(n, -np.inf), np.full(n, -1)
    values[:len(order)], ids[:len(order)] = x[order], order
    m = x.max()
    return values, ids, m / temperature + np.log(np.exp((x - m) / temperature).sum()), True


def distill_row(s, ids, logits, lse, temperature, weight):
    """(loss, gradient [V], details) of one row; ids are draft ids, -1: no entry."""
    s = np.asarray(s, np.float64)
    grad = np.zeros(len(s))
    members = np.asarray(ids)[np.asarray(ids) >= 0]
    if weight == 0 or len(members) == 0:
        return 0.0, grad, None
    z = np.asarray(logits, np.float64)[np.asarray(ids) >= 0] / temperature
    if lse is None:
        logp = z - z.max() - np.log(np.exp(z - z.max()).sum())
        p = np.exp(logp)
        p_r = 0.0
    else:
        logp = z - np.float64(lse)
        p = np.exp(logp)
        p_r = max(0.0, 1.0 - p.sum())
    if np.isnan(s).any() or np.isposinf(s).any() or not np.isfinite(s).any():
        return np.nan, grad, None
    m = s.max()
    e = np.exp((s - m) / temperature)
    logq = (s - m) / temperature - np.log(e.sum())
    q = e / e.sum()
    outside = np.ones(len(s), bool)
    outside[members] = False
    q_r = q[outside].sum()
    with np.errstate(invalid="ignore"):
        terms = np.where(p > 0, p * (logp - logq[members]), 0.0)
    loss = terms.sum()
    tail = p_r > 0 and q_r > 0
    if tail:
        loss += p_r * np.log(p_r / q_r)
    mass = p.sum() + p_r
    grad = q * (mass - (p_r / q_r if tail else 0.0))
    grad[members] = mass * q[members] - p
    details = dict(p=p, logp=logp, logq=logq[members], p_r=p_r, q_r=q_r, q=q, m=m, members=members, mass=mass,
                   ratio=p_r / q_r if tail else 0.0)
    return weight * loss, weight / temperature * grad, details
