"""Float64 oracle of what trains on decoded tokens: token log-probabilities and entropies, the policy and preference
losses, their gradients, clipping -- written from the formulas in include/dspark.h."""
from __future__ import annotations

import numpy as np


def token_row(x, y, temperature):
    """One row's distribution at its token: a dict, or None where it cannot be normalised."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or not np.isfinite(x).any():
        return None
    s = x / temperature
    others = np.delete(s, y)
    m = d = -np.inf                                          # d: log of the others' mass over the token's
    if len(others) and np.isfinite(others).any():
        m = others.max()
        d = (m - s[y]) + np.log(np.exp(others - m).sum())
    # from the largest logit, which may be far larger than what the logarithm adds
    logp = (s - s.max()) - np.log(np.exp(s - s.max()).sum())
    logp[y] = -np.logaddexp(0, d)                            # to its last bits for a token that has nearly all the mass
    with np.errstate(over="ignore"):
        q = 1 / (1 + np.exp(-d))
    if s[y] == -np.inf:
        logp[y], q = -np.inf, 1.0
    p = np.exp(logp)
    entropy = -(p[p > 0] * logp[p > 0]).sum()
    return dict(s=s, y=y, p=p, logp=logp, q=q, d=d, entropy=entropy, m=m)


def token_grad(r, a, h, temperature):
    """The gradient of a log p(y) + h H by the logits."""
    with np.errstate(invalid="ignore"):
        inner = np.where(r["p"] > 0, r["logp"] + r["entropy"], 0.0)
    g = -r["p"] * (a + h * inner)
    g[r["y"]] = a * r["q"] - (h * r["p"][r["y"]] * inner[r["y"]])
    return g / temperature


def policy_row(logp, entropy, old, advantage, ref, weight, low, high, kl_coef, entropy_coef):
    """(loss, dL/dlog p, dL/dH, KL) of one row."""
    with np.errstate(over="ignore"):
        rho = np.exp(logp - old)
    gain, slope = 0.0, 0.0
    if advantage != 0:
        plain, clipped = rho * advantage, min(max(rho, 1 - low), 1 + high) * advantage
        gain = min(plain, clipped)
        slope = -plain if plain <= clipped else 0.0
    loss, kl = -gain, 0.0
    if ref is not None:
        D = ref - logp
        kl = np.expm1(D) - D
        loss += kl_coef * kl
        slope -= kl_coef * np.expm1(D)
    loss -= entropy_coef * entropy
    return weight * loss, weight * slope, -weight * entropy_coef, kl


def preference_pair(sums, counts, beta, margin, smoothing, mean, weight):
    """(loss, rewards (2), dL/dlog p of a token of each sequence) from the two sums of log ratios and token counts."""
    n = [max(c, 1) if mean else 1 for c in counts]
    rewards = [beta * s / k for s, k in zip(sums, n)]
    z = rewards[0] - rewards[1] - margin
    loss = weight * ((1 - smoothing) * np.logaddexp(0, -z) + smoothing * np.logaddexp(0, z))
    slope = weight * (smoothing * np.exp(-np.logaddexp(0, -z)) - (1 - smoothing) * np.exp(-np.logaddexp(0, z)))
    return loss, rewards, (slope * beta / n[0], -slope * beta / n[1])


def clip(grads, max_norm):
    """(norm, scaled gradients)."""
    norm = np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads))
    factor = max_norm / norm if norm > max_norm else 1.0
    return norm, [np.asarray(g, np.float64) * factor for g in grads]
