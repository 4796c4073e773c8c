"""Measured cases of the operators that train on decoded tokens.

  logprobs    log-probability of one token of every row, the entropy of its distribution: "forward"
              (scoring a rollout), "two_call" (then the gradient from upstream gradients of both)
  policy      clipped policy loss with a KL term and an entropy bonus: "forward" (loss alone),
              "fused" (loss and gradient in one call), "two_call" (loss, then the gradient from an
              upstream gradient: the autograd form)
  preference  loss of paired log ratios of whole sequences, in the same three forms
  clip        norm of many gradients together, and the gradients scaled to a largest norm

Vocabularies are those of the repository's workloads (4096, 32000, 151936, 262144) and odd
neighbours; logits are N(0, 3^2) with the row's token raised by up to 24, so that its probability
runs from next to nothing to next to one, as a trained model's does on its own tokens.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_binding = None


def _framework():
    global _binding
    if _binding is None:
        from sample_verify_epilogue_gb300 import binding
        _binding = binding
    return _binding


def listed():
    return [
        # one verified request of eight drafts scored under the reference policy: latency counts
        dict(name="logprobs_one_request", op="logprobs", form="forward", R=9, V=151936, dtype="bf16", entropy=False,
             temperature=1.0, masked=0.0),
        # fp32 rows of an odd vocabulary with their entropies, and the gradient of both
        dict(name="logprobs_fp32_odd", op="logprobs", form="two_call", R=509, V=50001, dtype="fp32", entropy=True,
             temperature=0.7, masked=0.1),
        # a packed batch of rollouts scored under the reference policy
        dict(name="logprobs_batch", op="logprobs", form="forward", R=4096, V=151936, dtype="bf16", entropy=True,
             temperature=1.0, masked=0.1),
        # one short rollout of a drafter with a reduced vocabulary
        dict(name="policy_one_rollout", op="policy", form="fused", R=37, V=32000, dtype="bf16", kl=0.0, entropy=0.0,
             temperature=1.0, masked=0.0),
        # training through autograd, fp32 rows of an odd vocabulary, every term of the loss
        dict(name="policy_fp32_odd", op="policy", form="two_call", R=1021, V=32003, dtype="fp32", kl=0.05, entropy=0.01,
             temperature=1.3, masked=0.1),
        # a drafter's training step over many short rollouts
        dict(name="policy_drafter", op="policy", form="fused", R=4096, V=32000, dtype="bf16", kl=0.02, entropy=0.0,
             temperature=1.0, masked=0.1),
        # the largest training step: a packed batch of rollouts over the full vocabulary
        dict(name="policy_batch", op="policy", form="fused", R=4096, V=151936, dtype="bf16", kl=0.02, entropy=0.01,
             temperature=1.0, masked=0.1),
        # evaluation on two pairs of short answers
        dict(name="preference_eval", op="preference", form="forward", pairs=2, length=45, V=32000, dtype="bf16", mean=False,
             smoothing=0.0, reference=True, temperature=1.0),
        # fp32 rows of an odd vocabulary through autograd: no reference, mean over the answer, a margin
        dict(name="preference_fp32_odd", op="preference", form="two_call", pairs=5, length=101, V=32003, dtype="fp32", mean=True,
             smoothing=0.1, reference=False, temperature=1.0),
        # a training step on pairs of long answers over the full vocabulary
        dict(name="preference_batch", op="preference", form="fused", pairs=8, length=240, V=151936, dtype="bf16", mean=False,
             smoothing=0.0, reference=True, temperature=1.0),
        # the gradients of a drafter's head alone: latency counts
        dict(name="clip_head", op="clip", layers=0, hidden=16, vocab=8000, dtype="fp32", out="same", largest=1.0, size=0.02),
        # a drafter of four layers with bf16 gradients, into the fp32 buffers that its optimizer reads
        dict(name="clip_drafter", op="clip", layers=4, hidden=2048, vocab=32000, dtype="bf16", out="fp32", largest=1.0, size=1e-3),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("logprobs", "policy", "preference", "clip"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "clip":
        return dict(op=op, layers=rng.randint(0, 4), hidden=_log_int(rng, 16, 2048), vocab=_log_int(rng, 4096, 32000),
                    dtype=dtype, out=rng.choice(("same", "fp32")), largest=rng.choice((0.5, 1.0)),
                    size=rng.choice((1e-6, 1e-3, 0.02)))
    V = _log_int(rng, 4096, 262144)
    temperature = rng.choice((1.0, 0.7, 1.3))
    form = rng.choice(("forward", "fused", "two_call"))
    most = 300_000_000 // V
    if op == "preference":
        pairs = _log_int(rng, 1, 32)
        length = max(1, min(_log_int(rng, 8, 512), most // (4 * pairs)))
        return dict(op=op, form=form, pairs=pairs, length=length, V=V, dtype=dtype, mean=rng.random() < 0.4,
                    smoothing=rng.choice((0.0, 0.1)), reference=rng.random() < 0.7, temperature=temperature)
    R = min(_log_int(rng, 1, 4096), max(1, most))
    masked = rng.choice((0.0, 0.1)) if R > 20 else 0.0
    if op == "logprobs":
        return dict(op=op, form=rng.choice(("forward", "two_call")), R=R, V=V, dtype=dtype, entropy=rng.random() < 0.5,
                    temperature=temperature, masked=masked)
    return dict(op=op, form=form, R=R, V=V, dtype=dtype, kl=rng.choice((0.0, 0.05)), entropy=rng.choice((0.0, 0.01)),
                temperature=temperature, masked=masked)


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(case, R, seed):
    """Logits, a token of each row and the log-probabilities that a policy gives it that is a step away."""
    g, V = _generator(seed), case["V"]
    logits = torch.empty(R, V, dtype=_DTYPES[case["dtype"]], device="cuda")
    tokens = torch.randint(0, V, (R,), generator=g, device="cuda")
    raised = torch.rand(R, 1, generator=g, device="cuda") * 24
    logp = torch.empty(R, device="cuda")
    step = max(1, 200_000_000 // V)
    for lo in range(0, R, step):
        x = torch.randn(min(step, R - lo), V, generator=g, device="cuda") * 3
        x.scatter_add_(1, tokens[lo:lo + step, None], raised[lo:lo + step])
        if V > 64:
            x[::7, V // 2:V // 2 + V // 16] = -math.inf      # tokens that a grammar has masked
        x.scatter_(1, tokens[lo:lo + step, None], x.gather(1, tokens[lo:lo + step, None]).clamp(min=-30))
        logits[lo:lo + step] = x.to(logits.dtype)
        x = logits[lo:lo + step].float() / case["temperature"]
        at = x.gather(1, tokens[lo:lo + step, None])
        logp[lo:lo + step] = -torch.log(torch.exp(x - at).sum(-1, dtype=torch.float64)).float()
    return g, logits, tokens.to(torch.int32), logp


def _masked(case, R, g, tokens):
    if case["masked"]:                                       # tokens of the prompt, padding
        tokens[torch.rand(R, generator=g, device="cuda") < case["masked"]] = -1


def _outputs(R, V, logits, form):
    return dict(status=torch.zeros(R, dtype=torch.int32, device="cuda"), logprobs=torch.empty(R, device="cuda"),
                saved=torch.empty(R, 8, device="cuda"), grad=None if form == "forward" else torch.empty_like(logits))


def _prepare_logprobs(case, seed):
    R, V = case["R"], case["V"]
    g, logits, tokens, _ = _rows(case, R, seed)
    _masked(case, R, g, tokens)
    ups = torch.randn(2, R, generator=g, device="cuda")
    return dict(case=case, logits=logits, tokens=tokens, entropy=torch.empty(R, device="cuda") if case["entropy"] else None,
                up=ups[0].clone(), up_entropy=ups[1].clone() if case["entropy"] else None,
                **_outputs(R, V, logits, case["form"]))


_CLIP_LOW, _CLIP_HIGH = 0.2, 0.28


def _prepare_policy(case, seed):
    R, V = case["R"], case["V"]
    g, logits, tokens, logp = _rows(case, R, seed)
    # the policy has moved since the rollout; a ratio within 1e-4 of where clipping begins would make the
    # gradient a matter of the last bit, and is moved on
    move = torch.randn(R, generator=g, device="cuda") * 0.25
    for border in (math.log1p(-_CLIP_LOW), math.log1p(_CLIP_HIGH)):
        move = torch.where((move - border).abs() < 1e-4, border + 3e-4, move)
    ref = logp + torch.randn(R, generator=g, device="cuda") * 0.3
    weights = torch.rand(R, generator=g, device="cuda") + 0.5
    _masked(case, R, g, tokens)
    return dict(case=case, logits=logits, tokens=tokens, old=logp - move, ref=ref if case["kl"] else None,
                advantages=torch.randn(R, generator=g, device="cuda"), weights=weights,
                up=torch.rand(R, generator=g, device="cuda") + 0.5, loss=torch.empty(R, device="cuda"),
                **_outputs(R, V, logits, case["form"]))


def _lengths(case):
    """Rows of each sequence: ragged around the case's length, chosen and rejected in turn."""
    return [max(1, case["length"] * (5 + (3 * i) % 7) // 8) for i in range(2 * case["pairs"])]


def _pair_rows(case):
    n = sum(_lengths(case))
    return n + n // 40                                       # rows behind the last sequence: padding


def _prepare_preference(case, seed):
    R, V, P = _pair_rows(case), case["V"], case["pairs"]
    g, logits, tokens, logp = _rows(case, R, seed)
    lengths = _lengths(case)
    off = np.concatenate([[0], np.cumsum(lengths)])
    for s, n in enumerate(lengths):
        tokens[int(off[s]):int(off[s]) + n // 6] = -1        # the prompt's rows are not scored
    tokens[int(off[-1]):] = -1
    ref = logp + torch.randn(R, generator=g, device="cuda") * 0.2
    ref[tokens < 0] = 0.0
    return dict(case=case, logits=logits, tokens=tokens, offsets=torch.from_numpy(off.astype(np.int32)).cuda(),
                ref=ref if case["reference"] else None, weights=torch.rand(P, generator=g, device="cuda") + 0.5,
                up=torch.rand(P, generator=g, device="cuda") + 0.5, loss=torch.empty(P, device="cuda"),
                rewards=torch.empty(P, 2, device="cuda"), pair_status=torch.zeros(P, dtype=torch.int32, device="cuda"),
                **_outputs(R, V, logits, case["form"]))


def _shapes(case):
    """A drafter's parameters: embedding and head, and for each layer the attention's and the feed-forward
    block's matrices, their biases and norms."""
    h, wide, out = case["hidden"], case["hidden"] * 4, []
    for _ in range(case["layers"]):
        out += [(h,), (h, h), (h // 4 + 1, h), (h // 4 + 1, h), (h, h), (h,), (wide, h), (wide, h), (h, wide), (wide,)]
    return out + [(case["vocab"], h), (h,), (case["vocab"], h), (case["vocab"],)]


def _prepare_clip(case, seed):
    g = _generator(seed)
    grads = []
    for k, shape in enumerate(_shapes(case)):
        t = torch.randn(shape, generator=g, device="cuda") * (case["size"] * (0.5 + k % 4))
        if k == 10 * case["layers"]:
            t[::3] = 0.0                                     # rows of the embedding that no token has touched
        grads.append(t.to(_DTYPES[case["dtype"]]))
    out = [torch.empty_like(t, dtype=torch.float32 if case["out"] == "fp32" else t.dtype) for t in grads]
    s = dict(case=case, grads=grads, out=out, norm=torch.empty(1, device="cuda"),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if own:
        _plan_clip(s)
    return s


def _plan_clip(s):
    b = _framework()
    s["table"] = b.GradTable(s["grads"], s["out"])
    s["workspace"] = torch.empty(b.dspark_clip_workspace_bytes(s["table"]), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    return {"logprobs": _prepare_logprobs, "policy": _prepare_policy, "preference": _prepare_preference,
            "clip": _prepare_clip}[case["op"]](case, seed)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if op == "logprobs":
        return _own_logprobs(state) if own else _plain_logprobs(state)
    if op == "policy":
        return _own_policy(state) if own else _plain_policy(state)
    if op == "preference":
        return _own_preference(state) if own else _plain_preference(state)
    return _own_clip(state) if own else _plain_clip(state)


def _own_logprobs(s):
    c, b = s["case"], _framework()
    two = c["form"] == "two_call"
    b.dspark_token_logprobs(s["logits"], s["tokens"], logprobs=s["logprobs"], entropy=s["entropy"], row_status=s["status"],
                            saved=s["saved"] if two else None, temperature=c["temperature"])
    out = {"logprobs": s["logprobs"], "status": s["status"]} | ({} if s["entropy"] is None else {"entropy": s["entropy"]})
    if two:
        b.dspark_token_logprobs_backward(s["logits"], s["tokens"], saved=s["saved"], grad=s["grad"], grad_logprobs=s["up"],
                                         grad_entropy=s["up_entropy"], temperature=c["temperature"])
        out["grad"] = s["grad"]
    return out


def _own_policy(s):
    c, b = s["case"], _framework()
    given = dict(ref_logprobs=s["ref"], weights=s["weights"], clip_low=_CLIP_LOW, clip_high=_CLIP_HIGH, kl_coef=c["kl"],
                 entropy_coef=c["entropy"], temperature=c["temperature"])
    two = c["form"] == "two_call"
    b.dspark_policy_loss(s["logits"], s["tokens"], s["old"], s["advantages"], loss=s["loss"], logprobs=s["logprobs"],
                         row_status=s["status"], saved=None if c["form"] == "forward" else s["saved"],
                         grad=s["grad"] if c["form"] == "fused" else None, **given)
    if two:
        b.dspark_policy_loss_backward(s["logits"], s["tokens"], s["old"], s["advantages"], saved=s["saved"], grad=s["grad"],
                                      grad_loss=s["up"], **given)
    return {"loss": s["loss"], "logprobs": s["logprobs"], "status": s["status"]} | \
        ({} if s["grad"] is None else {"grad": s["grad"]})


_BETA, _MARGIN = 0.1, 0.05


def _own_preference(s):
    c, b = s["case"], _framework()
    two = c["form"] == "two_call"
    b.dspark_preference_loss(s["logits"], s["tokens"], s["offsets"], loss=s["loss"], logprobs=s["logprobs"],
                             row_status=s["status"], pair_status=s["pair_status"], rewards=s["rewards"],
                             saved=s["saved"], grad=s["grad"] if c["form"] == "fused" else None, ref_logprobs=s["ref"],
                             weights=s["weights"], beta=_BETA, margin=_MARGIN, label_smoothing=c["smoothing"], mean=c["mean"],
                             temperature=c["temperature"])
    if two:
        b.dspark_preference_loss_backward(s["logits"], s["tokens"], saved=s["saved"], grad=s["grad"], grad_loss=s["up"],
                                          temperature=c["temperature"])
    return {"loss": s["loss"], "rewards": s["rewards"], "logprobs": s["logprobs"], "status": s["status"],
            "pair_status": s["pair_status"]} | ({} if s["grad"] is None else {"grad": s["grad"]})


def _own_clip(s):
    b = _framework()
    if "table" not in s:
        _plan_clip(s)
    b.dspark_clip_grads(s["table"], s["case"]["largest"], norm=s["norm"], status=s["status"], workspace=s["workspace"])
    return {"grads": s["out"], "norm": s["norm"], "status": s["status"]}


def _softplus(d):
    return d.clamp(min=0) + torch.log1p(torch.exp(-d.abs()))


def _plain_rows(s, want_entropy):
    """Per row, with the sums in 64 bits: d = log sum of the other tokens' exponentials less the token's logit,
    log p, entropy; and the exponentials with what makes probabilities of them."""
    x, T = s["logits"], s["case"]["temperature"]
    live = s["tokens"] >= 0
    at = s["tokens"].long().clamp(min=0)[:, None]
    z = x.float() / T
    z = z - z.amax(-1, keepdim=True)
    e = torch.exp(z)
    zy = z.gather(1, at).double()
    rest = e.scatter(1, at, 0.0).sum(-1, keepdim=True, dtype=torch.float64)
    d = torch.log(rest) - zy
    logp = -_softplus(d)
    logz = torch.log(rest + torch.exp(zy))
    H = None
    if want_entropy:
        mean = torch.where(e > 0, e * z, 0.0).sum(-1, keepdim=True, dtype=torch.float64) * torch.exp(-logz)
        H = logz - mean
    return dict(live=live[:, None], at=at, z=z, e=e, d=d, logp=logp, logz=logz, entropy=H)


def _plain_grad(s, r, a, h):
    """(a (1[v = y] - p_v) - h p_v (log p_v + H)) / T of live rows; a and h [R, 1] in 64 bits."""
    T, logits = s["case"]["temperature"], s["logits"]
    a = torch.where(r["live"], a, 0.0) / T
    scale = torch.exp(-r["logz"])
    if h is None:
        grad = r["e"] * (-a * scale).float()
        at_y = torch.zeros_like(a)
    else:
        h = torch.where(r["live"], h, 0.0) / T
        level = (r["entropy"] - r["logz"]).float()
        p = r["e"] * scale.float()
        inner = torch.where(p > 0, r["z"] + level, 0.0)
        grad = p * (-a.float() - h.float() * inner)
        at_y = -h * torch.exp(r["logp"]) * (r["logp"] + r["entropy"])
    # at the token itself 1 - p without the difference of two near ones
    at_y = at_y + a * torch.exp(-_softplus(-r["d"]))
    grad.scatter_(1, r["at"], torch.where(r["live"], at_y, 0.0).float())
    return grad.to(logits.dtype)


def _plain_logprobs(s):
    c = s["case"]
    r = _plain_rows(s, c["entropy"])
    out = {"logprobs": torch.where(r["live"], r["logp"], 0.0)[:, 0].float(), "status": torch.zeros_like(s["status"])}
    if c["entropy"]:
        out["entropy"] = torch.where(r["live"], r["entropy"], 0.0)[:, 0].float()
    if c["form"] == "two_call":
        h = s["up_entropy"].double()[:, None] if c["entropy"] else None
        out["grad"] = _plain_grad(s, r, s["up"].double()[:, None], h)
    return out


def _plain_policy(s):
    c = s["case"]
    r = _plain_rows(s, c["entropy"] != 0)
    logp, w = r["logp"], s["weights"].double()[:, None]
    A, ratio = s["advantages"].double()[:, None], torch.exp(logp - s["old"].double()[:, None])
    plain, clipped = ratio * A, ratio.clamp(1 - _CLIP_LOW, 1 + _CLIP_HIGH) * A
    loss = -torch.minimum(plain, clipped)
    a = torch.where(plain <= clipped, -plain, 0.0)
    if s["ref"] is not None:
        D = s["ref"].double()[:, None] - logp
        loss = loss + c["kl"] * (torch.expm1(D) - D)
        a = a - c["kl"] * torch.expm1(D)
    h = None
    if c["entropy"]:
        loss = loss - c["entropy"] * r["entropy"]
        h = -c["entropy"] * w
    out = {"loss": torch.where(r["live"], w * loss, 0.0)[:, 0].float(),
           "logprobs": torch.where(r["live"], logp, 0.0)[:, 0].float(), "status": torch.zeros_like(s["status"])}
    if c["form"] == "forward":
        return out
    up = s["up"].double()[:, None] if c["form"] == "two_call" else 1.0
    return out | {"grad": _plain_grad(s, r, a * w * up, None if h is None else h * up)}


def _plain_preference(s):
    c, P = s["case"], s["case"]["pairs"]
    r = _plain_rows(s, False)
    logp = torch.where(r["live"], r["logp"], 0.0)[:, 0]
    gain = logp if s["ref"] is None else torch.where(r["live"][:, 0], logp - s["ref"].double(), 0.0)
    R = len(gain)
    off = s["offsets"].long()
    rows = torch.arange(R, device=gain.device)
    seq = (rows[:, None] >= off[None, 1:]).sum(-1)           # 2 * pairs behind the last sequence
    total = torch.zeros(2 * P + 1, dtype=torch.float64, device=gain.device).index_add_(0, seq, gain)
    count = torch.zeros_like(total).index_add_(0, seq, r["live"][:, 0].double())
    norm = 1 / count.clamp(min=1) if c["mean"] else torch.ones_like(total)
    reward = (_BETA * total * norm)[:2 * P].view(P, 2)
    z = reward[:, 0] - reward[:, 1] - _MARGIN
    smooth, w = c["smoothing"], s["weights"].double()
    loss = w * ((1 - smooth) * _softplus(-z) + smooth * _softplus(z))
    out = {"loss": loss.float(), "rewards": reward.float(), "logprobs": logp.float(), "status": torch.zeros_like(s["status"]),
           "pair_status": torch.zeros_like(s["pair_status"])}
    if c["form"] == "forward":
        return out
    by_z = w * (smooth * torch.sigmoid(z) - (1 - smooth) * torch.sigmoid(-z))
    if c["form"] == "two_call":
        by_z = by_z * s["up"].double()
    by_seq = torch.zeros_like(total)
    by_seq[0:2 * P:2], by_seq[1:2 * P:2] = by_z, -by_z
    a = (by_seq * norm * _BETA)[seq]
    return out | {"grad": _plain_grad(s, r, a[:, None], None)}


def _plain_clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        total = total + (g.float() * g.float()).sum(dtype=torch.float64)
    norm = torch.sqrt(total)
    scale = torch.where(norm > s["case"]["largest"], s["case"]["largest"] / norm, 1.0).float()
    out = [(g.float() * scale).to(o.dtype) for g, o in zip(s["grads"], s["out"])]
    return {"grads": out, "norm": norm.float()[None], "status": torch.zeros_like(s["status"])}


# ---------------------------------------------------------------- work and exact results
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip":
        n = sum(math.prod(shape) for shape in _shapes(case))
        return {"bytes": n * (size + (4.0 if case["out"] == "fp32" else size)), "flops": 3.0 * n}
    V = case["V"]
    if case["op"] == "preference":
        R = _pair_rows(case)
        live = sum(n - n // 6 for n in _lengths(case))
    else:
        R = case["R"]
        live = R * (1 - case["masked"])
    # the logits once a call; the gradient of every row
    reads = 2 if case["form"] == "two_call" else 1
    writes = 0 if case["form"] == "forward" else 1
    per = 4.0 + (2.0 if case.get("entropy") else 0.0)
    return {"bytes": live * V * size * reads + R * V * size * writes + 24.0 * R, "flops": per * live * V * (1 + writes)}


def exact(case, seed):
    if case["op"] == "clip":
        return _exact_clip(prepare(case, seed))
    s = prepare(case, seed)
    if s["logits"].numel() > 700_000_000:
        return None
    return {"logprobs": _exact_logprobs, "policy": _exact_policy, "preference": _exact_preference}[case["op"]](s)


def _exact_clip(s):
    squares = [g.double().square().sum() for g in s["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    factor = min(1.0, s["case"]["largest"] / float(norm)) if float(norm) > 0 else 1.0
    return {"grads": [g.double() * factor for g in s["grads"]], "norm": norm.reshape(1), "status": None}


def _exact_scores(s):
    """(log p of the token, entropy) of every row from the whole log-softmax in 64 bits, a few rows at a time."""
    x, T = s["logits"], s["case"]["temperature"]
    R, V = x.shape
    logp, H = torch.zeros(R, dtype=torch.float64, device="cuda"), torch.zeros(R, dtype=torch.float64, device="cuda")
    for lo, lp, ids in _exact_slices(s):
        logp[lo:lo + len(lp)] = lp.gather(1, ids.clamp(min=0)[:, None])[:, 0]
        p = torch.exp(lp)
        H[lo:lo + len(lp)] = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    return logp, H


def _exact_slices(s):
    x, T = s["logits"], s["case"]["temperature"]
    step = max(1, 100_000_000 // x.shape[1])
    for lo in range(0, len(x), step):
        lp = x[lo:lo + step].double() / T
        lp -= torch.logsumexp(lp, -1, keepdim=True)
        yield lo, lp, s["tokens"][lo:lo + step].long()


def _exact_grad(s, a, h, H):
    """From dL/dlog p (a) and dL/dentropy (h) of every row, 0 where the row counts for nothing."""
    T = s["case"]["temperature"]
    grad = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
    for lo, lp, ids in _exact_slices(s):
        hi = lo + len(lp)
        p = torch.exp(lp)
        g = -a[lo:hi, None] * p
        g.scatter_add_(1, ids.clamp(min=0)[:, None], a[lo:hi, None])
        if h is not None:
            g -= h[lo:hi, None] * torch.where(p > 0, p * (lp + H[lo:hi, None]), 0.0)
        grad[lo:hi] = torch.where(ids[:, None] >= 0, g / T, 0.0)
    return grad


def _exact_logprobs(s):
    live = s["tokens"] >= 0
    logp, H = _exact_scores(s)
    out = {"logprobs": torch.where(live, logp, 0.0), "status": None}
    if s["case"]["entropy"]:
        out["entropy"] = torch.where(live, H, 0.0)
    if s["case"]["form"] == "two_call":
        out["grad"] = _exact_grad(s, s["up"].double(), s["up_entropy"].double() if s["case"]["entropy"] else None, H)
    return out


def _exact_policy(s):
    c, live = s["case"], s["tokens"] >= 0
    logp, H = _exact_scores(s)
    A, w = s["advantages"].double(), s["weights"].double()
    rho = torch.exp(logp - s["old"].double())
    # the smaller of two products: clipping binds above for a gain, below for a loss
    bound = torch.where(A > 0, 1 + _CLIP_HIGH, 1 - _CLIP_LOW)
    binds = torch.where(A > 0, rho > bound, rho < bound)
    loss = -torch.where(binds, bound, rho) * A
    a = torch.where(binds, 0.0, -rho * A)
    if s["ref"] is not None:
        gap = s["ref"].double() - logp
        loss += c["kl"] * (torch.exp(gap) - gap - 1)
        a += c["kl"] * (1 - torch.exp(gap))
    loss -= c["entropy"] * H
    out = {"loss": torch.where(live, w * loss, 0.0), "logprobs": torch.where(live, logp, 0.0), "status": None}
    if c["form"] != "forward":
        w = w * s["up"].double() if c["form"] == "two_call" else w
        out["grad"] = _exact_grad(s, a * w, -c["entropy"] * w if c["entropy"] else None, H)
    return out


def _exact_preference(s):
    c, live = s["case"], s["tokens"] >= 0
    logp, _ = _exact_scores(s)
    logp = torch.where(live, logp, 0.0)
    off = s["offsets"].tolist()
    ref = torch.zeros_like(logp) if s["ref"] is None else s["ref"].double()
    a = torch.zeros_like(logp)
    losses, rewards = [], []
    for p in range(c["pairs"]):
        both = []
        for k in (2 * p, 2 * p + 1):
            part = slice(off[k], off[k + 1])
            scored = live[part]
            n = int(scored.sum()) if c["mean"] else 1
            both.append((part, n, _BETA * float(((logp - ref)[part])[scored].sum()) / max(n, 1)))
        z = both[0][2] - both[1][2] - _MARGIN
        log_up, log_down = -float(np.logaddexp(0, -z)), -float(np.logaddexp(0, z))   # of sigma(z), sigma(-z)
        w, eps = float(s["weights"][p]), c["smoothing"]
        losses.append(-w * ((1 - eps) * log_up + eps * log_down))
        rewards.append([both[0][2], both[1][2]])
        slope = w * (eps * math.exp(log_up) - (1 - eps) * math.exp(log_down)) * (float(s["up"][p]) if c["form"] == "two_call" else 1.0)
        for (part, n, _), sign in zip(both, (1, -1)):
            a[part] = sign * slope * _BETA / max(n, 1)
    out = {"loss": torch.tensor(losses, dtype=torch.float64, device="cuda"),
           "rewards": torch.tensor(rewards, dtype=torch.float64, device="cuda"), "logprobs": logp, "status": None,
           "pair_status": None}
    if c["form"] != "forward":
        out["grad"] = _exact_grad(s, torch.where(live, a, 0.0), None, None)
    return out
