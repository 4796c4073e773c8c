"""Measured cases of the operators around the verify-and-sample epilogue.

  process   repetition / presence / frequency penalties, biases and grammar masks on the
            target logits of every verify position (before the epilogue)
  top       the n largest logits of every row with their ids and the log-sum-exp (the record
            a drafter is trained on)
  distill   the divergence between a teacher's top logits and a drafter's logits: "forward"
            (loss alone, evaluation), "fused" (loss and gradient in one call), "two_call"
            (loss, then the gradient from an upstream gradient: the autograd form)

Vocabularies are those of the repository's workloads (4096, 32000, 151936, 262144) and odd
neighbours; logits are N(0, 3^2), the drafter's are the teacher's with N(0, 1) noise between.
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
        # one request of a constrained chat decoding token by token: latency counts
        dict(name="process_one_token", op="process", B=1, K=0, V=32000, dtype="bf16", history=200, bias=4,
             grammar=True, ragged=False),
        # fp32 logits of an odd vocabulary, requests with fewer drafts than the batch's most
        dict(name="process_fp32_ragged", op="process", B=7, K=3, V=151935, dtype="fp32", history=1000, bias=300,
             grammar=True, ragged=True),
        # a serving batch with penalties and biases, no grammar
        dict(name="process_penalties", op="process", B=16, K=4, V=151936, dtype="bf16", history=2048, bias=64,
             grammar=False, ragged=False),
        # the benchmark's batch: long histories, a grammar on three rows of four
        dict(name="process_batch", op="process", B=64, K=8, V=262144, dtype="bf16", history=4096, bias=64,
             grammar=True, ragged=False),
        # the teacher record of one verified request
        dict(name="top_one_request", op="top", R=9, V=151936, dtype="bf16", n=20, temperature=1.0),
        # fp32 rows of an odd vocabulary, a long record
        dict(name="top_fp32_odd", op="top", R=333, V=50001, dtype="fp32", n=128, temperature=2.0),
        # the record of a whole verified batch
        dict(name="top_batch", op="top", R=576, V=262144, dtype="bf16", n=64, temperature=1.0),
        # evaluation of a drafter with a reduced vocabulary on a few rows
        dict(name="distill_eval", op="distill", form="forward", R=64, V=32000, target_V=151936, dtype="bf16", n=20,
             temperature=1.0, tail=True, masked=0.0),
        # evaluation over a long sequence
        dict(name="distill_eval_long", op="distill", form="forward", R=2048, V=151936, target_V=0, dtype="bf16", n=64,
             temperature=2.0, tail=False, masked=0.1),
        # fp32 training rows of an odd vocabulary
        dict(name="distill_fp32_odd", op="distill", form="fused", R=509, V=32003, target_V=0, dtype="fp32", n=100,
             temperature=1.5, tail=True, masked=0.1),
        # training through autograd: loss, then the gradient; reduced draft vocabulary
        dict(name="distill_two_call", op="distill", form="two_call", R=2048, V=32000, target_V=262144, dtype="bf16",
             n=32, temperature=1.0, tail=False, masked=0.0),
        # the largest training step: a packed batch over the full vocabulary
        dict(name="distill_batch", op="distill", form="fused", R=4096, V=151936, target_V=0, dtype="bf16", n=64,
             temperature=1.0, tail=True, masked=0.1),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("process", "top", "distill"))
    V = _log_int(rng, 4096, 262144)
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "process":
        K = rng.randint(0, 8)
        B = min(_log_int(rng, 1, 64), max(1, 150_000_000 // (V * (K + 1))))
        return dict(op=op, B=B, K=K, V=V, dtype=dtype, history=_log_int(rng, 1, 4096), bias=rng.randint(0, 300),
                    grammar=rng.random() < 0.7, ragged=rng.random() < 0.5)
    if op == "top":
        R = min(_log_int(rng, 1, 576), max(1, 150_000_000 // V))
        return dict(op=op, R=R, V=V, dtype=dtype, n=_log_int(rng, 1, 256), temperature=rng.choice((1.0, 0.7, 2.0)))
    R = min(_log_int(rng, 16, 4096), max(1, 300_000_000 // V))
    target = rng.choice((0, 0, min(262144, 2 * V + rng.randint(0, 99))))
    if target:
        R = min(R, max(1, 300_000_000 // target))
    return dict(op=op, form=rng.choice(("forward", "fused", "two_call")), R=R, V=V, target_V=target, dtype=dtype,
                n=_log_int(rng, 4, 256), temperature=rng.choice((1.0, 1.5, 2.0)), tail=rng.random() < 0.5,
                masked=rng.choice((0.0, 0.1)))


# ---------------------------------------------------------------- inputs
def _num_drafts(case):
    """Drafts of each request: all K, or (ragged) fewer for most."""
    return [case["K"] - (b % (case["K"] + 1) if case["ragged"] else 0) for b in range(case["B"])]


def _mask_kind(i):
    """Grammar of verify row i: none, a few tokens (inside a literal), almost all (free text)."""
    return ("none", "few", "most", "few")[i % 4]


_FEW, _MOST = 1.0 / 512, 0.97


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _csr(lists, dtype):
    """Offsets and the concatenated columns of per-request tuples of arrays, on the GPU."""
    off = np.zeros(len(lists) + 1, np.int32)
    off[1:] = np.cumsum([len(x[0]) for x in lists])
    cols = [np.concatenate([x[k] for x in lists]).astype(t) for k, t in enumerate(dtype)]
    return tuple(torch.from_numpy(a).cuda() for a in [off] + [c if len(c) else np.zeros(1, c.dtype) for c in cols])


def _prepare_process(case, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    B, K, V, W = case["B"], case["K"], case["V"], case["K"] + 1
    logits = (torch.randn(B, W, V, generator=g, device="cuda") * 3).to(_DTYPES[case["dtype"]])
    cdf = np.cumsum(np.arange(1, V + 1, dtype=np.float64) ** -1.1)
    perm = rng.permutation(V)
    hist, bias = [], []
    for b in range(B):
        tokens = perm[np.minimum(np.searchsorted(cdf / cdf[-1], rng.random(case["history"])), V - 1)]
        ids, counts = np.unique(tokens, return_counts=True)
        counts[rng.random(len(ids)) < 0.25] = 0          # tokens of the prompt alone
        hist.append((ids, counts))
        ids = np.unique(rng.integers(0, V, case["bias"]))
        values = rng.normal(0, 4, len(ids))
        values[rng.random(len(ids)) < 0.1] = -np.inf     # banned tokens
        bias.append((ids, values))
    n_bias = sum(len(x[0]) for x in bias)
    hist = _csr(hist, (np.int32, np.int32))
    bias = _csr(bias, (np.int32, np.float32))
    drafts = rng.integers(0, V, (B, max(K, 1)))
    repeated = rng.random(drafts.shape) < 0.3            # drafts repeat the history's frequent tokens
    drafts[repeated] = perm[rng.integers(0, 20, int(repeated.sum()))]
    nd = _num_drafts(case)
    rows = np.zeros(B, np.dtype([("repetition", "f4"), ("presence", "f4"), ("frequency", "f4"), ("drafts", "i4")]))
    rows["repetition"] = rng.choice([1.0, 1.1, 1.3], B)
    rows["presence"] = rng.choice([0.0, 0.2, 0.5], B)
    rows["frequency"] = rng.choice([0.0, 0.2, 0.3], B)
    rows["drafts"] = nd
    mask = mask_rows = None
    if case["grammar"]:
        kinds = [_mask_kind(i + 1) for i in range(B * W)]
        index = np.full(B * W, -1, np.int32)
        used = [i for i, k in enumerate(kinds) if k != "none"]
        index[used] = np.arange(len(used))
        words = (V + 31) // 32
        share = torch.tensor([_FEW if kinds[i] == "few" else _MOST for i in used], device="cuda")
        if case["ragged"] and len(used) > 1:
            share[1] = 0.0                               # a grammar that allows nothing at this position
        bits = torch.rand(len(used), words, 32, generator=g, device="cuda") < share[:, None, None]
        place = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
        packed = (bits * place).sum(-1)
        mask = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
        mask_rows = torch.from_numpy(index).cuda()
    return dict(case=case, logits=logits, hist=hist, bias=bias, n_bias=n_bias, mask=mask, mask_rows=mask_rows,
                drafts=torch.from_numpy(drafts.astype(np.int32)).cuda() if K else None,
                rows=torch.from_numpy(rows.view(np.uint8).copy()).cuda(), out=torch.zeros_like(logits),
                status=torch.zeros(B, dtype=torch.int32, device="cuda"))


def _prepare_top(case, seed):
    R, V, n = case["R"], case["V"], case["n"]
    logits = (torch.randn(R, V, generator=_generator(seed), device="cuda") * 3).to(_DTYPES[case["dtype"]])
    logits[:, V // 2:V // 2 + V // 16] = -math.inf       # tokens a grammar has masked
    return dict(case=case, logits=logits, values=torch.empty(R, n, device="cuda"),
                ids=torch.empty(R, n, dtype=torch.int32, device="cuda"), lse=torch.empty(R, device="cuda"),
                status=torch.empty(R, dtype=torch.int32, device="cuda"))


def _prepare_distill(case, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    R, V, n, T = case["R"], case["V"], case["n"], case["temperature"]
    target_V = case["target_V"] or V
    t2d = subset = None
    if case["target_V"]:
        subset = torch.from_numpy(np.sort(rng.choice(target_V, V, replace=False))).cuda()
        t2d = torch.full((target_V,), -1, dtype=torch.int32, device="cuda")
        t2d[subset] = torch.arange(V, dtype=torch.int32, device="cuda")
    student = torch.empty(R, V, dtype=_DTYPES[case["dtype"]], device="cuda")
    ids = torch.empty(R, n, dtype=torch.int32, device="cuda")
    values = torch.empty(R, n, device="cuda")
    lse = torch.empty(R, device="cuda")
    step = max(1, 200_000_000 // target_V)
    for lo in range(0, R, step):
        hi = min(R, lo + step)
        teacher = torch.randn(hi - lo, target_V, generator=g, device="cuda") * 3
        if subset is not None:
            teacher[:, subset] += 2                      # the frequent tokens a reduced vocabulary keeps
        v, i = torch.topk(teacher, n, dim=-1)
        values[lo:hi], ids[lo:hi] = v, i.to(torch.int32)
        lse[lo:hi] = torch.logsumexp(teacher / T, -1)
        near = teacher if subset is None else teacher[:, subset]
        student[lo:hi] = (near + torch.randn(hi - lo, V, generator=g, device="cuda")).to(student.dtype)
    ids[::5, -1] = -1                                    # a record shorter than the others
    weights = torch.rand(R, generator=g, device="cuda") + 0.5
    if case["masked"]:
        weights[torch.rand(R, generator=g, device="cuda") < case["masked"]] = 0.0   # prompt tokens, padding
    return dict(case=case, student=student, ids=ids, values=values, lse=lse if case["tail"] else None, t2d=t2d,
                weights=weights, upstream=torch.rand(R, generator=g, device="cuda") + 0.5,
                loss=torch.empty(R, device="cuda"), saved=torch.empty(R, 4, device="cuda"),
                grad=None if case["form"] == "forward" else torch.empty_like(student),
                status=torch.empty(R, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    return {"process": _prepare_process, "top": _prepare_top, "distill": _prepare_distill}[case["op"]](case, seed)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if op == "process":
        return _own_process(state) if own else _plain_process(state)
    if op == "top":
        return _own_top(state) if own else _plain_top(state)
    return _own_distill(state) if own else _plain_distill(state)


def _own_process(s):
    _framework().dspark_process_logits(s["logits"], s["rows"], out=s["out"], row_status=s["status"],
                                       draft_ids=s["drafts"], history=s["hist"], bias=s["bias"], mask=s["mask"],
                                       mask_rows=s["mask_rows"])
    return {"logits": s["out"], "status": s["status"]}


def _own_top(s):
    _framework().dspark_top_logits(s["logits"], values=s["values"], ids=s["ids"], lse=s["lse"],
                                   row_status=s["status"], temperature=s["case"]["temperature"])
    return {"values": s["values"], "ids": s["ids"], "lse": s["lse"], "status": s["status"]}


def _own_distill(s):
    c, b = s["case"], _framework()
    given = dict(temperature=c["temperature"], teacher_lse=s["lse"], t2d=s["t2d"], weights=s["weights"],
                 row_status=s["status"])
    if c["form"] == "two_call":
        b.dspark_distill(s["student"], s["ids"], s["values"], loss=s["loss"], saved=s["saved"], **given)
        b.dspark_distill_backward(s["student"], s["ids"], s["values"], saved=s["saved"], grad_loss=s["upstream"],
                                  grad=s["grad"], **given)
    else:
        b.dspark_distill(s["student"], s["ids"], s["values"], loss=s["loss"], grad=s["grad"], **given)
    return {"loss": s["loss"], "status": s["status"]} | ({} if s["grad"] is None else {"grad": s["grad"]})


def _plain_process(s):
    x, (B, W, V) = s["logits"], s["logits"].shape
    rows = s["rows"].view(torch.float32).view(B, 4)
    drafts_of = s["rows"].view(torch.int32).view(B, 4)[:, 3]
    rep, pres, freq = (rows[:, k].view(B, 1, 1) for k in range(3))
    owner = torch.arange(B, device=x.device)
    off, ids, counts = s["hist"]
    at = torch.repeat_interleave(owner, (off[1:] - off[:-1]).long(), output_size=len(ids)), ids.long()
    count = torch.zeros(B, W, V, dtype=torch.int32, device=x.device)
    if W > 1:                                            # draft i counts from position i + 1 on
        j = torch.arange(W - 1, device=x.device)
        count.index_put_((owner[:, None], j + 1, s["drafts"].long()), torch.ones((), dtype=torch.int32, device=x.device))
        count = torch.cumsum(count, 1, dtype=torch.int32)
    seen = torch.zeros(B, V, dtype=torch.bool, device=x.device)
    seen[at] = True
    base = torch.zeros(B, V, dtype=torch.int32, device=x.device)
    base[at] = counts
    count += base[:, None]
    y = x.float()
    y = torch.where(seen[:, None] | (count > 0), torch.where(y > 0, y / rep, y * rep), y)
    y = torch.where(count > 0, y - (freq * count + pres), y)
    off, ids, values = s["bias"]
    total = s["n_bias"]
    at = torch.repeat_interleave(owner, (off[1:] - off[:-1]).long(), output_size=total), ids[:total].long()
    bias = torch.zeros(B, V, device=x.device)
    bias[at] = values[:total]
    y = y + bias[:, None]
    if s["mask"] is not None:
        bit = (s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=x.device)) & 1
        allowed = bit.view(len(s["mask"]), -1)[:, :V].bool()
        which = s["mask_rows"].view(B, W).long()
        y = torch.where((which < 0)[:, :, None] | allowed[which.clamp(min=0)], y, -math.inf)
    active = torch.arange(W, device=x.device) <= drafts_of[:, None]
    return {"logits": torch.where(active[:, :, None], y, 0.0).to(x.dtype), "status": torch.zeros_like(s["status"])}


def _plain_top(s):
    x, n = s["logits"].float(), s["case"]["n"]
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits)          # ordered as the values are
    V = x.shape[-1]
    top = torch.topk(order * (1 << 25) + (V - 1 - torch.arange(V, device=x.device)), n, dim=-1).values
    ids = V - 1 - (top & ((1 << 25) - 1))
    values = x.gather(-1, ids)
    z = x / s["case"]["temperature"]
    m = z.amax(-1, keepdim=True)
    lse = m[:, 0] + torch.exp(z - m).sum(-1).log()
    return {"values": values, "ids": torch.where(values > -math.inf, ids, -1).to(torch.int32), "lse": lse,
            "status": torch.zeros_like(s["status"])}


def _plain_distill(s):
    c, x = s["case"], s["student"]
    (R, V), T = x.shape, c["temperature"]
    ids = s["ids"].long()
    if s["t2d"] is not None:
        ids = torch.where(ids >= 0, s["t2d"].long()[ids.clamp(min=0)], -1)
    valid, at = ids >= 0, torch.where(ids >= 0, ids, V)
    z = torch.where(valid, s["values"].double() / T, -math.inf)
    if s["lse"] is None:
        zmax = z.amax(-1, keepdim=True).clamp(min=-1e30)
        part = torch.exp(z - zmax).sum(-1, keepdim=True)
        logp = z - zmax - torch.log(part)
    else:
        logp = z - s["lse"].double()[:, None]
    p = torch.exp(logp)
    p_rest = (1 - p.sum(-1)).clamp(min=0) if s["lse"] is not None else torch.zeros(R, dtype=torch.float64, device=x.device)
    y = x.float()
    m = y.amax(-1, keepdim=True)
    e = torch.exp((y - m) / T)
    inside = torch.zeros(R, V + 1, dtype=torch.bool, device=x.device).scatter_(1, at, True)[:, :V]
    rest = torch.where(inside, 0.0, e).sum(-1, dtype=torch.float64)
    total = e.sum(-1, dtype=torch.float64)
    y_at = y.gather(1, ids.clamp(min=0)).double()
    logq = (y_at - m.double()) / T - torch.log(total)[:, None]
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(-1)
    tail = (p_rest > 0) & (rest > 0)
    loss = loss + torch.where(tail, p_rest * (torch.log(p_rest) - torch.log(rest / total)), 0.0)
    used = (s["weights"] != 0) & valid.any(-1)
    w = torch.where(used, s["weights"].double(), 0.0)
    out = {"loss": torch.where(used, w * loss, 0.0).float(), "status": torch.zeros_like(s["status"])}
    if c["form"] == "forward":
        return out
    if c["form"] == "two_call":
        w = w * s["upstream"].double()
    mass = p.sum(-1) + p_rest
    scale_in = (w / T * mass / total).float()[:, None]
    scale_out = (w / T * (mass / total - torch.where(tail, p_rest / rest, 0.0))).float()[:, None]
    grad = e * torch.where(inside, scale_in, scale_out)
    put = torch.where(valid, -p * (w / T)[:, None], 0.0).float()
    grad.scatter_add_(1, ids.clamp(min=0), put)
    return out | {"grad": grad.to(x.dtype)}


# ---------------------------------------------------------------- work and exact results
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    V = case["V"]
    if case["op"] == "process":
        W, moved, touched = case["K"] + 1, 0.0, 0.0
        for b, nd in enumerate(_num_drafts(case)):
            for j in range(nd + 1):
                kind = _mask_kind(b * W + j + 1) if case["grammar"] else "none"
                moved += V * size + (V / 8 if kind != "none" else 0)
                # inside a literal only the allowed tokens' 32-byte sectors have to be read
                moved += V * size if kind != "few" else min(V * size, V * _FEW * 32)
                touched += V
            moved += 8 * (case["history"] + case["bias"])
        return {"bytes": moved, "flops": touched}
    if case["op"] == "top":
        return {"bytes": case["R"] * (V * size + 8.0 * case["n"] + 8), "flops": 4.0 * case["R"] * V}
    R = case["R"] * (1 - case["masked"])
    reads = {"forward": 1, "fused": 1, "two_call": 2}[case["form"]]
    writes = 0 if case["form"] == "forward" else 1
    return {"bytes": R * V * size * reads + case["R"] * V * size * writes + case["R"] * (8.0 * case["n"] + 20),
            "flops": 4.0 * R * V * (reads + writes)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"process": _exact_process, "top": _exact_top, "distill": _exact_distill}[case["op"]](s)


def _exact_process(s):
    x = s["logits"].double()
    B, W, V = x.shape
    rows = s["rows"].cpu().numpy().view([("r", "f4"), ("p", "f4"), ("f", "f4"), ("k", "i4")])
    hoff, hids, hcnt = (a.cpu().numpy() for a in s["hist"])
    boff, bids, bval = (a.cpu().numpy() for a in s["bias"])
    drafts = None if s["drafts"] is None else s["drafts"].cpu().numpy()
    out = torch.zeros_like(x)
    for b in range(B):
        r, p, f, k = (float(rows[n][b]) for n in "rpfk")
        for j in range(int(k) + 1):
            counts = dict(zip(hids[hoff[b]:hoff[b + 1]].tolist(), hcnt[hoff[b]:hoff[b + 1]].tolist()))
            for t in [] if drafts is None else drafts[b, :j].tolist():
                counts[t] = counts.get(t, 0) + 1
            row = x[b, j].clone()
            if counts:
                t = torch.tensor(list(counts), device=x.device)
                n = torch.tensor(list(counts.values()), device=x.device, dtype=torch.float64)
                v = row[t]
                v = torch.where(v > 0, v / r, v * r)
                row[t] = torch.where(n > 0, v - (f * n + p), v)
            t = torch.from_numpy(bids[boff[b]:boff[b + 1]]).long().to(x.device)
            row[t] += torch.from_numpy(bval[boff[b]:boff[b + 1]]).double().to(x.device)
            which = -1 if s["mask"] is None else int(s["mask_rows"][b * W + j])
            if which >= 0:
                words = s["mask"][which].cpu().numpy().view(np.uint8)
                keep = np.unpackbits(words, bitorder="little")[:V].astype(bool)
                row[torch.from_numpy(~keep).to(x.device)] = -math.inf
            out[b, j] = row
    return {"logits": out, "status": None}


def _exact_top(s):
    x, n = s["logits"].double(), s["case"]["n"]
    values = torch.empty(len(x), n, dtype=torch.float64, device=x.device)
    lse = torch.empty(len(x), dtype=torch.float64, device=x.device)
    for r in range(len(x)):
        values[r] = torch.sort(x[r], descending=True).values[:n]
        z = x[r] / s["case"]["temperature"]
        lse[r] = torch.log(torch.exp(z - z.max()).sum()) + z.max()
    return {"values": values, "ids": None, "lse": lse, "status": None}


def _exact_distill(s):
    c, T = s["case"], s["case"]["temperature"]
    R, V = s["student"].shape
    if R * V > 700_000_000:
        return None
    loss = torch.zeros(R, dtype=torch.float64, device="cuda")
    grad = None if c["form"] == "forward" else torch.empty(R, V, dtype=torch.float64, device="cuda")
    step = max(1, 100_000_000 // V)
    for lo in range(0, R, step):
        hi = min(R, lo + step)
        z = s["student"][lo:hi].double() / T
        logq = z - z.amax(-1, keepdim=True)
        logq = logq - torch.log(torch.exp(logq).sum(-1, keepdim=True))
        # the teacher's probabilities spread over the student's vocabulary; -inf: not in the record
        logp = torch.full((hi - lo, V + 1), -math.inf, dtype=torch.float64, device="cuda")
        ids = s["ids"][lo:hi].long()
        if s["t2d"] is not None:
            ids = torch.where(ids < 0, ids, s["t2d"][ids.clamp(min=0)].long())
        logp.scatter_(1, torch.where(ids < 0, V, ids), s["values"][lo:hi].double() / T)
        logp = logp[:, :V]
        member = torch.isfinite(logp)
        if s["lse"] is None:
            logp = logp - torch.logsumexp(logp, -1, keepdim=True)
            p = torch.where(member, torch.exp(logp), 0.0)
            left = torch.zeros(hi - lo, 1, dtype=torch.float64, device="cuda")
        else:
            logp = logp - s["lse"][lo:hi, None].double()
            p = torch.where(member, torch.exp(logp), 0.0)
            left = (1 - p.sum(-1, keepdim=True)).clamp(min=0)
        q = torch.exp(logq)
        q_left = torch.where(member, 0.0, q).sum(-1, keepdim=True)
        live = (left > 0) & (q_left > 0)
        kl = torch.where(member & (p > 0), p * (logp - logq), 0.0).sum(-1, keepdim=True)
        kl = kl + torch.where(live, left * torch.log(left / q_left), 0.0)
        w = s["weights"][lo:hi, None].double()
        w = torch.where(member.any(-1, keepdim=True), w, 0.0)
        loss[lo:hi] = torch.where(w != 0, w * kl, 0.0)[:, 0]
        if grad is not None:
            if c["form"] == "two_call":
                w = w * s["upstream"][lo:hi, None].double()
            push = torch.where(member, p, torch.where(live, left / q_left, 0.0) * q)
            grad[lo:hi] = w / T * ((p.sum(-1, keepdim=True) + left) * q - push)
    return {"loss": loss, "status": None} | ({} if grad is None else {"grad": grad})
