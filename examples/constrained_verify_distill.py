#!/usr/bin/env python3
"""Constrained speculative decoding with a drafter that learns from what is verified.

Each round, for B requests and K drafted tokens:
  1. the drafter proposes tokens over its reduced vocabulary;
  2. dspark_process_logits turns the target's logits into the distribution to sample from:
     repetition penalty over the history and the drafts so far, biases, a grammar mask for each
     position;
  3. dspark_verify_sample accepts drafts and draws the next token;
  4. dspark_top_logits records the target's largest logits at the verified positions;
  5. the drafter takes a step on the distillation loss of that record, its gradient clipped by
     dspark_clip_grads.

The "models" are one linear head each over given hidden states: there is no network to load.

  python examples/constrained_verify_distill.py [--rounds N]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sample_verify_epilogue_gb300 import binding  # noqa: E402
from sample_verify_epilogue_gb300.distill import distill_loss  # noqa: E402
from sample_verify_epilogue_gb300.training import clip_grads_  # noqa: E402


def run(rounds=30, B=32, K=4, V=32000, draft_V=8000, hidden=16, n=64, seed=0, say=print):
    """Plays the rounds; returns the loss of each, the accepted lengths and whether every emitted token
    was allowed by its grammar."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    W = K + 1
    target_head = torch.randn(hidden, V, generator=g, device=dev)
    subset = torch.sort(torch.randperm(V, generator=g, device=dev)[:draft_V]).values     # the draft vocabulary
    d2t = (subset - torch.arange(draft_V, device=dev)).to(torch.int32)
    t2d = torch.full((V,), -1, dtype=torch.int32, device=dev)
    t2d[subset] = torch.arange(draft_V, dtype=torch.int32, device=dev)
    frequent = torch.zeros(V, device=dev)
    frequent[subset] = 4.0                                                               # the tokens it keeps
    head = (target_head[:, subset] + 0.7 * torch.randn(hidden, draft_V, generator=g, device=dev)).requires_grad_()
    optimizer = torch.optim.Adam([head], lr=0.05)

    process_rows = np.zeros(B, binding.PROCESS_ROW_DTYPE)
    process_rows["repetition_penalty"], process_rows["frequency_penalty"], process_rows["num_drafts"] = 1.1, 0.1, K
    sampling = np.zeros(B, binding.ROW_PARAMS_DTYPE)
    sampling["temperature"], sampling["top_p"], sampling["num_drafts"] = 0.8, 0.95, K

    def packed(rows):
        return torch.from_numpy(rows.view(np.uint8).copy()).to(dev)

    process_rows, sampling = packed(process_rows), packed(sampling)
    history = [torch.zeros(0, dtype=torch.int64, device=dev) for _ in range(B)]
    banned = torch.tensor([7], dtype=torch.int32, device=dev)
    bias = (torch.arange(B + 1, dtype=torch.int32, device=dev), banned.repeat(B), torch.full((B,), -np.inf, device=dev))
    bit = torch.ones((), dtype=torch.int64, device=dev) << torch.arange(32, device=dev)

    def i32(*shape):
        return torch.empty(*shape, dtype=torch.int32, device=dev)

    processed = torch.empty(B, W, V, dtype=torch.bfloat16, device=dev)
    out = {"accept_len": i32(B), "tokens": i32(B, W)}
    status, row_status = i32(B), i32(B, W)
    values, ids, lse = torch.empty(B, W, n, device=dev), i32(B, W, n), torch.empty(B, W, device=dev)
    extras = binding.make_extras(q_layout="reduced", q_row_len=draft_V, d2t=d2t.data_ptr())
    workspace = torch.empty(binding.dspark_workspace_bytes(B, K, V, "bf16", extras=extras), dtype=torch.uint8, device=dev)

    losses, accepted, legal = [], [], True
    for r in range(rounds):
        states = torch.randn(B, W, hidden, generator=g, device=dev)
        logits = (states @ target_head + frequent).to(torch.bfloat16)
        student = states[:, :K] @ head                                     # [B, K, draft_V]
        q = torch.softmax(student.detach(), -1)
        drafts = torch.multinomial(q.view(-1, draft_V), 1, generator=g).view(B, K)
        drafts = subset[drafts].to(torch.int32)

        # the grammar of the moment: one position in two is free, the others allow nine tokens in ten
        allowed = torch.rand(B * W, (V + 31) // 32, 32, generator=g, device=dev) < 0.9
        words = (allowed * bit).sum(-1)
        mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        mask_rows = torch.arange(B * W, dtype=torch.int32, device=dev).view(B, W)
        mask_rows[:, ::2] = -1
        counted = [torch.unique(h, return_counts=True) for h in history]
        offsets = torch.tensor([0] + [len(t) for t, _ in counted], device=dev).cumsum(0).to(torch.int32)
        seen = (offsets, torch.cat([t for t, _ in counted]).to(torch.int32), torch.cat([c for _, c in counted]).to(torch.int32))

        binding.dspark_process_logits(logits, process_rows, out=processed, row_status=status, draft_ids=drafts,
                                      history=seen if r else None, bias=bias, mask=mask, mask_rows=mask_rows)
        binding.dspark_verify_sample(processed, q, drafts, None, sampling, torch.rand(B, W, 2, generator=g, device=dev),
                                     out=out, row_status=status, workspace=workspace, extras=extras)
        binding.dspark_top_logits(logits, values=values, ids=ids, lse=lse, row_status=row_status)
        record = (a[:, :K].contiguous() for a in (ids, values, lse))       # the drafter has K of the K + 1 positions
        loss, _ = distill_loss(student, *record, t2d=t2d)
        optimizer.zero_grad()
        loss.mean().backward()
        clip_grads_([head], 1.0)
        optimizer.step()

        losses.append(float(loss.detach().mean()))
        lengths = out["accept_len"].tolist()
        accepted.append(sum(lengths) / B)
        tokens = out["tokens"].tolist()
        flat = allowed.view(B, W, -1)
        for b in range(B):
            emitted = tokens[b][:lengths[b] + 1]
            legal = legal and lengths[b] >= 0 and all(
                t != 7 and (j % 2 == 0 or bool(flat[b, j, t])) for j, t in enumerate(emitted))
            history[b] = torch.cat([history[b], torch.tensor(emitted, device=dev)])
        say(f"round {r:2d}: loss {losses[-1]:.4f}, {accepted[-1]:.2f} of {K} drafts accepted")
    return losses, accepted, legal


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=30)
    losses, _, legal = run(ap.parse_args().rounds)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; every emitted token legal: {legal}")


if __name__ == "__main__":
    main()
