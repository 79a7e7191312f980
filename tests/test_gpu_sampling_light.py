"""A nucleus that ends among tokens which weigh two or three steps of 2^-44.

There a weight's rounding (documented: to 2^-45 of the largest) is a fair part of it,
so the rule is restated on the rounded weights: W = rint(2^44 exp((x - max) / T)), whose
sums are whole numbers.  None of the weights below lies near a half."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from block_diffusion_speculative_propose_b200 import sample_tokens, verify_sampled

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, TIES, KEPT = 393216, 1100, 1090
TOP_P = np.float32(1 - 2.0 ** -24)


def light_row():
    """One heavy token, 10 steps each for some, 3.45 for TIES equal ones of which the
    nucleus keeps KEPT, 2.6 (rounded to 3) for the rest, which it leaves out; in
    vocabulary order the rest, the equal ones, the ten-step ones, the heavy one."""
    rest = 349500
    for _ in range(4):                                   # where the tail passes 1 - top_p
        total = 2 ** 44 + 10 * (V - 1 - TIES - rest) + 3 * (TIES + rest)
        rest = (total - math.ceil(float(TOP_P) * total)) // 3 - (TIES - KEPT)
    x = np.zeros(V, np.float32)
    x[:rest] = math.log(2.6 / 2 ** 44)
    x[rest:rest + TIES] = math.log(3.45 / 2 ** 44)
    x[rest + TIES:V - 1] = math.log(10 / 2 ** 44)
    w = np.rint(np.exp(x.astype(np.float64)) * 2.0 ** 44)
    assert sorted(set(w)) == [3, 10, 2 ** 44]
    order = np.argsort(-x, kind="stable")
    cum = np.cumsum(w[order])                            # whole numbers below 2^53
    n = int(np.sum(cum - w[order] < float(TOP_P) * cum[-1]))
    assert n == V - TIES - rest + KEPT
    kept = np.sort(order[:n])
    return x, kept, w[kept], rest


def test_the_nucleus_ends_at_the_right_tie():
    x, ids, w, rest = light_row()
    cum = np.cumsum(w)
    # the first, the last kept tie, the first behind the ties, the heavy token
    goals = [0.0, 3 * (KEPT - 0.5), 3 * KEPT + 5, 2.0 ** 43]
    u = np.array([g / cum[-1] for g in goals], np.float32)
    want = [int(ids[np.sum(cum <= float(v) * cum[-1])]) for v in u]
    assert want == [rest, rest + KEPT - 1, rest + TIES, V - 1]
    n = len(u)
    logits = torch.from_numpy(x).to(DEV).expand(n, V).contiguous()
    par = dict(top_p=torch.full((n,), float(TOP_P), device=DEV))
    tok = torch.full((n,), -77, dtype=torch.int32, device=DEV)
    prob = torch.full((n,), -7.0, device=DEV)
    sample_tokens(logits, torch.from_numpy(u).to(DEV), tokens=tok, probs=prob, **par)
    assert tok.tolist() == want
    share = np.array([3, 3, 10, 2.0 ** 44]) / cum[-1]
    assert (np.abs(prob.cpu().numpy() - share) <= 2.0 ** -24 * share).all()
    # as the row behind an accepted draft: the same draws
    both = torch.stack([logits, logits], 1)
    drafts = torch.full((n, 1), V - 1, dtype=torch.int32, device=DEV)
    out = torch.full((n, 2), -77, dtype=torch.int32, device=DEV)
    num, bonus = (torch.full((n,), -77, dtype=torch.int32, device=DEV) for _ in range(2))
    verify_sampled(drafts, both, torch.zeros(n, 1, device=DEV), torch.from_numpy(u).to(DEV),
                   out_tokens=out, num_accepted=num, bonus=bonus, **par)
    assert out.tolist() == [[V - 1, t] for t in want]
    assert num.tolist() == [1] * n and bonus.tolist() == want
