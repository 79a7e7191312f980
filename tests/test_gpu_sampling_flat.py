"""Rows whose filters end in the bulk of the vocabulary: flat logits, where top_p
and min_p cut where many tokens weigh nearly the same.

Tokens are compared exactly with the rules in 64 bits (tests/_sampling.py), under
the same reservation as in test_gpu_sampling.py; outputs are filled beforehand with
values that no draw gives, so one that is never written shows."""

from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from block_diffusion_speculative_propose_b200 import sample_tokens, verify_sampled
from tests import _sampling as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LIST = 1024                # tokens that the kernels gather for a border
SETTINGS = [*itertools.product((1.0, 1.5, 3.0), (0.02, 0.05), (0.999, 0.9995), (0, 5000)),
            (1.3, 0.05, 0.99, 0), (2.0, 0.2, 0.98, 0),
            *itertools.product((2.0, 3.0), (0.1, 0.15, 0.2, 0.3), (0.9999,), (0,))]
# (temperature, min_p, top_p, top_k)


def flat(rows, V, std, seed, rounded):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = std * torch.randn(rows, V, generator=g, device=DEV)
    return x.to(torch.bfloat16).float() if rounded else x


def tensors(settings):
    t, m, p, k = zip(*settings)
    f = lambda v: torch.tensor(v, device=DEV)  # noqa: E731
    return dict(temperature=f(t), min_p=f(m), top_p=f(p), top_k=f(k).int())


def host(par, r):
    return {k: v[r].item() for k, v in par.items()}


def border_bin(x, temperature, min_p, top_p, **_):
    """(tokens, tokens that min_p leaves) of the bin, of 2047 linear ones over the 31.9
    units of (max - x) / T that weigh anything, in which the top_p of the row ends."""
    ids, _ = S.kept(x, temperature, 0, top_p, min_p)
    scale = np.float32(2047) / (np.float32(31.9) * np.float32(temperature))
    b = np.rint((x.max() - x).astype(np.float64) * scale)
    inside = b == b[ids].max()
    return int(inside.sum()), int(inside[S.kept(x, temperature, 0, 1.0, min_p)[0]].sum())


CASES = pytest.mark.parametrize("V,std,rounded", list(itertools.product(
    (128256, 151936, 262144), (1.0, 2.0), (False, True))))


@CASES
def test_draws(V, std, rounded):
    rows = len(SETTINGS)
    x = flat(rows, V, std, V, rounded)
    g = torch.Generator(device=DEV)
    g.manual_seed(V + 1)
    u = torch.rand(rows, generator=g, device=DEV)
    par = tensors(SETTINGS)
    tok = torch.full((rows,), -77, dtype=torch.int32, device=DEV)
    prob = torch.full((rows,), -7.0, device=DEV)
    sample_tokens(x, u, tokens=tok, probs=prob, **par)
    tok, prob, xs, us = tok.cpu().numpy(), prob.cpu().numpy(), x.cpu().numpy(), u.cpu().numpy()
    reached = 0
    for r in range(rows):
        want, p = S.draw(*S.kept(xs[r], **host(par, r)), us[r])
        assert tok[r] == want, (host(par, r), tok[r], want)
        assert abs(prob[r] - p) <= 2.0 ** -24 * p + 2.0 ** -45 * V, (host(par, r), prob[r], p)
        if SETTINGS[r][3] == 0:
            every, left = border_bin(xs[r], **host(par, r))
            reached += left < LIST - 16 and every > LIST
    # rows in which min_p took so many tokens of the border's bin away that a list has
    # room for what is left but not for all
    assert reached or std > 1 or rounded


@CASES
def test_verify(V, std, rounded):
    B, K = len(SETTINGS), 2
    x = flat(B * (K + 1), V, std, V + 2, rounded).view(B, K + 1, V)
    g = torch.Generator(device=DEV)
    g.manual_seed(V + 3)
    drafts = x[:, :K].argmax(2).int()
    ua = torch.rand(B, K, generator=g, device=DEV)
    ua[::2, 0] = 0.0                       # accepted: the second row decides
    us = torch.rand(B, generator=g, device=DEV)
    par = tensors(SETTINGS)
    out = torch.full((B, K + 1), -77, dtype=torch.int32, device=DEV)
    n, bonus = (torch.full((B,), -77, dtype=torch.int32, device=DEV) for _ in range(2))
    verify_sampled(drafts, x, ua, us, out_tokens=out, num_accepted=n, bonus=bonus, **par)
    out, n, bonus = out.cpu().numpy(), n.cpu().numpy(), bonus.cpu().numpy()
    for b in range(B):
        want = S.verify(drafts[b].cpu().numpy(), x[b].cpu().numpy(), ua[b].cpu().numpy(),
                        us[b].item(), **host(par, b))
        assert (out[b] == want[0]).all() and n[b] == want[1] and bonus[b] == want[2], \
            (host(par, b), out[b], want)
