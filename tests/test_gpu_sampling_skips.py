"""Verification rows that have nothing to say: the rows behind a request's first refusal,
most of which are left out, by clusters that start in large numbers and end at once."""

from __future__ import annotations

import pytest
import torch

from block_diffusion_speculative_propose_b200 import verify_sampled

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("B,K,V", [(300, 31, 64), (64, 128, 9), (1, 128, 5000), (1000, 15, 33)])
@pytest.mark.parametrize("at", [0, 3])
def test_all_rows_behind_a_refusal(B, K, V, at):
    """Drafts are the only token a row has, until a draft that is none: row `at` refuses,
    and what it draws is its only token."""
    only = torch.arange(B * (K + 1), device=DEV).view(B, K + 1) % V
    logits = torch.full((B, K + 1, V), -float("inf"), device=DEV)
    logits.scatter_(2, only[:, :, None], 1.0)
    drafts = only[:, :K].int().contiguous()
    drafts[:, at] = -1
    ua, us = torch.zeros(B, K, device=DEV), torch.rand(B, device=DEV)
    want = torch.full((B, K + 1), -1, dtype=torch.int32, device=DEV)
    want[:, :at + 1] = only[:, :at + 1].int()
    for _ in range(20):
        out = torch.full((B, K + 1), -77, dtype=torch.int32, device=DEV)
        n, bonus = (torch.full((B,), -77, dtype=torch.int32, device=DEV) for _ in range(2))
        verify_sampled(drafts, logits, ua, us, out_tokens=out, num_accepted=n, bonus=bonus)
        assert torch.equal(out, want) and (n == at).all()
        assert torch.equal(bonus, only[:, at].int())
