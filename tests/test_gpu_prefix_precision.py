"""dflash_prefix_attention holds weights and partial results to the precision of
dflash_block_attention.

Bound per element, derived: with weights p_k (sum 1) and A = sum p_k |v_k|,
  - a weight is the sum of two bf16: the first leaves 2^-8 of it, the second 2^-8 of
    that: 2^-16 A;
  - scores and exponents: 2^-12 A (as in test_gpu_prefix_attention.py);
  - a sum over n <= 4096 keys in fp32 makes 2 n / 16 additions of products, each off by
    2^-23 of what is summed so far: 2^-14 A; joining parts is far below that;
  - the output is rounded to fp16: 2^-11 of itself, 2^-25 where it is subnormal.
Over a whole output the last dominates: a rounding is even within a step, whose width is
between 2^-11 and 2^-10 of the value, so its 2-norm stays below 2^-10 / sqrt(12) of the
result's, 2.82e-4; 3e-4 with the rest, whose roundings are independent too."""

from __future__ import annotations

import pytest
import torch

from tests.test_gpu_prefix_attention import case, handle, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("hq,hkv,d,q_len", [(32, 8, 128, 1), (32, 8, 128, 16), (8, 2, 64, 5),
                                            (5, 1, 128, 3), (4, 4, 64, 40)])
@pytest.mark.parametrize("prefix_pages,own,B", [(0, 300, 4), (9, 150, 3), (64, 40, 40),
                                                (20, 1500, 8), (100, 0, 5)])
def test_against_64_bits(hq, hkv, d, q_len, prefix_pages, own, B, causal):
    h = handle(hq, hkv, d)
    seq = [16 * prefix_pages + own * (b + 1) // B for b in range(B)]
    q, seq, table, kc, vc = case(hq, hkv, d, q_len, seq, prefix_pages, seed=31)
    got = h.prefix_attention(q, seq, table, prefix_pages, kc, vc, causal=causal).double()
    want, mag = reference(q, seq, table, prefix_pages, kc, vc, causal)
    err = (got - want).abs()
    bound = 2.0 ** -11 * want.abs() + 2.0 ** -25 + (2.0 ** -12 + 2.0 ** -14 + 2.0 ** -16) * mag
    assert (err <= bound).all(), float((err / bound).max())
    assert float(err.norm() / want.norm()) <= 3e-4
    assert h.check_device_errors() == 0


def test_weights_far_above_the_first_keys_lose_nothing():
    """The reference of a row is the first maximum that it meets: later weights of up to
    2^32 are held in two halves like the others."""
    h = handle(32, 8, 128)
    q, seq, table, kc, vc = case(32, 8, 128, 2, [500, 700, 900], 16, seed=32)
    for b in range(3):
        for j in range(16, -(-(int(seq[b]) + 2) // 16)):
            kc[table[b, j]] *= 1.0 + 0.02 * j
    got = h.prefix_attention(q, seq, table, 16, kc, vc).double()
    want, _ = reference(q, seq, table, 16, kc, vc, False)
    assert float((got - want).norm() / want.norm()) <= 3e-4
