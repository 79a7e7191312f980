"""dflash_prefix_attention holds weights and partial results to the precision of
dflash_block_attention.

Bound per element, derived: with weights p_k (sum 1) and A = sum p_k |v_k|,
  - a weight is the sum of two bf16: the first is cut off and leaves 2^-7 of it, the
    second is off by 2^-8 of that, and adds 2^-20: 2^-15 A + 2^-20 A;
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
    bound = 2.0 ** -11 * want.abs() + 2.0 ** -25 + (2.0 ** -12 + 2.0 ** -14 + 2.0 ** -15 + 2.0 ** -20) * mag
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


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("hq,hkv,d,q_len", [(32, 8, 128, 1), (32, 8, 128, 16), (4, 2, 64, 3)])
@pytest.mark.parametrize("key", [5, 70, 200, 255, 256, 300])
def test_an_infinite_value_that_is_seen(hq, hkv, d, q_len, key, value):
    """A key's infinite V is infinite in every row that sees it, in that head and column
    alone (weights are small, equal to 1 and between; none is 0)."""
    h = handle(hq, hkv, d)
    q, seq, table, kc, vc = case(hq, hkv, d, q_len, [300, 330, 350], 16, seed=33, spread=0.3)
    kc[table[0, 0], :, 3] = 0                        # a score of exactly 0
    for b in range(1 if key < 256 else 3):
        vc[table[b, key // 16], hkv - 1, key % 16, 7] = value
    for causal in (False, True):
        got = h.prefix_attention(q, seq, table, 16, kc, vc, causal=causal).double()
        want, _ = reference(q, seq, table, 16, kc, vc, causal)
        inf = want.isinf()
        assert inf.any() and torch.equal(got[inf], want[inf])
        err, fin = (got - want)[~inf].abs(), want[~inf]
        assert float(err.norm() / fin.norm()) <= 3e-4
    # one key: a weight of exactly 1, whose second half is nothing but the addition
    q, seq, table, kc, vc = case(hq, hkv, d, 1, [0, 0], 0, seed=34)
    vc[table[0, 0], 0, 0, 2] = value
    got = h.prefix_attention(q, seq, table, 0, kc, vc).double()
    want, _ = reference(q, seq, table, 0, kc, vc, False)
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got[got.isinf()], want[want.isinf()])
