"""dflash_prefix_attention against softmax(q K^T / sqrt(d)) V in 64 bits.

Tolerance per element, derived: with weights p_k (sum 1) and A = sum p_k |v_k|,
  - each weight is rounded to bf16 once: 2^-8 of itself, so 2^-8 A;
  - a score is an fp32 sum of exact products (|q||k| <= 60 in these tests: off
    by less than 2^-24 * 128 * 60 = 2^-11 before the scale 1/sqrt(d) <= 1/8), the
    exponent one fma (2^-24 of at most 2^7) and ex2 (2^-22): below 2^-13 in all,
    for numerator and denominator: 2^-12 A;
  - each part of the keys leaves its own average in fp16, 2^-11 of itself, and
    the parts' averages add up to at most A: 2^-11 A;
  - the output is rounded to fp16: 2^-11 of itself.
The roundings of different keys are independent, so over a whole output their
2-norm stays below 2^-8 / sqrt(3) of the result's for V without a common part:
3e-3 with the rest."""

from __future__ import annotations

import math

import pytest
import torch

from block_diffusion_speculative_propose_b200 import DFlash, DFlashError, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
_HANDLES = {}


def handle(hq, hkv, d, bs=2):
    key = (hq, hkv, d, bs)
    if key not in _HANDLES:
        cfg = dict(hidden=256, n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                   intermediate=256, vocab=1024, n_target_layers=1, block_size=bs,
                   mask_token_id=1023, page_size=16, rms_eps=1e-6, rope_theta=1e6)
        _HANDLES[key] = DFlash(cfg, synth.make_weights(cfg, device=DEV), max_position=64)
    return _HANDLES[key]


def case(hq, hkv, d, q_len, seq, prefix_pages, width=None, seed=0, fill=float("nan"), spread=1.5):
    """Inputs whose unused slots and pages hold `fill`."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B = len(seq)
    need = max([prefix_pages] + [-(-(s + q_len) // 16) for s in seq])
    W = need if width is None else width
    own = W - prefix_pages
    pages = prefix_pages + B * own + 3
    ids = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((B, W), -5, dtype=torch.int32, device=DEV)     # never read where unused
    kc = torch.full((pages, hkv, 16, d), fill, device=DEV)
    vc = torch.full((pages, hkv, 16, d), fill, device=DEV)
    at = 0
    for j in range(prefix_pages):
        table[0, j] = ids[at]
        at += 1
    for b, s in enumerate(seq):
        for j in range(prefix_pages, -(-(s + q_len) // 16)):
            table[b, j] = ids[at]
            at += 1
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    ends = []
    for j in range(prefix_pages):
        ends.append((int(table[0, j]), 16))
    for b, s in enumerate(seq):
        for j in range(prefix_pages, -(-(s + q_len) // 16)):
            ends.append((int(table[b, j]), min(16, s + q_len - 16 * j)))
    for p, n in ends:
        kc[p, :, :n] = rn(hkv, n, d)
        vc[p, :, :n] = rn(hkv, n, d)
    q = (spread * rn(B * q_len, hq, d)).to(BF)
    return (q, torch.tensor(seq, dtype=torch.int32, device=DEV), table, kc.to(BF), vc.to(BF))


def reference(q, seq, table, prefix_pages, kc, vc, causal):
    """(o, A) in 64 bits."""
    B = seq.shape[0]
    T, hq, d = q.shape[0] // B, q.shape[1], q.shape[2]
    hkv = kc.shape[1]
    G = hq // hkv
    out = torch.zeros(B, T, hq, d, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    for b, s in enumerate(seq.tolist()):
        if s < 0:
            continue
        n = s + T
        row = table[b].clone()
        row[:prefix_pages] = table[0, :prefix_pages]
        pages = row[:-(-n // 16)].long()
        k = kc[pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        v = vc[pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        sc = torch.einsum("thd,hkd->htk", q.view(B, T, hq, d)[b].double(), k) / math.sqrt(d)
        if causal:
            late = torch.arange(n, device=DEV) > s + torch.arange(T, device=DEV)[:, None]
            sc = sc.masked_fill(late, -math.inf)
        p = sc.softmax(-1)
        out[b] = torch.einsum("htk,hkd->thd", p, v)
        mag[b] = torch.einsum("htk,hkd->thd", p, v.abs())
    return out.view(B * T, hq * d), mag.view(B * T, hq * d)


def check(h, q, seq, table, prefix_pages, kc, vc, causal=False, norm=True, **kw):
    o = torch.full((q.shape[0], q.shape[1] * q.shape[2]), 7.0, dtype=torch.float16, device=DEV)
    got = h.prefix_attention(q, seq, table, prefix_pages, kc, vc, causal=causal, o=o, **kw)
    torch.cuda.synchronize()
    assert h.check_device_errors() == 0
    want, mag = reference(q, seq, table, prefix_pages, kc, vc, causal)
    T = q.shape[0] // seq.shape[0]
    real = (seq >= 0).repeat_interleave(T)
    err = (got.double() - want).abs()[real]
    bound = (2.0 ** -11 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * mag * (1 + 2.0 ** -11))[real]
    assert (err <= bound).all(), (float((err / bound).max()), (err > bound).nonzero()[:4].tolist())
    if norm and real.any():
        assert float(err.norm() / want[real].norm()) <= 3e-3
    assert (got[~real] == 7.0).all()
    return got


SHAPES = [(32, 8, 128), (4, 2, 64), (8, 1, 128), (5, 1, 64), (10, 2, 128), (3, 3, 128), (2, 2, 64)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("q_len", [1, 2, 7, 16])
@pytest.mark.parametrize("causal", [False, True])
def test_prefix_and_own_keys(hq, hkv, d, q_len, causal):
    h = handle(hq, hkv, d)
    for prefix_pages, lo, B in ((0, 0, 3), (1, 16, 1), (3, 48, 5), (9, 150, 9), (40, 640, 33)):
        seq = [lo + 11 * b % 90 for b in range(B)]
        check(h, *_with(case(hq, hkv, d, q_len, seq, prefix_pages, seed=B), prefix_pages),
              causal=causal)


def _with(c, prefix_pages):
    q, seq, table, kc, vc = c
    return q, seq, table, prefix_pages, kc, vc


@pytest.mark.parametrize("hq,hkv,d,q_len", [(32, 8, 128, 32), (4, 2, 64, 64), (5, 1, 128, 25),
                                            (2, 2, 64, 64), (16, 2, 64, 16)])
def test_whole_row_tiles(hq, hkv, d, q_len):
    for causal in (False, True):
        check(handle(hq, hkv, d),
              *_with(case(hq, hkv, d, q_len, [70, 64, 101], 4, seed=q_len), 4), causal=causal)


@pytest.mark.parametrize("causal", [False, True])
def test_requests_that_end_inside_the_prefix(causal):
    h = handle(32, 8, 128)
    seq = [0, 1, 5, 30, 31, 32, 100, 127, 128, 129, 200]
    for q_len in (1, 4):
        check(h, *_with(case(32, 8, 128, q_len, seq, 8, seed=3), 8), causal=causal)
    # only the first rows see anything of the last tiles
    check(h, *_with(case(32, 8, 128, 3, [2] * 40 + [500], 32, seed=4), 32), causal=causal)


def test_no_prefix_and_the_first_token():
    h = handle(4, 2, 64)
    check(h, *_with(case(4, 2, 64, 1, [0], 0), 0))
    check(h, *_with(case(4, 2, 64, 1, [15, 16, 17], 0), 0))
    check(h, *_with(case(4, 2, 64, 1, [0, 3], 1), 1))
    # the table ends with the prefix
    check(h, *_with(case(4, 2, 64, 2, [5, 9, 14], 1, width=1), 1))


def test_long_own_keys_and_wide_tables():
    h = handle(32, 8, 128)
    check(h, *_with(case(32, 8, 128, 2, [3000, 160, 1029], 9, seed=5), 9))
    check(h, *_with(case(32, 8, 128, 1, [9000], 2, width=2000, seed=6), 2))
    check(h, *_with(case(32, 8, 128, 1, [40000], 2400, seed=6), 2400))


def test_pages_past_32_bits_of_a_pool():
    h = handle(32, 8, 128)
    for q_len, B in ((1, 2), (4, 40)):
        q, seq, table, kc, vc = case(32, 8, 128, q_len, [200 + b for b in range(B)], 8, seed=27)
        pages = 2 ** 31 // (8 * 16 * 128) + kc.shape[0]
        big_k = torch.empty(pages, 8, 16, 128, dtype=BF, device=DEV)
        big_v = torch.empty_like(big_k)
        first = pages - kc.shape[0]              # every page past element 2^31
        big_k[first:], big_v[first:] = kc, vc
        moved = torch.where(table >= 0, table + first, table)
        want = h.prefix_attention(q, seq, table, 8, kc, vc, causal=True)
        got = h.prefix_attention(q, seq, moved, 8, big_k, big_v, causal=True)
        assert torch.equal(got, want)
        check(h, q, seq, table, 8, kc, vc, causal=True)
        # a masked value that is not finite is found there too
        last = int(seq[1]) + q_len - 1
        page = int(moved[1, last // 16])
        big_v[page, :, last % 16] = float("nan")
        got = h.prefix_attention(q, seq, moved, 8, big_k, big_v, causal=True)
        exact, mag = reference(q, seq, table, 8, kc, vc, True)
        bound = 2.0 ** -11 * exact.abs() + (2.0 ** -8 + 2.0 ** -10) * mag
        near = ((got.double() - exact).abs() <= bound).view(B, q_len, -1)
        assert near[1, :-1].all()
        assert torch.equal(got.view(B, q_len, -1)[2:], want.view(B, q_len, -1)[2:])
    assert h.check_device_errors() == 0


def test_padding_requests_keep_their_rows():
    h = handle(32, 8, 128)
    c = case(32, 8, 128, 4, [60, 64, 75, 90, 48, 50], 3, seed=7)
    seq = c[1].clone()
    seq[2] = seq[5] = -1
    check(h, c[0], seq, c[2], 3, c[3], c[4])
    seq[:] = -7
    check(h, c[0], seq, c[2], 3, c[3], c[4])


def test_scores_that_grow_and_lie_far_apart():
    """Later keys outgrow the first reference again and again (by up to 2^80 a
    tile); |q||k| is scaled by a power of two in K alone, so scores stay exact."""
    h = handle(32, 8, 128)
    for prefix_pages, q_len, B in ((64, 2, 40), (64, 1, 4), (0, 4, 3)):
        q, seq, table, kc, vc = case(32, 8, 128, q_len, [1100 + b for b in range(B)],
                                     prefix_pages, seed=8, fill=0.0)
        q.zero_()
        q[:, :, 0] = 8.0
        kc.zero_()
        order = torch.cat([table[0, :prefix_pages], table[0, prefix_pages:]]).long()
        kc[:, :, :, 0] = -100.0
        for n, pg in enumerate(order.tolist()):
            if pg >= 0:
                kc[pg, :, :, 0] = float(n) * 2 - 60
        check(h, q, seq, table, prefix_pages, kc, vc, norm=False)


def test_minus_infinity_and_nan_in_keys():
    h = handle(4, 2, 64)
    q, seq, table, kc, vc = case(4, 2, 64, 2, [40, 45], 2, seed=9)
    kc[table[0, 1].long(), 1, 3] = float("nan")          # seen by both requests, kv head 1
    o = h.prefix_attention(q, seq, table, 2, kc, vc).view(4, 4, 64)
    assert o[:, 2:].isnan().all() and o[:, :2].isfinite().all()
    q, seq, table, kc, vc = case(4, 2, 64, 2, [40, 45], 2, seed=9)
    kc[table[1, 2].long(), 0, 14] = float("nan")         # key 46: request 1's last slot
    o = h.prefix_attention(q, seq, table, 2, kc, vc, causal=True).view(2, 2, 4, 64)
    assert o[0].isfinite().all() and o[1, 0].isfinite().all() and o[1, 1, :2].isnan().all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (5, 1, 64), (8, 1, 128)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(value, hq, hkv, d):
    h = handle(hq, hkv, d)
    # the last position of a causal block, in one kv head
    q, seq, table, kc, vc = case(hq, hkv, d, 4, [40, 45, 61], 2, seed=25)
    clean = check(h, q, seq, table, 2, kc, vc, causal=True)
    vc[table[1, 3].long(), 0, 0, 5] = value              # key 48: the last of request 1
    o = h.prefix_attention(q, seq, table, 2, kc, vc, causal=True)
    G = hq // hkv
    hit = torch.zeros(12, hq, d, dtype=torch.bool, device=DEV)
    hit[7, :G, 5] = True
    assert not o.view(12, hq, d)[hit].isfinite().any()
    # rows that do not see it: right within the same bounds; other requests: the same bits
    rest = ~hit.view(12, -1)
    vc[table[1, 3].long(), 0, 0, 5] = 0.0
    want, mag = reference(q, seq, table, 2, kc, vc, True)
    bound = 2.0 ** -11 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag
    assert ((o.double() - want).abs() <= bound)[rest].all()
    assert torch.equal(o[:4], clean[:4]) and torch.equal(o[8:], clean[8:])
    # requests that end inside the prefix, whose last pages hold nothing yet
    for B, q_len in ((1, 1), (1, 16), (30, 12)):
        seq_l = [100 - 2 * b for b in range(B)]
        q, seq, table, kc, vc = case(hq, hkv, d, q_len, seq_l, 12, seed=26)
        tail = 100 + q_len
        for j in range(tail // 16, 12):
            vc[int(table[0, j]), :, tail - 16 * j if tail > 16 * j else 0:] = value
            kc[int(table[0, j]), :, tail - 16 * j if tail > 16 * j else 0:] = value
        for causal in (False, True):
            check(h, q, seq, table, 12, kc, vc, causal=causal)
    assert h.check_device_errors() == 0


@pytest.mark.parametrize("bs", [4, 16])
def test_agrees_with_block_attention(bs):
    h = handle(32, 8, 128, bs)
    q, seq, table, kc, vc = case(32, 8, 128, bs, [300, 257, 400], 16, seed=10)
    a = check(h, q, seq, table, 16, kc, vc)
    table[1:, :16] = table[0, :16]
    b = h.block_attention(q, seq, table, kc, vc)
    want, mag = reference(q, seq, table, 16, kc, vc, False)
    assert ((a.double() - b.double()).abs() <= 2.0 ** -10 * want.abs() + 2.0 ** -7 * mag).all()
    assert torch.equal(a, h.prefix_attention(q, seq, table, 16, kc, vc))     # same bits again


def test_streams_graph_and_shared_workspace():
    h = handle(32, 8, 128)
    a = _with(case(32, 8, 128, 3, [200, 260, 333] * 8, 12, seed=11), 12)
    b = _with(case(32, 8, 128, 1, [500, 40], 2, seed=12), 2)
    wa, wb = check(h, *a), check(h, *b)
    # two captured graphs over one workspace, replayed in turn
    need = max(h.prefix_attention_workspace_bytes(24, 3, a[2].shape[1], 12),
               h.prefix_attention_workspace_bytes(2, 1, b[2].shape[1], 2))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        h.prefix_attention(*a, o=oa, workspace=ws)
    with torch.cuda.graph(gb):
        h.prefix_attention(*b, o=ob, workspace=ws)
    for _ in range(3):
        oa.zero_(), ob.zero_()
        ga.replay(), gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o = h.prefix_attention(*a, stream=st)
    st.synchronize()
    assert torch.equal(o, wa) and h.check_device_errors() == 0


@pytest.mark.parametrize("B", [2, 40])
def test_parts_past_the_output_type(B):
    """V of one part is past fp16 while the whole is inside it: those rows' parts are
    left in bf16, another 2^-9 of their share of A."""
    h = handle(32, 8, 128)
    q, seq, table, kc, vc = case(32, 8, 128, 4, [300 + b for b in range(B)], 18, seed=B)
    for page in (int(table[0, 17]), int(table[1, 18]), int(table[1, 19])):
        vc[page, :, :, 40] = 90000.0        # shared keys 272.., own keys of request 1
    o = h.prefix_attention(q, seq, table, 18, kc, vc)
    torch.cuda.synchronize()
    want, mag = reference(q, seq, table, 18, kc, vc, False)
    assert float(want.abs().max()) < 65504 and float(want.abs().max()) > 2000
    bound = 2.0 ** -11 * want.abs() + (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11) * 1.01 * mag
    assert ((o.double() - want).abs() <= bound).all()


def test_captured_call_outlives_a_larger_eager_one():
    h = handle(32, 8, 128, 3)               # a handle with no scratch yet
    a = _with(case(32, 8, 128, 1, [40, 50], 2, seed=21), 2)
    o = torch.zeros(2, 32 * 128, dtype=torch.float16, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.prefix_attention(*a, o=o)
    big = _with(case(32, 8, 128, 16, [900] * 40, 50, seed=22), 50)
    want_big = check(h, *big)
    want = check(h, *a)
    for _ in range(2):
        o.zero_()
        g.replay()
        got_big = h.prefix_attention(*big)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(got_big, want_big)


def test_first_request_may_be_padding():
    h = handle(32, 8, 128)
    c = case(32, 8, 128, 2, [60, 64, 75], 3, seed=23)
    seq = c[1].clone()
    seq[0] = -1                              # its table row still names the prefix
    check(h, c[0], seq, c[2], 3, c[3], c[4])


def test_tensor_parallel_shard_has_its_own_heads():
    cfg = dict(hidden=256, n_layers=1, n_q_heads=8, n_kv_heads=4, head_dim=64, intermediate=256,
               vocab=1024, n_target_layers=1, block_size=2, mask_token_id=1023, page_size=16,
               rms_eps=1e-6, rope_theta=1e6)
    h = DFlash(cfg, synth.make_weights(cfg, device=DEV), max_position=512, tp=(1, 2))
    q, seq, table, kc, vc = case(4, 2, 64, 3, [70, 33, 64], 2, seed=24)
    check(h, q, seq, table, 2, kc, vc)
    with pytest.raises(ValueError):
        h.prefix_attention(torch.zeros(9, 8, 64, dtype=BF, device=DEV), seq, table, 2, kc, vc)
    k = torch.randn(5, 2, 64, device=DEV).to(BF)
    slots = torch.arange(5, device=DEV)
    h.append_kv(k, k, slots, slots, kc, vc)
    assert torch.equal(vc[0, :, :5], k.transpose(0, 1))
    h.close()


def test_bad_pages_are_reported_and_not_read():
    h = handle(4, 2, 64)
    q, seq, table, kc, vc = case(4, 2, 64, 1, [40, 45], 2, seed=13, fill=0.0)
    bad = table.clone()
    bad[1, 2] = kc.shape[0]
    h.prefix_attention(q, seq, bad, 2, kc, vc)
    assert h.check_device_errors() == 2
    bad = table.clone()
    bad[0, 1] = -1
    h.prefix_attention(q, seq, bad, 2, kc, vc)
    assert h.check_device_errors() == 2
    seq[1] = 16 * table.shape[1]                # one token past the table
    h.prefix_attention(q, seq, table, 2, kc, vc)
    assert h.check_device_errors() & 4
    seq[1] = 2 ** 31 - 1
    h.prefix_attention(q, seq, table, 2, kc, vc)
    assert h.check_device_errors() & 4
    seq[1] = 45
    check(h, q, seq, table, 2, kc, vc)


def test_refusals():
    h = handle(32, 8, 128)
    q, seq, table, kc, vc = case(32, 8, 128, 2, [40, 45], 2, seed=14)
    o = h.prefix_attention(q[:0], seq[:0], table[:0], 2, kc, vc)
    assert o.shape[0] == 0
    with pytest.raises(ValueError):
        h.prefix_attention(q[:3], seq, table, 2, kc, vc)
    with pytest.raises(ValueError):
        h.prefix_attention(q.half(), seq, table, 2, kc, vc)
    with pytest.raises(ValueError):
        h.prefix_attention(q, seq.long(), table, 2, kc, vc)
    with pytest.raises(ValueError):
        h.prefix_attention(q, seq, table[:1], 2, kc, vc)
    with pytest.raises(ValueError):
        h.prefix_attention(q, seq, table, 2, kc[:, :4].contiguous(), vc)
    with pytest.raises(ValueError):
        h.prefix_attention(q, seq, table, 2, kc, vc, o=torch.empty(3, device=DEV).half())
    for pages in (-1, table.shape[1] + 1):
        with pytest.raises(DFlashError):
            h.prefix_attention(q, seq, table, pages, kc, vc)
    with pytest.raises(DFlashError):
        h.prefix_attention(q, seq, table, 2, kc, vc,
                           workspace=torch.empty(512, dtype=torch.uint8, device=DEV))
    with pytest.raises(DFlashError):             # 33 rows x 4 heads of a kv group
        h.prefix_attention(torch.zeros(66, 32, 128, dtype=BF, device=DEV), seq, table, 2, kc, vc)
    flat = torch.zeros(4 * 4096 + 4, dtype=BF, device=DEV)[4:].view(4, 32, 128)
    with pytest.raises(DFlashError):             # 8-byte aligned only
        h.prefix_attention(flat, seq, table, 2, kc, vc)
    torch.cuda.synchronize()
    assert h.check_device_errors() == 0
