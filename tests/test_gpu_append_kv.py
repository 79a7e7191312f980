"""dflash_append_kv against the formula in 64 bits, through the C ABI.

Tolerance: the kernel computes in fp32 and rounds once to bf16.  With a', b' the
(normed) pair in 64 bits, the fp32 path (a sum of D squares, rsqrt, two products
by the weight and the rotation, one addition, cos/sin held in fp32) is off by
less than 16 roundings, d = 2^-20 (|a'| + |b'|); the store adds half a bf16 step,
2^-8 of the value.  Values are copied: exact."""

from __future__ import annotations

import pytest
import torch

from block_diffusion_speculative_propose_b200 import DFlash, DFlashError, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
MAXPOS = 4096
EPS, THETA = 1e-6, 1e6


def handle(hq, hkv, d):
    cfg = dict(hidden=256, n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, intermediate=256,
               vocab=1024, n_target_layers=1, block_size=2, mask_token_id=1023, page_size=16,
               rms_eps=EPS, rope_theta=THETA)
    return DFlash(cfg, synth.make_weights(cfg, device=DEV), max_position=MAXPOS)


def formula(x, w, pos):
    """(value, bound) in 64 bits."""
    d = x.shape[-1]
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    inv = THETA ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
    ang = pos.double()[:, None, None] * inv
    a, b = x[..., :d // 2], x[..., d // 2:]
    y = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    slack = 2.0 ** -20 * (a.abs() + b.abs()).repeat(*([1] * (x.dim() - 1)), 2)
    return y, 2.0 ** -8 * (y.abs() + slack) + slack


def inputs(n, hq, hkv, d, seed=0, fused=True, spread=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    qkv = (spread * torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV)).to(BF)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pages = n // 16 + 4
    kc = torch.randn(pages, hkv, 16, d, generator=g, device=DEV).to(BF)
    vc = torch.randn(pages, hkv, 16, d, generator=g, device=DEV).to(BF)
    slots = torch.randperm(pages * 16, generator=g, device=DEV)[:n]
    pos = torch.randint(0, MAXPOS, (n,), generator=g, device=DEV)
    kn = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(BF)
    qn = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(BF)
    return q, k, v, kc, vc, slots, pos, kn, qn


def check(h, q, k, v, kc, vc, slots, pos, kn, qn, good=None, **kw):
    good = (slots >= 0) if good is None else good
    k0, v0 = kc.clone(), vc.clone()
    sentinel = torch.full((k.shape[0], h.cfg["n_q_heads"], h.cfg["head_dim"]), 3.25, dtype=BF,
                          device=DEV) if q is not None else None
    before = None if sentinel is None else sentinel.clone()
    got = h.append_kv(k, v, pos, slots, kc, vc, k_norm=kn, q=q, q_norm=qn, q_out=sentinel, **kw)
    torch.cuda.synchronize()
    page, off = slots[good] // 16, slots[good] % 16
    want, bound = formula(k[good], kn, pos[good])
    assert ((kc[page, :, off].double() - want).abs() <= bound).all()
    assert torch.equal(vc[page, :, off], v[good])
    # every other slot keeps its bits
    k0[page, :, off] = kc[page, :, off]
    v0[page, :, off] = v[good]
    assert torch.equal(k0, kc) and torch.equal(v0, vc)
    if q is not None:
        want, bound = formula(q[good], qn, pos[good])
        assert ((got[good].double() - want).abs() <= bound).all()
        assert torch.equal(got[~good], before[~good])


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64), (5, 1, 128), (3, 3, 64), (1, 1, 128)])
@pytest.mark.parametrize("n", [1, 2, 33, 700])
@pytest.mark.parametrize("norm,with_q,fused", [(True, True, True), (False, True, False),
                                               (True, False, True), (False, False, False)])
def test_against_the_formula(hq, hkv, d, n, norm, with_q, fused):
    h = handle(hq, hkv, d)
    q, k, v, kc, vc, slots, pos, kn, qn = inputs(n, hq, hkv, d, seed=n, fused=fused)
    check(h, q if with_q else None, k, v, kc, vc, slots, pos, kn if norm else None,
          qn if norm and with_q else None)
    assert h.check_device_errors() == 0
    h.close()


def test_many_rows_and_one_norm_only():
    h = handle(32, 8, 128)
    a = inputs(6000, 32, 8, 128, seed=5)
    check(h, *a[:8], None)                       # keys normed, queries not
    a = inputs(6001, 32, 8, 128, seed=6)
    check(h, *a[:7], None, a[8])                 # queries normed, keys not
    h.close()


def test_padding_and_bad_rows_are_skipped():
    h = handle(4, 2, 64)
    q, k, v, kc, vc, slots, pos, kn, qn = inputs(64, 4, 2, 64, seed=9)
    slots[::5] = -1
    pos[5] = -77                                 # never looked at: row 5 is padding
    check(h, q, k, v, kc, vc, slots, pos, kn, qn)
    assert h.check_device_errors() == 0
    good = slots >= 0
    slots[1] = kc.shape[0] * 16                  # one past the pool
    good[1] = False
    check(h, q, k, v, kc, vc, slots, pos, kn, qn, good=good)
    assert h.check_device_errors() == 2
    pos[2], pos[3], pos[4] = MAXPOS, -1, MAXPOS - 1
    good[2] = good[3] = False
    check(h, q, k, v, kc, vc, slots, pos, kn, qn, good=good)
    assert h.check_device_errors() == 2 | 16
    h.close()


def test_zeros_and_infinities_stay_in_their_heads():
    h = handle(4, 2, 64)
    q, k, v, kc, vc, slots, pos, kn, qn = inputs(8, 4, 2, 64, seed=3, fused=False)
    k[0] = 0
    check(h, q, k, v, kc, vc, slots, pos, kn, qn)
    k[1, 0, 3] = float("inf")
    v[2, 1, 5] = float("nan")
    h.append_kv(k, v, pos, slots, kc, vc, k_norm=kn)
    page, off = slots // 16, slots % 16
    got = kc[page, :, off]
    assert not got[1, 0].isfinite().all() and got[1, 1].isfinite().all()
    assert vc[page, :, off][2].isnan().sum() == 1
    h.close()


def test_offsets_past_32_bits():
    """Rows 2^30 elements apart, slots past element 2^31 of the pools."""
    hq, hkv, d, n = 32, 8, 128, 5
    h = handle(hq, hkv, d)
    q, k, v, _, _, _, pos, kn, qn = inputs(n, hq, hkv, d, seed=9, fused=False)
    far = torch.empty((n - 1) * 2 ** 30 + hq * d, dtype=BF, device=DEV)
    rows = lambda x: far.as_strided((n, *x.shape[1:]), (2 ** 30, d, 1))  # noqa: E731
    pages = 2 ** 31 // (hkv * 16 * d) + 40
    kc = torch.empty(pages, hkv, 16, d, dtype=BF, device=DEV)
    vc = torch.empty_like(kc)
    slots = torch.tensor([3, pages * 16 - 1, pages * 16 - 200, 2 ** 31 // (hkv * d), 700], device=DEV)
    page, off = slots // 16, slots % 16
    for x in (k, v):                              # keys far apart, then values
        rows(x).copy_(x)
        h.append_kv(rows(k) if x is k else k, rows(v) if x is v else v, pos, slots, kc, vc,
                    k_norm=kn)
        want, bound = formula(k, kn, pos)
        assert ((kc[page, :, off].double() - want).abs() <= bound).all()
        assert torch.equal(vc[page, :, off], v)
    rows(q).copy_(q)
    got = h.append_kv(k, v, pos, slots, kc, vc, k_norm=kn, q=rows(q), q_norm=qn)
    want, bound = formula(q, qn, pos)
    assert ((got.double() - want).abs() <= bound).all()
    assert h.check_device_errors() == 0
    h.close()


def test_in_place_query_other_stream_and_graph():
    h = handle(8, 2, 128)
    q, k, v, kc, vc, slots, pos, kn, qn = inputs(40, 8, 2, 128, seed=4, fused=False)
    want, bound = formula(q, qn, pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    x = q.clone()
    torch.cuda.current_stream().synchronize()
    out = h.append_kv(k, v, pos, slots, kc, vc, k_norm=kn, q=x, q_norm=qn, q_out=x, stream=st)
    st.synchronize()
    assert out.data_ptr() == x.data_ptr() and ((x.double() - want).abs() <= bound).all()
    g = torch.cuda.CUDAGraph()
    y = torch.zeros_like(q)
    with torch.cuda.graph(g):
        h.append_kv(k, v, pos, slots, kc, vc, k_norm=kn, q=q, q_norm=qn, q_out=y)
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, y)
    wk, bk = formula(k, kn, pos)
    assert ((kc[slots // 16, :, slots % 16].double() - wk).abs() <= bk).all()
    h.close()


def test_refusals():
    h = handle(4, 2, 64)
    q, k, v, kc, vc, slots, pos, kn, qn = inputs(8, 4, 2, 64, fused=False)
    kept = kc.clone()
    h.append_kv(k[:0], v[:0], pos[:0], slots[:0], kc, vc)            # nothing to do
    with pytest.raises(ValueError):
        h.append_kv(k.float(), v, pos, slots, kc, vc)
    with pytest.raises(ValueError):
        h.append_kv(k, v, pos.int(), slots, kc, vc)
    with pytest.raises(ValueError):
        h.append_kv(k, v[:4], pos, slots, kc, vc)
    with pytest.raises(ValueError):
        h.append_kv(k.transpose(1, 2).contiguous().transpose(1, 2), v, pos, slots, kc, vc)
    with pytest.raises(ValueError):
        h.append_kv(k, v, pos, slots, kc[:, :1].contiguous(), vc)
    with pytest.raises(DFlashError):
        h.append_kv(k, v, pos, slots, kc, vc, q_norm=qn)             # a norm without queries
    with pytest.raises(DFlashError):
        h.append_kv(k[:1].expand(8, 2, 64), v, pos, slots, kc, vc)   # rows on top of each other
    odd = torch.empty(8 * 132, dtype=BF, device=DEV).as_strided((8, 2, 64), (132, 64, 1))
    with pytest.raises(DFlashError):
        h.append_kv(odd, v, pos, slots, kc, vc)                      # stride not a multiple of 8
    off = torch.empty(8 * 128 + 4, dtype=BF, device=DEV)[4:].view(8, 2, 64)
    with pytest.raises(DFlashError):
        h.append_kv(k, off, pos, slots, kc, vc)                      # 8-byte aligned only
    wide = torch.empty(8, 6, 64, dtype=BF, device=DEV)
    with pytest.raises(DFlashError):                                 # in place, not packed
        L = __import__("block_diffusion_speculative_propose_b200").lib()
        from block_diffusion_speculative_propose_b200.dflash import _check
        _check(L.dflash_append_kv(h.h, k.data_ptr(), 128, v.data_ptr(), 128, None,
                                  wide.data_ptr(), 6 * 64, None, wide.data_ptr(), pos.data_ptr(),
                                  slots.data_ptr(), 8, kc.data_ptr(), vc.data_ptr(),
                                  kc.shape[0], None), "dflash_append_kv")
    torch.cuda.synchronize()
    assert torch.equal(kept, kc)
    h.close()
