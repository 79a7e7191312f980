"""The handle's scratch and the streams that use it: what a queued call still writes is
not handed to another allocation, and what a captured call has stays its graph's."""

from __future__ import annotations

import contextlib

import pytest
import torch

from block_diffusion_speculative_propose_b200 import DFlash, synth, verify_sampled

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, D, BS = 4, 2, 64, 2


@pytest.fixture
def handle():
    cfg = dict(hidden=256, n_layers=1, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D,
               intermediate=256, vocab=1024, n_target_layers=1, block_size=BS,
               mask_token_id=1023, page_size=16, rms_eps=1e-6, rope_theta=1e6)
    h = DFlash(cfg, synth.make_weights(cfg, device=DEV), max_position=64)
    yield h
    h.close()


def inputs(B, W):
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    table = torch.randperm(B * W, generator=g, device=DEV).int().view(B, W)
    seq = torch.full((B,), 16 * W - BS, dtype=torch.int32, device=DEV)
    return rn(B * BS, HQ, D), seq, table, rn(B * W, HKV, 16, D), rn(B * W, HKV, 16, D)


def call(h, kind, args, **kw):
    q, seq, table, kc, vc = args
    if kind == "prefix":
        return h.prefix_attention(q, seq, table, 0, kc, vc, **kw)
    return h.block_attention(q, seq, table, kc, vc, **kw)


class Watch:
    """The byte tensors that torch.empty gave."""

    def __init__(self, monkeypatch):
        self.seen, self.patch, self.empty = [], monkeypatch, torch.empty

    def __enter__(self):
        def watched(*a, **kw):
            t = self.empty(*a, **kw)
            if kw.get("dtype") == torch.uint8:
                self.seen.append((t.data_ptr(), t.numel()))
            return t
        self.patch.setattr(torch, "empty", watched)
        return self

    def __exit__(self, *exc):
        self.patch.setattr(torch, "empty", self.empty)


@pytest.mark.parametrize("kind", ["prefix", "block"])
@pytest.mark.parametrize("how", ["given", "raw", "current"])
def test_scratch_that_grows_while_a_stream_is_busy(handle, monkeypatch, kind, how):
    small, large = inputs(1, 4), inputs(6, 64)
    want = [call(handle, kind, a) for a in (small, large)]
    torch.cuda.synchronize()
    handle.ws.__init__(handle.device)
    call(handle, kind, small)                      # the scratch is the default stream's
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)             # about 0.1 s
    kw = {} if how == "current" else {"stream": side if how == "given" else side.cuda_stream}
    with Watch(monkeypatch) as w:
        w.seen.append((handle.ws.buf.data_ptr(), handle.ws.buf.numel()))
        with torch.cuda.stream(side) if how == "current" else contextlib.nullcontext():
            got = [call(handle, kind, a, **kw) for a in (small, large)]
    assert not side.query()
    for at, n in w.seen:
        taken = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(16)]
        assert all(abs(t.data_ptr() - at) >= n for t in taken)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_captured_on_a_given_stream_has_its_own_scratch(handle, monkeypatch, raw):
    small, large = inputs(1, 4), inputs(6, 64)
    o = call(handle, "prefix", small)
    want = o.clone()
    torch.cuda.synchronize()
    s, other, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with Watch(monkeypatch) as w:
        with torch.cuda.graph(g, stream=s):
            with torch.cuda.stream(other):         # not the one that is captured
                call(handle, "prefix", small, o=o, stream=s.cuda_stream if raw else s)
    held = (handle.ws.buf.data_ptr(), handle.ws.buf.numel())
    assert len(w.seen) == 1 and w.seen[0][0] != held[0]
    call(handle, "prefix", large)                  # the handle's own is replaced
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _, n in (*w.seen, held)
            for _ in range(8)]
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    assert all(bool((t == 255).all()) for t in junk)


@pytest.mark.parametrize("raw", [False, True])
def test_a_verification_captured_on_a_given_stream_has_its_own_scratch(raw):
    B, K, V = 8, 4, 1000
    logits = torch.randn(B, K + 1, V, device=DEV)
    drafts = torch.randint(0, V, (B, K), device=DEV, dtype=torch.int32)
    ua, us = torch.rand(B, K, device=DEV), torch.rand(B, device=DEV)
    temp = torch.ones(B, device=DEV)
    outs = verify_sampled(drafts, logits, ua, us, temperature=temp)
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    s, other, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(other):             # not the one that is captured
            verify_sampled(drafts, logits, ua, us, temperature=temp, out_tokens=outs[0],
                           num_accepted=outs[1], bonus=outs[2],
                           stream=s.cuda_stream if raw else s)
    with torch.cuda.stream(other):                 # whose memory the scratch would be
        junk = [torch.full((512,), 255, dtype=torch.uint8, device=DEV) for _ in range(64)]
    torch.cuda.synchronize()
    for t in outs:
        t.fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(bool((t == 255).all()) for t in junk)
