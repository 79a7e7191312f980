"""dflash_sample_tokens and dflash_verify_sampled against the rules in 64 bits.

Tokens and counts are compared exactly.  The kernels hold weights to 2^-45 of
the largest and sum them exactly, so a token can differ from the 64-bit rule
only where u, min_p or top_p lies within about 2^-35 of a border; the seeds
are fixed.  A probability is one division rounded to fp32 of sums that are
exact to 2^-35: 2^-24 relative, plus 2^-45 * V / (sum >= 1) absolute."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from block_diffusion_speculative_propose_b200 import (DFlashError, prepare_proposal_inputs,
                                                      sample_tokens, verify_greedy,
                                                      verify_sampled)
from tests import _sampling as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def lm_logits(rows, V, seed, std=2.0):
    g = rng(seed)
    x = std * torch.randn(rows, V, generator=g, device=DEV)
    few = min(20, V)
    at = torch.randint(0, V, (rows, few), generator=g, device=DEV)
    return x.scatter_add_(1, at, 10 * torch.rand(rows, few, generator=g, device=DEV))


def full(n, v, dt=torch.float32):
    return torch.full((n,), v, dtype=dt, device=DEV)


def settings_of(n, t=None, k=None, p=None, m=None):
    return dict(temperature=None if t is None else full(n, t),
                top_k=None if k is None else full(n, k, torch.int32),
                top_p=None if p is None else full(n, p), min_p=None if m is None else full(n, m))


def check(x, u, **par):
    rows, V = x.shape
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tok, prob = sample_tokens(x, u, return_probs=True, device_error=err, **par)
    torch.cuda.synchronize()
    xs, us = x.cpu().numpy(), u.cpu().numpy()
    host = {k: (None if v is None else v.cpu().numpy()) for k, v in par.items()}
    tok, prob = tok.cpu().numpy(), prob.cpu().numpy()
    empty = False
    for r in range(rows):
        kw = {k: v[r] for k, v in host.items() if v is not None}
        want, p = S.draw(*S.kept(xs[r], **kw), us[r])
        assert tok[r] == want, (r, tok[r], want, kw, us[r])
        assert abs(prob[r] - p) <= 2.0 ** -24 * p + 2.0 ** -45 * V, (r, prob[r], p)
        empty |= want < 0
    assert int(err.item()) == (0x20 if empty else 0)


GRID = [dict(), dict(t=0.0), dict(t=0.7, k=20, p=0.8), dict(k=1), dict(t=1.5, k=50), dict(p=0.9),
        dict(t=1.3, p=0.99), dict(t=0.5, p=0.3), dict(m=0.05), dict(t=2.0, k=1000, p=0.95, m=0.001),
        dict(t=1.0, k=5000), dict(t=1.2, k=3000, p=0.97, m=1e-4), dict(p=0.0), dict(m=1.0),
        dict(t=20.0, p=0.5), dict(t=1e-3, k=7), dict(t=1e30, p=0.25), dict(t=float("nan")),
        dict(t=float("inf"), p=0.5), dict(t=float("inf"), k=9)]


@pytest.mark.parametrize("V", [1, 2, 5, 33, 1000, 1024, 8191, 8193, 32000, 50257, 151936])
@pytest.mark.parametrize("par", GRID, ids=lambda d: "_".join(f"{k}{v}" for k, v in d.items()) or "off")
def test_rules(V, par):
    rows = 5 if V > 20000 else 9
    u = torch.rand(rows, generator=rng(V + 1), device=DEV)
    u[0], u[1] = 0.0, 1.0 - 2.0 ** -24
    check(lm_logits(rows, V, V), u, **settings_of(rows, **par))


@pytest.mark.parametrize("V", [262144, 300001, 393216])
def test_large_vocabularies(V):
    u = torch.rand(2, generator=rng(1), device=DEV)
    for par in (dict(), dict(k=40, p=0.9), dict(t=1.5, p=0.9)):
        check(lm_logits(2, V, V), u, **settings_of(2, **par))


def test_every_row_its_own_settings_and_rows_apart():
    rows, V, ld = 64, 50257, 50304
    g = rng(3)
    buf = torch.full((rows, ld), float("nan"), device=DEV)
    buf[:, :V] = lm_logits(rows, V, 4)
    pick = lambda v, dt=torch.float32: torch.tensor(v, dtype=dt, device=DEV)[  # noqa: E731
        torch.randint(0, len(v), (rows,), generator=g, device=DEV)]
    par = dict(temperature=pick([0.0, 0.4, 1.0, 1.7]), top_k=pick([0, 1, 10, 2000], torch.int32),
               top_p=pick([1.0, 0.9, 0.5]), min_p=pick([0.0, 0.1]))
    u = torch.rand(rows, generator=g, device=DEV)
    check(buf[:, :V], u, **par)
    odd = torch.full((rows, ld + 1), float("nan"), device=DEV)   # rows that start anywhere
    odd[:, :V] = buf[:, :V]
    check(odd[:, :V], u, **par)


def test_bad_values_masks_and_ties():
    V = 20000
    x = lm_logits(16, V, 11)
    inf = float("inf")
    x[0, ::2] = -inf
    x[1] = -inf                       # nothing left
    x[2] = float("nan")
    x[3, 5] = float("nan")
    x[4] = torch.finfo(torch.float32).min
    x[5, 100:] = torch.finfo(torch.float32).min
    x[6, 7] = x[6, 19000] = inf
    x[7] = 1.25                       # all equal
    x[8] = x[8].round()               # many ties
    x[9] = x[9].to(torch.bfloat16).float()
    x[10] = 0.0
    x[10, ::3] = -0.0
    x[11] = -inf
    x[11, V - 1] = -3.0               # one token left
    x[12] *= 1e30
    x[13] *= 1e-30
    x[14] = inf
    x[15, :V // 2] = 1e30             # a plateau far above the rest
    u = torch.rand(16, generator=rng(12), device=DEV)
    for par in GRID:
        check(x, u, **settings_of(16, **par))


def test_u_outside_the_unit_interval():
    x = lm_logits(6, 1000, 21)
    u = torch.tensor([-1.0, 1.0, 2.0, float("nan"), float("inf"), -0.0], device=DEV)
    check(x, u)
    check(x, u, **settings_of(6, k=10))


def test_distribution():
    """Evenly spaced u on one row visit each token as often as its probability says."""
    n, V = 4096, 64
    x = lm_logits(1, V, 31).expand(n, V).contiguous()
    u = (torch.arange(n, device=DEV) + 0.5) / n
    tok = sample_tokens(x, u, **settings_of(n, t=1.2, k=10, p=0.9))
    ids, w = S.kept(x[0].cpu().numpy(), np.float32(1.2), 10, np.float32(0.9))
    got = torch.bincount(tok.long(), minlength=V).cpu().numpy() / n
    want = np.zeros(V)
    want[ids] = w / w.sum()
    assert np.abs(got - want).max() <= 1.0 / n


# ------------------------------------------------------------------ verification
def verify_inputs(B, K, V, seed, likely=0.8):
    g = rng(seed)
    logits = lm_logits(B * (K + 1), V, seed).view(B, K + 1, V)
    hit = torch.rand(B, K, generator=g, device=DEV) < likely
    other = torch.randint(0, V, (B, K), generator=g, device=DEV)
    drafts = torch.where(hit, logits[:, :K].argmax(2), other).to(torch.int32)
    return (drafts, logits, torch.rand(B, K, generator=g, device=DEV),
            torch.rand(B, generator=g, device=DEV))


def check_verify(drafts, logits, ua, us, err_bits=0, **par):
    B = drafts.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, n, bonus = verify_sampled(drafts, logits, ua, us, device_error=err, **par)
    torch.cuda.synchronize()
    host = {k: (None if v is None else v.cpu().numpy()) for k, v in par.items()}
    d, x = drafts.cpu().numpy(), logits.cpu().numpy()
    a, s = ua.cpu().numpy(), us.cpu().numpy()
    for b in range(B):
        kw = {k: v[b] for k, v in host.items() if v is not None}
        want = S.verify(d[b], x[b], a[b], s[b], **kw)
        assert (out[b].cpu().numpy() == want[0]).all(), (b, out[b], want)
        assert int(n[b]) == want[1] and int(bonus[b]) == want[2]
    assert int(err.item()) == err_bits
    return out, n, bonus


@pytest.mark.parametrize("B,K,V", [(1, 15, 151936), (3, 0, 1000), (7, 1, 33), (40, 9, 1024),
                                   (5, 15, 32000), (300, 3, 200), (2, 128, 64)])
@pytest.mark.parametrize("par", [dict(t=0.6, k=20, p=0.95), dict(), dict(t=0.0), dict(p=0.9),
                                 dict(k=1), dict(t=1.4, p=0.97, m=1e-3), dict(k=2000)],
                         ids=lambda d: "_".join(f"{k}{v}" for k, v in d.items()) or "off")
def test_verify_rules(B, K, V, par):
    check_verify(*verify_inputs(B, K, V, seed=B + K), **settings_of(B, **par))


def test_rows_past_32_bits():
    V, ld = 5000, 2 ** 30
    far = torch.empty(2 * ld + V, device=DEV)
    drafts, logits, ua, us = verify_inputs(1, 2, V, 41, likely=1.0)
    ua.zero_()                                    # the last row decides
    rows = far.as_strided((3, V), (ld, 1))
    rows.copy_(logits[0])
    u = torch.rand(3, generator=rng(42), device=DEV)
    for par in (dict(), dict(k=20, p=0.9), dict(p=0.8), dict(t=0.0)):
        check(rows, u, **settings_of(3, **par))
        want = verify_sampled(drafts, logits, ua, us, **settings_of(1, **par))
        got = verify_sampled(drafts, rows.view(1, 3, V), ua, us, **settings_of(1, **par))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_verify_greedy_rows_decide_as_verify_greedy():
    drafts, logits, ua, us = verify_inputs(9, 15, 5000, 2, likely=0.9)
    logits[2, 3] = logits[2, 3].round()
    logits[3, 1, 17] = float("nan")
    got = verify_sampled(drafts, logits, ua, us, temperature=full(9, 0.0))
    for a, b in zip(got, verify_greedy(drafts, logits)):
        assert torch.equal(a, b)


def test_verify_edges():
    B, K, V = 8, 4, 3000
    drafts, logits, ua, us = verify_inputs(B, K, V, 5, likely=1.0)
    logits[0, 0] = -float("inf")                 # nothing to draw from: -1
    logits[1, 0] = -float("inf")
    logits[1, 0, drafts[1, 0].long()] = 2.0      # the draft holds everything
    ua[1, 0] = 1.0
    drafts[2, 0], drafts[3, 1], drafts[4, 2] = -1, V, 2 ** 31 - 1
    ua[5, 0] = float("nan")
    ua[6] = 0.0                                  # accepted wherever it weighs anything
    logits[7, 2, drafts[7, 2].long()] = float("inf")
    for par in (dict(), dict(k=5, p=0.9), dict(p=0.95), dict(t=1.5)):
        check_verify(drafts, logits, ua, us, err_bits=0x20, **settings_of(B, **par))


def test_verify_residual_leaves_the_draft_out():
    """Over even u, refused drafts never come back and the rest keep their shares."""
    n, V = 2048, 50
    x = lm_logits(1, V, 41)
    d = int(x[0].argmax())
    logits = x.view(1, 1, V).expand(n, 2, V).contiguous()
    drafts = torch.full((n, 1), d, dtype=torch.int32, device=DEV)
    us = (torch.arange(n, device=DEV) + 0.5) / n
    out, num, bonus = verify_sampled(drafts, logits, torch.full((n, 1), 0.9999999, device=DEV), us)
    assert int(num.max()) == 0 and not (bonus == d).any()
    w = np.exp(x[0].double().cpu().numpy())
    w[d] = 0
    got = torch.bincount(bonus.long(), minlength=V).cpu().numpy() / n
    assert np.abs(got - w / w.sum()).max() <= 1.0 / n


def test_streams_graphs_and_repeats():
    drafts, logits, ua, us = verify_inputs(33, 7, 40000, 6)
    par = settings_of(33, t=0.9, p=0.9)
    want = verify_sampled(drafts, logits, ua, us, **par)
    x, u = logits.view(-1, 40000), torch.rand(33 * 8, generator=rng(8), device=DEV)
    want_s = sample_tokens(x, u)
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):                           # two calls at once
        for st in sts:
            outs.append((verify_sampled(drafts, logits, ua, us, stream=st, **par),
                         sample_tokens(x, u, stream=st)))
    torch.cuda.synchronize()
    for v, s in outs:
        assert all(torch.equal(a, b) for a, b in zip(v, want)) and torch.equal(s, want_s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v = verify_sampled(drafts, logits, ua, us, **par)
        s = sample_tokens(x, u)
    for _ in range(2):
        for t in (*v, s):
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(v, want)) and torch.equal(s, want_s)


def test_outputs_feed_the_preparation():
    """verify_sampled's outputs in the place of verify_greedy's."""
    B, K, V = 6, 3, 2000
    drafts, logits, ua, us = verify_inputs(B, K, V, 7)
    out, n, bonus = verify_sampled(drafts, logits, ua, us, temperature=full(B, 0.8))
    start = torch.arange(B, device=DEV) * 10 + 5
    pos = (start[:, None] + torch.arange(K + 1, device=DEV)).reshape(-1)
    last = (torch.arange(B, device=DEV, dtype=torch.int32) + 1) * (K + 1) - 1
    table = torch.arange(B * 8, dtype=torch.int32, device=DEV).view(B, 8)
    nd = torch.full((B,), K, dtype=torch.int32, device=DEV)
    _, _, seq, b2 = prepare_proposal_inputs(pos, last, out, nd, table, 16, V)
    assert torch.equal(b2, bonus) and torch.equal(seq.long(), start + n.long() + 1)


def test_refusals():
    x, u = lm_logits(4, 100, 1), torch.rand(4, device=DEV)
    assert sample_tokens(x[:0], u[:0]).numel() == 0
    for bad in (lambda: sample_tokens(x.half(), u), lambda: sample_tokens(x, u.double()),
                lambda: sample_tokens(x, u[:3]), lambda: sample_tokens(x, u, top_k=full(4, 1.0)),
                lambda: sample_tokens(x, u, temperature=full(3, 1.0)),
                lambda: sample_tokens(x.t().contiguous().t(), u),
                lambda: sample_tokens(x, u, tokens=torch.empty(3, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(DFlashError):
        sample_tokens(x[:1].expand(4, 100), u)                     # rows on top of each other
    with pytest.raises(DFlashError):
        sample_tokens(torch.empty(1, 393217, device=DEV), u[:1])
    drafts, logits, ua, us = verify_inputs(3, 2, 100, 1)
    for bad in (lambda: verify_sampled(drafts.long(), logits, ua, us),
                lambda: verify_sampled(drafts[:, :1], logits, ua, us),
                lambda: verify_sampled(drafts, logits, ua, us[:2]),
                lambda: verify_sampled(drafts, logits.transpose(0, 1).contiguous().transpose(0, 1),
                                       ua, us)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(DFlashError):
        verify_sampled(drafts, logits, ua, us, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("raw", [False, True])
def test_verify_keeps_its_scratch_while_another_stream_runs(monkeypatch, raw):
    """The scratch of a call on a given stream is not handed to the next
    allocation before that stream has passed the call."""
    B, K, V = 8, 4, 1000
    logits = torch.randn(B, K + 1, V, device=DEV)
    drafts = torch.randint(0, V, (B, K), device=DEV, dtype=torch.int32)
    ua, us = torch.rand(B, K, device=DEV), torch.rand(B, device=DEV)
    temp = torch.ones(B, device=DEV)
    want = verify_sampled(drafts, logits, ua, us, temperature=temp)
    torch.cuda.synchronize()
    scratch, empty = [], torch.empty

    def watched(*a, **kw):
        t = empty(*a, **kw)
        if kw.get("dtype") == torch.uint8:
            scratch.append((t.data_ptr(), t.numel()))
        return t

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)           # about 0.1 s
    monkeypatch.setattr(torch, "empty", watched)
    got = verify_sampled(drafts, logits, ua, us, temperature=temp,
                         stream=side.cuda_stream if raw else side)
    monkeypatch.setattr(torch, "empty", empty)
    assert not side.query() and len(scratch) == 1
    taken = [torch.empty(scratch[0][1], dtype=torch.uint8, device=DEV) for _ in range(32)]
    assert scratch[0][0] not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_tensors_of_another_device_are_refused():
    x, u = torch.randn(2, 50, device=DEV), torch.rand(2, device=DEV)
    for bad in (lambda: sample_tokens(x.cpu(), u), lambda: sample_tokens(x, u.cpu()),
                lambda: sample_tokens(x, u, temperature=full(2, 1.0).cpu()),
                lambda: sample_tokens(x, u, tokens=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
