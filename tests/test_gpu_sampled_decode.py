"""The operators around a sampled draft block run together, as a decode loop runs
them: a batch whose requests share a prompt has its prompt appended once, then
every step appends the block's keys and values, attends (shared prefix, causal
block), and verifies the drafts against the target's sampled distribution; what
was accepted moves each request on.

The target here is one attention layer between random tables.  Every step's
outputs are checked against the rules in 64 bits on the very tensors the step
saw, and a greedy run emits what plain greedy decoding of the same target does."""

from __future__ import annotations

import pytest
import torch

from block_diffusion_speculative_propose_b200 import (DFlash, paged_slots, sample_tokens, synth,
                                                      verify_greedy, verify_sampled)
from tests import _sampling as S
from tests.test_gpu_append_kv import formula
from tests.test_gpu_prefix_attention import reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
HQ, HKV, D, H, V = 8, 2, 64, 256, 512


class Loop:
    """The batch, its pools and its one-layer target."""

    def __init__(self, B, K, prompt, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        cfg = dict(hidden=H, n_layers=1, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D,
                   intermediate=256, vocab=1024, n_target_layers=1, block_size=K + 1,
                   mask_token_id=1023, page_size=16, rms_eps=1e-6, rope_theta=1e6)
        self.h = DFlash(cfg, synth.make_weights(cfg, device=DEV), max_position=1024)
        self.B, self.K = B, K
        self.embed, self.wqkv = rn(V, H), rn(H, (HQ + 2 * HKV) * D) / 16
        self.head = rn(HQ * D, V) / 8
        self.kn, self.qn = (1 + 0.1 * rn(D)).to(BF), (1 + 0.1 * rn(D)).to(BF)
        self.prefix_pages = prompt // 16
        own = 12
        pages = self.prefix_pages + B * own
        ids = torch.randperm(pages, generator=g, device=DEV).int()
        self.table = torch.empty(B, self.prefix_pages + own, dtype=torch.int32, device=DEV)
        self.table[:, :self.prefix_pages] = ids[:self.prefix_pages]
        self.table[:, self.prefix_pages:] = ids[self.prefix_pages:].view(B, own)
        shape = (pages, HKV, 16, D)
        self.kc = torch.full(shape, float("nan"), dtype=BF, device=DEV)
        self.vc = torch.full(shape, float("nan"), dtype=BF, device=DEV)
        self.prompt = torch.randint(0, V, (prompt,), generator=g, device=DEV)
        pos = torch.arange(prompt, device=DEV)
        slots = paged_slots(pos, torch.zeros_like(pos), self.table)
        _, k, v = self.project(self.prompt)
        self.h.append_kv(k, v, pos, slots, self.kc, self.vc, k_norm=self.kn)   # once for all
        self.seq = torch.full((B,), prompt, dtype=torch.int32, device=DEV)

    def project(self, tokens):
        x = (self.embed[tokens] @ self.wqkv).to(BF).view(-1, HQ + 2 * HKV, D)
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def block(self, tokens):
        """Logits [B, T, V] after each of the block's tokens [B, T]."""
        B, T = tokens.shape
        pos = (self.seq.long()[:, None] + torch.arange(T, device=DEV)).reshape(-1)
        req = torch.arange(B, device=DEV).repeat_interleave(T)
        slots = paged_slots(pos, req, self.table)
        q, k, v = self.project(tokens.reshape(-1))
        q = self.h.append_kv(k, v, pos, slots, self.kc, self.vc, k_norm=self.kn, q=q,
                             q_norm=self.qn)
        o = self.h.prefix_attention(q, self.seq, self.table, self.prefix_pages, self.kc, self.vc,
                                    causal=True)
        self.seen = (pos, slots, q, k, v, o, tokens)
        return (o.float() @ self.head).view(B, T, V)

    def check_block(self):
        pos, slots, q, k, v, o, tokens = self.seen
        kept = self.kc[slots // 16, :, slots % 16]
        want, bound = formula(k, self.kn, pos)
        assert ((kept.double() - want).abs() <= bound).all()
        assert torch.equal(self.vc[slots // 16, :, slots % 16], v)
        want, bound = formula(self.project(tokens.reshape(-1))[0], self.qn, pos)
        assert ((q.double() - want).abs() <= bound).all()
        want, mag = reference(q, self.seq, self.table, self.prefix_pages, self.kc, self.vc, True)
        bound = 2.0 ** -11 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag
        assert ((o.double() - want).abs() <= bound).all()
        assert self.h.check_device_errors() == 0


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_sampled_decode_of_a_batch_with_a_shared_prompt(temperature):
    B, K, steps = 5, 3, 6
    L = Loop(B, K, prompt=96, seed=3)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    par = dict(temperature=torch.full((B,), temperature, device=DEV),
               top_k=torch.full((B,), 40, dtype=torch.int32, device=DEV),
               top_p=torch.full((B,), 0.95, device=DEV))
    # the first token: one row a request, from the prompt's last token
    first = L.prompt[-1].expand(B, 1).contiguous()
    L.seq -= 1                                  # its own slot is written again, unchanged
    logits = L.block(first)
    L.check_block()
    L.seq += 1
    u = torch.rand(B, generator=g, device=DEV)
    bonus = sample_tokens(logits[:, 0], u, **par)
    for b in range(B):
        kw = {k: v[b].item() for k, v in par.items()}
        assert int(bonus[b]) == S.draw(*S.kept(logits[b, 0].cpu().numpy(), **kw),
                                       u[b].item())[0]
    emitted = [[int(t)] for t in bonus]
    for _ in range(steps):
        drafts = torch.randint(0, V, (B, K), generator=g, device=DEV, dtype=torch.int32)
        # two requests get the target's own greedy continuation as drafts
        tokens = torch.cat([bonus[:, None], drafts], 1).long()
        for j in range(K):
            guess = L.block(tokens)[:2, j].argmax(1)
            drafts[:2, j], tokens[:2, j + 1] = guess.int(), guess
        logits = L.block(tokens)
        L.check_block()
        ua = torch.rand(B, K, generator=g, device=DEV)
        us = torch.rand(B, generator=g, device=DEV)
        out, n, bonus = verify_sampled(drafts, logits, ua, us, **par)
        if temperature == 0.0:
            for a, b in zip((out, n, bonus), verify_greedy(drafts, logits)):
                assert torch.equal(a, b)
        for b in range(B):
            kw = {k: v[b].item() for k, v in par.items()}
            want = S.verify(drafts[b].cpu().numpy(), logits[b].cpu().numpy(),
                            ua[b].cpu().numpy(), us[b].item(), **kw)
            assert (out[b].cpu().numpy() == want[0]).all() and int(n[b]) == want[1]
            emitted[b] += [int(t) for t in out[b] if int(t) >= 0]
        if temperature == 0.0:
            assert int(n[:2].min()) == K         # its own continuation is accepted whole
        L.seq += n + 1
    # the caches of rejected rows are overwritten by what comes next
    assert all(len(e) == int(s) - 96 + 1 for e, s in zip(emitted, L.seq))
    if temperature == 0.0:
        # plain greedy decoding, one token a step, gives the same tokens
        P = Loop(B, 1, prompt=96, seed=3)
        P.seq -= 1
        tok = P.block(L.prompt[-1].expand(B, 1).contiguous())[:, 0].argmax(1)
        P.seq += 1
        plain, gaps = [[int(t)] for t in tok], []
        for _ in range(max(len(e) for e in emitted) - 1):
            logits = P.block(tok[:, None])[:, 0]
            top = logits.topk(2).values
            gaps.append((top[:, 0] - top[:, 1]) / logits.std(1))
            tok = logits.argmax(1)
            P.seq += 1
            for b in range(B):
                plain[b].append(int(tok[b]))
        # the same tokens, up to where two logits are closer than the roundings
        # of a block and of single tokens (2^-7 of the logits' spread) tell apart
        for b, e in enumerate(emitted):
            apart = [i for i, (x, y) in enumerate(zip(e, plain[b])) if x != y]
            assert not apart or (apart[0] > 0 and float(gaps[apart[0] - 1][b]) < 2.0 ** -7), b
        P.h.close()
    L.h.close()
