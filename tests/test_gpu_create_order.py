"""A handle is built of its weights as the work that was queued before leaves them, on
whichever stream that is."""

from __future__ import annotations

import contextlib

import pytest
import torch

from block_diffusion_speculative_propose_b200 import DFlash, TargetModel, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def each(W, f):
    return {k: [f(x) for x in v] if isinstance(v, list) else f(v) for k, v in W.items()}


@contextlib.contextmanager
def queued(W, where):
    """Weights whose values are still being written: zeros now, `W` a while later."""
    late = each(W, torch.zeros_like)
    torch.cuda.synchronize()
    st = torch.cuda.Stream() if where == "side" else torch.cuda.current_stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(400_000_000)             # about 0.2 s
        for k, v in W.items():
            for a, b in zip(late[k], v) if isinstance(v, list) else ((late[k], v),):
                a.copy_(b, non_blocking=True)
    assert not st.query()
    yield late
    torch.cuda.synchronize()


@pytest.mark.parametrize("where", ["current", "side"])
def test_draft(where):
    cfg = synth.model_config("tiny")
    W = synth.make_weights(cfg, device=DEV)
    L, bs, V = cfg["n_layers"], cfg["block_size"], cfg["vocab"]
    shape = (4, cfg["n_kv_heads"], 16, cfg["head_dim"])
    aux = torch.randn(20, cfg["n_target_layers"] * cfg["hidden"], device=DEV).bfloat16()
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)

    def logits(h):
        kc, vc = ([torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(L)]
                  for _ in range(2))
        at = torch.arange(20, device=DEV)
        h.inject_context(aux, at, at, kc, vc)
        out = torch.empty(bs - 1, V, device=DEV)
        h.propose(torch.tensor([3], dtype=torch.int32, device=DEV),
                  torch.tensor([20], dtype=torch.int32, device=DEV), table, kc, vc, logits_out=out)
        torch.cuda.synchronize()
        h.close()
        return out

    want = logits(DFlash(cfg, W, max_position=128))
    assert want.abs().max() > 0
    with queued(W, where) as late:
        h = DFlash(cfg, late, max_position=128)
    assert torch.equal(logits(h), want)


@pytest.mark.parametrize("where", ["current", "side"])
def test_target(where):
    tcfg = synth.target_config(synth.model_config("tiny"), 2)
    W = synth.make_target_weights(tcfg, device=DEV)
    tokens = torch.tensor([5, 17, 2, 40], dtype=torch.int32, device=DEV)

    def logits(t):
        out = t.forward(tokens, 0)[0]
        torch.cuda.synchronize()
        t.close()
        return out

    want = logits(TargetModel(tcfg, W, [], 64))
    assert want.abs().max() > 0
    with queued(W, where) as late:
        t = TargetModel(tcfg, late, [], 64)
    assert torch.equal(logits(t), want)
