"""Cases of the operators around a draft block at temperature > 0 and over a shared prompt.

    append   DFlash.append_kv          new keys/values (and queries): per-head norm, rotation, paged scatter
    prefix   DFlash.prefix_attention   block attention of a batch whose prompts share their first pages
    sample   sample_tokens             temperature, top-k, min-p, top-p, one draw per row
    verify   verify_sampled            acceptance of greedy drafts against the target's sampled distribution

``run`` computes each in elementary torch operations, or calls the package where
``own`` is true.  All inputs are drawn from the seed alone.
"""

import functools
import math

import numpy as np
import torch

own = False

PAGE = 16
THETA = 1e6
EPS = 1e-6
MAX_POSITION = 65536


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one request, as a target's decode step appends it
        dict(name="append_token", op="append", n=1, hq=32, hkv=8, d=128, q=True, norm=True,
             fused=True, pad=0.0),
        # a verified block of 16 rows for each of 128 requests, some rows padding
        dict(name="append_blocks", op="append", n=2048, hq=32, hkv=8, d=128, q=True, norm=True,
             fused=True, pad=0.1),
        # one long prompt's context rows, keys and values only
        dict(name="append_prompt", op="append", n=32768, hq=32, hkv=8, d=128, q=False,
             norm=False, fused=False, pad=0.0),
        # single tokens of a few requests under one system prompt
        dict(name="prefix_decode", op="prefix", batch=16, q_len=1, causal=False, hq=32, hkv=8,
             d=128, prefix=2048, lo=1, hi=512),
        # draft blocks of 16 slots over a long shared document
        dict(name="prefix_blocks", op="prefix", batch=32, q_len=16, causal=False, hq=32, hkv=8,
             d=128, prefix=8192, lo=128, hi=2048),
        # a full batch's causal verification rows (block 10) over a longer one
        dict(name="prefix_batch", op="prefix", batch=128, q_len=10, causal=True, hq=32, hkv=8,
             d=128, prefix=16384, lo=64, hi=1024),
        # the next token of one request
        dict(name="sample_one", op="sample", rows=1, vocab=151936, temperature=0.7, top_k=20,
             top_p=0.8, min_p=0.0, mixed=False),
        # a serving batch in which every request has its own settings
        dict(name="sample_mixed", op="sample", rows=128, vocab=151936, temperature=1.0, top_k=50,
             top_p=0.95, min_p=0.05, mixed=True),
        # plain sampling at temperature 1 from the whole distribution
        dict(name="sample_plain", op="sample", rows=512, vocab=128256, temperature=1.0, top_k=0,
             top_p=1.0, min_p=0.0, mixed=False),
        # one request's block of 15 drafts
        dict(name="verify_one", op="verify", batch=1, k=15, vocab=151936, temperature=0.6,
             top_k=20, top_p=0.95, min_p=0.0, mixed=False, likely=0.8),
        # blocks of 9 drafts, nucleus only
        dict(name="verify_nucleus", op="verify", batch=32, k=9, vocab=128256, temperature=1.0,
             top_k=0, top_p=0.9, min_p=0.0, mixed=False, likely=0.8),
        # a full batch with settings of every request's own
        dict(name="verify_batch", op="verify", batch=128, k=15, vocab=151936, temperature=0.8,
             top_k=40, top_p=0.95, min_p=0.02, mixed=True, likely=0.85),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sampling(rng):
    return dict(temperature=rng.choice([0.0, 0.3, 0.6, 0.8, 1.0, 1.0, 1.3]),
                top_k=rng.choice([0, 0, 1, 5, 20, 50, 64, 200, 1000, 5000]),
                top_p=rng.choice([1.0, 1.0, 0.99, 0.95, 0.9, 0.7, 0.3]),
                min_p=rng.choice([0.0, 0.0, 0.02, 0.05, 0.2]),
                mixed=rng.random() < 0.4)


def draw(rng):
    op = rng.choice(["append", "prefix", "sample", "verify"])
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, n=_log_int(rng, 1, 16384), hq=hkv * rng.choice([1, 2, 4, 5, 8]),
                    hkv=hkv, d=rng.choice([64, 128]), q=rng.random() < 0.6,
                    norm=rng.random() < 0.5, fused=rng.random() < 0.5,
                    pad=rng.choice([0.0, 0.05, 0.3]))
    if op == "prefix":
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 4, 5, 8])
        q_len = rng.choice([1, 2, 3, 4, 7, 10, 16])
        batch = _log_int(rng, 1, 128)
        prefix = PAGE * _log_int(rng, 1, 1024 if batch <= 64 else 512)
        lo = _log_int(rng, 1, 256)
        return dict(op=op, batch=batch, q_len=min(q_len, 128 // g), causal=rng.random() < 0.4,
                    hq=hkv * g, hkv=hkv, d=rng.choice([64, 128, 128]), prefix=prefix, lo=lo,
                    hi=lo + _log_int(rng, 1, 700))
    vocab = rng.choice([1024, 32000, 50257, 128256, 151936, 151936])
    if op == "sample":
        return dict(op=op, rows=_log_int(rng, 1, 400), vocab=vocab, **_sampling(rng))
    return dict(op=op, batch=_log_int(rng, 1, 64), k=rng.choice([1, 3, 4, 9, 15]), vocab=vocab,
                likely=rng.choice([0.3, 0.7, 0.9]), **_sampling(rng))


# ------------------------------------------------------------------ the inputs
@functools.lru_cache(maxsize=None)
def _handle(hq, hkv, d):
    """The library handle that a program creates once: heads and rotation table."""
    from block_diffusion_speculative_propose_b200 import DFlash, synth
    cfg = dict(hidden=256, n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
               intermediate=256, vocab=1024, n_target_layers=1, block_size=4,
               mask_token_id=1023, page_size=PAGE, rms_eps=EPS, rope_theta=THETA)
    return DFlash(cfg, synth.make_weights(cfg, device="cuda"), max_position=MAX_POSITION)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_append(c, seed):
    g = _generator(seed)
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    dev = "cuda"
    bf = torch.bfloat16
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if c["fused"]:     # slices of one projection output
        qkv = rn(n, hq + 2 * hkv, d).to(bf)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = rn(n, hq, d).to(bf), rn(n, hkv, d).to(bf), rn(n, hkv, d).to(bf)
    pages = -(-n // PAGE) + 3
    # one spare page behind the pool, where the plain form writes its padding rows
    kbuf, vbuf = rn(pages + 1, hkv, PAGE, d).to(bf), rn(pages + 1, hkv, PAGE, d).to(bf)
    slots = torch.randperm(pages * PAGE, generator=g, device=dev)[:n]
    slots = slots.sort().values if seed % 2 else slots
    pad = torch.rand(n, generator=g, device=dev) < c["pad"]
    slots = torch.where(pad, torch.full_like(slots, -1), slots)
    start = torch.randint(0, MAX_POSITION - n + 1, (1,), generator=g, device=dev)
    positions = start + torch.arange(n, device=dev)
    s = dict(op="append", q=q if c["q"] else None, k=k, v=v, kbuf=kbuf, vbuf=vbuf,
             k_cache=kbuf[:pages], v_cache=vbuf[:pages], slots=slots, positions=positions,
             k_norm=(1 + 0.1 * rn(d)).to(bf) if c["norm"] else None,
             q_norm=(1 + 0.1 * rn(d)).to(bf) if c["norm"] and c["q"] else None,
             q_out=rn(n, hq, d).to(bf) if c["q"] else None)
    if own:
        s["h"] = _handle(hq, hkv, d)
    return s


def _prepare_prefix(c, seed):
    g = _generator(seed)
    B, T, hq, hkv, d = c["batch"], c["q_len"], c["hq"], c["hkv"], c["d"]
    dev, bf = "cuda", torch.bfloat16
    P = c["prefix"] // PAGE
    seq = c["prefix"] + torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device=dev)
    width = P + -(-(c["hi"] + T) // PAGE)
    num_pages = P + B * (width - P) + 1
    ids = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    table = torch.empty(B, width, dtype=torch.int32, device=dev)
    table[:, :P] = ids[:P]
    table[:, P:] = ids[P:P + B * (width - P)].view(B, width - P)
    shape = (num_pages, hkv, PAGE, d)
    s = dict(op="prefix", seq=seq.to(torch.int32), table=table, prefix_pages=P, q_len=T,
             causal=c["causal"],
             k_cache=torch.randn(shape, generator=g, device=dev).to(bf),
             v_cache=torch.randn(shape, generator=g, device=dev).to(bf),
             q=(1.5 * torch.randn(B * T, hq, d, generator=g, device=dev)).to(bf))
    if own:
        s["h"] = _handle(hq, hkv, d)
    return s


def _logits(g, rows, vocab):
    """Rows of a language model's logits: a broad bulk and a few raised tokens,
    from near-certain rows to open ones."""
    x = 2.0 * torch.randn(rows, vocab, generator=g, device="cuda")
    few = min(64, vocab)
    at = torch.randint(0, vocab, (rows, few), generator=g, device="cuda")
    peak = 8.0 * torch.rand(rows, 1, generator=g, device="cuda")
    up = 4.0 + peak * torch.rand(rows, few, generator=g, device="cuda")
    return x.scatter_add_(1, at, up)


def _settings(c, n, g):
    """Per-request sampling settings; in a mixed batch every request has its own."""
    dev = "cuda"
    f = lambda v: torch.full((n,), v, dtype=torch.float32, device=dev)  # noqa: E731
    if not c["mixed"]:
        return dict(temperature=f(c["temperature"]), top_p=f(c["top_p"]), min_p=f(c["min_p"]),
                    top_k=torch.full((n,), c["top_k"], dtype=torch.int32, device=dev))
    pick = lambda vals, dt: torch.tensor(vals, dtype=dt, device=dev)[  # noqa: E731
        torch.randint(0, len(vals), (n,), generator=g, device=dev)]
    return dict(temperature=pick([0.0, 0.5, 0.8, 1.0, c["temperature"]], torch.float32),
                top_k=pick([0, 1, 20, c["top_k"], c["top_k"]], torch.int32),
                top_p=pick([1.0, 0.9, c["top_p"], c["top_p"]], torch.float32),
                min_p=pick([0.0, 0.0, c["min_p"]], torch.float32))


def _prepare_sample(c, seed):
    g = _generator(seed)
    return dict(op="sample", logits=_logits(g, c["rows"], c["vocab"]),
                u=torch.rand(c["rows"], generator=g, device="cuda"),
                **_settings(c, c["rows"], g))


def _prepare_verify(c, seed):
    g = _generator(seed)
    B, K, V = c["batch"], c["k"], c["vocab"]
    logits = _logits(g, B * (K + 1), V).view(B, K + 1, V)
    hit = torch.rand(B, K, generator=g, device="cuda") < c["likely"]
    other = torch.randint(0, V, (B, K), generator=g, device="cuda")
    drafts = torch.where(hit, logits[:, :K].argmax(2), other).to(torch.int32)
    return dict(op="verify", logits=logits, drafts=drafts,
                u_accept=torch.rand(B, K, generator=g, device="cuda"),
                u_sample=torch.rand(B, generator=g, device="cuda"), **_settings(c, B, g))


def prepare(case, seed):
    return {"append": _prepare_append, "prefix": _prepare_prefix, "sample": _prepare_sample,
            "verify": _prepare_verify}[case["op"]](case, seed)


# ------------------------------------------------------------- the plain forms
def _rotated(x, w, positions):
    """RMSNorm over the head (with w), then rotation of the pairs (i, i + d/2)."""
    d = x.shape[-1]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    inv = THETA ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
    angle = positions.double()[:, None] * inv
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)


def _append(s):
    if own:
        s["h"].append_kv(s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                         k_norm=s["k_norm"], q=s["q"], q_norm=s["q_norm"], q_out=s["q_out"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], q=s["q_out"])
    pad = s["slots"] < 0
    spare = s["k_cache"].shape[0]
    page = torch.where(pad, spare, s["slots"] // PAGE)
    off = s["slots"] % PAGE
    s["kbuf"][page, :, off] = _rotated(s["k"], s["k_norm"], s["positions"])
    s["vbuf"][page, :, off] = s["v"]
    if s["q"] is not None:
        s["q_out"].copy_(torch.where(pad[:, None, None], s["q_out"],
                                     _rotated(s["q"], s["q_norm"], s["positions"])))
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], q=s["q_out"])


def _prefix(s):
    if own:
        return s["h"].prefix_attention(s["q"], s["seq"], s["table"], s["prefix_pages"],
                                       s["k_cache"], s["v_cache"], causal=s["causal"])
    B, T = s["seq"].shape[0], s["q_len"]
    hkv, d = s["k_cache"].shape[1], s["k_cache"].shape[3]
    G = s["q"].shape[1] // hkv
    keys = s["table"].shape[1] * PAGE
    gather = lambda c: c[s["table"].long()].transpose(1, 2).reshape(B, hkv, keys, d)  # noqa: E731
    q = s["q"].view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d).float()
    sc = q @ gather(s["k_cache"]).float().transpose(2, 3)
    sc *= 1.0 / math.sqrt(d)
    row = torch.arange(T, device=q.device).repeat_interleave(G)
    seen = s["seq"][:, None] + (row + 1 if s["causal"] else torch.full_like(row, T))
    sc.masked_fill_(torch.arange(keys, device=q.device) >= seen[:, None, :, None], -math.inf)
    sc -= sc.amax(-1, keepdim=True)
    sc.exp_()
    o = (sc @ gather(s["v_cache"]).float()) / sc.sum(-1, keepdim=True)
    o = o.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B * T, hkv * G * d)
    return o.to(torch.float16)


def _weights(x, temperature, top_k, top_p, min_p):
    """Unnormalised probabilities in 64 bits after temperature, min-p, top-k and
    top-p, zero where a token is filtered out.  x: [rows, V], settings: [rows]."""
    x = torch.where(x.isnan(), -math.inf, x)
    V = x.shape[1]
    xs, order = x.sort(dim=1, descending=True, stable=True)
    top = xs[:, :1].double()
    t = temperature.double()[:, None]
    greedy = ~(t > 0)
    w = torch.where(xs == top, 1.0, ((xs.double() - top) / torch.where(greedy, 1.0, t)).exp())
    rank = torch.arange(V, device=x.device)
    k = torch.where(greedy, 1, torch.where(top_k[:, None] > 0, top_k[:, None], V))
    first = rank == 0
    keep = (rank < k) & ((w >= min_p.double()[:, None]) | first) & (xs > -math.inf)
    w *= keep
    cum = w.cumsum(1)
    w *= ((cum - w) < top_p.double()[:, None] * cum[:, -1:]) | first
    return torch.zeros_like(w).scatter_(1, order, w)


def _drawn(w, u):
    """The first token whose running sum of w passes u * sum(w); -1 where nothing is left."""
    cum = w.cumsum(1)
    total = cum[:, -1:]
    at = torch.searchsorted(cum, u.double()[:, None] * total, right=True)
    at = at.clamp_max(w.shape[1] - 1)
    prob = (w.gather(1, at) / total)[:, 0]
    empty = total[:, 0] == 0
    return (torch.where(empty, -1, at[:, 0]).to(torch.int32),
            torch.where(empty, 0.0, prob).float())


def _sample(s):
    par = {k: s[k] for k in ("temperature", "top_k", "top_p", "min_p")}
    if own:
        from block_diffusion_speculative_propose_b200 import sample_tokens
        return sample_tokens(s["logits"], s["u"], return_probs=True, **par)
    return _drawn(_weights(s["logits"], **par), s["u"])


def _verify(s):
    par = {k: s[k] for k in ("temperature", "top_k", "top_p", "min_p")}
    if own:
        from block_diffusion_speculative_propose_b200 import verify_sampled
        return verify_sampled(s["drafts"], s["logits"], s["u_accept"], s["u_sample"], **par)
    B, K1, V = s["logits"].shape
    K = K1 - 1
    w = _weights(s["logits"].view(B * K1, V),
                 **{k: v.repeat_interleave(K1) for k, v in par.items()}).view(B, K1, V)
    drafts = s["drafts"].long()
    p = w[:, :K].gather(2, drafts[:, :, None])[:, :, 0] / w[:, :K].sum(2)
    n = (s["u_accept"].double() < p).to(torch.int64).cumprod(1).sum(1)
    last = w.gather(1, n[:, None, None].expand(B, 1, V))[:, 0]
    # a rejected draft's probability is what is left out of the residual
    token = torch.arange(V, device=w.device)
    refused = drafts.gather(1, n.clamp_max(K - 1)[:, None])
    last = torch.where((token == refused) & (n < K)[:, None], 0.0, last)
    bonus = _drawn(last, s["u_sample"])[0]
    slot = torch.arange(K1, device=w.device)
    out = torch.where(slot < n[:, None], torch.nn.functional.pad(s["drafts"], (0, 1)), -1)
    out = torch.where(slot == n[:, None], bonus[:, None], out)
    return out.to(torch.int32), n.to(torch.int32), bonus


def run(state):
    return {"append": _append, "prefix": _prefix, "sample": _sample,
            "verify": _verify}[state["op"]](state)


# -------------------------------------------------------------------- the work
def work(case):
    c = case
    if c["op"] == "append":
        real = c["n"] * (1 - c["pad"])
        heads = 2 * c["hkv"] + (c["hq"] if c["q"] else 0)
        rotated = c["hkv"] + (c["hq"] if c["q"] else 0)
        return dict(bytes=real * (heads * c["d"] * 4 + 8 + c["d"] * 4) + 8 * c["n"],
                    flops=real * rotated * c["d"] * (6 if c["norm"] else 3))
    if c["op"] == "prefix":
        B, T, d = c["batch"], c["q_len"], c["d"]
        own_keys = B * ((c["lo"] + c["hi"]) / 2 + T)
        return dict(bytes=(c["prefix"] + own_keys) * c["hkv"] * d * 4 + B * T * c["hq"] * d * 4,
                    flops=4.0 * T * c["hq"] * d * (B * c["prefix"] + own_keys))
    if c["op"] == "sample":
        rows = c["rows"]
    else:   # the rows behind the first refused draft need not be looked at
        a = c["likely"] * 0.5
        rows = c["batch"] * sum(a ** i for i in range(c["k"] + 1))
    return dict(bytes=rows * c["vocab"] * 4.0, flops=rows * c["vocab"] * 4.0)


# --------------------------------------------------- the definitions in 64 bits
def _exact_append(c, s):
    def head(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        half = x.shape[-1] // 2
        i = torch.arange(half, device=x.device, dtype=torch.float64)
        ang = s["positions"].double()[:, None, None] * torch.exp(-i / half * math.log(THETA))
        z = torch.complex(x[..., :half], x[..., half:]) * torch.polar(torch.ones_like(ang), ang)
        return torch.cat([z.real, z.imag], -1)
    kept = (s["slots"] >= 0).nonzero()[:, 0]
    page, off = s["slots"][kept] // PAGE, s["slots"][kept] % PAGE
    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[page, :, off] = head(s["k"], s["k_norm"])[kept]
    v[page, :, off] = s["v"].double()[kept]
    q = None
    if s["q"] is not None:
        q = s["q_out"].double()
        q[kept] = head(s["q"], s["q_norm"])[kept]
    return dict(k_cache=k, v_cache=v, q=q)


def _exact_prefix(c, s):
    B, T, d, G = c["batch"], c["q_len"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty(B, T, c["hkv"], G, d, dtype=torch.float64, device="cuda")
    q = s["q"].view(B, T, c["hkv"], G, d).double()
    for b, L in enumerate(s["seq"].tolist()):
        pages = s["table"][b, :-(-(L + T) // PAGE)].long()
        k = s["k_cache"][pages].double().transpose(0, 1).reshape(c["hkv"], -1, d)[:, :L + T]
        v = s["v_cache"][pages].double().transpose(0, 1).reshape(c["hkv"], -1, d)[:, :L + T]
        sc = torch.einsum("thgd,hkd->htgk", q[b], k) / d ** 0.5
        if c["causal"]:
            late = torch.arange(L + T, device="cuda") > L + torch.arange(T, device="cuda")[:, None]
            sc = sc.masked_fill(late[None, :, None], -math.inf)
        out[b] = torch.einsum("htgk,hkd->thgd", sc.softmax(-1), v)
    return out.view(B * T, -1)


def _exact_row(x, t, k, p, m):
    """(tokens in the order of the vocabulary, their weights) that one row keeps."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if not len(order):
        return order, x[:0]
    if not t > 0:
        return order[:1], np.ones(1)
    order = order[:k] if k > 0 else order
    w = np.exp((x[order] - x[order[0]]) / t)
    n = max(1, int(np.sum(w >= m)))
    run_ = np.concatenate([[0.0], np.cumsum(w[:n])])
    n = max(1, int(np.sum(run_[:-1] < p * run_[-1])))
    at = np.argsort(order[:n])
    return order[at], w[at]


def _exact_draw(ids, w, u):
    if not len(ids) or w.sum() == 0:
        return -1, 0.0
    cum = np.cumsum(w)
    j = min(int(np.sum(cum <= float(u) * cum[-1])), len(ids) - 1)
    return int(ids[j]), w[j] / cum[-1]


def _exact_settings(s):
    names = ("temperature", "top_k", "top_p", "min_p")
    return list(zip(*[s[n].cpu().numpy().astype(np.float64) for n in names]))


def _exact_sample(c, s):
    if c["rows"] * c["vocab"] > 60e6:
        return None
    u, par = s["u"].cpu().numpy(), _exact_settings(s)
    got = []
    for r in range(c["rows"]):
        t, k, p, m = par[r]
        got.append(_exact_draw(*_exact_row(s["logits"][r].cpu().numpy(), t, int(k), p, m), u[r]))
    tokens = torch.tensor([a for a, _ in got], dtype=torch.int32)
    return tokens, torch.tensor([b for _, b in got], dtype=torch.float64)


def _exact_verify(c, s):
    B, K = c["batch"], c["k"]
    if B * c["vocab"] > 6e6:
        return None
    par, drafts = _exact_settings(s), s["drafts"].cpu().numpy()
    ua, us = s["u_accept"].cpu().numpy(), s["u_sample"].cpu().numpy()
    out, num, bonus = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        t, k, p, m = par[b]
        for i in range(K + 1):
            ids, w = _exact_row(s["logits"][b, i].cpu().numpy(), t, int(k), p, m)
            if i < K:
                hit = ids == drafts[b, i]
                if len(ids) and float(ua[b, i]) < w[hit].sum() / w.sum():
                    out[b, i] = drafts[b, i]
                    continue
                ids, w = ids[~hit], w[~hit]
            num[b], bonus[b] = i, _exact_draw(ids, w, us[b])[0]
            out[b, i] = bonus[b]
            break
    return tuple(torch.from_numpy(a) for a in (out, num, bonus))


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "prefix": _exact_prefix, "sample": _exact_sample,
            "verify": _exact_verify}[case["op"]](case, s)
