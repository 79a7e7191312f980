"""The sampling rules in 64 bits, row by row (numpy), for the tests of
dflash_sample_tokens and dflash_verify_sampled."""

from __future__ import annotations

import numpy as np


def kept(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(ids in vocabulary order, their weights) that the row keeps."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if not len(order):
        return order, np.zeros(0)
    if not temperature > 0:
        return order[:1], np.ones(1)
    if 0 < top_k < len(order):
        order = order[:top_k]
    m = x[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == m, 1.0, np.exp((x[order] - m) / float(temperature)))
    w[np.isnan(w)] = 0.0        # infinitely far below, at an infinite temperature
    if min_p > 0:
        ok = w >= float(min_p)
        ok[0] = True
        order, w = order[ok], w[ok]
    if top_p < 1:
        cum = np.cumsum(w)
        ok = (cum - w) < max(float(top_p), 0.0) * cum[-1]
        ok[0] = True
        order, w = order[ok], w[ok]
    at = np.argsort(order)
    return order[at], w[at]


def unit(u):
    u = float(np.float32(u))
    return min(u, 1.0 - 2.0 ** -24) if u > 0 else 0.0


def draw(ids, w, u):
    if not len(ids) or not w.sum() > 0:
        return -1, 0.0
    cum = np.cumsum(w)
    j = min(int(np.sum(cum <= unit(u) * cum[-1])), len(ids) - 1)
    return int(ids[j]), float(w[j] / cum[-1])


def verify(drafts, logits, u_accept, u_sample, **settings):
    """One request: (out_tokens, num_accepted, bonus)."""
    K = len(drafts)
    out = np.full(K + 1, -1, np.int64)
    for j in range(K + 1):
        ids, w = kept(logits[j], **settings)
        if j < K:
            hit = ids == drafts[j]
            if len(ids) and hit.any():
                p = w[hit].sum() / w.sum()
                if float(np.float32(u_accept[j])) < p or hit.all():
                    out[j] = drafts[j]
                    continue
            ids, w = ids[~hit], w[~hit]
        out[j] = draw(ids, w, u_sample)[0]
        return out, j, out[j]
