"""float64 restatement of the chunk calls: attention of a chunk of new tokens
over one (layer, KV head)'s cache, the attention weight its entries received,
and the eviction by that weight.  One (b, l, h) at a time, entries in index
order (the chunk's own tokens are the last n entries)."""
from __future__ import annotations

import numpy as np

LOG2E = 1.0 / np.log(2.0)


def chunk_scores(q, K, logm, pos, n0, pos_new, softcap=0.0, window=0.0, slopes=None):
    """Natural-log scores [G, n, N] of a chunk's queries q [G, n, d] over the
    n0 + n entries (-inf where token t may not look)."""
    q, K = np.asarray(q, np.float64), np.asarray(K, np.float64)
    G, n, d = q.shape
    s = q @ K.T / np.sqrt(d)
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    s = s + np.asarray(logm, np.float64)
    gap = (float(pos_new) + np.arange(n))[:, None] - np.asarray(pos, np.float64)[None]
    if slopes is not None:
        s = s - np.asarray(slopes, np.float64)[:, None, None] * gap
    see = np.arange(K.shape[0])[None] <= n0 + np.arange(n)[:, None]
    if window > 0:
        see = see & (gap < window)
    return np.where(see, s, -np.inf)


def chunk_softmax(s):
    """(probabilities, base-2 log-sum-exp) of scores over their last axis; a row
    with nothing to see gives zeros and -inf."""
    m = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isinf(m), 0.0, m))
    t = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = ((m + np.log(t)) * LOG2E)[..., 0]
    return p / np.where(t > 0, t, 1.0), lse


def chunk_attn(q, K, V, logm, pos, n0, pos_new, softcap=0.0, window=0.0, slopes=None):
    """(out [G, n, d], base-2 lse [G, n], probabilities [G, n, N])."""
    p, lse = chunk_softmax(chunk_scores(q, K, logm, pos, n0, pos_new, softcap, window, slopes))
    return p @ np.asarray(V, np.float64), lse, p


def chunk_mass(mass, n0, s, lse, decay):
    """decay * mass of the first n0 entries (the chunk's own start from 0) plus the
    weight 2^(s log2 e - lse) of every query row; rows with lse = -inf add nothing."""
    lse = np.asarray(lse, np.float64)
    live = ~np.isinf(lse)
    w = np.exp2(s * LOG2E - np.where(live, lse, 0.0)[..., None])
    out = np.where(live[..., None], w, 0.0).sum((0, 1))
    out[:n0] += decay * np.asarray(mass, np.float64)[:n0]
    return out


def mass_evict(mass, pos, keep, safe_from):
    """(B, holes, movers): the length after the eviction, the evicted entries below
    it and the staying entries at or above it.  Entries with pos >= safe_from stay;
    then the largest mass, ties to the lower index, NaN below everything."""
    mass, pos = np.asarray(mass, np.float64), np.asarray(pos, np.float64)
    n = len(mass)
    safe = pos >= safe_from
    B = min(n, max(max(0, int(keep)), int(safe.sum())))
    nan = np.isnan(mass)
    order = np.lexsort((np.arange(n), -np.where(nan, -np.inf, mass), nan, ~safe))
    stays = np.zeros(n, bool)
    stays[order[:B]] = True
    i = np.arange(n)
    return B, i[(i < B) & ~stays], i[(i >= B) & stays]
