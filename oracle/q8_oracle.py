"""Restatement of the calls on the 8-bit cache, one (b, l, h) at a time: e4m3 values,
page scales and bounds (bit for bit: fp32 rotation, every operation rounded by itself),
the choice of pages (integers and two roundings to fp32), and attention in float64 over
chunk_oracle's softmax."""
from __future__ import annotations

import numpy as np

from .chunk_oracle import chunk_softmax

MIN_EXP, MAX_EXP, TOP = -40, 40, 448.0


def e4m3_round(v):
    """Values rounded to e4m3 (to nearest, ties to even, saturating at 448)."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), TOP)
    _, e = np.frexp(a)                                   # a = f 2^e, f in [1/2, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, TOP), v)


def e4m3_decode(code):
    """Values of e4m3 codes (uint8); 0x7f and 0xff are not numbers."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v) * np.where(c & 128, -1.0, 1.0)
    return v[np.asarray(code, np.int64)]


def scale_exp(top):
    """The least x with top <= 448 2^x, held to -40 .. 40; -40 for 0."""
    top = float(top)
    if top == 0.0:
        return MIN_EXP
    f, e = np.frexp(top)
    return int(min(MAX_EXP, max(MIN_EXP, e - 9 + (f > 0.875))))


def rope(x, cos, sin):
    """Rows [.., d] by table rows cos, sin [.., d/2]: fp32, each operation rounded by itself."""
    x, cos, sin = (np.asarray(t, np.float32) for t in (x, cos, sin))
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)


def bounds(values):
    """[2, d] least and largest rint(value / 4) of a page's entries (values in units of the scale)."""
    i = np.rint(np.asarray(values, np.float64) / 4)
    return np.stack([i.min(0), i.max(0)])


def page_append(old, old_exp, new):
    """A page's values in units of its scale after `new` rows (fp32) join the `old` ones
    (in units of 2^old_exp), and its exponent."""
    x = scale_exp(np.abs(new).max())
    if len(old):
        x = max(x, old_exp)
        old = e4m3_round(old * 2.0 ** (old_exp - x))
    return np.concatenate([np.reshape(old, (-1, new.shape[1])), e4m3_round(np.asarray(new, np.float64) * 2.0 ** -x)]), x


def pick_pages(q, page_bounds, page_scale, own, n_sel, first, recent):
    """Pages (ascending) of a token whose G query rows are q, own page `own`; page_bounds
    [own + 1, 2, d] integers, page_scale [own + 1]."""
    if own < n_sel:
        return np.arange(own + 1)
    q = np.asarray(q, np.float32)
    a = np.abs(q).max(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(a > 0, np.float32(127) * (np.float32(1) / a), np.float32(0)).astype(np.float32)
    i = np.rint(q * inv[:, None]).astype(np.int64)
    b = np.asarray(page_bounds, np.int64)
    D = np.maximum(i[:, None] * b[None, :, 0], i[:, None] * b[None, :, 1]).sum(-1)          # [G, pages]
    s = (D.astype(np.float32) * np.asarray(page_scale, np.float32)) * a[:, None]
    key = s.max(0).astype(np.float64)
    j = np.arange(own + 1)
    key[(j < first) | (j > own - recent)] = np.inf
    return np.sort(np.lexsort((j, -key))[:n_sel])


def q8_scores(q, K, logm, n0, page_rows, pages=None):
    """Natural-log scores [G, n, N] of q [G, n, d] over the N = n0 + n entries; pages: for
    every token the page numbers it looks at (None: all)."""
    q, K = np.asarray(q, np.float64), np.asarray(K, np.float64)
    G, n, d = q.shape
    s = q @ K.T / np.sqrt(d) + np.asarray(logm, np.float64)
    e = np.arange(len(K))
    see = e[None] <= n0 + np.arange(n)[:, None]
    if pages is not None:
        for t in range(n):
            see[t] &= np.isin(e // page_rows, pages[t])
    return np.where(see, s, -np.inf)


def q8_attn(q, K, V, logm, n0, page_rows, pages=None):
    """(out [G, n, d], base-2 lse [G, n], probabilities [G, n, N])."""
    p, lse = chunk_softmax(q8_scores(q, K, logm, n0, page_rows, pages))
    return p @ np.asarray(V, np.float64), lse, p
