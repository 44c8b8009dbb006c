"""kvc_q8_attn on both sides of the sizes where its form changes, and its streaming forms to the rounding
of their own numerators (11 bits in bf16)."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from tests.chunk_cases import EPS
from tests.q8_cases import Q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


def _expands(c):
    """Whether a bf16 call goes through expanded rows: more than 64 rows of a (b, l, h), and more than 12288 groups
    of 16 entries to do in blocks of 32 rows, by what the table's pages hold."""
    blocks = -(-c.T // (32 // c.G))
    return c.G * c.T > 64 and len(c.units) * blocks * c.table.shape[1] * c.page // 16 > 12288


def _check_numerators(c, s, pages=None):
    """As check_attn of q8_cases, with 11 bits (fp32: 22) whatever the number of rows: numerators rounded to half a
    step of 2^-11, subnormal ones by 2^-29 of the largest; scores off by the fp32 sums of d products."""
    out = s["out"].double().cpu().numpy()
    half = 2.0 ** -22 if c.dtype == "f32" else 2.0 ** -11
    for u in c.units:
        b, lr, h, hs, n, n0 = c.where(u)
        if n == 0:
            continue
        K, V, lm = c.entries(u)
        q = c.q[b, lr, hs, :n].double().numpy()
        o, _, p = Q.q8_attn(q, K, V, lm, n0, c.page, None if pages is None else pages[u])
        N = len(K)
        dots = np.abs(q) @ np.abs(K).T / np.sqrt(c.d)
        top = np.abs(q).max(-1, keepdims=True) * np.abs(K).sum(-1) / np.sqrt(c.d)
        de = c.d * 2.0 ** -23 * dots + 2.0 ** -33 * top + 2.0 ** -21 * (dots + np.abs(np.where(np.isinf(lm), 0.0, lm)))
        dbar = (p * de).sum(-1)
        pn = half + 2.0 ** -21 + N * 2.0 ** -23
        tol = (np.einsum("gtn,nd->gtd", p * (de + pn) + 2.0 ** -29 * p.max(-1, keepdims=True) * (p > 0), np.abs(V))
               + (dbar + N * 2.0 ** -24 + 2.0 ** -21)[..., None] * np.abs(o) + 1.01 * EPS[c.dtype] * np.abs(o) + 1e-30)
        err = np.abs(out[b, lr, hs, :n] - o)
        assert (err <= tol).all(), (u, err.max(), (err / tol).max())


def _attn(kvc, c, pick=None):
    c.fill_new()
    s = c.upload()
    if pick:
        c.select(s, *pick)
    c.attn(s, s.get("sel"))
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    return s


# ------------------------------------------------------------------ an item for every warp, or fewer
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [-8, 0, 8])
def test_items_around_the_number_of_warps(kvc, dtype, more):
    """One token over as many caches as the grid has warps, a few fewer and a few more."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    items = sms * (3 if dtype == "bf16" else 2) * 4 + more
    c = Q8(kvc, np.arange(items) * 7 % 61, [1], L=items // 8, H=8, G=2, d=64, dtype=dtype)
    s = _attn(kvc, c)
    c.check_attn(s)
    _check_numerators(c, s)


@pytest.mark.parametrize("T", [227, 228, 229, 299, 300])
def test_picked_pages_around_the_number_of_warps(kvc, T):
    c = Q8(kvc, np.arange(8) * 37 % 200, [T], H=8, G=1, d=64)
    s = _attn(kvc, c, (3, 1, 1))
    picks = c.all_picks(3, 1, 1)
    c.check_select(s, picks)
    c.check_attn(s, picks)
    _check_numerators(c, s, picks)


# ------------------------------------------------------------------ precision of the streaming forms
STREAMED = {
    "four row tiles, 333 tokens": dict(lens=[600, 129], n_new=[333], H=2, page=128),
    "four row tiles, G 8": dict(lens=[100, 333], n_new=[130], H=2, G=8, page=32),
    "four row tiles, layer range": dict(lens=[5, 70, 200, 130, 64, 9], n_new=[90, 61], B=2, L=3, layers=(1, 3), page=64),
    "four row tiles, sharp": dict(lens=[300, 700], n_new=[60], H=2, qscale=20.0, page=64),
    "three row tiles, pieces": dict(lens=[9000, 20011], n_new=[5], H=2, page=64),
    "two row tiles, pieces": dict(lens=[9000, 20011], n_new=[3], H=2, page=128),
    "one row tile, pieces": dict(lens=[9000, 20011], n_new=[1], H=2, page=64),
    "a table wider than its entries": dict(lens=[300, 50], n_new=[7], H=2, max_pages=1500),
}


@pytest.mark.parametrize("name", list(STREAMED))
def test_numerators_keep_11_bits(kvc, name):
    c = Q8(kvc, seed=list(STREAMED).index(name), **STREAMED[name])
    s = _attn(kvc, c)
    assert not _expands(c)
    _check_numerators(c, s)
