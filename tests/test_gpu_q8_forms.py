"""kvc_q8_attn on both sides of the sizes where its form changes."""
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
