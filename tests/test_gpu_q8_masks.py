"""kvc_q8_attn with entries masked by ln m: -inf, the types' lowest values and other large negative ones, which
all leave an entry no weight beside one that is not masked; whole groups, tiles and rows of them."""
import numpy as np
import pytest
import torch

from tests.q8_cases import Q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


FORMS = {
    "cluster": dict(n_new=[1], H=4),
    "cluster, four row tiles": dict(n_new=[9, 7], B=2, H=2),
    "cluster, picked pages": dict(n_new=[3], H=4, pick=(30, 1, 2)),
    "pieces": dict(n_new=[1], H=4, max_pages=1500),
    "pieces, two row tiles": dict(n_new=[4], H=4, max_pages=1500),
    "a warp an item": dict(n_new=[500], H=4, G=1, d=64, pick=(4, 1, 1)),
    "expanded": dict(n_new=[40], H=4, max_pages=1500),
}
MASKS = {"-inf": -np.inf, "fp32 lowest": -3.4028234663852886e38, "bf16 lowest": -3.3895313892515355e38, "-1e30": -1e30,
         "-1e9": -1e9, "fp16 lowest": -65504.0}


def _device_error(kvc):
    torch.cuda.synchronize()
    return kvc.kvc_device_error()


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("form,dtype", [(f, t) for f in FORMS for t in ("bf16", "f32") if (f, t) != ("expanded", "f32")])
def test_masked_entries_have_no_weight(kvc, form, dtype, mask):
    """Masked: the first 200 entries, single ones, a run past a tile's length, and all but one entry of the second (b, l, h)'s
    cache of before."""
    kw = dict(FORMS[form])
    pick = kw.pop("pick", None)
    c = Q8(kvc, [1300, 700, 90, 1000], dtype=dtype, logm=True, seed=3, **kw)
    c.fill_new()
    masked = np.zeros(c.n_pages * c.page, bool)
    for u in range(c.U):
        e = np.arange(int(c.lens[u]))
        dead = (e < 200) | (e % 5 == 2) | ((e >= 400) & (e < 700))
        if u == 1:
            dead = e != 650
        masked[c.table[u][e // c.page] * c.page + e % c.page] = dead
    normal = c.logm.copy()
    c.logm[masked] = MASKS[mask]
    s = c.upload()
    picks = None
    if pick:
        c.select(s, *pick)
        picks = c.all_picks(*pick)
    c.attn(s, s.get("sel"))
    assert _device_error(kvc) == 0
    c.logm = np.where(masked, -np.inf, normal).astype(np.float32)
    c.check_attn(s, picks)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("mask", ["-1e30", "-1e9"])
def test_rows_of_masked_entries_alone(kvc, form, mask):
    """All of a row's entries masked by a finite value whose steps in fp32 exceed the products: the scores are equal, so
    out is the values' average (numerators are equal, of 11 bits or, expanded, of 8), as the definition's."""
    kw = dict(FORMS[form])
    pick = kw.pop("pick", None)
    c = Q8(kvc, [1300, 700, 90, 1000], logm=True, seed=4, qscale=2.0 ** -12, **kw)
    c.fill_new()
    c.logm[:] = MASKS[mask]
    s = c.upload()
    picks = None
    if pick:
        c.select(s, *pick)
        picks = c.all_picks(*pick)
    c.attn(s, s.get("sel"))
    assert _device_error(kvc) == 0
    out = s["out"].double().cpu().numpy()
    for u in c.units:
        b, lr, h, hs, n, n0 = c.where(u)
        V = c.entries(u)[1]
        for t in {0, n - 1}:
            see = np.arange(len(V)) <= n0 + t
            if picks is not None:
                see &= np.isin(np.arange(len(V)) // c.page, picks[u][t])
            o, size, N = V[see].mean(0), np.abs(V[see]).mean(0), see.sum()
            tol = (N * 2.0 ** -23 + 2.0 ** -8) * size + (N * 2.0 ** -24 + 2.0 ** -20 + 1.01 * 2.0 ** -8) * np.abs(o) + 1e-30
            assert (np.abs(out[b, lr, hs, t] - o) <= tol).all(), (u, t)
