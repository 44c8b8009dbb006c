"""The calls on the 8-bit cache against the oracle: types, head layouts, lengths around pages and
groups, ragged chunks, layer ranges, scales that grow, dead entries; unused rows hold codes that
are not numbers.  Codes, scales, bounds and picked pages are compared bit for bit."""
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


EDGE = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 255, 500]
CASES = {
    "one token": dict(lens=EDGE, n_new=[1, 1], B=2, L=4, H=2),
    "one token, page 64": dict(lens=EDGE, n_new=[1], L=4, H=4, page=64),
    "one token, page 128, d 64": dict(lens=EDGE, n_new=[1], L=4, H=4, d=64, page=128),
    "one token, G 1": dict(lens=EDGE, n_new=[1], L=8, H=2, G=1, page=32),
    "one token, G 8": dict(lens=EDGE, n_new=[1], L=8, H=2, G=8, page=32),
    "one token, long": dict(lens=[9000, 5, 20011, 300], n_new=[1], L=2, H=2, page=64),
    "no log m": dict(lens=[70, 500], n_new=[1], H=2, logm=False),
    "empty cache": dict(lens=[0, 0], n_new=[1], H=2),
    "empty cache, chunk": dict(lens=[0, 0], n_new=[77], H=2, page=32),
    "two tokens": dict(lens=[0, 3, 128, 200], n_new=[2], H=4, G=2),
    "ragged chunks": dict(lens=[40, 0, 130, 300, 17, 64, 1, 255], n_new=[1, 17, 0, 33], B=4, H=2, page=32),
    "no new tokens anywhere": dict(lens=[40, 0], n_new=[0], H=2, T=4),
    "drafts, G 8": dict(lens=[0, 15, 64, 65, 130, 300], n_new=[5, 3], B=2, H=3, G=8, page=64),
    "long chunk": dict(lens=[600, 129], n_new=[333], H=2, page=128),
    "long chunk, G 1": dict(lens=[100], n_new=[700], G=1, page=64),
    "long chunk, G 2, d 64": dict(lens=[100, 0], n_new=[300], H=2, G=2, d=64),
    "long chunk, G 8": dict(lens=[100, 333], n_new=[130], H=2, G=8, page=32),
    "many units": dict(lens=np.arange(7 * 3 * 16) * 3 % 211, n_new=[1, 2, 3, 4, 5, 6, 7], B=7, L=3, H=16, G=2),
    "runs of short units": dict(lens=np.where(np.arange(600) % 7 == 3, 300, np.arange(600) % 50), n_new=[1], L=50,
                                H=12, G=1, d=64),
    # tables wider than the cache needs (then an item's groups are not known to be few), by row tiles
    "wide table": dict(lens=[300, 50, 700, 129], n_new=[1], H=4, max_pages=700),
    "wide table, two tiles": dict(lens=[300, 50, 700, 129], n_new=[4], H=4, max_pages=700),
    "wide table, three tiles": dict(lens=[300, 50, 700, 129], n_new=[5, 3], B=2, H=2, page=32, max_pages=300),
    "wide table, four tiles": dict(lens=[300, 50, 700, 129], n_new=[7, 8], B=2, H=2, max_pages=700),
    "wide table, G 8, d 64": dict(lens=[300, 50, 700, 129], n_new=[2, 1], B=2, H=2, G=8, d=64, page=64, max_pages=200),
    # many rows and wide tables: expanded rows
    "expanded": dict(lens=[600, 129], n_new=[333], H=2, page=128, max_pages=40),
    "expanded, G 1": dict(lens=[100], n_new=[700], G=1, page=64, max_pages=300),
    "expanded, G 2, d 64": dict(lens=[100, 0], n_new=[300], H=2, G=2, d=64, max_pages=400),
    "expanded, G 8": dict(lens=[100, 333], n_new=[130], H=2, G=8, page=32, max_pages=100),
    "expanded, layer range": dict(lens=[5, 70, 200, 130, 64, 9, 0, 31, 77], n_new=[90, 61, 0], B=3, L=3, layers=(1, 3),
                                  page=64, max_pages=100),
    "expanded, scales of all sizes": dict(lens=[300, 50, 129], n_new=[40], H=3, spread=6.0, max_pages=900),
    "expanded, dead entries": dict(lens=[300, 129], n_new=[40], H=2, dead=0.7, logm=True, max_pages=1300),
    "expanded, no log m": dict(lens=[300, 129], n_new=[40], H=2, logm=False, max_pages=1300),
    "expanded, unit by unit": dict(lens=[70, 300, 0], n_new=[20], H=3, page=128, max_pages=16384),
    # more items than warps
    "many items": dict(lens=np.arange(2500) % 37, n_new=[1], L=125, H=20, d=64),
    "many tokens": dict(lens=np.arange(32) * 7 % 150, n_new=[80, 79, 80, 70], B=4, H=8, G=2, d=64),
    "layer range": dict(lens=[5, 70, 200, 130, 64, 9, 1, 300], n_new=[9, 20], B=2, L=4, layers=(1, 3)),
    "layer range, long": dict(lens=[5, 70, 200, 130, 64, 9], n_new=[90, 61], B=2, L=3, layers=(1, 3), page=64),
    "no n_new": dict(lens=[5, 70], n_new=[9, 9], B=2, pass_n_new=False),
    "scales of all sizes": dict(lens=[300, 50, 129], n_new=[20], H=3, spread=6.0),
    "scales of all sizes, one token": dict(lens=[300, 50, 129], n_new=[1], H=3, spread=6.0, page=32),
    "dead entries": dict(lens=[300, 129], n_new=[20], H=2, dead=0.7),
    "sharp": dict(lens=[300, 700], n_new=[60], H=2, qscale=20.0, page=64),
    "sharp, one token": dict(lens=[300, 700], n_new=[1], H=2, qscale=20.0, page=64),
}
F32 = ("one token", "one token, page 128, d 64", "ragged chunks", "drafts, G 8", "long chunk", "layer range",
       "scales of all sizes", "dead entries", "sharp", "no new tokens anywhere", "empty cache", "wide table",
       "wide table, four tiles", "wide table, G 8, d 64", "many items", "many tokens")
ALL = [(n, "bf16") for n in CASES] + [(n, "f32") for n in F32]
IDS = [f"{n}-{t}" for n, t in ALL]


def _seed(name):
    return list(CASES).index(name)


@pytest.mark.parametrize("name,dtype", ALL, ids=IDS)
def test_append(kvc, name, dtype):
    c = Q8(kvc, dtype=dtype, seed=_seed(name), **CASES[name])
    s = c.upload()
    c.append(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    c.check_append(s, name)


@pytest.mark.parametrize("name,dtype", ALL, ids=IDS)
def test_attention(kvc, name, dtype):
    c = Q8(kvc, dtype=dtype, seed=50 + _seed(name), **CASES[name])
    c.fill_new()
    s = c.upload()
    c.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    c.check_attn(s, what=name)


PICKS = [(1, 0, 1), (4, 1, 2), (7, 2, 1), (20, 0, 4)]


@pytest.mark.parametrize("name,dtype", ALL, ids=IDS)
def test_picked_pages_and_attention_over_them(kvc, name, dtype):
    c = Q8(kvc, dtype=dtype, seed=100 + _seed(name), **CASES[name])
    c.fill_new()
    s = c.upload()
    pick = PICKS[_seed(name) % len(PICKS)]
    c.select(s, *pick)
    c.attn(s, s["sel"])
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    picks = c.all_picks(*pick)
    c.check_select(s, picks, what=name)
    c.check_attn(s, picks, what=name)
