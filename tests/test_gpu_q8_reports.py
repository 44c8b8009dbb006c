"""kvc_q8_select and kvc_q8_attn report every (b, l, h) with lengths or pages out of range, whichever
it is and in each form of the kernel, and skip that one alone."""
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
    "cluster": dict(n=1), "cluster, two row blocks": dict(n=40), "cluster, fp32": dict(n=3, dtype="f32"),
    "pieces": dict(n=1, wide=1500), "four row tiles": dict(n=7, wide=700), "expanded": dict(n=40, wide=4000),
    "picked pages": dict(n=2, pick=(3, 1, 1)),
}
BAD = {                                                    # (length before, length after) of a unit with n tokens
    "a length below 0": lambda n: (-1, n - 1),
    "fewer after than before": lambda n: (60, 59),
    "more than T tokens": lambda n: (60, 60 + n + 1),
    "past the table": lambda n: (1 << 30, (1 << 30) + n),
}


@pytest.mark.parametrize("what", list(BAD))
@pytest.mark.parametrize("form", list(FORMS))
def test_lengths_out_of_range_of_any_unit(kvc, form, what):
    f = dict(FORMS[form])
    n, wide, pick, dtype = f["n"], f.get("wide"), f.get("pick"), f.get("dtype", "bf16")
    c = Q8(kvc, [50, 60, 70, 80, 90], [n], H=5, page=16, dtype=dtype, max_pages=wide)
    c.fill_new()
    good = c.upload()
    if pick:
        c.select(good, *pick)
    c.attn(good, good.get("sel"))
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    for u in (1, 2, 4):
        s = c.upload()
        s["len"].view(-1)[u], s["new"].view(-1)[u] = BAD[what](n)
        if pick:
            c.select(s, *pick)
            torch.cuda.synchronize()
            assert kvc.kvc_device_error() == kvc.KVC_EDEVICE, u
            assert (s["sel"][0, 0, u] == -9).all()
            s["sel"][0, 0, u] = 0
        c.attn(s, s.get("sel"))
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == kvc.KVC_EDEVICE, u
        others = [h for h in range(20) if h // 4 != u]
        assert (s["out"][0, 0, 4 * u:4 * u + 4] == 7.0).all() and (s["lse"][0, 0, 4 * u:4 * u + 4] == 7.0).all()
        for k in ("out", "lse"):
            assert torch.equal(s[k][0, 0, others], good[k][0, 0, others]), (u, k)


@pytest.mark.parametrize("form", list(FORMS))
def test_pages_out_of_range_of_any_unit(kvc, form):
    f = dict(FORMS[form])
    n, wide, pick, dtype = f["n"], f.get("wide"), f.get("pick"), f.get("dtype", "bf16")
    c = Q8(kvc, [50, 60, 70, 80, 90], [n], H=5, page=16, dtype=dtype, max_pages=wide)
    c.fill_new()
    good = c.upload()
    if pick:
        c.select(good, *pick)
    c.attn(good, good.get("sel"))
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    for u in (1, 4):
        s = c.upload()
        if pick:
            s["sel"] = good["sel"].clone()
        s["c"]._keep[0].view(5, -1)[u, 0] = c.n_pages
        c.attn(s, s.get("sel"))
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == kvc.KVC_EDEVICE, u
        others = [h for h in range(20) if h // 4 != u]
        for k in ("out", "lse"):
            assert torch.equal(s[k][0, 0, others], good[k][0, 0, others]), (u, k)


@pytest.mark.parametrize("off", [2 ** 63 - 1, 2 ** 63 - 90, 2 ** 62, -2 ** 63, -1])
def test_pack_skips_offsets_of_any_size(kvc, off):
    """An offset near 2^63 is out of range, whatever it and the length add up to."""
    c = Q8(kvc, [90, 40], [0], H=2, page=16, T=1)
    s = c.upload()
    rows = 200
    g = torch.Generator(device="cuda").manual_seed(3)
    Kp, Vp = (torch.randn((rows, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    lm = torch.zeros(rows, device="cuda")
    offs = torch.tensor([off, 150], device="cuda")
    old = s["K"].clone()
    kvc.kvc_q8_pack(s["p"], s["c"], s["x"], Kp, Vp, lm, s["len"], offs, s["cap"], s["len_out"])
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == kvc.KVC_EDEVICE
    assert s["len_out"].view(-1).tolist() == [0, 40]
    for p in c.table[0][c.table[0] >= 0]:
        assert torch.equal(s["K"][p * 16:(p + 1) * 16], old[p * 16:(p + 1) * 16])


@pytest.mark.parametrize("units", [1, 250])
def test_picked_pages_behind_their_places(kvc, units):
    """A token that sees two pages has its list in the first two places; a page further on is reported."""
    U = 8 * units
    c = Q8(kvc, [20] * U, [1], L=units, H=8, page=16, logm=False)
    c.fill_new()
    s = c.upload()
    for places, code in (([1, 0, -1, -1], 0), ([-1, 1, 5, -7], 0), ([0, -1, 1 << 30, 2], 0), ([-1, 0, 1, -1], kvc.KVC_EDEVICE),
                         ([0, 9, -1, 1], kvc.KVC_EDEVICE)):
        lists = np.tile(np.array([0, 1, -1, -1], np.int32), (U, 1))
        lists[U - 1] = places
        s["sel"] = torch.from_numpy(lists).cuda().view(1, units, 8, 1, 4)
        s["out"].fill_(7.0), s["lse"].fill_(7.0)
        c.attn(s, s["sel"])
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == code, places
        c.check_attn(s, {u: [[j for j in lists[u][:2] if 0 <= j <= 1]] for u in range(U)})
