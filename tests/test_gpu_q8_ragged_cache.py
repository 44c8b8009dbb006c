"""A QuantizedCache with room of its own for every (b, l, h), as Compressor.to_q8 builds it: pages for what
each one holds, results as with the same room for all."""
import numpy as np
import pytest
import torch

from synth import workloads as W
from tests.gpu_helpers import upload_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n_sel", [0, 5])
def test_a_compressed_cache_with_full_heads(kvc, n_sel):
    """Half of the heads are kept whole: the 8-bit cache has pages for each one's entries and the reserve, and less
    than the packed cache's bytes; entries and steps are those of a cache with the largest length for all."""
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    cfg = W.small_config(B=2, L=2, H=2, n=3000, n_min=2500, n_decode=40, budget_ratio=0.6)
    wl = W.make_workload(cfg)
    p, comp, dev, _ = upload_workload(wl, head_full_frac=0.5)
    comp.compress(dev["K"], dev["V"], dev["Qp"], dev["bounds"], dev["n_slots"], dev["sens"])
    ctx = torch.tensor([float(s.n) for s in wl.seqs], device="cuda")
    R, reserve = 32, 40
    kw = dict(T=20, page_rows=R, n_sel=n_sel)
    cache = comp.to_q8(reserve, ctx, **kw)
    lens = comp.len_lh.cpu().numpy()
    assert lens.max() > 2 * lens.min()
    rows = int((-(-(lens + reserve) // R) * R).sum())
    assert cache.K.shape[0] == cache.V.shape[0] == rows and cache.p.packed_rows == rows
    # a code is half a packed element; pages add less than R entries and the reserve to each (b, l, h)
    assert rows * cfg.d < lens.sum() * cfg.d + lens.size * (R + reserve) * cfg.d < 2 * lens.sum() * cfg.d
    same = QuantizedCache(p, int(lens.max()) + reserve, logm=True, n_pos=p.n_max + reserve, **kw)
    same.pack(comp.Kp, comp.Vp, comp.logm, comp.len_lh, comp.off_lh, ctx)
    assert same.table.shape == cache.table.shape

    def entries():
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        assert torch.equal(cache.len_lh, same.len_lh)
        for b, l, h in np.ndindex(2, 2, 2):
            for x, y in zip(cache.entries(b, l, h), same.entries(b, l, h)):
                np.testing.assert_array_equal(x, y)
    entries()
    g = torch.Generator(device="cuda").manual_seed(2)
    for T in (20, 1, 7):
        q, k, v = (torch.randn((2, 2, n, T, cfg.d), generator=g, device="cuda").to(comp.Kp.dtype) for n in (2 * cfg.G, 2, 2))
        a, b = torch.empty_like(q), torch.empty_like(q)
        cache.step(q, k, v, a)
        same.step(q, k, v, b)
        entries()
        assert torch.equal(a, b)
    assert (cache.len_lh.cpu() == torch.from_numpy(lens) + 28).all()


def test_room_of_its_own_for_each(kvc):
    """Every (b, l, h) takes tokens until its own pages are full, and those alone are reported."""
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    p = kvc.make_params(B=1, L=2, H=2, G=4, d=128, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16)
    cache = QuantizedCache(p, [[[16, 33], [1, 64]]], T=20, page_rows=16, n_pos=200)
    assert cache.cap_lh.view(-1).tolist() == [16, 48, 16, 64] and cache.K.shape[0] == 144
    assert cache.table.view(4, -1).tolist() == [[0, -1, -1, -1], [1, 2, 3, -1], [4, -1, -1, -1], [5, 6, 7, 8]]
    g = torch.Generator(device="cuda").manual_seed(3)
    want = [[16, 16, 16, 16], [16, 32, 16, 32], [16, 48, 16, 48], [16, 48, 16, 64], [16, 48, 16, 64]]
    for step, lens in enumerate(want):
        q, k, v = (torch.randn((1, 2, n, 16, 128), generator=g, device="cuda").bfloat16() for n in (8, 2, 2))
        out = torch.full_like(q, 7.0)
        cache.step(q, k, v, out)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == (0 if step == 0 else kvc.KVC_ECAPACITY)
        assert cache.len_lh.view(-1).tolist() == lens
        for u in range(4):
            took = step == 0 or lens[u] > want[step - 1][u]
            assert (out.view(4, 4, 16, 128)[u] == 7.0).all() == (not took)
    for bad in ([[[16, 33], [0, 64]]], [[16, 33], [1, 64]], [16, 33, 1, 64]):
        with pytest.raises(ValueError):
            QuantizedCache(p, bad, T=20, page_rows=16)
