"""What a call of QuantizedCache.step or pack would refuse is refused before the cache changes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


def _params(kvc, **over):
    kw = dict(B=2, L=2, H=2, G=4, d=128, P=1, W=1, dtype=kvc.KVC_BF16, n_max=64, S_max=1)
    return kvc.make_params(**{**kw, **over})


def _shifted(t, elements):
    """t's values in memory that begins that many elements after an aligned place."""
    x = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)[elements:].view(t.shape)
    return x.copy_(t)


STATE = ("K", "V", "k_scale", "v_scale", "len_lh", "pos_next")


@pytest.mark.parametrize("n_sel", [0, 4])
def test_a_refused_step_leaves_the_cache_as_it_was(kvc, n_sel):
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    cache = QuantizedCache(_params(kvc), 64, T=4, page_rows=16, n_sel=n_sel)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((2, 2, n, 3, 128), generator=g, device="cuda").bfloat16() for n in (8, 2, 2))
    out = torch.empty_like(q)
    cache.step(q, k, v, out)
    torch.cuda.synchronize()
    old = {n: getattr(cache, n).clone() for n in STATE}
    lse = torch.empty((2, 2, 8, 3), device="cuda")
    q, k, v = 4 * q, 4 * k, 4 * v                           # appended, these would change scales too
    bad = {
        "out off a 32-byte boundary": (q, k, v, _shifted(out, 8), None),
        "out not contiguous": (q, k, v, torch.empty((2, 2, 8, 3, 256), dtype=q.dtype, device="cuda")[..., ::2], None),
        "out in host memory": (q, k, v, out.cpu(), None),
        "lse not contiguous": (q, k, v, out, torch.empty((2, 2, 8, 6), device="cuda")[..., ::2]),
        "lse in host memory": (q, k, v, out, lse.cpu()),
        "keys not contiguous": (q, torch.empty((2, 2, 2, 3, 256), dtype=q.dtype, device="cuda")[..., ::2], v, out, lse),
    }
    for what, (a, b, c, o, x) in bad.items():
        with pytest.raises(ValueError):
            cache.step(a, b, c, o, lse=x)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        for n in STATE:
            assert torch.equal(getattr(cache, n), old[n]), (what, n)
    with pytest.raises(kvc.KvcError):                       # the append's own refusal, its first call
        cache.step(q, _shifted(k, 4), v, out)
    torch.cuda.synchronize()
    for n in STATE:
        assert torch.equal(getattr(cache, n), old[n]), n
    cache.step(q, k, v, out, lse=lse)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0 and (cache.len_lh == 6).all()


def test_sizes_and_positions(kvc):
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    with pytest.raises(ValueError, match="no cache of these sizes"):
        QuantizedCache(_params(kvc, d=96), 64)
    cache = QuantizedCache(_params(kvc), 64, logm=True)
    Kp = torch.randn((100, 128), device="cuda").bfloat16()
    lens = torch.full((2, 2, 2), 5, dtype=torch.int32, device="cuda")
    off = torch.arange(8, device="cuda").view(2, 2, 2) * 5
    for pos in (torch.zeros(3, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros((2, 1), device="cuda")):
        with pytest.raises(ValueError, match="pos_next"):
            cache.pack(Kp, Kp, torch.zeros(100, device="cuda"), lens, off, pos)
    torch.cuda.synchronize()
    assert (cache.len_lh == 0).all() and (cache.K == 0).all()
    cache.pack(Kp, Kp, torch.zeros(100, device="cuda"), lens, off, torch.tensor([5.0, 7.0], device="cuda"))
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0 and (cache.len_lh == 5).all() and cache.pos_next.tolist() == [5.0, 7.0]
