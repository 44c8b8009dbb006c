"""Host-side checks of the chunk calls' further forms (no GPU: the fake pointers are
never dereferenced)."""
import ctypes

import pytest
import torch

from kv_cache_compression_probe_gb300 import kvc
from tests.test_chunk_host import BAD_CHUNK, BAD_PARAMS, PAGED, VP, _chunk, _fake, _params


@pytest.fixture(scope="module")
def lib():
    from kv_cache_compression_probe_gb300 import build
    build.build()
    return kvc.lib()


# ------------------------------------------------------------------ mass with capacities
def _mass_cap(lib, p, c, ptrs=None, ws=VP(1 << 20), nb=1 << 40, decay=1.0):
    a = ptrs or _fake(10)
    return lib.kvc_chunk_mass_cap(ctypes.byref(p), ctypes.byref(c) if c else None, *a[:9], ctypes.c_float(decay),
                                  a[9], ws, ctypes.c_size_t(nb), None)


def test_mass_with_capacities_checks_its_arguments(lib):
    p, c = _params(), _chunk()
    for bad in BAD_CHUNK:
        assert _mass_cap(lib, p, _chunk(**bad)) == kvc.KVC_EINVAL, bad
    for bad in BAD_PARAMS:
        assert _mass_cap(lib, _params(**bad), c) == kvc.KVC_EINVAL, bad
    assert _mass_cap(lib, p, None) == kvc.KVC_EINVAL
    for i in range(10):                                 # the capacities may be missing, and off_lh with pages
        ptrs = _fake(10)
        ptrs[i] = None
        want = kvc.KVC_EWORKSPACE if i == 6 else kvc.KVC_EINVAL
        assert _mass_cap(lib, p, c, ptrs, None) == want, i
        if i == 7:
            assert _mass_cap(lib, p, _chunk(**PAGED), ptrs, None) == kvc.KVC_EWORKSPACE
    for decay in (-0.1, 1.1, float("nan")):
        assert _mass_cap(lib, p, c, decay=decay) == kvc.KVC_EINVAL


def test_a_step_hands_its_capacities_to_both_calls(monkeypatch):
    """ChunkedCache: what attention skips for want of room, the mass call skips as well."""
    from kv_cache_compression_probe_gb300 import pipeline
    cache = _cpu_cache(monkeypatch, pipeline)
    seen = {}
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_attn", lambda *a: seen.update(attn=a))
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_mass", lambda *a: seen.update(mass=a))
    monkeypatch.setattr(pipeline.kvc, "kvc_mass_evict", lambda *a: None)
    cache.step(**_tokens(4))
    assert any(x is cache.cap_lh for x in seen["attn"]) and seen["mass"][14] is cache.cap_lh


def _cpu_cache(monkeypatch, pipeline, **kw):
    """A ChunkedCache in host memory; the library's calls are to be replaced."""
    monkeypatch.setattr(pipeline.kvc, "make_chunk", lambda T, l0, l1, **mods: (T, l0, l1))
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_workspace_bytes", lambda p, c: 256)
    monkeypatch.setattr(pipeline.kvc, "kvc_mass_evict_workspace_bytes", lambda p, c, n: 256)
    p = kvc.make_params(B=2, L=2, H=2, G=4, d=128, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16)
    return pipeline.ChunkedCache(p, **dict(dict(budget=32, T=8, page_rows=16, recent=4, device="cpu"), **kw))


def _tokens(T):
    return {n: torch.zeros(2, 2, h, T, 128, dtype=torch.bfloat16)
            for n, h in (("q", 8), ("k_new", 2), ("v_new", 2), ("out", 8))}


# ------------------------------------------------------------------ ChunkedCache.step
def _quiet(monkeypatch, pipeline, calls):
    for n in ("kvc_chunk_attn", "kvc_chunk_mass", "kvc_mass_evict"):
        monkeypatch.setattr(pipeline.kvc, n, lambda *a, n=n: calls.append(n))


BAD_COUNTS = {
    "64 bits": torch.tensor([3, 1]),
    "floats": torch.tensor([3.0, 1.5]),
    "one for all": torch.tensor([3], dtype=torch.int32),
    "a number": torch.tensor(3, dtype=torch.int32),
    "a sequence more": torch.tensor([3, 1, 2], dtype=torch.int32),
    "two dimensions": torch.tensor([[3, 1]], dtype=torch.int32),
}


@pytest.mark.parametrize("name", list(BAD_COUNTS))
def test_step_refuses_counts_of_another_type_or_shape(monkeypatch, name):
    from kv_cache_compression_probe_gb300 import pipeline
    cache, calls = _cpu_cache(monkeypatch, pipeline), []
    _quiet(monkeypatch, pipeline, calls)
    with pytest.raises(ValueError):
        cache.step(n_new=BAD_COUNTS[name], **_tokens(4))
    assert not calls and not cache.n_new.any() and not cache.pos_next.any()
    cache.step(n_new=torch.tensor([3, 1], dtype=torch.int32), **_tokens(4))
    assert len(calls) == 3 and cache.n_new.tolist() == [3, 1]


@pytest.mark.parametrize("evict", [True, False])
def test_positions_advance_only_with_the_tokens_taken(monkeypatch, evict):
    """A sequence whose units the device skipped (a count above T, or no room) keeps its next
    position, so that its later tokens get theirs."""
    from kv_cache_compression_probe_gb300 import pipeline
    cache = _cpu_cache(monkeypatch, pipeline)
    _quiet(monkeypatch, pipeline, [])

    def attn(p, c, q, k, v, pos_new, K, V, logm, pos, len_lh, cap_lh, off, out, lse, len_out, ws, stream):
        n = cache.n_new[:, None, None]
        took = (n <= q.shape[3]) & (len_lh + n <= cap_lh)
        len_out.copy_(torch.where(took, len_lh + n, len_lh))
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_attn", attn)
    monkeypatch.setattr(pipeline.kvc, "kvc_mass_evict", lambda *a: a[12].copy_(a[10]))
    at = [0, 0]
    for ns, took in (([4, 4], [4, 4]), ([9, 2], [0, 2]), ([1, 0], [1, 0]), ([8, 8], [8, 8]), ([8, 8], [8, 8]),
                     ([8, 8], [8, 8]), ([8, 8], [8, 8]), ([8, 8], [8, 8]), ([8, 2], [0, 2])):
        if ns == [8, 2]:                                # 45 and 46 of the 48 rows are taken
            assert cache.len_lh[:, 0, 0].tolist() == [45, 46]
        cache.step(n_new=torch.tensor(ns, dtype=torch.int32), evict=evict, **_tokens(max(1, min(8, max(ns)))))
        at = [a + t for a, t in zip(at, took)]
        assert cache.pos_next.tolist() == at
        assert cache.len_lh[:, 1, 1].tolist() == at


# ------------------------------------------------------------------ streams and devices
class _Stream:
    """A stream of device `dev`, as far as the binding looks at it."""

    def __init__(self, dev, handle):
        self.device_index, self.cuda_stream = dev, handle


class _Tensor:
    def __init__(self, dev):
        self.dev, self.nbytes = dev, 1 << 20

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096 * (self.dev + 1)


class _Lib:
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        return lambda *a: self.streams.append(a[-1]) or kvc.KVC_OK


@pytest.fixture
def two_devices(monkeypatch):
    """The binding as it would be with device 1 current and stream 77 on it; returns the library."""
    fake = _Lib()
    monkeypatch.setattr(kvc.torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(kvc.torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(kvc.torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + 7 * d, raising=False)
    monkeypatch.setattr(kvc.torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(kvc, "lib", lambda: fake)
    return fake


def _calls(c, dev, stream):
    t = _Tensor(dev)
    yield lambda: kvc.kvc_chunk_attn(None, c, *[t] * 15, stream)
    yield lambda: kvc.kvc_chunk_mass(None, c, *[t] * 8, 1.0, t, t, stream)
    yield lambda: kvc.kvc_mass_evict(None, c, t, t, 4, *[t] * 8, 100, t, stream)


def test_streams_and_tensors_of_another_device_are_refused(two_devices):
    for stream in (None, _Stream(1, 5), 9):
        for call in _calls(_chunk(), 1, stream):
            call()
    assert two_devices.streams == [77] * 3 + [5] * 3 + [9] * 3
    other = _chunk()
    other._devices = (0,)                               # a page table, say
    both = _chunk()
    both._devices = (0, 1)
    for c, dev, stream in ((_chunk(), 1, _Stream(0, 5)), (_chunk(), 0, None), (other, 1, None), (both, 1, None)):
        for call in _calls(c, dev, stream):
            with pytest.raises(ValueError):
                call()
    assert len(two_devices.streams) == 9


def test_step_refuses_a_stream_that_is_not_the_current_one(monkeypatch, two_devices):
    from kv_cache_compression_probe_gb300 import pipeline
    cache, calls = _cpu_cache(monkeypatch, pipeline), []
    _quiet(monkeypatch, pipeline, calls)
    for stream in (_Stream(1, 5), 5, _Stream(0, 77)):
        with pytest.raises(ValueError):
            cache.step(stream=stream, **_tokens(4))
    assert not calls and not cache.pos_next.any()
    for stream in (_Stream(1, 77), 77, None):
        cache.step(stream=stream, **_tokens(4))
    assert len(calls) == 9


# ------------------------------------------------------------------ workspaces
def test_workspace_depends_on_the_units_only(lib):
    """As much as the kernels use (without a GPU the library counts one SM): a record and a tile
    number per (b,l,h), and two partial results per CTA, of 256 rows (bf16) or 64 (fp32, two CTAs)."""
    for dtype, rows in ((kvc.KVC_BF16, 512), (kvc.KVC_F32, 256)):
        for d in (64, 128):
            for B, L, H in ((1, 1, 1), (2, 4, 2), (16, 32, 8)):
                p = _params(B=B, L=L, H=H, d=d, dtype=dtype, packed_rows=1 << 20)
                sizes = {kvc.kvc_chunk_workspace_bytes(p, _chunk(T=T, layer_end=L, **more))
                         for T in (1, 40, 2048, 65536) for more in ({}, PAGED, dict(window=5.0, softcap=3.0))}
                units = B * L * H
                need = 16 * units + 4 * units + 16 + rows * (d + 2) * 4
                assert len(sizes) == 1
                if not torch.cuda.is_available():
                    assert need <= sizes.pop() <= need + 5 * 256


def test_extend_grows_its_workspace_with_the_layers(monkeypatch, lib):
    """With the library's own sizes: a larger layer range outgrows the workspace, which stays alive for
    calls captured with it; more tokens do not."""
    from kv_cache_compression_probe_gb300 import pipeline
    used = []
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_attn", lambda *a: used.append(a[-2]))
    comp = object.__new__(pipeline.Compressor)
    comp.p = kvc.make_params(B=4, L=32, H=8, G=1, d=64, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16)
    comp.device, comp._ws_chunk, comp._ws_outgrown = "cpu", None, []
    comp.Kp = torch.zeros(64, 64)
    for name in ("Vp", "logm", "pos", "len_lh", "cap_lh", "off_lh"):
        setattr(comp, name, None)
    for T, layers in ((1, (0, 1)), (9, (3, 4)), (1, (0, 32)), (9, None), (2, (5, 6))):
        n = 32 if layers is None else layers[1] - layers[0]
        q = torch.zeros(4, n, 8, T, 64, dtype=torch.bfloat16)
        comp.extend(q, q, q, q, torch.zeros(4), layers=layers)
    assert used[0] is used[1] and used[2] is used[3] and used[3] is used[4] and used[0] is not used[2]
    assert len(comp._ws_outgrown) == 1 and comp._ws_outgrown[0] is used[0]


# ------------------------------------------------------------------ no step ends half way
def test_what_a_later_call_of_a_step_would_refuse_is_refused_first(monkeypatch):
    """The eviction takes up to 65535 (b,l,h) and the mass call a decay in 0..1: a step that cannot end
    does not begin."""
    from kv_cache_compression_probe_gb300 import pipeline
    for decay in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError):
            _cpu_cache(monkeypatch, pipeline, decay=decay)
    cache, calls = _cpu_cache(monkeypatch, pipeline), []
    _quiet(monkeypatch, pipeline, calls)
    cache.p.B = 16384                                   # 65536 (b,l,h)
    x = {n: t[:1].expand(16384, *t.shape[1:]) for n, t in _tokens(1).items()}
    with pytest.raises(ValueError):
        cache.step(**x)
    assert not calls and not cache.pos_next.any()
    cache.step(evict=False, **x)
    assert calls == ["kvc_chunk_attn", "kvc_chunk_mass"]
