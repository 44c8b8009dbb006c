"""The chunk calls' oracle pins and host-side refusals (no GPU: the fake pointers
are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from kv_cache_compression_probe_gb300 import kvc

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from kv_cache_compression_probe_gb300 import build
    build.build()
    return kvc.lib()


# ------------------------------------------------------------------ oracle
def _head(seed, n0=50, n=7, G=3, d=16):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((G, n, d)), rng.standard_normal((n0 + n, d)), rng.standard_normal((n0 + n, d)),
            np.where(np.arange(n0 + n) < n0, rng.uniform(0, 2, n0 + n), 0.0),
            np.r_[np.sort(rng.integers(0, 400, n0)) / 2, 300.0 + np.arange(n)], n0)


def test_oracle_chunk_equals_its_decode_steps():
    """Without extras, token t of the chunk is a decode step over the entries before it."""
    q, K, V, lm, pos, n0 = _head(0)
    out, lse, p = O.chunk_attn(q, K, V, lm, pos, n0, 300.0)
    for t in range(q.shape[1]):
        c = n0 + t
        want, *_ = O.decode_step_head(q[:, t], K[c], V[c], K[:c], V[:c], lm[:c])
        np.testing.assert_allclose(out[:, t], want, rtol=1e-12)
    np.testing.assert_allclose(p.sum(-1), 1.0, rtol=1e-12)


def test_oracle_scores_against_torch():
    q, K, V, lm, pos, n0 = _head(1)
    sl = np.asarray([0.5, 0.25, 0.125])
    s = O.chunk_scores(q, K, lm, pos, n0, 300.0, softcap=2.0, window=120.0, slopes=sl)
    tq, tk = torch.from_numpy(q), torch.from_numpy(K)
    x = 2.0 * torch.tanh(torch.einsum("gtd,nd->gtn", tq, tk) / 4.0 / 2.0) + torch.from_numpy(lm)
    gap = (300.0 + torch.arange(7.0, dtype=torch.float64))[:, None] - torch.from_numpy(pos)
    x = x - torch.from_numpy(sl)[:, None, None] * gap
    x[:, gap >= 120.0] = -np.inf
    for t in range(7):
        x[:, t, n0 + t + 1:] = -np.inf
    np.testing.assert_allclose(s, x.numpy(), rtol=1e-12)
    p, lse = O.chunk_softmax(s)
    np.testing.assert_allclose(p, torch.softmax(x, -1).numpy(), rtol=1e-11, atol=1e-300)
    np.testing.assert_allclose(lse, torch.logsumexp(x, -1).numpy() / np.log(2), rtol=1e-12)


def test_oracle_mass_adds_probabilities():
    q, K, V, lm, pos, n0 = _head(2)
    s = O.chunk_scores(q, K, lm, pos, n0, 300.0)
    p, lse = O.chunk_softmax(s)
    old = np.full(len(K), 5.0)
    m = O.chunk_mass(old, n0, s, lse, 0.5)
    np.testing.assert_allclose(m, p.sum((0, 1)) + np.where(np.arange(len(K)) < n0, 2.5, 0.0), rtol=1e-12)
    assert abs((m - np.where(np.arange(len(K)) < n0, 2.5, 0.0)).sum() - q.shape[0] * q.shape[1]) < 1e-9
    lse[0, 0] = -np.inf
    m2 = O.chunk_mass(old, n0, s, lse, 0.5)
    np.testing.assert_allclose(m - m2, p[0, 0], atol=1e-12)


@pytest.mark.parametrize("seed", range(6))
def test_oracle_evict_is_a_brute_force_sort(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(0, 60))
    mass = rng.choice([0.0, 0.5, 1.0, np.nan, np.inf], n)
    pos = rng.permutation(n).astype(float)
    keep, safe = int(rng.integers(-2, n + 5)), float(rng.integers(0, n + 3))
    B, holes, movers = O.mass_evict(mass, pos, keep, safe)
    prot = [i for i in range(n) if pos[i] >= safe]
    rest = sorted((i for i in range(n) if pos[i] < safe),
                  key=lambda i: (np.isnan(mass[i]), -mass[i] if not np.isnan(mass[i]) else 0.0, i))
    assert B == min(n, max(keep, len(prot), 0))
    stay = set((prot + rest)[:B])
    final = [i if i in stay else None for i in range(B)]
    assert list(holes) == [i for i in range(B) if final[i] is None]
    assert list(movers) == sorted(i for i in stay if i >= B) and len(holes) == len(movers)


# ------------------------------------------------------------------ refusals
def _params(**over):
    kw = dict(B=2, L=4, H=2, G=4, d=128, P=1, W=1, dtype=kvc.KVC_BF16, n_max=64, S_max=1, packed_rows=4096)
    kw.update(over)
    return kvc.make_params(**kw)


def _chunk(**over):
    c = kvc.kvc_chunk()
    kw = dict(T=4, layer_begin=0, layer_end=4, page_rows=0, max_pages=0, softcap=0.0, window=0.0)
    kw.update(over)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _fake(k):
    return [VP(4096 * (i + 1)) for i in range(k)]


def _attn(lib, p, c, ptrs=None, ws=VP(1 << 20), nb=1 << 40):
    return lib.kvc_chunk_attn(ctypes.byref(p), ctypes.byref(c) if c else None, *(ptrs or _fake(14)), ws,
                              ctypes.c_size_t(nb), None)


def _mass(lib, p, c, ptrs=None, ws=VP(1 << 20), nb=1 << 40, decay=1.0):
    a = ptrs or _fake(9)
    return lib.kvc_chunk_mass(ctypes.byref(p), ctypes.byref(c) if c else None, *a[:8], ctypes.c_float(decay), a[8],
                              ws, ctypes.c_size_t(nb), None)


def _evict(lib, p, c, ptrs=None, ws=VP(1 << 20), nb=1 << 40, recent=0, max_len=100):
    a = ptrs or _fake(10)
    return lib.kvc_mass_evict(ctypes.byref(p), ctypes.byref(c) if c else None, a[0], a[1], recent, *a[2:10], max_len,
                              ws, ctypes.c_size_t(nb), None)


CALLS = {"attn": _attn, "mass": _mass, "evict": _evict}
PAGED = dict(page_rows=64, max_pages=8, page_table=VP(4096))
BAD_CHUNK = [dict(T=0), dict(T=-1), dict(T=65537), dict(layer_begin=-1), dict(layer_begin=4), dict(layer_end=5),
             dict(layer_begin=2, layer_end=2), dict(page_rows=48, max_pages=8, page_table=VP(4096)),
             dict(page_rows=8, max_pages=8, page_table=VP(4096)),
             dict(page_rows=2048, max_pages=8, page_table=VP(4096)), dict(page_rows=-64),
             dict(page_rows=64, max_pages=0, page_table=VP(4096)), dict(page_rows=64, max_pages=8),
             dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(window=-1.0),
             dict(window=float("nan")), dict(window=float("inf"))]
BAD_PARAMS = [dict(B=0), dict(G=3), dict(d=96), dict(dtype=5), dict(packed_rows=0), dict(packed_rows=1 << 31),
              dict(packed_rows=-1), dict(B=1 << 16, H=1 << 10)]


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_blocks_are_rejected(lib, name):
    for bad in BAD_CHUNK:
        assert CALLS[name](lib, _params(), _chunk(**bad)) == kvc.KVC_EINVAL, bad
        assert lib.kvc_chunk_workspace_bytes(ctypes.byref(_params()), ctypes.byref(_chunk(**bad))) == 0
    for bad in BAD_PARAMS:
        assert CALLS[name](lib, _params(**bad), _chunk()) == kvc.KVC_EINVAL, bad
    assert CALLS[name](lib, _params(), None) == kvc.KVC_EINVAL
    assert CALLS[name](lib, _params(packed_rows=32), _chunk(**PAGED)) == kvc.KVC_EINVAL


# pointer positions that may be NULL: off_lh with pages; lse and len_out of the attention
OPTIONAL = {"attn": {12, 13}, "mass": set(), "evict": set()}
OFF = {"attn": 10, "mass": 6, "evict": 8}
N_PTR = {"attn": 14, "mass": 9, "evict": 10}


@pytest.mark.parametrize("name", list(CALLS))
def test_missing_pointers_and_bad_workspaces(lib, name):
    p = _params()
    for i in range(N_PTR[name]):
        ptrs = _fake(N_PTR[name])
        ptrs[i] = None
        if i not in OPTIONAL[name]:
            assert CALLS[name](lib, p, _chunk(), ptrs) == kvc.KVC_EINVAL, i
        if i == OFF[name]:                              # with pages the row offsets are not needed
            assert CALLS[name](lib, p, _chunk(**PAGED), ptrs, None) == kvc.KVC_EWORKSPACE
    c = _chunk()
    need = (kvc.kvc_mass_evict_workspace_bytes(p, c, 100) if name == "evict" else kvc.kvc_chunk_workspace_bytes(p, c))
    assert need > 0
    assert CALLS[name](lib, p, c, None, None) == kvc.KVC_EWORKSPACE
    assert CALLS[name](lib, p, c, None, VP(1 << 20), need - 1) == kvc.KVC_EWORKSPACE
    assert CALLS[name](lib, p, c, None, VP((1 << 20) + 16), need) == kvc.KVC_EWORKSPACE


@pytest.mark.parametrize("name,idx", [("attn", i) for i in (0, 1, 2, 4, 5, 11)] + [("mass", 0), ("mass", 1),
                                                                                   ("evict", 3), ("evict", 4)])
def test_row_arrays_off_a_16_byte_boundary_are_rejected(lib, name, idx):
    ptrs = _fake(N_PTR[name])
    ptrs[idx] = VP(4096 * (idx + 1) + 8)
    assert CALLS[name](lib, _params(), _chunk(), ptrs) == kvc.KVC_EINVAL


def test_output_is_written_in_whole_sectors(lib):
    ptrs = _fake(14)
    ptrs[11] = VP(4096 * 12 + 16)
    assert _attn(lib, _params(), _chunk(), ptrs) == kvc.KVC_EINVAL


def test_scalars_are_checked(lib):
    p, c = _params(), _chunk()
    for decay in (-0.1, 1.1, float("nan")):
        assert _mass(lib, p, c, decay=decay) == kvc.KVC_EINVAL
    assert _evict(lib, p, c, recent=-1) == kvc.KVC_EINVAL
    assert _evict(lib, p, c, max_len=0) == kvc.KVC_EINVAL
    assert kvc.kvc_mass_evict_workspace_bytes(p, c, 0) == 0
    assert _evict(lib, _params(B=9000), c) == kvc.KVC_EINVAL   # 72000 (b,l,h): one grid dimension each


def test_chunk_struct_layout(lib):
    assert ctypes.sizeof(kvc.kvc_chunk) == 56
    assert kvc.kvc_chunk.page_table.offset == 32 and kvc.kvc_chunk.slopes.offset == 48


def test_make_chunk_checks_types():
    with pytest.raises(TypeError):
        kvc.make_chunk(1, n_new=torch.zeros(1, dtype=torch.int64))
    c = kvc.make_chunk(3, 1, 2, softcap=5.0, window=7.0)
    assert (c.T, c.layer_begin, c.layer_end, c.page_rows, c.max_pages) == (3, 1, 2, 0, 0)
    assert c.page_table is None and c.n_new is None and c.slopes is None


def test_extend_keeps_an_outgrown_workspace(monkeypatch):
    # a call captured with the smaller workspace replays with it after a larger turn
    from kv_cache_compression_probe_gb300 import kvc, pipeline
    used = []
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_attn", lambda *a: used.append(a[-2].data_ptr()))
    comp = object.__new__(pipeline.Compressor)
    comp.p = kvc.make_params(B=1, L=2, H=2, G=4, d=128, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16)
    comp.device, comp._ws_chunk, comp._ws_outgrown = "cpu", None, []
    comp.Kp = torch.zeros(64, 128)
    for name in ("Vp", "logm", "pos", "len_lh", "cap_lh", "off_lh"):
        setattr(comp, name, None)
    sizes = {1: 256, 40: 1024, 2: 256, 300: 4096}
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_workspace_bytes", lambda p, c: sizes[c.T])
    for T in (1, 40, 2, 300):
        q, k = (torch.zeros(1, 2, n, T, 128, dtype=torch.bfloat16) for n in (8, 2))
        comp.extend(q, k, k, q, torch.zeros(1))
    assert used[1] == used[2] and len(set(used)) == 3
    assert [w.data_ptr() for w in comp._ws_outgrown] + [comp._ws_chunk.data_ptr()] == [used[0], used[1], used[3]]


BAD_CHUNKS = {
    "q of another type": dict(q=torch.zeros(1, 2, 8, 4, 128)),
    "q of four dimensions": dict(q=torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)),
    "q of three dimensions": dict(q=torch.zeros(8, 4, 128, dtype=torch.bfloat16)),
    "no token": {n: torch.zeros(1, 2, h, 0, 128, dtype=torch.bfloat16)
                 for n, h in (("q", 8), ("k_new", 2), ("v_new", 2), ("out", 8))},
    "fewer keys than queries": dict(k_new=torch.zeros(1, 2, 2, 3, 128, dtype=torch.bfloat16)),
    "values for every query head": dict(v_new=torch.zeros(1, 2, 8, 4, 128, dtype=torch.bfloat16)),
    "a short out": dict(out=torch.zeros(1, 2, 8, 3, 128, dtype=torch.bfloat16)),
    "a layer less": dict(out=torch.zeros(1, 1, 8, 4, 128, dtype=torch.bfloat16)),
    "counts of 64 bits": dict(n_new=torch.zeros(1, dtype=torch.int64)),
    "counts of another batch": dict(n_new=torch.zeros(2, dtype=torch.int32)),
}


@pytest.mark.parametrize("name", list(BAD_CHUNKS))
def test_extend_and_step_refuse_tensors_of_other_shapes(monkeypatch, name):
    from kv_cache_compression_probe_gb300 import pipeline
    calls = []
    monkeypatch.setattr(pipeline.kvc, "kvc_chunk_attn", lambda *a: calls.append(a))
    p = kvc.make_params(B=1, L=2, H=2, G=4, d=128, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16)
    x = {n: torch.zeros(1, 2, h, 4, 128, dtype=torch.bfloat16)
         for n, h in (("q", 8), ("k_new", 2), ("v_new", 2), ("out", 8))}
    x.update(BAD_CHUNKS[name])
    comp = object.__new__(pipeline.Compressor)
    comp.p, comp.device, comp._ws_chunk, comp.Kp = p, "cpu", None, torch.zeros(64, 128)
    with pytest.raises(ValueError):
        comp.extend(pos_new=torch.zeros(1), **x)
    if "n_new" not in x:                                # (the cache copies the counts into its own)
        cache = object.__new__(pipeline.ChunkedCache)
        cache.p, cache.T = p, 40
        with pytest.raises(ValueError):
            cache.step(**x)
    assert not calls
