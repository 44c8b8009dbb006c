"""The 8-bit cache's oracle pins and host-side refusals (no GPU: the fake pointers are
never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

from kv_cache_compression_probe_gb300 import kvc
from oracle import q8_oracle as Q

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from kv_cache_compression_probe_gb300 import build
    build.build()
    return kvc.lib()


# ------------------------------------------------------------------ oracle
def test_oracle_e4m3_is_torchs():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 9, 4000), np.arange(-500, 500) / 2.0 ** 10,
                        [0.0, 448.0, 448.1, -1000.0, 2.0 ** -10, 3 * 2.0 ** -10, 464.0]]).astype(np.float32)
    t = torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(Q.e4m3_round(v), t.double().numpy())
    np.testing.assert_array_equal(Q.e4m3_decode(t.view(torch.uint8).numpy()), t.double().numpy())


def test_oracle_scale_is_the_least_that_holds():
    for top in (448.0, np.nextafter(np.float32(448), np.float32(449)), 447.0, 1.0, 0.875, 0.876, 3.5, 1e-3, 300.7):
        x = Q.scale_exp(top)
        assert top <= 448 * 2.0 ** x and top > 448 * 2.0 ** (x - 1)
    assert Q.scale_exp(0.0) == Q.scale_exp(1e-30) == -40 and Q.scale_exp(1e30) == 40


def test_oracle_page_grows_in_parts_as_at_once():
    """Up to codes that become subnormal on the way, a page filled in parts holds the same
    values as one filled at once."""
    rng = np.random.default_rng(1)
    w = (rng.standard_normal((16, 8)) * 2.0 ** np.arange(16)[:, None] / 64).astype(np.float32)
    whole, x = Q.page_append(np.zeros((0, 8)), 0, w)
    parts, y = np.zeros((0, 8)), 0
    for r in range(16):
        parts, y = Q.page_append(parts, y, w[r:r + 1])
    assert x == y
    big = np.abs(whole) >= 2.0 ** -6
    np.testing.assert_array_equal(parts[big], whole[big])
    assert np.abs(parts - whole).max() <= 16 * 2.0 ** -10
    np.testing.assert_array_equal(Q.bounds(whole)[1], np.rint(whole.max(0) / 4))


def test_oracle_rotation_is_complex_multiplication():
    rng = np.random.default_rng(2)
    x, th = rng.standard_normal((5, 8)), rng.uniform(0, 6, (5, 4))
    z = (x[:, :4] + 1j * x[:, 4:]) * np.exp(1j * th)
    got = Q.rope(x, np.cos(th), np.sin(th))
    np.testing.assert_allclose(got, np.concatenate([z.real, z.imag], 1), atol=1e-6)


def test_oracle_score_bounds_the_products():
    """With integer keys and queries the score is an upper bound, and pages with the key nearest
    to a query are picked."""
    rng = np.random.default_rng(3)
    K = rng.integers(-100, 101, (40, 16, 32)) * 4.0
    q = rng.integers(-127, 128, (2, 32)).astype(np.float32)
    q[:, 0] = 127
    bd = np.stack([Q.bounds(k) for k in K])
    D = np.maximum(q[:, None] * bd[None, :, 0] * 4, q[:, None] * bd[None, :, 1] * 4).sum(-1)
    assert (np.einsum("gd,prd->gpr", q, K).max(-1) <= D).all()
    got = Q.pick_pages(q, bd, np.ones(40, np.float32), 39, 6, 1, 2)
    assert len(got) == 6 and {0, 38, 39} <= set(got) and (np.diff(got) > 0).all()
    rest = [j for j in np.argsort(-D.max(0), kind="stable") if j not in (0, 38, 39)][:3]
    assert set(got) == {0, 38, 39, *rest}
    np.testing.assert_array_equal(Q.pick_pages(q * 0, bd, np.ones(40, np.float32), 39, 6, 1, 2), [0, 1, 2, 3, 38, 39])


def test_oracle_attention_over_all_picked_pages_is_attention():
    rng = np.random.default_rng(4)
    q, K, V, lm = rng.standard_normal((2, 3, 8)), rng.standard_normal((40, 8)), rng.standard_normal((40, 8)), rng.uniform(0, 1, 40)
    a, b = Q.q8_attn(q, K, V, lm, 37, 16), Q.q8_attn(q, K, V, lm, 37, 16, [[0, 1, 2]] * 3)
    np.testing.assert_array_equal(a[0], b[0])
    s = torch.einsum("gtd,nd->gtn", *map(torch.from_numpy, (q, K))) / 8 ** 0.5 + torch.from_numpy(lm)
    s[:, 0, 38:], s[:, 1, 39:] = -np.inf, -np.inf
    np.testing.assert_allclose(a[0], (torch.softmax(s, -1) @ torch.from_numpy(V)).numpy(), rtol=1e-11)
    np.testing.assert_allclose(a[1], torch.logsumexp(s, -1).numpy() / np.log(2), rtol=1e-12)


# ------------------------------------------------------------------ refusals
def _params(**over):
    kw = dict(B=2, L=4, H=2, G=4, d=128, P=1, W=1, dtype=kvc.KVC_BF16, n_max=64, S_max=1, packed_rows=4096)
    kw.update(over)
    return kvc.make_params(**kw)


def _chunk(**over):
    c = kvc.kvc_chunk()
    kw = dict(T=4, layer_begin=0, layer_end=4, page_rows=64, max_pages=8, page_table=VP(4096))
    kw.update(over)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _cache(**over):
    x = kvc.kvc_q8()
    kw = {n: 4096 * (i + 40) for i, n in enumerate(("K", "V", "k_scale", "v_scale", "bounds", "logm"))}
    kw.update(over)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def _fake(k):
    return [VP(4096 * (i + 1)) for i in range(k)]


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _append(lib, p, c, x, ptrs=None, n_half=100):
    a = ptrs or _fake(10)
    return lib.kvc_q8_append(_ref(p), _ref(c), _ref(x), a[0], a[1], n_half, *a[2:], None)


def _pack(lib, p, c, x, ptrs=None, rows=100):
    a = ptrs or _fake(7)
    return lib.kvc_q8_pack(_ref(p), _ref(c), _ref(x), *a[:3], rows, *a[3:], None)


def _select(lib, p, c, x, ptrs=None, n_sel=8, first=1, recent=2):
    a = ptrs or _fake(4)
    return lib.kvc_q8_select(_ref(p), _ref(c), _ref(x), *a[:3], n_sel, first, recent, a[3], None)


def _attn(lib, p, c, x, ptrs=None, n_sel=8, ws=VP(1 << 20), nb=1 << 40):
    a = ptrs or _fake(6)
    return lib.kvc_q8_attn(_ref(p), _ref(c), _ref(x), *a[:4], n_sel, a[4], a[5], ws, ctypes.c_size_t(nb), None)


CALLS = {"append": _append, "pack": _pack, "select": _select, "attn": _attn}
BAD_CHUNK = [dict(T=0), dict(T=65537), dict(layer_begin=-1), dict(layer_begin=4), dict(layer_end=5), dict(page_rows=0),
             dict(page_rows=8), dict(page_rows=48), dict(page_rows=256), dict(page_rows=1024), dict(max_pages=0),
             dict(page_table=None), dict(softcap=1.0), dict(window=5.0), dict(slopes=VP(4096)), dict(softcap=float("nan")),
             dict(max_pages=1 << 24)]
BAD_PARAMS = [dict(B=0), dict(G=3), dict(d=96), dict(dtype=5), dict(packed_rows=0), dict(packed_rows=1 << 31),
              dict(packed_rows=32), dict(B=1 << 16, H=1 << 10)]
BAD_CACHE = [dict(K=None), dict(V=None), dict(k_scale=None), dict(v_scale=None), dict(K=4096 * 40 + 8), dict(V=4096 * 41 + 4),
             dict(bounds=4096 * 44 + 8)]


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_blocks_are_refused(lib, name):
    call = CALLS[name]
    for bad in BAD_CHUNK:
        assert call(lib, _params(), _chunk(**bad), _cache()) == kvc.KVC_EINVAL, bad
    for bad in BAD_PARAMS:
        assert call(lib, _params(**bad), _chunk(), _cache()) == kvc.KVC_EINVAL, bad
    for bad in BAD_CACHE:
        assert call(lib, _params(), _chunk(), _cache(**bad)) == kvc.KVC_EINVAL, bad
    assert call(lib, None, _chunk(), _cache()) == kvc.KVC_EINVAL
    assert call(lib, _params(), None, _cache()) == kvc.KVC_EINVAL
    assert call(lib, _params(), _chunk(), None) == kvc.KVC_EINVAL


# positions that may be missing (lse); those that go together are tested below
N_PTR = {"append": 10, "pack": 7, "select": 4, "attn": 6}


@pytest.mark.parametrize("name", list(CALLS))
def test_missing_pointers_are_refused(lib, name):
    for i in range(N_PTR[name]):
        if (name, i) == ("attn", 5):
            continue
        ptrs = _fake(N_PTR[name])
        ptrs[i] = None
        assert CALLS[name](lib, _params(), _chunk(), _cache(), ptrs) == kvc.KVC_EINVAL, i


@pytest.mark.parametrize("name,idx", [("append", i) for i in (0, 1, 2, 3, 4, 6)] + [("pack", 0), ("pack", 1), ("select", 0),
                                                                                  ("attn", 0), ("attn", 4)])
def test_row_arrays_off_their_boundary_are_refused(lib, name, idx):
    ptrs = _fake(N_PTR[name])
    ptrs[idx] = VP(4096 * (idx + 1) + 8)
    assert CALLS[name](lib, _params(), _chunk(), _cache(), ptrs) == kvc.KVC_EINVAL


def test_arguments_that_go_together(lib):
    p, c, x = _params(), _chunk(), _cache()
    a = _fake(10)
    assert _append(lib, p, c, x, a[:9] + [a[7]]) == kvc.KVC_EINVAL             # len_out = len_lh
    assert _append(lib, p, c, x, n_half=0) == kvc.KVC_EINVAL
    b = _fake(7)
    assert _pack(lib, p, c, x, b[:6] + [b[3]]) == kvc.KVC_EINVAL
    assert _pack(lib, p, c, _cache(logm=None)) == kvc.KVC_EINVAL               # log m has nowhere to go
    assert _pack(lib, p, c, x, rows=0) == kvc.KVC_EINVAL
    assert _select(lib, p, c, _cache(bounds=None)) == kvc.KVC_EINVAL
    for bad in (dict(n_sel=0), dict(n_sel=-1), dict(n_sel=32769), dict(first=-1), dict(recent=0), dict(first=7, recent=2),
                dict(first=2 ** 31 - 1, recent=2)):
        assert _select(lib, p, c, x, **bad) == kvc.KVC_EINVAL, bad
    assert _select(lib, _params(packed_rows=1 << 24), _chunk(page_rows=16, max_pages=32769), x) == kvc.KVC_EINVAL
    for bad in (-1, 0):
        assert _attn(lib, p, c, x, n_sel=bad) == kvc.KVC_EINVAL
    d = _fake(6)
    d[3] = None
    assert _attn(lib, p, c, x, d, n_sel=0, ws=None) == kvc.KVC_EWORKSPACE
    assert _attn(lib, p, c, x, d, n_sel=4) == kvc.KVC_EINVAL


@pytest.mark.parametrize("n_sel", [0, 8])
def test_workspaces(lib, n_sel):
    p, c, x = _params(), _chunk(), _cache()
    need = kvc.kvc_q8_workspace_bytes(p, c, n_sel)
    assert need > 0
    ptrs = _fake(6)
    if n_sel == 0:
        ptrs[3] = None
    for ws, nb in ((None, need), (VP(1 << 20), need - 1), (VP((1 << 20) + 64), need)):
        assert _attn(lib, p, c, x, ptrs, n_sel, ws, nb) == kvc.KVC_EWORKSPACE
    for bad in (dict(page_rows=0), dict(page_rows=256), dict(T=0)):
        assert kvc.kvc_q8_workspace_bytes(p, _chunk(**bad), n_sel) == 0
    assert kvc.kvc_q8_workspace_bytes(p, c, -1) == 0
    assert kvc.kvc_q8_workspace_bytes(_params(d=32), c, n_sel) == 0


def test_struct_layout_and_types():
    assert ctypes.sizeof(kvc.kvc_q8) == 48 and kvc.kvc_q8.logm.offset == 40
    z = torch.zeros(16, 128, dtype=torch.uint8)
    with pytest.raises(TypeError):
        kvc.make_q8(z.float(), z, z, z)
    with pytest.raises(ValueError):
        kvc.make_q8(z, z, torch.ones(1), torch.ones(1))                        # not on a GPU
