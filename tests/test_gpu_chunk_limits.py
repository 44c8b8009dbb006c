"""The chunk calls at the ends of what they accept: caps of every size, caches without
room, windows that are no multiple of 1/2, values of 2^64.  Small cases against the
float64 oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.chunk_cases import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()                           # buffers full of NaN stay with this module


# ------------------------------------------------------------------ caps
FAST_CAP = 64.0                                        # up to here bf16 attention may use the short form


class Capped(Chunk):
    def score_error(self, u):
        """Bound on the error of each natural-log score that does not grow with the cap: the d
        products in fp32 (as in Chunk), cap * tanh(s / cap) off by at most 2^-21 of its
        value (tanh by 9e-8, a product and a sum, each half a step of 2^-24), ln m and bias a
        handful of half steps.  The short form cap - 2 cap / (1 + e^2y) adds the errors of e^2y
        (2^-22 of it), of the sum (2^-24), the reciprocal (2^-23) and of two roundings at the
        cap's size: 4.5 * 2^-23 of the cap, up to FAST_CAP and on the bf16 path only."""
        K, V, lm, pos, q, (b, lr, hs, n, n0) = self.entries(u)
        dots = np.abs(q) @ np.abs(K).T / np.sqrt(self.d)
        size = dots + np.abs(np.where(np.isinf(lm), 0.0, lm))
        if self.slopes is not None:
            gap = np.abs((float(self.pos_new[b]) + np.arange(n))[:, None] - pos[None])
            size = size + self.slopes_of(u)[:, None, None] * gap
        short = 4.5 * 2.0 ** -23 * self.softcap if self.dtype == "bf16" and self.softcap <= FAST_CAP else 0.0
        return self.d * 2.0 ** -23 * dots + 2.0 ** -21 * size + short


CAPS = (1e-30, 30.0, 64.0, 65.0, 1e3, 1e5, 1e7, 1e20, 3e38)
CAP_CASES = {
    "one token": (dict(lens=[300, 1025], n_new=[1], H=2), "bf16"),
    "one token, slopes, window, paged": (dict(lens=[300, 1025], n_new=[1], H=2, slopes=True, window=700.0, page=64), "bf16"),
    "chunk": (dict(lens=[300, 50], n_new=[140], H=2), "bf16"),
    "chunk, slopes, d 64": (dict(lens=[300, 50], n_new=[150], H=2, slopes=True, d=64), "bf16"),
    "f32 chunk": (dict(lens=[300, 50], n_new=[40], H=2, slopes=True), "f32"),
}


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("name", list(CAP_CASES))
def test_caps_of_every_size(kvc, name, cap):
    """Attention, then the mass from its lse: both match the oracle, and the weights of all
    rows add up to their number."""
    kw, dtype = CAP_CASES[name]
    ch = Capped(kvc, dtype=dtype, softcap=cap, qscale=2.0, seed=11, **kw)
    s = ch.upload()
    ch.attn(s)
    ch.run_mass(s, 0.0)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s, name)
    lse = s["lse"].cpu().numpy()
    ch.check_mass(s, lse, 0.0, name)
    mass = s["mass"].double().cpu().numpy()
    for u in ch.units:
        where = ch.entries(u)[5]
        n, n0 = where[3], where[4]
        r = ch.rows(u, n0 + n)
        # a row's weights: the error of every score twice (lse and mass form it anew), of the lse
        # (half a step of its value) and of 2^x and the sums
        rows = ch.G * n
        tol = rows * (2 * ch.score_error(u).max() + 2.0 ** -23 * (np.abs(lse[lse != 7.0]).max() + 1)
                      + 2.0 ** -20 + (n0 + n) * 2.0 ** -24)
        assert abs(mass[r].sum() - rows) <= tol, (name, u, mass[r].sum() - rows, tol)


# ------------------------------------------------------------------ no room
def _full(kvc, page, dtype, **kw):
    """Four sequences, the second without room for its tokens; its rows end where the third's begin
    (with a reserve: that many rows before)."""
    ch = Chunk(kvc, [100, 90, 300, 64], [5, 2, 3, 4], B=4, H=1, T=5, page=page, dtype=dtype, seed=9, **kw)
    ch.n[1] = 5                                        # the capacity is for two
    ch.n_u = np.repeat(ch.n, ch.L * ch.H)
    for t in (ch.q, ch.k_new, ch.v_new):
        t[1] = torch.randn(t[1].shape).to(t.dtype)
    ch.caps = ch.caps - kw.get("reserve", 0)
    return ch


def _mass(kvc, ch, s, decay, cap):
    kvc.kvc_chunk_mass(s["p"], s["c"], s["q"], s["K"], s["logm"], s["pos"], s["pos_new"], s["len"],
                       None if ch.page else s["off"], s["lse"], decay, s["mass"], s["ws"], None, cap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["packed", "packed, capacities not passed", "spread", "paged", "window"])
def test_a_full_unit_is_left_out_of_the_mass_too(kvc, how, dtype):
    """Attention skips a unit without room; the mass call after it leaves that unit's mass and
    its neighbours' alone."""
    page = 16 if how == "paged" else 0
    kw = dict(reserve=8) if how == "spread" else dict(window=50.0) if how == "window" else {}
    ch = _full(kvc, page, dtype, **kw)
    s = ch.upload()
    ch.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == kvc.KVC_ECAPACITY
    _mass(kvc, ch, s, 0.5, None if "not passed" in how else s["cap"])
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == kvc.KVC_ECAPACITY
    ch.units = [0, 2, 3]                               # check_mass: every other row as it was
    ch.check_mass(s, s["lse"].cpu().numpy(), 0.5, how)


def test_mass_with_room_everywhere_is_the_same_with_capacities(kvc):
    ch = Chunk(kvc, [100, 90, 300, 64], [5, 3], B=2, H=2, reserve=1)
    s = ch.upload()
    ch.attn(s)
    m0 = s["mass"].clone()
    _mass(kvc, ch, s, 0.5, None)
    m1 = s["mass"].clone()
    s["mass"].copy_(m0)
    _mass(kvc, ch, s, 0.5, s["cap"])
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    assert torch.equal(s["mass"].view(torch.int32), m1.view(torch.int32))
    ch.check_mass(s, s["lse"].cpu().numpy(), 0.5)


# ------------------------------------------------------------------ windows
def _next(x):
    return float(np.nextafter(np.float32(x), np.float32(np.inf)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [33.7, _next(33.0), _next(0.0), 0.25])
def test_windows_between_the_half_integers(kvc, window, dtype):
    """Positions are multiples of 1/2, a window need not be: an entry just inside it is seen,
    whatever pos_token - window rounds to."""
    ch = Chunk(kvc, [300, 50], [140], H=2, dtype=dtype, window=window, seed=3)
    s = ch.upload()
    ch.attn(s)
    ch.run_mass(s, 0.5)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s, window)
    ch.check_mass(s, s["lse"].cpu().numpy(), 0.5, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_edge_at_a_far_position(kvc, dtype):
    """The only visible old entry lies alone in its tile, half a position inside the window, at a
    position where fp32 keeps halves only."""
    ch = Chunk(kvc, [700], [3], dtype=dtype, window=33.7, seed=4)
    ch.pos_new[:] = 5000001.0
    r = ch.rows(0, 700)
    ch.pos[r] = 4000000.0 + np.arange(700)
    ch.pos[r[200]] = 4999967.5                         # 33.5 before the first new token
    s = ch.upload()
    ch.attn(s)
    ch.run_mass(s, 0.5)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s, "edge")
    ch.check_mass(s, s["lse"].cpu().numpy(), 0.5, "edge")


# ------------------------------------------------------------------ large values
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("natural", [37.1, -37.1, 90.0, 19.0])
def test_values_up_to_2_64(kvc, natural, n, dtype):
    """All scores far from 0 and |v| up to 2^64: nothing overflows on the way to the average."""
    ch = Chunk(kvc, [5000], [n], dtype=dtype, seed=5)
    r = ch.rows(0, 5000)
    k = natural * np.sqrt(ch.d) / ch.d
    ch.q[:], ch.K[r], ch.k_new[:] = 1.0, k, k
    ch.logm[r] = 0.0
    ch.V[r] = (ch.V[r].float().abs().clamp(0.25, 1.0) * 2.0 ** 64).to(ch.V.dtype)
    ch.v_new[:] = (ch.v_new.float().abs().clamp(0.25, 1.0) * 2.0 ** 64).to(ch.V.dtype)
    s = ch.upload()
    ch.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s, natural)


# ------------------------------------------------------------------ a step that is skipped
def test_a_skipped_step_leaves_no_gap(kvc):
    """A cache that is asked for more than it has room for goes on as if it had not been asked."""
    from kv_cache_compression_probe_gb300.pipeline import ChunkedCache

    def make():
        p = kvc.make_params(B=2, L=2, H=2, G=4, d=64, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16)
        sl = 2.0 ** -torch.arange(1, 9, dtype=torch.float32, device="cuda")
        return ChunkedCache(p, budget=32, T=8, page_rows=16, recent=4, slopes=sl, window=40.0)
    g = torch.Generator().manual_seed(2)
    caches, outs = (make(), make()), ([], [])
    for ns, evict, refused in (([8, 8], True, False), ([8, 5], False, False), ([8, 8], False, False),
                               ([8, 8], False, False), ([8, 8], False, False), ([8, 8], False, False),
                               ([8, 1], False, True), ([9, 0], False, True), ([0, 2], True, False), ([8, 8], True, False)):
        x = [torch.randn((2, 2, h, 8, 64), generator=g).to(torch.bfloat16).cuda() for h in (8, 2, 2)]
        for k, cache in enumerate(caches):
            n = torch.tensor([0, ns[1]] if refused and k else ns, dtype=torch.int32, device="cuda")
            if refused and k and ns[1] == 0:           # the other cache is not asked at all
                continue
            out = torch.zeros_like(x[0])
            cache.step(*x, out, n, evict=evict)
            torch.cuda.synchronize()
            code = kvc.kvc_device_error()
            if refused and k == 0:
                assert code == (kvc.KVC_ECAPACITY if ns[0] == 8 else kvc.KVC_EDEVICE)
            else:
                assert code == 0
                if not refused:
                    outs[k].append(out)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(caches[0].pos_next, caches[1].pos_next) and caches[0].pos_next.tolist() == [56.0, 56.0]
    assert torch.equal(caches[0].len_lh, caches[1].len_lh)


# ------------------------------------------------------------------ far rows
FAR = 17_000_000                                       # rows: 2^31 elements of d 128 lie before them


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 64])
def test_rows_past_32_bit_offsets(kvc, page, dtype):
    """Attention, mass and eviction of a cache whose rows begin beyond 2^31 elements."""
    n = [5, 40]
    ch = Chunk(kvc, [100, 300, 64, 700], n, B=2, H=2, dtype=dtype, page=page, window=200.0, slopes=True, seed=6)
    s = ch.upload()
    base = -(-FAR // 1024) * 1024
    small = {k: s[k] for k in ("K", "V", "logm", "pos", "mass")}
    for k, t in small.items():
        s[k] = torch.empty((base + t.shape[0], *t.shape[1:]), dtype=t.dtype, device="cuda")
        s[k][base:] = t
    s["p"].packed_rows = base + ch.rows_total
    s["off"] += base
    if page:
        s["c"]._keep[0].add_(base // page)
    ch.attn(s)
    ch.run_mass(s, 0.5)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(dict(s, **{k: s[k][base:] for k in small}), "far")
    ch.check_mass(dict(s, mass=s["mass"][base:]), s["lse"].cpu().numpy(), 0.5, "far")
    got = {k: s[k][base:].cpu() for k in small}        # and the eviction, from here
    keep = s["len_out"] // 2
    ws = torch.empty(kvc.kvc_mass_evict_workspace_bytes(s["p"], s["c"], 800), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(s["len_out"])
    kvc.kvc_mass_evict(s["p"], s["c"], s["mass"], keep, 8, s["pos_new"], s["K"], s["V"], s["logm"], s["pos"],
                       s["len_out"], None if page else s["off"], out, 800, ws)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    for u in ch.units:
        b = u // 2
        r = ch.rows(u, int(ch.lens[u]) + n[b])
        B, holes, movers = O.mass_evict(got["mass"].numpy()[r], got["pos"].numpy()[r], len(r) // 2,
                                        ch.pos_new[b] - np.float32(8))
        assert int(out.view(-1)[u]) == B
        for k, t in got.items():
            t[r[holes]] = t[r[movers]]
    for k, t in got.items():
        bits = torch.int16 if t.element_size() == 2 else torch.int32
        assert torch.equal(s[k][base:].cpu().view(bits), t.view(bits)), k


# ------------------------------------------------------------------ long chunks
LONG = {
    "slopes": dict(lens=[500, 130], n_new=[700], H=2, slopes=True, page=64),
    "window": dict(lens=[500, 130], n_new=[700], H=2, window=300.0),
    "cap": dict(lens=[500, 130], n_new=[700], H=2, softcap=20.0, qscale=3.0),
    "all of it, ragged": dict(lens=[500, 130, 0, 900], n_new=[700, 333], B=2, H=2, softcap=50.0, slopes=True,
                              window=411.5, page=128, qscale=3.0),
    "4000 tokens": dict(lens=[300], n_new=[4000], G=1, d=64, slopes=True),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(LONG))
def test_modified_scores_over_long_chunks(kvc, name, dtype):
    """Many row tiles with a bias, a window or a cap: attention, and the mass from its lse."""
    ch = Chunk(kvc, dtype=dtype, seed=30 + list(LONG).index(name), **LONG[name])
    s = ch.upload()
    ch.attn(s)
    ch.run_mass(s, 0.9)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s, name)
    ch.check_mass(s, s["lse"].cpu().numpy(), 0.9, name)
