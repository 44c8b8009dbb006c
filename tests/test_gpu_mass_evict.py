"""kvc_mass_evict against the float64 oracle: the kept set, the moves and the new
lengths bit for bit, over ties, NaN, infinities, protection, pages and lengths."""
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


def _run(kvc, ch, keep, recent, max_len=None, in_place=False, stream=None, ws=None, s=None):
    s = s or ch.upload()
    max_len = int(max_len or max(1, ch.lens.max()))
    ws = ws if ws is not None else torch.empty(
        kvc.kvc_mass_evict_workspace_bytes(s["p"], s["c"], max_len), dtype=torch.uint8, device="cuda").fill_(0xFF)
    k = torch.from_numpy(np.asarray(keep, np.int32).reshape(ch.B, ch.L, ch.H)).cuda()
    kvc.kvc_mass_evict(s["p"], s["c"], s["mass"], k, recent, s["pos_new"], s["K"], s["V"], s["logm"],
                       s["pos"], s["len"], None if ch.page else s["off"],
                       s["len"] if in_place else s["len_out"], max_len, ws, stream)
    return s


def _check(ch, s, keep, recent, in_place=False):
    K, V = ch.K.clone(), ch.V.clone()
    arr = {k: getattr(ch, k).copy() for k in ("logm", "pos", "mass")}
    lens = (ch.lens if in_place else np.full(len(ch.lens), -3)).copy()
    keep = np.asarray(keep).reshape(-1)
    for u in ch.units:
        n = int(ch.lens[u])
        r = ch.rows(u, n)
        B, holes, movers = O.mass_evict(ch.mass[r], ch.pos[r], keep[u],
                                        ch.pos_new[u // (ch.L * ch.H)] - np.float32(recent))
        lens[u] = B
        assert len(holes) == len(movers)
        K[r[holes]], V[r[holes]] = K[r[movers]], V[r[movers]]
        for a in arr.values():
            a[r[holes]] = a[r[movers]]
    bits = torch.int16 if ch.dtype == "bf16" else torch.int32
    np.testing.assert_array_equal(s["len" if in_place else "len_out"].cpu().numpy().reshape(-1), lens)
    for k, a in arr.items():
        np.testing.assert_array_equal(s[k].cpu().numpy(), a, err_msg=k)
    assert torch.equal(s["K"].cpu().view(bits), K.view(bits)) and torch.equal(s["V"].cpu().view(bits), V.view(bits))


CASES = {
    "edges": (dict(lens=[0, 1, 2, 31, 32, 33, 500, 1023, 1024, 1025, 2049, 5000], n_new=[0, 0], B=2, L=3, H=2), 0.5, 16),
    "f32, d 64": (dict(lens=[0, 1, 700, 3000], n_new=[0], H=4, dtype="f32", d=64), 0.3, 10),
    "f32, d 128": (dict(lens=[90, 700], n_new=[0], H=2, dtype="f32"), 0.9, 0),
    "paged 16": (dict(lens=[0, 15, 16, 17, 300, 1000], n_new=[0, 0], B=2, H=3, page=16), 0.6, 32),
    "paged 128": (dict(lens=[700, 3000], n_new=[0], H=2, page=128), 0.25, 200),
    "keep everything": (dict(lens=[700, 30], n_new=[0], H=2), 1.5, 3),
    "keep nothing": (dict(lens=[700, 30], n_new=[0], H=2), 0.0, 0),
    "below zero": (dict(lens=[700, 30], n_new=[0], H=2), -0.1, 0),
    "protection above the target": (dict(lens=[700, 30], n_new=[0], H=2), 0.1, 400),
    "all protected": (dict(lens=[700, 30], n_new=[0], H=2), 0.1, 100000),
    "layer range": (dict(lens=[5, 70, 200, 130, 64, 9, 1, 300], n_new=[0, 0], B=2, L=4, layers=(1, 3)), 0.5, 8),
    "long": (dict(lens=[70001, 40], n_new=[0], H=2), 0.4, 1000),
    "long, spread over a cluster": (dict(lens=[70001, 5000, 4097, 8191, 3, 0, 20000, 12345], n_new=[0], H=8, d=64), 0.4, 1000),
    "longer than shared memory": (dict(lens=[410003, 1000], n_new=[0], H=2, d=64), 0.7, 100),
    "one unit per CTA, long": (dict(lens=[60001] + [10] * 23, n_new=[0], H=24, d=64), 0.3, 100),
    "many units": (dict(lens=np.arange(600) * 7 % 301, n_new=[0, 0], B=2, L=20, H=15), 0.7, 20),
}


@pytest.mark.parametrize("masses", ["distinct", "ties", "odd"])
@pytest.mark.parametrize("name", list(CASES))
def test_eviction(kvc, name, masses):
    kw, frac, recent = CASES[name]
    ch = Chunk(kvc, seed=list(CASES).index(name), T=1, **kw)
    rng = np.random.default_rng(3)
    if masses == "ties":                                # a handful of values: ties at the cut
        ch.mass[:] = np.where(np.isnan(ch.mass), np.nan, rng.integers(0, 3, len(ch.mass)) * 0.25)
    elif masses == "odd":                               # NaN, infinities, both zeros, negative masses
        some = np.asarray([np.nan, np.inf, -np.inf, -0.0, 0.0, -1.0, 1e-45, 3e38], np.float32)
        ch.mass[:] = np.where(np.isnan(ch.mass), np.nan, some[rng.integers(0, 8, len(ch.mass))])
    keep = np.floor(ch.lens * frac).astype(np.int64)
    s = _run(kvc, ch, keep, recent)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    _check(ch, s, keep, recent)


@pytest.mark.parametrize("recent", [0, 50])
@pytest.mark.parametrize("step", [1 << 21, 1 << 10, 1])
def test_the_cut_falls_at_every_level_of_the_search(kvc, step, recent):
    # masses in pairs whose bit patterns are `step` apart: their codes part in the first, second
    # or last digit of the search; an even target keeps whole pairs, an odd one parts a pair
    ch = Chunk(kvc, [400, 401, 6001, 2], [0], H=4, T=1, seed=step % 97)
    rng = np.random.default_rng(5)
    for u in range(4):
        r = ch.rows(u, int(ch.lens[u]))
        bits = np.uint32(0x04000000) + np.uint32(step) * (np.arange(len(r), dtype=np.uint32) // 2 % 900)
        ch.mass[r] = rng.permutation(bits).view(np.float32)
    for keep in (100, 101, 399, 5000, 5001):
        s = _run(kvc, ch, [keep] * 4, recent)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        _check(ch, s, [keep] * 4, recent)


def test_in_place_lengths_and_a_second_eviction(kvc):
    ch = Chunk(kvc, [700, 30, 1025, 64], [0, 0], B=2, H=2, T=1)
    keep = np.asarray([500, 30, 800, 10])
    s = _run(kvc, ch, keep, 16, in_place=True)
    torch.cuda.synchronize()
    _check(ch, s, keep, 16, in_place=True)
    for k in ("logm", "pos", "mass"):                   # evict again from what is left
        setattr(ch, k, s[k].cpu().numpy())
    ch.K, ch.V = s["K"].cpu(), s["V"].cpu()
    ch.lens = s["len"].cpu().numpy().astype(np.int64).reshape(-1)
    s2 = _run(kvc, ch, keep // 2, 16)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    _check(ch, s2, keep // 2, 16)


def test_bad_units_keep_their_length(kvc):
    for what in ("length", "max_len", "rows", "page"):
        ch = Chunk(kvc, [700, 300, 64, 90], [0], H=4, T=1, page=64 if what == "page" else 0)
        if what == "length":
            ch.lens[1] = -5
        elif what == "rows":
            ch.off[1] = ch.rows_total - 10
        elif what == "page":
            ch.table[1, 2] = 1 << 20
        s = ch.upload()
        before = {k: s[k].clone() for k in ("mass", "pos", "logm")}
        _run(kvc, ch, [350, 100, 32, 45], 4, max_len=699 if what == "max_len" else 700, s=s)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == kvc.KVC_EDEVICE, what
        bad = 0 if what == "max_len" else 1
        got = s["len_out"].view(-1).tolist()
        assert got[bad] == s["len"].view(-1)[bad], what
        want = {0: 350, 1: 100, 2: 32, 3: 45}
        assert all(got[u] == want[u] for u in range(4) if u != bad), (what, got)
        if what in ("max_len",):
            r = torch.from_numpy(ch.rows(0, 700)).cuda()
            for k, v in before.items():
                assert torch.equal(v[r], s[k][r])


def test_captured_eviction_replays(kvc):
    ch = Chunk(kvc, [700, 30, 1025, 64], [0, 0], B=2, H=2, T=1, page=16)
    keep = np.asarray([500, 30, 800, 10])
    s = ch.upload()
    ws = torch.empty(kvc.kvc_mass_evict_workspace_bytes(s["p"], s["c"], 1025), dtype=torch.uint8, device="cuda")
    k = torch.from_numpy(keep.astype(np.int32)).cuda()
    kvc.kvc_device_error()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kvc.kvc_mass_evict(s["p"], s["c"], s["mass"], k, 16, s["pos_new"], s["K"], s["V"], s["logm"], s["pos"],
                           s["len"], None, s["len_out"], 1025, ws, side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        e = ch.upload()
        for n in ("K", "V", "logm", "pos", "mass"):
            s[n].copy_(e[n])
        g.replay()
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        _check(ch, s, keep, 16)
