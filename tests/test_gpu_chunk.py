"""kvc_chunk_attn and kvc_chunk_mass against the float64 oracle: types, head
layouts, lengths from none to several tiles, ragged chunks, pages that end inside
a tile, caps, distance bias, windows, layer ranges; unused rows hold NaN."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()                           # buffers full of NaN stay with this module


EDGE = [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]
CASES = {
    # one token: every length around the tiles
    "one token": dict(lens=EDGE, n_new=[1, 1], B=2, L=3, H=2),
    "one token, d 64": dict(lens=EDGE, n_new=[1], L=4, H=3, d=64),
    "one token, G 1": dict(lens=EDGE, n_new=[1], L=6, H=2, G=1),
    "one token, G 8, paged": dict(lens=EDGE, n_new=[1], L=6, H=2, G=8, page=16),
    "one token, long": dict(lens=[9000, 5, 20011, 300], n_new=[1], L=2, H=2),
    "empty cache": dict(lens=[0, 0], n_new=[1], H=2),
    "empty cache, chunk": dict(lens=[0, 0], n_new=[77], H=2),
    # chunks
    "two tokens": dict(lens=[0, 3, 128, 200], n_new=[2], H=4, G=2),
    "ragged chunks": dict(lens=[40, 0, 130, 300, 17, 64, 1, 255], n_new=[1, 17, 0, 33], B=4, H=2),
    "no new tokens anywhere": dict(lens=[40, 0], n_new=[0], H=2, T=4),
    "paged 16": dict(lens=[0, 15, 16, 17, 130, 300], n_new=[5, 21], B=2, H=3, page=16),
    "paged 64, G 8": dict(lens=[0, 15, 64, 65, 130, 300], n_new=[50, 21], B=2, H=3, G=8, page=64),
    "paged 128": dict(lens=[100, 700], n_new=[150], H=2, page=128),
    "paged 1024": dict(lens=[100, 1500], n_new=[40], H=2, page=1024),
    "paged 32, d 64": dict(lens=[31, 33], n_new=[130], H=2, d=64, page=32),
    "long chunk": dict(lens=[600, 129], n_new=[333], H=2),
    "long chunk, G 1": dict(lens=[100], n_new=[700], G=1),
    "long chunk, G 2, d 64": dict(lens=[100, 0], n_new=[300], H=2, G=2, d=64),
    "many units": dict(lens=np.arange(7 * 3 * 16) * 3 % 211, n_new=[1, 2, 3, 4, 5, 6, 7], B=7, L=3, H=16, G=2),
    "row tiles of every count": dict(lens=np.arange(24) * 97 % 1500 + 300, n_new=[1, 65, 129, 194], B=4, L=3, H=2,
                                     G=2, d=64, page=64, softcap=30.0),
    "runs of short units": dict(lens=np.where(np.arange(3000) % 7 == 3, 300, np.arange(3000) % 90), n_new=[1], L=250,
                                H=12, G=1, d=64),
    "runs of short units, paged": dict(lens=np.where(np.arange(1500) % 19 == 3, 500, np.arange(1500) % 60),
                                       n_new=[3, 1, 0], B=3, L=50, H=10, G=2, page=16),
    "layer range": dict(lens=[5, 70, 200, 130, 64, 9, 1, 300], n_new=[9, 20], B=2, L=4, layers=(1, 3)),
    "no n_new": dict(lens=[5, 70], n_new=[9, 9], B=2, pass_n_new=False),
    # scores
    "cap": dict(lens=[300, 50], n_new=[40], H=2, softcap=5.0, qscale=4.0),
    "cap, one token": dict(lens=[300, 50], n_new=[1], H=2, softcap=3.0, qscale=8.0),
    "slopes": dict(lens=[300, 50], n_new=[40], H=2, slopes=True, pos_gap=3.0),
    "slopes, one token, paged": dict(lens=[300, 50, 900], n_new=[1], H=3, slopes=True, page=16),
    "window": dict(lens=[300, 50], n_new=[40], H=2, window=33.5),
    "window 1: only itself": dict(lens=[300, 50], n_new=[40], H=2, window=1.0),
    "window, one token": dict(lens=[700, 50], n_new=[1], H=2, window=100.0, pos_gap=4.0),
    "window, long chunk": dict(lens=[900, 50], n_new=[290], H=2, window=150.0),
    "all of it": dict(lens=[300, 50, 0, 131], n_new=[140, 3], B=2, H=2, window=200.0, softcap=8.0,
                      slopes=True, page=64, pos_gap=2.0, qscale=3.0),
    "dead entries": dict(lens=[300, 129], n_new=[20], H=2, dead=0.7),
    "all entries dead": dict(lens=[300, 129], n_new=[1], H=2, dead=1.1),
    "sharp": dict(lens=[300, 700], n_new=[60], H=2, qscale=30.0),
}
F32 = ("one token", "one token, G 8, paged", "ragged chunks", "paged 64, G 8", "long chunk",
       "long chunk, G 2, d 64", "layer range", "cap", "slopes", "window", "all of it", "dead entries",
       "all entries dead", "sharp", "no new tokens anywhere")
ALL = [(n, "bf16") for n in CASES] + [(n, "f32") for n in F32]


@pytest.mark.parametrize("name,dtype", ALL, ids=[f"{n}-{t}" for n, t in ALL])
def test_chunk_attention(kvc, name, dtype):
    ch = Chunk(kvc, dtype=dtype, seed=list(CASES).index(name), **CASES[name])
    s = ch.upload()
    ch.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s, name)


@pytest.mark.parametrize("name,dtype", ALL, ids=[f"{n}-{t}" for n, t in ALL])
def test_chunk_mass(kvc, name, dtype):
    ch = Chunk(kvc, dtype=dtype, seed=100 + list(CASES).index(name), **CASES[name])
    s = ch.upload()
    lse = ch.set_lse(s)
    ch.run_mass(s, 0.75)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_mass(s, lse, 0.75, name)


def test_lengths_in_place_and_optional_outputs(kvc):
    """len_out may be len_lh itself, and lse and len_out may be left out; a call is
    repeatable bit for bit."""
    ch = Chunk(kvc, [100, 0, 300, 64], [7, 12], B=2, H=2)
    a, b, c = ch.upload(), ch.upload(), ch.upload()
    ch.attn(a)
    ch.attn(b, len_out="len", lse=None)
    ch.attn(c, len_out=None)
    ch.attn(c)
    torch.cuda.synchronize()
    assert torch.equal(b["len"], a["len_out"]) and (b["lse"] == 7.0).all()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["out"], c["out"])
    assert torch.equal(a["lse"], c["lse"]) and torch.equal(a["len_out"], c["len_out"])
    ch.check_attn(a)


def test_a_chunk_equals_its_tokens_one_by_one(kvc):
    """Causality across calls: a chunk's rows match the same tokens given one call each
    (to the tolerance of one rounding each way)."""
    n = 19
    ch = Chunk(kvc, [150, 63], [n], H=2, dtype="f32")
    s = ch.upload()
    ch.attn(s)
    one = ch.upload()
    c1 = kvc.make_chunk(1, 0, 1)
    for t in range(n):
        o = torch.empty((1, 1, ch.H * ch.G, 1, ch.d), device="cuda")
        kvc.kvc_chunk_attn(one["p"], c1, one["q"][:, :, :, t:t + 1].contiguous(),
                           one["k_new"][:, :, :, t:t + 1].contiguous(),
                           one["v_new"][:, :, :, t:t + 1].contiguous(), one["pos_new"] + t, one["K"],
                           one["V"], one["logm"], one["pos"], one["len"], one["cap"], one["off"], o,
                           None, one["len"], one["ws"])
        torch.testing.assert_close(o[:, :, :, 0], s["out"][:, :, :, t], rtol=1e-5, atol=1e-5)
    assert torch.equal(one["len"], s["len_out"])
    assert torch.equal(one["K"].view(torch.int32), s["K"].view(torch.int32))


def test_matches_the_decode_call(kvc):
    """T = 1 without extras is kvc_decode_attn_lse, and its lse feeds kvc_chunk_mass."""
    ch = Chunk(kvc, [150, 0, 700, 64], [1], L=2, H=2, reserve=2)
    s, d = ch.upload(), ch.upload()
    ch.attn(s)
    ws = kvc.workspace(kvc.KVC_WS_DECODE, ch.params(n_max=1024), zero=True)
    out, lse = torch.empty_like(d["out"][:, :, :, 0]), torch.empty(4, 4, device="cuda")
    kvc.kvc_decode_attn_lse(ch.params(n_max=1024), d["q"][:, :, :, 0].contiguous(),
                            d["k_new"][:, :, :, 0].contiguous(), d["v_new"][:, :, :, 0].contiguous(),
                            d["pos_new"], d["K"], d["V"], d["logm"], d["pos"], d["len"], d["cap"],
                            d["off"], out, lse, None, ws)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    torch.testing.assert_close(s["out"][:, :, :, 0], out, rtol=2 ** -7, atol=2 ** -7)
    torch.testing.assert_close(s["lse"].view(4, 4), lse, rtol=0, atol=2 ** -8)
    assert torch.equal(s["len_out"], d["len"])
    assert torch.equal(s["K"].view(torch.int16), d["K"].view(torch.int16))


BAD = {
    "length": lambda ch: ch.lens.__setitem__(1, -1),
    "n_new": lambda ch: ch.n.__setitem__(0, ch.T + 1),
    "page number": lambda ch: ch.table.__setitem__((1, 0), 1 << 20),
    "negative page": lambda ch: ch.table.__setitem__((1, 1), -1),
    "rows": lambda ch: ch.off.__setitem__(1, ch.rows_total - 4),
    "capacity": lambda ch: ch.caps.__setitem__(1, ch.lens[1]),
}


@pytest.mark.parametrize("what", list(BAD))
def test_bad_units_are_skipped_and_reported(kvc, what):
    """The unit at fault appends nothing and keeps its outputs; the others are served."""
    paged = "page" in what
    ch = Chunk(kvc, [100, 90, 300, 64], [5, 3], B=2, H=2, page=64 if paged else 0)
    ref = ch.upload()
    ch.attn(ref)
    BAD[what](ch)
    skip = {0, 1} if what == "n_new" else {1}
    s = ch.upload()
    ch.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == (kvc.KVC_ECAPACITY if what == "capacity" else kvc.KVC_EDEVICE)
    for u in range(4):
        b, h = u // 2, u % 2
        got, want = s["out"][b, 0, h * 4:h * 4 + 4], ref["out"][b, 0, h * 4:h * 4 + 4]
        if u in skip:
            assert (got == 7.0).all() and (s["lse"][b, 0, h * 4:h * 4 + 4] == 7.0).all()
            assert s["len_out"][b, 0, h] == s["len"][b, 0, h]
        else:
            tol = 2 ** -7
            torch.testing.assert_close(got, want, rtol=tol, atol=tol)
            assert s["len_out"][b, 0, h] == ref["len_out"][b, 0, h]
    m0 = s["mass"].clone()
    if what != "capacity":                              # the mass call checks the same things
        ch.run_mass(s, 0.5)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == kvc.KVC_EDEVICE
        if what != "n_new" and what != "length" and not paged:
            r = torch.from_numpy(np.arange(ch.off[0], ch.off[0] + ch.lens[0])).cuda()
            assert not torch.equal(m0[r], s["mass"][r])


def test_captured_calls_replay(kvc):
    """Attention and mass in one CUDA graph on another stream, replayed over new inputs."""
    ch = Chunk(kvc, [100, 0, 300, 64], [7, 12], B=2, H=2, page=64, slopes=True)
    s = ch.upload()
    kvc.kvc_device_error()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ch.attn(s, stream=side)
        ch.run_mass(s, 0.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2):
        new = Chunk(kvc, [100, 0, 300, 64], [7, 12], B=2, H=2, page=64, slopes=True, seed=seed)
        e = new.upload()
        for k in ("K", "V", "logm", "pos", "mass", "q", "k_new", "v_new"):
            s[k].copy_(e[k])
        ch2 = new
        # the page table is baked into the graph: the new case's rows go where the old table says
        ch2.table = ch.table
        base = Chunk(kvc, [100, 0, 300, 64], [7, 12], B=2, H=2, page=64, slopes=True, seed=0)
        for k in ("K", "V", "logm", "pos", "mass"):
            setattr(ch2, k, getattr(base, k))
            x = getattr(base, k)
            s[k].copy_(x if isinstance(x, torch.Tensor) else torch.from_numpy(x))
        s["out"].fill_(7.0)
        s["lse"].fill_(7.0)
        s["len_out"].fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        ch2.check_attn(s, f"replay {seed}")
        ch2.check_mass(s, s["lse"].cpu().numpy(), 0.5, f"replay {seed}")


def test_two_streams_with_their_own_workspaces(kvc):
    chs = [Chunk(kvc, [700, 90, 1300, 64], [40, 21], B=2, H=2, seed=k) for k in range(2)]
    ss = [c.upload() for c in chs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chs]
    for _ in range(4):
        for c, s, st in zip(chs, ss, streams):
            c.attn(s, stream=st)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    for c, s in zip(chs, ss):
        c.check_attn(s)


def test_mass_is_deterministic(kvc):
    ch = Chunk(kvc, [700, 90, 1300, 64], [140, 21], B=2, H=2)
    got = []
    for _ in range(3):
        s = ch.upload()
        ch.attn(s)
        ch.run_mass(s, 0.9)
        got.append((s["mass"].clone(), s["out"].clone()))
    for m, o in got[1:]:
        assert torch.equal(m.view(torch.int32), got[0][0].view(torch.int32)) and torch.equal(o, got[0][1])


def test_waits_give_up_and_the_next_call_is_right(kvc):
    """Copies withheld: every consumer's wait can only end by its limit.  The calls
    report it, and the same calls are right afterwards."""
    kvc.kvc_device_error()
    for kw in (dict(lens=[700, 90, 1300, 64], n_new=[40, 21], B=2, H=2),
               dict(lens=[700, 90, 1300, 64], n_new=[1, 1], B=2, H=2, page=64)):
        ch = Chunk(kvc, **kw)
        kvc.kvc_set_wait_limit(200_000, True)           # 0.2 ms
        try:
            for call in (ch.attn, lambda s: ch.run_mass(s, 0.5)):
                s = ch.upload()
                call(s)
                torch.cuda.synchronize()
                assert kvc.kvc_device_error() == kvc.KVC_ETIMEOUT
        finally:
            kvc.kvc_set_wait_limit(2_000_000_000, False)
        s = ch.upload()
        ch.attn(s)
        ch.run_mass(s, 0.5)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        ch.check_attn(s)
        ch.check_mass(s, s["lse"].cpu().numpy(), 0.5)


def test_the_binding_refuses_tensors_it_cannot_pass(kvc):
    ch = Chunk(kvc, [100, 64], [3], H=2)
    for name, bad in (("q", lambda t: t.cpu()), ("K", lambda t: t.t()), ("out", lambda t: t.transpose(2, 3)),
                      ("len", lambda t: t.cpu())):
        s = ch.upload()
        s[name] = bad(s[name])
        with pytest.raises(ValueError):
            ch.attn(s)
    s = ch.upload()
    s["pos"] = 5
    with pytest.raises(TypeError):
        ch.run_mass(s, 0.5)


def test_repeated_calls_share_a_workspace(kvc):
    """One workspace serves calls of every shape one after the other, back to back on a stream."""
    kws = [dict(lens=[700, 90, 1300, 64], n_new=[40, 21], B=2, H=2), dict(lens=[9000, 5], n_new=[1], H=2, seed=1),
           dict(lens=[0, 3, 128, 200], n_new=[2], H=4, G=2, d=64, seed=2),
           dict(lens=[300, 50], n_new=[40], H=2, window=33.5, seed=3),
           dict(lens=[90, 700], n_new=[5], H=2, dtype="f32", seed=4)]
    chs = [Chunk(kvc, **kw) for kw in kws]
    ss = [c.upload() for c in chs]
    ws = torch.empty(max(s["ws"].numel() for s in ss), dtype=torch.uint8, device="cuda")
    for s in ss:
        s["ws"] = ws
    for _ in range(3):
        for c, s in zip(chs, ss):
            s["mass"].copy_(torch.from_numpy(c.mass))
            c.attn(s)
            c.run_mass(s, 0.5)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    for c, s in zip(chs, ss):
        c.check_attn(s)
        c.check_mass(s, s["lse"].cpu().numpy(), 0.5)


def test_pages_shared_between_sequences(kvc):
    """Two sequences over the same pages of a common prompt (attention only reads them), each
    with a page of its own for the new tokens."""
    ch = Chunk(kvc, [128, 128], [9, 9], B=2, H=1, page=64, reserve=64)
    ch.table[1, :2] = ch.table[0, :2]
    s = ch.upload()
    ch.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    ch.check_attn(s)


def test_a_length_past_the_pages_is_reported(kvc):
    """More entries than the page table has columns for, and a cache row number that does not fit
    the extent's last, partial page."""
    ch = Chunk(kvc, [60, 70], [4], H=2, page=16)
    ch.table = ch.table[:, :4].copy()                   # 64 rows: the second unit needs 74
    s = ch.upload()
    ch.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == kvc.KVC_EDEVICE
    assert s["len_out"].view(-1).tolist() == [64, 70]
