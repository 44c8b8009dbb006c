"""The chunk calls as they are used together: a prompt streamed through a cache of
bounded size (ChunkedCache), decoding from it, and a follow-up turn over a compressed
cache (Compressor.extend), each step against the float64 oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from synth import workloads as W
from tests.chunk_cases import EPS
from tests.gpu_helpers import assert_bf16_close, upload_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()                           # buffers full of NaN stay with this module


def _cache(kvc, dtype, d=128, **kw):
    from kv_cache_compression_probe_gb300.pipeline import ChunkedCache
    p = kvc.make_params(B=2, L=2, H=2, G=4, d=d, P=1, W=1, n_max=64, S_max=1,
                        dtype=kvc.KVC_BF16 if dtype == "bf16" else kvc.KVC_F32)
    return p, ChunkedCache(p, **kw)


STREAMS = {
    "bf16": ("bf16", 128, dict(budget=96, T=40, page_rows=16, recent=16, decay=0.9), {}),
    "bf16, slopes and window": ("bf16", 128, dict(budget=200, T=70, page_rows=64, recent=8, window=150.0), {"slopes": True}),
    "bf16, d 64, cap": ("bf16", 64, dict(budget=64, T=33, page_rows=32, recent=0, softcap=8.0), {}),
    "f32": ("f32", 64, dict(budget=50, T=21, page_rows=16, recent=4, decay=0.5), {}),
}


@pytest.mark.parametrize("name", list(STREAMS))
def test_a_prompt_streams_through_and_decodes(kvc, name):
    dtype, d, kw, more = STREAMS[name]
    rng = np.random.default_rng(5)
    H, G, B, L = 2, 4, 2, 2
    sl = None
    if more.get("slopes"):
        sl = (2.0 ** -np.arange(1, H * G + 1)).astype(np.float32)
        kw = dict(kw, slopes=torch.from_numpy(sl).cuda())
    p, cache = _cache(kvc, dtype, d, **kw)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = kw["T"]
    chunks = [[T, T], [T, 7], [1, T], [T, T], [0, 3]] + [[1, 1]] * 4         # a prompt, then tokens
    held = {(b, l, h): (np.zeros((0, d)), np.zeros((0, d)), np.zeros(0), np.zeros(0))
            for b in range(B) for l in range(L) for h in range(H)}
    at = np.zeros(B)
    e = EPS[dtype]
    for step, ns in enumerate(chunks):
        Tc = max(max(ns), 1)
        def rnd(heads):
            return torch.from_numpy(rng.standard_normal((B, L, heads, Tc, d)).astype(np.float32)).to(dt)
        q, kn, vn = rnd(H * G), rnd(H), rnd(H)
        out = torch.full((B, L, H * G, Tc, d), 9.0, dtype=dt, device="cuda")
        n_new = torch.tensor(ns, dtype=torch.int32, device="cuda")
        cache.step(q.cuda(), kn.cuda(), vn.cuda(), out, n_new)
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        got = out.double().cpu().numpy()
        for (b, l, h), (K, V, pos, mass) in held.items():
            n, n0 = ns[b], len(K)
            K = np.concatenate([K, kn[b, l, h, :n].double().numpy()])
            V = np.concatenate([V, vn[b, l, h, :n].double().numpy()])
            pos = np.concatenate([pos, at[b] + np.arange(n)])
            hs = slice(h * G, (h + 1) * G)
            mods = dict(softcap=kw.get("softcap", 0.0), window=kw.get("window", 0.0),
                        slopes=None if sl is None else sl[hs])
            qs = q[b, l, hs, :n].double().numpy()
            s = O.chunk_scores(qs, K, np.zeros(len(K)), pos, n0, at[b], **mods)
            if n:
                o, lse, pr = O.chunk_attn(qs, K, V, np.zeros(len(K)), pos, n0, at[b], **mods)
                # fp32 scores of |q k| sums below 40 (d 128, unit normals), one rounding of the
                # numerators and of the result each
                ds = d * 2.0 ** -23 * 40
                tol = (np.einsum("gtn,nd->gtd", pr, np.abs(V)) * (2 * ds + (e if dtype == "bf16" else 0) + 2.0 ** -18)
                       + 1.01 * e * np.abs(o))
                assert (np.abs(got[b, l, hs, :n] - o) <= tol).all(), (name, step, b, l, h)
                m = O.chunk_mass(np.concatenate([mass, np.zeros(n)]), n0, s, lse, cache.decay)
            else:
                m = cache.decay * mass
            assert (got[b, l, hs, n:] == 9.0).all()
            # the eviction follows the device's masses: compare those first
            Kd, Vd, pd, md = cache.entries(b, l, h)
            # which entries the device kept (positions are distinct)
            where = {x: i for i, x in enumerate(pos)}
            kept = np.array([where[x] for x in pd], int)
            assert len(set(kept)) == len(kept)
            ds = d * 2.0 ** -23 * 40 * (2 if dtype == "bf16" else 1)
            tol_m = (2 * ds + 2.0 ** -18) * np.abs(m) + 1e-6
            assert (np.abs(md - m[kept]) <= tol_m[kept]).all(), (name, step, "mass")
            np.testing.assert_array_equal(Kd, K[kept])
            np.testing.assert_array_equal(Vd, V[kept])
            Bn = min(len(K), max(cache.budget, int((pos >= at[b] + n - cache.recent).sum())))
            assert len(kept) == Bn
            gone = np.setdiff1d(np.arange(len(K)), kept)
            safe = pos >= at[b] + n - cache.recent
            assert not safe[gone].any()
            rest = kept[~safe[kept]]
            if len(gone) and len(rest):                   # nothing that left outweighs what stayed
                assert m[gone].max() <= m[rest].min() + 2 * max(tol_m[gone].max(), tol_m[rest].max())
            held[b, l, h] = (K[kept], V[kept], pos[kept], md.astype(np.float64))
        at += ns
    assert (cache.len_lh.cpu().numpy() <= max(cache.budget, cache.recent)).all()


def test_steps_replay_from_a_graph(kvc):
    """The three calls of a step in one graph, replayed: bit for bit the eager run."""
    dt = torch.bfloat16
    kw = dict(budget=100, T=24, page_rows=16, recent=10, decay=0.8)
    g = torch.Generator().manual_seed(1)
    qs, ks, vs = (torch.randn((5, 2, 2, n, 24, 128), generator=g).to(dt).cuda() for n in (8, 2, 2))
    _, eager = _cache(kvc, "bf16", **kw)
    want = []
    for t in range(5):
        out = torch.empty_like(qs[t])
        eager.step(qs[t], ks[t], vs[t], out)
        want.append(out)
    _, cache = _cache(kvc, "bf16", **kw)
    q, k, v = qs[0].clone(), ks[0].clone(), vs[0].clone()
    out = torch.empty_like(q)
    kvc.kvc_device_error()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.step(q, k, v, out)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(5):
        for a, b in ((q, qs), (k, ks), (v, vs)):
            a.copy_(b[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[t]), t
    assert kvc.kvc_device_error() == 0
    for n in ("K", "V", "pos", "mass", "len_lh", "pos_next"):
        assert torch.equal(getattr(cache, n), getattr(eager, n)), n


def test_a_chunk_larger_than_the_cache_was_built_for_is_refused(kvc):
    _, cache = _cache(kvc, "bf16", budget=32, T=8, page_rows=16, recent=4)
    q = torch.zeros((2, 2, 8, 9, 128), dtype=torch.bfloat16, device="cuda")
    kn = torch.zeros((2, 2, 2, 9, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        cache.step(q, kn, kn, torch.empty_like(q))
    with pytest.raises(ValueError):
        _cache(kvc, "bf16", budget=32, T=8, recent=33)


@pytest.mark.parametrize("tc", [True, False], ids=["tcgen05", "simt"])
def test_follow_up_turn_over_a_compressed_cache(kvc, tc):
    """compress, a chunk of new tokens, then decode steps: every output against the
    oracle over the packed entries."""
    cfg = W.small_config(B=2, L=1, H=2, n=900, n_min=700, n_decode=40)
    wl = W.make_workload(cfg)
    p, comp, dev, _ = upload_workload(wl, tensor_cores=tc)
    comp.compress(dev["K"], dev["V"], dev["Qp"], dev["bounds"], dev["n_slots"], dev["sens"])
    torch.cuda.synchronize()
    lens, offs = comp.len_lh.cpu().numpy(), comp.off_lh.cpu().numpy()
    Kp, Vp = comp.Kp.double().cpu().numpy(), comp.Vp.double().cpu().numpy()
    lm, pos = comp.logm.double().cpu().numpy(), comp.pos.double().cpu().numpy()
    T, G, d = 30, cfg.G, cfg.d
    rng = np.random.default_rng(3)
    bf = torch.bfloat16

    def rnd(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(bf)
    q, kn, vn = rnd(2, 1, 2 * G, T, d), rnd(2, 1, 2, T, d), rnd(2, 1, 2, T, d)
    ctx = np.asarray([s.n for s in wl.seqs], np.float32)
    n_new = torch.tensor([T, 11], dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 1, 2 * G, T, d), dtype=bf, device="cuda")
    lse = torch.zeros((2, 1, 2 * G, T), device="cuda")
    comp.extend(q.cuda(), kn.cuda(), vn.cuda(), out, torch.from_numpy(ctx).cuda(), n_new, lse)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    got = out.float().cpu().numpy()
    held = {}
    for b in range(2):
        n = [T, 11][b]
        for h in range(2):
            o, m = int(offs[b, 0, h]), int(lens[b, 0, h])
            hs = slice(h * G, (h + 1) * G)
            K = np.concatenate([Kp[o:o + m], kn[b, 0, h, :n].double().numpy()])
            V = np.concatenate([Vp[o:o + m], vn[b, 0, h, :n].double().numpy()])
            l2 = np.concatenate([lm[o:o + m], np.zeros(n)])
            ps = np.concatenate([pos[o:o + m], ctx[b] + np.arange(n)])
            want, wl2, _ = O.chunk_attn(q[b, 0, hs, :n].double().numpy(), K, V, l2, ps, m, ctx[b])
            assert_bf16_close(got[b, 0, hs, :n], want, f"turn b={b} h={h}")
            np.testing.assert_allclose(lse[b, 0, hs, :n].cpu().numpy(), wl2, rtol=1e-5, atol=1e-4)
            held[b, h] = (K, V, l2)
    qd, kd, vd = rnd(2, 1, 2 * G, d), rnd(2, 1, 2, d), rnd(2, 1, 2, d)
    od = torch.empty((2, 1, 2 * G, d), dtype=bf, device="cuda")
    comp.decode(qd.cuda(), kd.cuda(), vd.cuda(), od)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    for (b, h), (K, V, l2) in held.items():
        hs = slice(h * G, (h + 1) * G)
        want, *_ = O.decode_step_head(qd[b, 0, hs].double().numpy(), kd[b, 0, h].double().numpy(),
                                      vd[b, 0, h].double().numpy(), K, V, l2)
        assert_bf16_close(od[b, 0, hs].float().cpu().numpy(), want, f"decode b={b} h={h}")
