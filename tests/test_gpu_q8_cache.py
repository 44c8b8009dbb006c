"""The calls on the 8-bit cache as they are used together (QuantizedCache): a prompt in chunks,
drafts and single tokens over all entries or picked pages, from empty or from a compressed
cache, each step against the oracle; steps in a graph."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from synth import workloads as W
from tests.gpu_helpers import upload_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


def _params(kvc, dtype="bf16", d=128, **kw):
    p = dict(B=2, L=2, H=2, G=4, d=d, P=1, W=1, n_max=64, S_max=1,
             dtype=kvc.KVC_BF16 if dtype == "bf16" else kvc.KVC_F32)
    return kvc.make_params(**{**p, **kw})


class Held:
    """What one (b, l, h) holds, by the oracle: values in units of their page's scale."""

    def __init__(self, page, d, base):
        self.page, self.d, self.base = page, d, base
        self.pages, self.exp, self.lm = {"K": [], "V": []}, {"K": [], "V": []}, np.zeros(0)

    def add(self, K, V, lm=None):
        n, at = len(K), 0
        while at < n:
            r = len(self.lm) % self.page
            c = min(self.page - r, n - at)
            for name, new in (("K", K[at:at + c]), ("V", V[at:at + c])):
                if r == 0:
                    self.pages[name].append(np.zeros((0, self.d)))
                    self.exp[name].append(0)
                self.pages[name][-1], self.exp[name][-1] = Q.page_append(self.pages[name][-1], self.exp[name][-1], new)
            self.lm = np.concatenate([self.lm, np.zeros(c) if lm is None else lm[at:at + c]])
            at += c

    def turn(self, x, pos):
        e = np.asarray(pos, np.float64)[:, None] * float(self.base) ** (-2.0 * np.arange(self.d // 2) / self.d)
        return Q.rope(x, np.cos(e).astype(np.float32), np.sin(e).astype(np.float32))

    def values(self, name):
        return np.concatenate([p * 2.0 ** x for p, x in zip(self.pages[name], self.exp[name])]) if len(self.lm) else np.zeros((0, self.d))

    def picks(self, q, n0, n_sel, first, recent):
        """Of every token; the bounds hold all of a page's entries, the chunk's later ones too."""
        bd = np.stack([Q.bounds(p) for p in self.pages["K"]])
        sc = np.exp2(np.asarray(self.exp["K"], np.float64))
        out = []
        for t in range(q.shape[1]):
            own = (n0 + t) // self.page
            out.append(Q.pick_pages(q[:, t], bd[:own + 1], sc[:own + 1], own, n_sel, first, recent))
        return out


def _check(held, q_rot, got, n0, picks, dtype, what):
    """Tolerance: fp32 scores of d products and their rounding, numerators of 11 bits (8 where there are
    more than 64 rows; fp32 22), one rounding of the result."""
    G, n, d = q_rot.shape
    K, V = held.values("K"), held.values("V")
    o, _, p = Q.q8_attn(q_rot, K, V, held.lm, n0, held.page, picks)
    dots = np.abs(q_rot.astype(np.float64)) @ np.abs(K).T / np.sqrt(d)
    de = d * 2.0 ** -23 * dots + 2.0 ** -20 * (dots + np.abs(held.lm))
    e = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    half = e if dtype == "bf16" else 2.0 ** -21
    N = len(K)
    tol = (np.einsum("gtn,nd->gtd", p * (2 * de + half + 2.0 ** -20 + N * 2.0 ** -22) + 2.0 ** -29, np.abs(V))
           + 1.01 * e * np.abs(o))
    err = np.abs(got - o)
    assert (err <= tol).all(), (what, err.max(), (err / tol).max())


RUNS = {
    "bf16": dict(kw=dict(tokens=300, T=70, page_rows=16)),
    "bf16, picked pages": dict(kw=dict(tokens=300, T=70, page_rows=16, n_sel=5, first=1, recent=2)),
    "bf16, d 64, large pages": dict(d=64, kw=dict(tokens=300, T=70, page_rows=128, n_sel=2, first=0, recent=1)),
    "f32, picked pages": dict(dtype="f32", kw=dict(tokens=300, T=70, page_rows=32, n_sel=3, first=1, recent=1)),
    "f32": dict(dtype="f32", d=64, kw=dict(tokens=300, T=70, page_rows=64)),
    "bf16, no rotation": dict(kw=dict(tokens=300, T=70, page_rows=32, rotate=False)),
}


@pytest.mark.parametrize("name", list(RUNS))
def test_a_prompt_drafts_and_tokens(kvc, name):
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    r = RUNS[name]
    dtype, d, kw = r.get("dtype", "bf16"), r.get("d", 128), r["kw"]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    p = _params(kvc, dtype, d)
    cache = QuantizedCache(p, **kw)
    rng = np.random.default_rng(6)
    held = {(b, l, h): Held(kw["page_rows"], d, p.rope_base) for b in range(2) for l in range(2) for h in range(2)}
    at = np.zeros(2, int)
    for step, ns in enumerate([[70, 33], [1, 70], [5, 4], [0, 3], [1, 1], [1, 1], [17, 2], [1, 1]]):
        T = max(ns)

        def rnd(heads):
            return torch.from_numpy(rng.standard_normal((2, 2, heads, T, d)).astype(np.float32)).to(dt)
        q, kn, vn = rnd(8), rnd(2), rnd(2)
        out = torch.full((2, 2, 8, T, d), 9.0, dtype=dt, device="cuda")
        cache.step(q.cuda(), kn.cuda(), vn.cuda(), out, torch.tensor(ns, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        got = out.double().cpu().numpy()
        for (b, l, h), x in held.items():
            n, n0, hs = ns[b], len(x.lm), slice(4 * h, 4 * h + 4)
            assert (got[b, l, hs, n:] == 9.0).all()
            if n == 0:
                continue
            pos = at[b] + np.arange(n)
            turn = x.turn if cache.rope_cos is not None else lambda v, _: v
            x.add(turn(kn[b, l, h, :n].float().numpy(), pos), vn[b, l, h, :n].float().numpy())
            K, V, _ = cache.entries(b, l, h)
            np.testing.assert_array_equal(K, x.values("K"), err_msg=f"{name} {step}")
            np.testing.assert_array_equal(V, x.values("V"), err_msg=f"{name} {step}")
            qr = torch.from_numpy(turn(q[b, l, hs, :n].float().numpy(), pos)).to(dt).float().numpy()
            picks = x.picks(qr, n0, kw["n_sel"], kw["first"], kw["recent"]) if kw.get("n_sel") else None
            if picks is not None:
                sel = cache.sel[:2 * 2 * 2 * T * cache.n_sel].view(2, 2, 2, T, -1)[b, l, h].cpu().numpy()
                for t in range(n):
                    assert [j for j in sel[t] if j >= 0] == list(picks[t]), (name, step, t)
            _check(x, qr, got[b, l, hs, :n], n0, picks, dtype, (name, step, b, l, h))
        at += ns
    assert cache.pos_next.tolist() == at.tolist()


def test_a_compressed_cache_in_8_bits(kvc):
    """compress, to_q8, a chunk of new tokens and single ones: entries and outputs."""
    cfg = W.small_config(B=2, L=1, H=2, n=900, n_min=700, n_decode=40)
    wl = W.make_workload(cfg)
    p, comp, dev, _ = upload_workload(wl)
    comp.compress(dev["K"], dev["V"], dev["Qp"], dev["bounds"], dev["n_slots"], dev["sens"])
    ctx = torch.tensor([float(s.n) for s in wl.seqs], device="cuda")
    cache = comp.to_q8(60, ctx, T=40, page_rows=32, n_sel=6, first=1, recent=2)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    lens, offs = comp.len_lh.cpu().numpy(), comp.off_lh.cpu().numpy()
    Kp, Vp, lm = comp.Kp.float().cpu().numpy(), comp.Vp.float().cpu().numpy(), comp.logm.cpu().numpy()
    held = {}
    for b in range(2):
        for h in range(2):
            o, n = int(offs[b, 0, h]), int(lens[b, 0, h])
            x = held[b, h] = Held(32, cfg.d, p.rope_base)
            x.add(Kp[o:o + n], Vp[o:o + n], lm[o:o + n].astype(np.float64))
            K, V, l2 = cache.entries(b, 0, h)
            np.testing.assert_array_equal(K, x.values("K"))
            np.testing.assert_array_equal(V, x.values("V"))
            np.testing.assert_array_equal(l2, lm[o:o + n])
    rng = np.random.default_rng(3)
    bf = torch.bfloat16
    at = np.asarray([s.n for s in wl.seqs])
    for ns in ([40, 13], [1, 1], [1, 1]):
        T = max(ns)
        q, kn, vn = (torch.from_numpy(rng.standard_normal((2, 1, k, T, cfg.d)).astype(np.float32)).to(bf) for k in (2 * cfg.G, 2, 2))
        out = torch.zeros((2, 1, 2 * cfg.G, T, cfg.d), dtype=bf, device="cuda")
        cache.step(q.cuda(), kn.cuda(), vn.cuda(), out, torch.tensor(ns, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        for (b, h), x in held.items():
            n, n0, hs = ns[b], len(x.lm), slice(h * cfg.G, (h + 1) * cfg.G)
            pos = at[b] + np.arange(n)
            x.add(x.turn(kn[b, 0, h, :n].float().numpy(), pos), vn[b, 0, h, :n].float().numpy())
            qr = torch.from_numpy(x.turn(q[b, 0, hs, :n].float().numpy(), pos)).to(bf).float().numpy()
            picks = x.picks(qr, n0, 6, 1, 2)
            _check(x, qr, out[b, 0, hs, :n].double().cpu().numpy(), n0, picks, "bf16", (ns, b, h))
        at = at + ns


@pytest.mark.parametrize("n_sel", [0, 4])
def test_steps_replay_from_a_graph(kvc, n_sel):
    """A step captured once and replayed: bit for bit the eager run; a full cache takes no more."""
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    kw = dict(tokens=128, T=20, page_rows=16, n_sel=n_sel, n_pos=400)
    g = torch.Generator().manual_seed(1)
    qs, ks, vs = (torch.randn((8, 2, 2, n, 20, 128), generator=g).bfloat16().cuda() for n in (8, 2, 2))
    eager, cache = QuantizedCache(_params(kvc), **kw), QuantizedCache(_params(kvc), **kw)
    want = []
    for t in range(6):
        out = torch.empty_like(qs[t])
        eager.step(qs[t], ks[t], vs[t], out)
        want.append(out)
    q, k, v = qs[0].clone(), ks[0].clone(), vs[0].clone()
    out = torch.empty_like(q)
    kvc.kvc_device_error()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.step(q, k, v, out)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(6):
        for a, b in ((q, qs), (k, ks), (v, vs)):
            a.copy_(b[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[t]), t
    assert kvc.kvc_device_error() == 0 and (cache.len_lh == 120).all()
    for n in ("K", "V", "k_scale", "v_scale", "len_lh", "pos_next"):
        assert torch.equal(getattr(cache, n), getattr(eager, n)), n
    out.fill_(3.0)
    graph.replay()                                         # 120 + 20 > 128
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == kvc.KVC_ECAPACITY
    assert (out == 3.0).all() and (cache.len_lh == 120).all() and (cache.pos_next == 120).all()
    one = torch.empty((2, 2, 8, 1, 128), dtype=torch.bfloat16, device="cuda")
    cache.step(*(x[0, :, :, :, :1].contiguous() for x in (qs, ks, vs)), one)   # one still fits
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0 and (cache.len_lh == 121).all()


def test_refusals(kvc):
    from kv_cache_compression_probe_gb300.pipeline import QuantizedCache
    with pytest.raises(ValueError):
        QuantizedCache(_params(kvc), 64, n_sel=2, first=1, recent=2)
    cache = QuantizedCache(_params(kvc), 64, T=4)
    q, k = (torch.zeros((2, 2, n, 5, 128), dtype=torch.bfloat16, device="cuda") for n in (8, 2))
    with pytest.raises(ValueError):
        cache.step(q, k, k, torch.empty_like(q))           # five tokens
    q, k = q[:, :, :, :4].contiguous(), k[:, :, :, :4].contiguous()
    with pytest.raises(ValueError):
        cache.step(q.float(), k, k, torch.empty_like(q))
    with pytest.raises(ValueError):
        cache.step(q, k, k, torch.empty_like(q), lse=torch.empty((2, 2, 8, 3), device="cuda"))
    with pytest.raises(ValueError):
        cache.step(q, k, k, torch.empty_like(q), stream=torch.cuda.Stream())
    assert (cache.len_lh == 0).all()
