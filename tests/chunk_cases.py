"""Seeded inputs of the chunk calls, their device copies, and the bounds on how far
the device may be from the float64 oracle."""
import numpy as np
import torch

import oracle as O

EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}        # half a step, relative
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Chunk:
    """lens: cache length of every (b, l, h); n_new: new tokens of every sequence."""

    def __init__(self, kvc, lens, n_new, B=1, L=1, H=1, G=4, d=128, dtype="bf16", T=None, page=0,
                 softcap=0.0, window=0.0, slopes=False, layers=None, seed=0, qscale=1.0,
                 dead=0.0, reserve=0, pos_gap=1.0, pass_n_new=True):
        rng = np.random.default_rng(seed)
        self.kvc, self.dtype, self.B, self.L, self.H, self.G, self.d = kvc, dtype, B, L, H, G, d
        U = B * L * H
        self.lens = np.asarray(lens, np.int64).reshape(U)
        self.n = np.asarray(n_new, np.int64).reshape(B)
        self.T = int(T or max(1, self.n.max()))
        self.layers = layers or (0, L)
        l0, l1 = self.layers
        self.units = [(b * L + l) * H + h for b in range(B) for l in range(l0, l1) for h in range(H)]
        dt = DT[dtype]

        def rnd(*shape, scale=1.0):
            x = torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dt)
            return x
        self.n_u = np.repeat(self.n, L * H)
        caps = self.lens + self.n_u + reserve
        self.page = page
        if page:
            pages = -(-caps // page)
            n_pages = int(pages.sum()) + 2
            ids = rng.permutation(n_pages).astype(np.int32)
            self.table = np.full((U, max(1, int(pages.max()))), -7, np.int32)
            at = 0
            for u in range(U):
                self.table[u, :pages[u]] = ids[at:at + pages[u]]
                at += pages[u]
            self.rows_total = n_pages * page
            off = np.zeros(U, np.int64)
        else:
            self.table = None
            off = np.cumsum(caps) - caps + 3           # rows before the first unit's
            self.rows_total = int(caps.sum()) + 5
        self.caps, self.off = caps, off
        R = self.rows_total
        self.K, self.V = torch.full((R, d), float("nan"), dtype=dt), torch.full((R, d), float("nan"), dtype=dt)
        self.logm = np.full(R, np.nan, np.float32)
        self.pos = np.full(R, np.nan, np.float32)
        self.mass = np.full(R, np.nan, np.float32)
        self.pos_new = (np.ceil(self.lens.reshape(B, -1).max(1) * pos_gap) + 7).astype(np.float32)
        for u in range(U):
            n0 = int(self.lens[u])
            r = self.rows(u, n0)
            self.K[r], self.V[r] = rnd(n0, d), rnd(n0, d)
            lm = np.where(rng.uniform(size=n0) < 0.6, 0.0, rng.uniform(0, 3, size=n0))
            lm[rng.uniform(size=n0) < dead] = -np.inf
            self.logm[r] = lm
            self.pos[r] = np.floor(2 * (np.arange(n0) * pos_gap + rng.uniform(0, 1, n0))) / 2
            self.mass[r] = rng.uniform(0, 2, n0)
        Lr = l1 - l0
        self.q = rnd(B, Lr, H * G, self.T, d, scale=qscale)
        self.k_new, self.v_new = rnd(B, Lr, H, self.T, d), rnd(B, Lr, H, self.T, d)
        for b in range(B):                             # rows past the sequence's tokens are not read
            for t in (self.q, self.k_new, self.v_new):
                t[b, :, :, int(self.n[b]):] = float("nan")
        self.softcap, self.window = float(softcap), float(window)
        self.slopes = (2.0 ** (-8.0 * np.arange(1, H * G + 1) / (H * G))).astype(np.float32) if slopes else None
        self.pass_n_new = pass_n_new

    def rows(self, u, n):
        e = np.arange(n)
        if self.page:
            return self.table[u][e // self.page].astype(np.int64) * self.page + e % self.page
        return self.off[u] + e

    # ------------------------------------------------------------ device side
    def params(self, **over):
        kw = dict(B=self.B, L=self.L, H=self.H, G=self.G, d=self.d, P=1, W=1,
                  dtype=self.kvc.KVC_BF16 if self.dtype == "bf16" else self.kvc.KVC_F32, n_max=64,
                  S_max=1, packed_rows=self.rows_total)
        kw.update(over)
        return self.kvc.make_params(**kw)

    def upload(self, device="cuda"):
        kvc = self.kvc

        def up(x, dt=None):
            x = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
            return (x.to(dt) if dt else x).to(device).contiguous()
        B, L, H = self.B, self.L, self.H
        dt = DT[self.dtype]
        s = dict(K=up(self.K).clone(), V=up(self.V).clone(), logm=up(self.logm), pos=up(self.pos),
                 mass=up(self.mass), len=up(self.lens.reshape(B, L, H), torch.int32),
                 cap=up(self.caps.reshape(B, L, H), torch.int32), off=up(self.off.reshape(B, L, H)),
                 q=up(self.q), k_new=up(self.k_new), v_new=up(self.v_new), pos_new=up(self.pos_new),
                 len_out=torch.full((B, L, H), -3, dtype=torch.int32, device=device))
        s["out"] = torch.full(self.q.shape, 7.0, dtype=dt, device=device)
        s["lse"] = torch.full(self.q.shape[:-1], 7.0, dtype=torch.float32, device=device)
        s["p"] = self.params()
        s["c"] = kvc.make_chunk(self.T, *self.layers, page_rows=self.page,
                                page_table=None if self.table is None else
                                up(self.table.reshape(B, L, H, -1)),
                                n_new=up(self.n, torch.int32) if self.pass_n_new else None,
                                softcap=self.softcap, window=self.window,
                                slopes=None if self.slopes is None else up(self.slopes))
        s["ws"] = torch.empty(kvc.kvc_chunk_workspace_bytes(s["p"], s["c"]), dtype=torch.uint8,
                              device=device).fill_(0xFF)
        return s

    def attn(self, s, len_out="len_out", lse="lse", stream=None):
        self.kvc.kvc_chunk_attn(s["p"], s["c"], s["q"], s["k_new"], s["v_new"], s["pos_new"], s["K"],
                                s["V"], s["logm"], s["pos"], s["len"], s["cap"],
                                None if self.page else s["off"], s["out"], s[lse] if lse else None,
                                s[len_out] if len_out else None, s["ws"], stream)

    def run_mass(self, s, decay, stream=None):
        self.kvc.kvc_chunk_mass(s["p"], s["c"], s["q"], s["K"], s["logm"], s["pos"], s["pos_new"],
                                s["len"], None if self.page else s["off"], s["lse"], decay, s["mass"],
                                s["ws"], stream)

    # ------------------------------------------------------------ oracle side
    def entries(self, u):
        """(K, V, logm, pos) in float64 of unit u after the append, its queries [G, n, d]
        and where they live in q ([b, l], head slice)."""
        L, H, G = self.L, self.H, self.G
        b, l, h = u // (L * H), (u // H) % L, u % H
        lr = l - self.layers[0]
        n, n0 = int(self.n[b]), int(self.lens[u])
        r = self.rows(u, n0)

        def f(x):
            return x.double().numpy()
        K = np.concatenate([f(self.K[r]), f(self.k_new[b, lr, h, :n])])
        V = np.concatenate([f(self.V[r]), f(self.v_new[b, lr, h, :n])])
        lm = np.concatenate([self.logm[r].astype(np.float64), np.zeros(n)])
        pos = np.concatenate([self.pos[r].astype(np.float64), self.pos_new[b] + np.arange(n)])
        q = f(self.q[b, lr, h * G:(h + 1) * G, :n])
        return K, V, lm, pos, q, (b, lr, slice(h * G, (h + 1) * G), n, n0)

    def slopes_of(self, u):
        h = u % self.H
        return None if self.slopes is None else self.slopes[h * self.G:(h + 1) * self.G]

    def scores(self, u):
        K, V, lm, pos, q, where = self.entries(u)
        return O.chunk_scores(q, K, lm, pos, where[4], self.pos_new[where[0]], self.softcap,
                              self.window, self.slopes_of(u))

    def score_error(self, u):
        """Bound on the error of each natural-log score: the d products are summed in
        fp32 (each addition off by at most one step 2^-23 of the partial sums, which
        stay below sum |q k|; tensor cores may truncate), the base-2 scaling, cap and
        biases are a handful of fp32 operations (8 half steps of 2^-24) on values up
        to |s| + |ln m| + |slope gap| + cap."""
        K, V, lm, pos, q, (b, lr, hs, n, n0) = self.entries(u)
        dots = np.abs(q) @ np.abs(K).T / np.sqrt(self.d)
        size = dots + np.abs(np.where(np.isinf(lm), 0.0, lm)) + self.softcap
        if self.slopes is not None:
            gap = np.abs((float(self.pos_new[b]) + np.arange(n))[:, None] - pos[None])
            size = size + self.slopes_of(u)[:, None, None] * gap
        return self.d * 2.0 ** -23 * dots + 8 * 2.0 ** -24 * size

    def check_attn(self, s, what=""):
        """out, lse, the appended rows, len_out and everything that must not change."""
        e = EPS[self.dtype]
        out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
        Kd, Vd = s["K"].cpu(), s["V"].cpu()
        lmd, posd = s["logm"].cpu().numpy(), s["pos"].cpu().numpy()
        K0, V0, lm0, pos0 = self.K.clone(), self.V.clone(), self.logm.copy(), self.pos.copy()
        want_len = np.full(len(self.lens), -3, np.int64)
        for u in self.units:
            K, V, lm, pos, q, (b, lr, hs, n, n0) = self.entries(u)
            want_len[u] = n0 + n
            assert (out[b, lr, hs, n:] == 7.0).all() and (lse[b, lr, hs, n:] == 7.0).all(), (what, u)
            r = self.rows(u, n0 + n)[n0:]
            h = u % self.H
            K0[r], V0[r] = self.k_new[b, lr, h, :n], self.v_new[b, lr, h, :n]
            lm0[r], pos0[r] = 0.0, pos[n0:]
            if n == 0:
                continue
            o, ls, p = O.chunk_attn(q, K, V, lm, pos, n0, self.pos_new[b], self.softcap, self.window,
                                    self.slopes_of(u))
            de = self.score_error(u)
            dbar = (p * de).sum(-1)
            N = n0 + n
            # lse: the scores' error, the sum of N numerators (each off by 2^-22), log2, rounding
            tol_l = (dbar + (N * 2.0 ** -24 + 2.0 ** -21)) * O.LOG2E + 2.0 ** -22 * (np.abs(ls) + 1)
            bad = np.abs(lse[b, lr, hs, :n] - ls) > tol_l
            assert not bad.any(), (what, u, "lse", np.abs(lse[b, lr, hs, :n] - ls).max(), tol_l.min())
            # out: each numerator's relative error (scores, one rounding to bf16 on the bf16
            # path), the fp32 sums, and the rounding of the result
            pn = (e if self.dtype == "bf16" else 0.0) + 2.0 ** -21 + N * 2.0 ** -23
            tol = (np.einsum("gtn,nd->gtd", p * (de + pn), np.abs(V))
                   + (dbar + N * 2.0 ** -24 + 2.0 ** -21)[..., None] * np.abs(o) + 1.01 * e * np.abs(o) + 1e-30)
            err = np.abs(out[b, lr, hs, :n] - o)
            assert (err <= tol).all(), (what, u, "out", err.max(), (err / tol).max())
        for a, w, name in ((Kd, K0, "K"), (Vd, V0, "V")):
            assert torch.equal(a.view(torch.int16 if self.dtype == "bf16" else torch.int32),
                               w.view(torch.int16 if self.dtype == "bf16" else torch.int32)), (what, name)
        np.testing.assert_array_equal(lmd, lm0, err_msg=what)
        np.testing.assert_array_equal(posd, pos0, err_msg=what)
        np.testing.assert_array_equal(s["len_out"].cpu().numpy().reshape(-1), want_len, err_msg=what)

    def set_lse(self, s):
        """Appends the chunk's rows and fills s["lse"] with the oracle's (rounded to fp32),
        so the mass can be checked by itself.  Returns the lse as the device has it."""
        lse = np.full(s["lse"].shape, 7.0, np.float32)
        for u in self.units:
            K, V, lm, pos, q, (b, lr, hs, n, n0) = self.entries(u)
            r = torch.from_numpy(self.rows(u, n0 + n)[n0:]).to(s["K"].device)
            h = u % self.H
            s["K"][r] = self.k_new[b, lr, h, :n].to(s["K"].device)
            s["logm"][r], s["pos"][r] = 0.0, torch.from_numpy(pos[n0:].astype(np.float32)).to(r.device)
            if n:
                lse[b, lr, hs, :n] = O.chunk_softmax(self.scores(u))[1]
        s["lse"].copy_(torch.from_numpy(lse))
        return lse

    def check_mass(self, s, lse, decay, what=""):
        got = s["mass"].double().cpu().numpy()
        want = self.mass.astype(np.float64)
        for u in self.units:
            K, V, lm, pos, q, (b, lr, hs, n, n0) = self.entries(u)
            r = self.rows(u, n0 + n)
            sc = self.scores(u)
            m = O.chunk_mass(self.mass[r], n0, sc, lse[b, lr, hs, :n], decay)
            w = np.exp2(sc * O.LOG2E - lse[b, lr, hs, :n].astype(np.float64)[..., None])
            # every term: the score's error, subtracting lse and 2^x (2^-22 and half a step of
            # |s - lse| each); the sum of R terms in fp32; one fused multiply-add with the old mass
            size = np.where(w > 0, np.abs(np.where(w > 0, sc, 0.0)) * O.LOG2E + np.abs(lse[b, lr, hs, :n][..., None]), 0.0)
            R = self.G * n
            tol = ((w * (self.score_error(u) + 2.0 ** -23 * size + 2.0 ** -21)).sum((0, 1)) if n else 0.0)
            tol = tol + (R + 4) * 2.0 ** -24 * np.abs(m) + 1e-30
            err = np.abs(got[r] - m)
            assert (err <= tol).all(), (what, u, err.max(), (err / tol).max())
            want[r] = got[r]
        np.testing.assert_array_equal(got, want, err_msg=what)   # every other row as it was
