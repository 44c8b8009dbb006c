"""Seeded inputs of the calls on the 8-bit cache, their device copies, and the checks
against the oracle (codes, scales, bounds and picked pages bit for bit)."""
import numpy as np
import torch

import oracle as O
from oracle import q8_oracle as Q
from tests.chunk_cases import DT, EPS

UNUSED = 0x7F                                      # the code that is not a number


class Q8:
    """A paged 8-bit cache with lens entries for every (b, l, h) and n_new tokens to come for
    every sequence.  Unused rows hold codes that are not numbers, unused pages NaN scales."""

    def __init__(self, kvc, lens, n_new, B=1, L=1, H=1, G=4, d=128, dtype="bf16", T=None, page=16,
                 layers=None, seed=0, qscale=1.0, dead=0.0, logm=True, reserve=0, pass_n_new=True,
                 spread=0.0, max_pages=None, rope=True, bounds=True):
        rng = np.random.default_rng(seed)
        self.kvc, self.dtype, self.B, self.L, self.H, self.G, self.d = kvc, dtype, B, L, H, G, d
        U = B * L * H
        self.U, self.page, self.rope, self.keep_bounds = U, page, rope, bounds
        self.lens = np.asarray(lens, np.int64).reshape(U)
        self.n = np.asarray(n_new, np.int64).reshape(B)
        self.T = int(T or max(1, self.n.max()))
        self.layers = layers or (0, L)
        l0, l1 = self.layers
        self.units = [(b * L + l) * H + h for b in range(B) for l in range(l0, l1) for h in range(H)]
        self.n_u = np.repeat(self.n, L * H)
        self.caps = self.lens + self.n_u + reserve
        pages = -(-self.caps // page)
        self.n_pages = int(pages.sum()) + 2
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((U, max_pages or max(1, int(pages.max()))), -7, np.int32)
        at = 0
        for u in range(U):
            self.table[u, :pages[u]] = ids[at:at + pages[u]]
            at += pages[u]
        dt = DT[dtype]
        chan = np.exp(0.7 * rng.standard_normal(d))
        # page contents: values in units of the scale, exponents; spread: scales of all sizes
        self.val = {n: np.full((self.n_pages, page, d), np.nan) for n in "KV"}
        self.exp = {n: np.zeros(self.n_pages, np.int64) for n in "KV"}
        self.logm = np.full(self.n_pages * page, np.nan, np.float32)
        self.used = np.zeros((self.n_pages, page), bool)
        for u in range(U):
            for j in range(-(-int(self.lens[u]) // page)):
                c = min(page, int(self.lens[u]) - j * page)
                p = self.table[u, j]
                self.used[p, :c] = True
                for n in "KV":
                    w = rng.standard_normal((c, d)) * chan * 2.0 ** (spread * rng.standard_normal())
                    self.val[n][p, :c], self.exp[n][p] = Q.page_append(np.zeros((0, d)), 0, w.astype(np.float32))
                lm = np.where(rng.uniform(size=c) < 0.6, 0.0, rng.uniform(0, 3, size=c))
                lm[rng.uniform(size=c) < dead] = -np.inf
                self.logm[p * page:p * page + c] = lm
        if not logm:
            self.logm = None
        Lr = l1 - l0

        def rnd(*shape, scale=1.0):
            return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dt)
        self.q = rnd(B, Lr, H * G, self.T, d, scale=qscale)
        grow = 2.0 ** (spread * rng.standard_normal())
        self.k_new = (rnd(B, Lr, H, self.T, d, scale=grow) * torch.from_numpy(chan)).to(dt)
        self.v_new = (rnd(B, Lr, H, self.T, d, scale=grow) * torch.from_numpy(chan)).to(dt)
        for b in range(B):                         # rows past the sequence's tokens are not read
            for t in (self.q, self.k_new, self.v_new):
                t[b, :, :, int(self.n[b]):] = float("nan")
        self.pos_new = (self.lens.reshape(B, -1).max(1) * 1.5).astype(np.float32)
        self.pos_new = np.floor(2 * self.pos_new) / 2
        self.n_half = int(2 * (self.pos_new.max() + self.T + 1))
        ang = 0.5 * np.arange(self.n_half)[:, None] * 10000.0 ** (-2.0 * np.arange(d // 2) / d)
        self.cos, self.sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        self.pass_n_new = pass_n_new

    # ------------------------------------------------------------ device side
    def params(self, **over):
        kw = dict(B=self.B, L=self.L, H=self.H, G=self.G, d=self.d, P=1, W=1,
                  dtype=self.kvc.KVC_BF16 if self.dtype == "bf16" else self.kvc.KVC_F32, n_max=64,
                  S_max=1, packed_rows=self.n_pages * self.page)
        kw.update(over)
        return self.kvc.make_params(**kw)

    def codes(self, name):
        """uint8 [pages, page, d] codes of the values held."""
        table = Q.e4m3_decode(np.arange(256))
        order = np.argsort(np.where(np.isnan(table), np.inf, table), kind="stable")[:254]
        v = self.val[name]
        at = np.searchsorted(table[order], np.where(np.isnan(v), 0.0, v))
        return np.where(np.isnan(v), UNUSED, order[np.minimum(at, 253)]).astype(np.uint8)

    def bound_array(self):
        out = np.full((self.n_pages, 2, self.d), -5, np.int8)
        for p in range(self.n_pages):
            if self.used[p].any():
                out[p] = Q.bounds(self.val["K"][p][self.used[p]])
        return out

    def scale_array(self, name):
        return np.where(self.used.any(1), 2.0 ** self.exp[name], np.nan).astype(np.float32)

    def upload(self, device="cuda"):
        kvc = self.kvc

        def up(x, dt=None):
            x = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
            return (x.to(dt) if dt else x).to(device).contiguous()
        B, L, H, d = self.B, self.L, self.H, self.d
        s = dict(K=up(self.codes("K")).view(-1, d), V=up(self.codes("V")).view(-1, d),
                 k_scale=up(self.scale_array("K")), v_scale=up(self.scale_array("V")),
                 bounds=up(self.bound_array()) if self.keep_bounds else None,
                 logm=None if self.logm is None else up(self.logm),
                 len=up(self.lens.reshape(B, L, H), torch.int32), cap=up(self.caps.reshape(B, L, H), torch.int32),
                 new=up((self.lens + self.n_u).reshape(B, L, H), torch.int32),
                 q=up(self.q), k_new=up(self.k_new), v_new=up(self.v_new), pos_new=up(self.pos_new, torch.float32),
                 cos=up(self.cos), sin=up(self.sin),
                 len_out=torch.full((B, L, H), -3, dtype=torch.int32, device=device))
        s["q_out"] = torch.full(self.q.shape, 5.0, dtype=self.q.dtype, device=device)
        s["out"] = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device=device)
        s["lse"] = torch.full(self.q.shape[:-1], 7.0, dtype=torch.float32, device=device)
        s["p"] = self.params()
        s["c"] = kvc.make_chunk(self.T, *self.layers, page_rows=self.page, page_table=up(self.table.reshape(B, L, H, -1)),
                                n_new=up(self.n, torch.int32) if self.pass_n_new else None)
        s["x"] = kvc.make_q8(s["K"], s["V"], s["k_scale"], s["v_scale"], s["bounds"], s["logm"])
        return s

    def append(self, s, stream=None, q=True):
        t = (s["cos"], s["sin"]) if self.rope else (None, None)
        self.kvc.kvc_q8_append(s["p"], s["c"], s["x"], *t, s["q"] if q else None, s["k_new"], s["v_new"],
                               s["pos_new"], s["q_out"] if q else None, s["len"], s["cap"], s["len_out"], stream)

    def workspace(self, s, n_sel=0):
        n = self.kvc.kvc_q8_workspace_bytes(s["p"], s["c"], n_sel)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["K"].device).fill_(0xFF)
        return s["ws"]

    def attn(self, s, sel=None, lse="lse", stream=None, q="q"):
        ws = self.workspace(s, 0 if sel is None else sel.shape[-1])
        self.kvc.kvc_q8_attn(s["p"], s["c"], s["x"], s[q], s["len"], s["new"], sel, s["out"],
                             s[lse] if lse else None, ws, stream)

    def select(self, s, n_sel, first, recent, stream=None, q="q"):
        s["sel"] = torch.full((*self.k_new.shape[:4], n_sel), -9, dtype=torch.int32, device=s["K"].device)
        self.kvc.kvc_q8_select(s["p"], s["c"], s["x"], s[q], s["len"], s["new"], first, recent, s["sel"], stream)
        return s["sel"]

    # ------------------------------------------------------------ oracle side
    def where(self, u):
        L, H, G = self.L, self.H, self.G
        b, l, h = u // (L * H), (u // H) % L, u % H
        return b, l - self.layers[0], h, slice(h * G, (h + 1) * G), int(self.n[b]), int(self.lens[u])

    def turned(self, x, b, n):
        """Rows [.., n, d] as they go on: rotated, or as they are, in fp32."""
        x = x.float().numpy()
        if not self.rope:
            return x
        e = (2 * self.pos_new[b]).astype(np.int64) + 2 * np.arange(n)
        return Q.rope(x, self.cos[e], self.sin[e])

    def do_append(self):
        """The append, on this object's own pages; the queries as they come out."""
        q = torch.full(self.q.shape, 5.0, dtype=self.q.dtype)
        for u in self.units:
            b, lr, h, hs, n, n0 = self.where(u)
            q[b, lr, hs, :n] = torch.from_numpy(self.turned(self.q[b, lr, hs, :n], b, n)).to(q.dtype)
            rows = {"K": self.turned(self.k_new[b, lr, h, :n], b, n), "V": self.v_new[b, lr, h, :n].float().numpy()}
            at = 0
            while at < n:
                j, r = divmod(n0 + at, self.page)
                c = min(self.page - r, n - at)
                p = self.table[u, j]
                for name in "KV":
                    v, self.exp[name][p] = Q.page_append(self.val[name][p, :r], self.exp[name][p], rows[name][at:at + c])
                    self.val[name][p, :r + c] = v
                self.used[p, r:r + c] = True
                if self.logm is not None:
                    self.logm[p * self.page + r:p * self.page + r + c] = 0.0
                at += c
        return q

    def check_cache(self, s, what=""):
        for name in "KV":
            got = Q.e4m3_decode(s[name].cpu().numpy().reshape(self.n_pages, self.page, self.d))
            np.testing.assert_array_equal(got, self.val[name], err_msg=f"{what} {name}")
            np.testing.assert_array_equal(s["k_scale" if name == "K" else "v_scale"].cpu().numpy(),
                                          self.scale_array(name), err_msg=f"{what} {name} scale")
        if s["bounds"] is not None:
            np.testing.assert_array_equal(s["bounds"].cpu().numpy(), self.bound_array(), err_msg=f"{what} bounds")
        if self.logm is not None:
            np.testing.assert_array_equal(s["logm"].cpu().numpy(), self.logm, err_msg=f"{what} logm")

    def check_append(self, s, what=""):
        q = self.do_append()
        assert torch.equal(s["q_out"].cpu(), q), what
        self.check_cache(s, what)
        want = np.full(self.U, -3, np.int64)
        want[self.units] = (self.lens + self.n_u)[self.units]
        np.testing.assert_array_equal(s["len_out"].cpu().numpy().reshape(-1), want, err_msg=what)

    def fill_new(self):
        """As if the new tokens had been appended as they are (for attention by itself)."""
        rope, self.rope = self.rope, False
        self.do_append()
        self.rope = rope

    def entries(self, u):
        """(K, V, ln m) in float64 of all entries of a unit, the new ones included."""
        N = int(self.lens[u] + self.n_u[u])
        e = np.arange(N)
        p, r = self.table[u][e // self.page], e % self.page
        K, V = (self.val[n][p, r] * 2.0 ** self.exp[n][p][:, None] for n in "KV")
        return K, V, (0.0 if self.logm is None else self.logm[p * self.page + r].astype(np.float64)) + np.zeros(N)

    def all_picks(self, n_sel, first, recent):
        """{unit: pages of every token}."""
        bd, sc = self.bound_array(), self.scale_array("K")
        return {u: self.picks(u, bd, sc, n_sel, first, recent) for u in self.units}

    def picks(self, u, bd, sc, n_sel, first, recent):
        b, lr, h, hs, n, n0 = self.where(u)
        out = []
        for t in range(n):
            own = (n0 + t) // self.page
            p = self.table[u, :own + 1]
            out.append(Q.pick_pages(self.q[b, lr, hs, t].float().numpy(), bd[p], sc[p], own, n_sel, first, recent))
        return out

    def check_select(self, s, picks, what=""):
        """picks: all_picks' answer."""
        want = np.full(s["sel"].shape, -9, np.int64)
        for u in self.units:
            b, lr, h, hs, n, n0 = self.where(u)
            for t, p in enumerate(picks[u]):
                want[b, lr, h, t] = -1
                want[b, lr, h, t, :len(p)] = p
        np.testing.assert_array_equal(s["sel"].cpu().numpy(), want, err_msg=what)

    def check_attn(self, s, pages=None, what=""):
        """pages: {unit: page numbers of every token}."""
        e = EPS[self.dtype]
        out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
        want_o, want_l = np.full(out.shape, 7.0), np.full(lse.shape, 7.0)
        for u in self.units:
            b, lr, h, hs, n, n0 = self.where(u)
            if n == 0:
                continue
            K, V, lm = self.entries(u)
            q = self.q[b, lr, hs, :n].double().numpy()
            pg = None if pages is None else pages[u]
            o, ls, p = Q.q8_attn(q, K, V, lm, n0, self.page, pg)
            N = len(K)
            dots = np.abs(q) @ np.abs(K).T / np.sqrt(self.d)
            # scores: fp32 sums of d products (a step 2^-23 of the partial sums each; tensor cores
            # may truncate), the query's fp16 parts (exact, or 2^-33 of the row's largest), the scale and
            # ln m in a handful of fp32 operations
            top = np.abs(q).max(-1, keepdims=True) * np.abs(K).sum(-1) / np.sqrt(self.d)
            size = dots + np.abs(np.where(np.isinf(lm), 0.0, lm))
            de = self.d * 2.0 ** -23 * dots + 2.0 ** -33 * top + 8 * 2.0 ** -24 * size
            dbar = (p * de).sum(-1)
            tol_l = (dbar + N * 2.0 ** -24 + 2.0 ** -21) / np.log(2) + 2.0 ** -22 * (np.abs(np.where(np.isinf(ls), 0, ls)) + 1)
            gl = lse[b, lr, hs, :n]
            with np.errstate(invalid="ignore"):
                bad = ~(np.abs(gl - ls) <= tol_l) & ~((gl == ls) & np.isinf(ls))
            assert not bad.any(), (what, u, "lse", gl[bad][:4], ls[bad][:4])
            # out: every numerator is off by its score's error, 2^x (2^-22) and half a step of
            # 11 bits (fp32: of 22; more than 64 rows in bf16: of 8), or, when subnormal in fp16, by
            # 2^-25 where the largest is 2^7 over 8 at least: 2^-29 of it; then the fp32 sums and the rounding of the result
            many = pages is None and self.G * self.T > 64
            half = 2.0 ** -22 if self.dtype != "bf16" else 2.0 ** -8 if many else 2.0 ** -11
            pn = half + 2.0 ** -21 + N * 2.0 ** -23
            pm = p.max(-1, keepdims=True)
            tol = (np.einsum("gtn,nd->gtd", p * (de + pn) + 2.0 ** -29 * pm * (p > 0), np.abs(V))
                   + (dbar + N * 2.0 ** -24 + 2.0 ** -21)[..., None] * np.abs(o) + 1.01 * e * np.abs(o) + 1e-30)
            go = out[b, lr, hs, :n]
            err = np.abs(go - o)
            assert (err <= tol).all(), (what, u, "out", err.max(), (err / tol).max())
            want_o[b, lr, hs, :n], want_l[b, lr, hs, :n] = go, gl
        np.testing.assert_array_equal(out, want_o, err_msg=what)        # rows of no token stay
        np.testing.assert_array_equal(lse, want_l, err_msg=what)
