"""kvc_q8_attn with scores far above one, where a step of fp32 is no longer small: every key of a
(b, l, h) is the same, so that all its scores are, and only ln m and the visible entries
decide the weights.  In each form of the kernel: one token by a cluster, cut into pieces, a warp an
item, several row tiles, picked pages, expanded rows."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from tests.chunk_cases import EPS
from tests.q8_cases import Q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


LENS = [1300, 700, 90, 3000]
LONG = np.linspace(2500, 4500, 32)                         # several groups a warp where the line is cut into pieces
FORMS = {
    "cluster": dict(lens=LENS, n_new=[1], H=4),
    "cluster, two row tiles": dict(lens=LENS, n_new=[3], H=4),
    "cluster, four row tiles": dict(lens=LENS, n_new=[9, 7], B=2, H=2),
    "cluster, picked pages": dict(lens=LENS, n_new=[3], H=4, pick=(60, 1, 2)),
    "pieces": dict(lens=LONG, n_new=[1], H=32, page=128),
    "pieces, three row tiles": dict(lens=LONG, n_new=[5], H=32, page=128),
    "a warp an item": dict(lens=60 + np.arange(2500) % 70, n_new=[1], L=125, H=20, d=64),
    "expanded": dict(lens=LONG[:24], n_new=[40], H=24, page=64, max_pages=400),
}
LARGE = ("pieces", "pieces, three row tiles", "a warp an item", "expanded")     # a few powers of these
ALL = [(f, "bf16") for f in FORMS] + [(f, "f32") for f in FORMS if f != "expanded"]
STREAMED = [(f, t) for f, t in ALL if f != "expanded"]


def _same_keys(kvc, form, dtype, seed, q_power, k_power=0, v_exps=(0,)):
    """The cache, with queries around 2^q_power, keys around 2^k_power, and its device copy."""
    kw = dict(FORMS[form])
    pick = kw.pop("pick", None)
    c = Q8(kvc, dtype=dtype, logm=False, seed=seed, **kw)
    c.fill_new()
    rng = np.random.default_rng(seed)
    key = Q.e4m3_round(rng.choice([-1.0, 1.0], c.d) * rng.uniform(0.5, 2.0, c.d))
    c.val["K"][c.used] = key
    pages = np.flatnonzero(c.used.any(1))
    c.exp["K"][pages] = k_power
    c.exp["V"][pages] = np.resize(v_exps, len(pages))
    c.q = (c.q.double() * 2.0 ** q_power).to(c.q.dtype)
    return c, pick


def _run(c, pick):
    s = c.upload()
    picks = None
    if pick:
        c.select(s, *pick)
        sel = s["sel"].cpu().numpy()
        picks = {u: [[int(j) for j in row if j >= 0] for row in sel[(*c.where(u)[:3],)][:c.where(u)[4]]] for u in c.units}
    c.attn(s, s.get("sel"))
    torch.cuda.synchronize()
    assert c.kvc.kvc_device_error() == 0
    return s, picks


def _check_averages(c, s, picks, numerator=0.0):
    """Equal scores: out is the average of the values seen.  Scores beyond 2^23 are whole numbers, so the
    numerators are the same power of two (2^-22 off at most; `numerator`: relative rounding of
    numerators that are not), and what is left is the fp32 sum of N values (a step 2^-23 of the
    partial sums each), that of the numerators, and the rounding of the result.  lse: the score's own
    error (fp32 sums of d products, scale), and the sum's."""
    out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
    for u in c.units:
        b, lr, h, hs, n, n0 = c.where(u)
        K, V, _ = c.entries(u)
        q = c.q[b, lr, hs, :n].double().numpy()
        for t in sorted({0, 1, n // 2, n - 1} & set(range(n))):
            see = np.arange(len(V)) <= n0 + t
            if picks is not None:
                see &= np.isin(np.arange(len(V)) // c.page, picks[u][t])
            N = see.sum()
            o, size = V[see].mean(0), np.abs(V[see]).mean(0)
            tol = (N * 2.0 ** -23 + 2.0 ** -20 + numerator) * size + (N * 2.0 ** -24 + 2.0 ** -21 + 1.01 * EPS[c.dtype]) * np.abs(o) + 1e-30
            err = np.abs(out[b, lr, hs, t] - o)
            assert (err <= tol).all(), (u, t, err.max(), (err / tol).max())
            ls = q[:, t] @ K[0] / np.sqrt(c.d) / np.log(2) + np.log2(N)
            dots = np.abs(q[:, t]) @ np.abs(K[0]) / np.sqrt(c.d) / np.log(2)
            tol_l = (c.d * 2.0 ** -23 + 2.0 ** -20) * dots + 2.0 ** -20
            assert (np.abs(lse[b, lr, hs, t] - ls) <= tol_l).all(), (u, t, lse[b, lr, hs, t], ls)


# ------------------------------------------------------------------ steps of 1 to 1024
@pytest.mark.parametrize("form,dtype,power", [(f, t, x) for f, t in STREAMED
                                              for x in ((25, 28) if f in LARGE else (24, 25, 26, 27, 28, 34))])
def test_equal_scores_over_pages_of_other_value_scales(kvc, form, dtype, power):
    """Neighbouring pages' value scales differ by 2 to 8: equal scores keep equal weights."""
    c, pick = _same_keys(kvc, form, dtype, 5 + power, power, v_exps=(0, -1, -3, -2, 0, 2, 1, -1))
    _check_averages(c, *_run(c, pick))


@pytest.mark.parametrize("form,dtype,power,step",
                         [(f, t, x, y) for f, t in STREAMED
                          for x, y in (((25, 8), (27, 16)) if f in LARGE else
                                       ((24, 8), (24, 16), (25, 8), (25, 16), (26, 8), (26, 16), (27, 16), (28, 32)))])
def test_ln_m_steps_on_large_scores(kvc, form, dtype, power, step):
    """ln m of 0 and step ln 2 in turn: a score may stand 16 above the reference exactly, where its numerator
    is not to pass fp16.  A row's result lies between the values' ends, whatever the rounding of its
    scores makes of the weights; and the log-sum-exp is known to that rounding."""
    c, pick = _same_keys(kvc, form, dtype, 50 + power, power)
    c.logm = np.full(c.n_pages * c.page, np.nan, np.float32)
    for u in range(c.U):
        e = np.arange(int(c.lens[u] + c.n_u[u]))
        c.logm[c.table[u][e // c.page] * c.page + e % c.page] = step * np.log(2.0) * (e // 48 % 2)
    s, picks = _run(c, pick)
    assert torch.isfinite(s["out"].float()).all() and torch.isfinite(s["lse"]).all()
    c.check_attn(s, picks)
    out = s["out"].double().cpu().numpy()
    for u in c.units:
        b, lr, h, hs, n, n0 = c.where(u)
        V = c.entries(u)[1]
        room = (2.0 * EPS[dtype] + len(V) * 2.0 ** -22 + 2.0 ** -10) * np.abs(V).max(0)
        assert (out[b, lr, hs, :n] <= V.max(0) + room).all() and (out[b, lr, hs, :n] >= V.min(0) - room).all()


# ------------------------------------------------------------------ scores of the largest sizes
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("form,dtype", ALL)
def test_scores_of_all_sizes_there_are(kvc, form, dtype, sign):
    """Queries around 2^62 and keys around 2^40, all products of a row's of one sign: scores near 2^107, which
    a row that has seen nothing is not to be taken for."""
    c, pick = _same_keys(kvc, form, dtype, 9, 62, 40, v_exps=(0, 0, -1))
    key = torch.from_numpy(np.sign(c.val["K"][c.used][0]))
    c.q = (c.q.double().abs().clamp(2.0 ** 58, 2.0 ** 64) * sign * key).to(c.q.dtype)
    s, picks = _run(c, pick)
    scores = s["lse"][s["lse"] != 7.0]
    assert (scores.abs() > 1e30).all() and ((scores < 0) == (sign < 0)).all()
    _check_averages(c, s, picks)
