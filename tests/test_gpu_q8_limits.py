"""The calls on the 8-bit cache at their ends: rows that see nothing, values and scales of all
sizes, full and invalid (b, l, h), optional arguments, other streams, graphs, packed
caches, rows beyond 2^31 elements."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from tests.chunk_cases import DT, EPS
from tests.q8_cases import UNUSED, Q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_probe_gb300 import build, kvc as K
    build.build()
    yield K
    torch.cuda.empty_cache()


def _done(kvc, code=0):
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == code


# ------------------------------------------------------------------ attention
WIDE = 4000                                            # table columns with which many rows are expanded


@pytest.mark.parametrize("n_new,wide", [(1, None), (7, None), (40, None), (40, WIDE)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(kvc, dtype, n_new, wide):
    """All of ln m is -inf: out 0, lse -inf; the other unit's rows as ever."""
    c = Q8(kvc, [200, 129], [n_new], H=2, dtype=dtype, page=32, max_pages=wide)
    c.fill_new()
    dead = c.table[0][:-(-(200 + n_new) // 32)]
    for p in dead:
        c.logm[p * 32:(p + 1) * 32] = -np.inf
    for pick in (None, (3, 1, 1)):
        s = c.upload()
        picks = None
        if pick:
            c.select(s, *pick)
            picks = c.all_picks(*pick)
        c.attn(s, s.get("sel"))
        _done(kvc)
        assert (s["out"][0, 0, :4] == 0).all() and (s["lse"][0, 0, :4] == -np.inf).all()
        c.check_attn(s, picks)


@pytest.mark.parametrize("T,wide", [(1, None), (3, None), (30, None), (30, WIDE)])
def test_masked_and_unused_places_may_hold_anything(kvc, T, wide):
    """Codes that are no numbers behind the last entry and in pages of nobody, NaN ln m and
    scales there, +-inf queries and NaN in rows of no token."""
    c = Q8(kvc, [77, 130, 16], [T], H=3, T=T + 2, page=64, max_pages=wide)
    c.fill_new()
    s = c.upload()
    assert (s["K"] == UNUSED).any() and torch.isnan(s["logm"]).any() and torch.isnan(s["k_scale"]).any()
    s["q"][..., T:, :] = float("inf")
    c.attn(s)
    _done(kvc)
    c.check_attn(s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,wide", [(1, None), (6, None), (50, None), (50, WIDE)])
def test_scales_at_their_ends(kvc, dtype, n, wide):
    """Pages whose values' scales are 2^-40 .. 2^40 side by side, keys likewise with queries that
    bring the scores back."""
    c = Q8(kvc, [200], [n], dtype=dtype, page=16, logm=False, max_pages=wide)
    c.fill_new()
    used = c.used.any(1)
    pages = np.flatnonzero(used)
    c.exp["V"][pages] = np.resize([-40, 40, 0, -3, -1, 3, -40, 12, 40], len(pages))
    c.exp["K"][pages] = -40
    c.q = (c.q.float() * 2.0 ** 38).to(DT[dtype])
    s = c.upload()
    c.attn(s)
    _done(kvc)
    c.check_attn(s)


def test_scores_that_rise_and_leap(kvc):
    """Scores of thousands, rising from page to page: the reference moves again and again."""
    for G, n, wide in ((4, 1, None), (2, 9, None), (8, 4, None), (4, 33, None), (4, 33, WIDE)):
        c = Q8(kvc, [400, 65], [n], H=2, G=G, page=16, logm=False, seed=G, max_pages=wide)
        c.fill_new()
        for j in range(c.table.shape[1]):
            for u in range(2):
                if c.table[u, j] >= 0:
                    c.exp["K"][c.table[u, j]] += j // 3
        s = c.upload()
        c.attn(s)
        _done(kvc)
        c.check_attn(s, what=f"G {G}")


def test_optional_outputs_and_repeats(kvc):
    """lse may be left out; the same call gives the same bits, whatever the workspace held."""
    for n_new, wide in (([1, 1], None), ([3, 5], None), ([40, 33], None), ([40, 33], WIDE)):
        c = Q8(kvc, [100, 0, 300, 64], n_new, B=2, H=2, page=32, max_pages=wide)
        c.fill_new()
        a, b = c.upload(), c.upload()
        c.attn(a)
        c.attn(b, lse=None)
        _done(kvc)
        assert torch.equal(a["out"], b["out"]) and (b["lse"] == 7.0).all()
        a["out"].fill_(7.0)
        ws = a["ws"]
        kvc.kvc_q8_attn(a["p"], a["c"], a["x"], a["q"], a["len"], a["new"], None, a["out"], a["lse"], ws)
        _done(kvc)
        assert torch.equal(a["out"], b["out"])
        c.check_attn(a)


def test_picked_pages_that_are_none(kvc):
    """Numbers of no visible page, in any order, are passed over; a row left with none sees nothing."""
    c = Q8(kvc, [150, 300], [2], H=2, page=16)
    c.fill_new()
    s = c.upload()
    own = [(150 + t) // 16 for t in range(2)], [(300 + t) // 16 for t in range(2)]
    lists = [[[own[0][0], -1, 3, 99999], [-5, 1 << 30, own[0][1] + 1, -1]], [[0, 2, 1, own[1][0]], [own[1][1], 5, -2, 4]]]
    s["sel"] = torch.tensor(lists, dtype=torch.int32, device="cuda").view(1, 1, 2, 2, 4)
    c.attn(s, s["sel"])
    _done(kvc)
    picks = {u: [[j for j in lists[u][t] if 0 <= j <= own[u][t]] for t in range(2)] for u in range(2)}
    assert picks[0][1] == []
    c.check_attn(s, picks)
    assert (s["out"][0, 0, :4, 1] == 0).all()


@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("what", ["inf", "nan", "scale", "all scales"])
def test_a_choice_among_scores_that_are_no_numbers(kvc, n, what):
    """Infinite or NaN queries and scales of one (l, h): its rows hold distinct pages that it sees,
    the first and last ones among them; nothing beyond its rows is written, the others choose as ever."""
    c = Q8(kvc, [400, 500, 300], [n], H=3, page=16)
    c.fill_new()
    s, good = c.upload(), c.upload()
    pages = s["c"]._keep[0].view(3, -1)[1, :500 // 16].long()
    if what in ("inf", "nan"):
        s["q"].view(1, 1, 3, 4, n, 128)[:, :, 1] = float(what)
    else:
        s["k_scale"][pages[::2] if what == "scale" else pages] = float("nan")
    c.select(s, 6, 1, 2)
    c.select(good, 6, 1, 2)
    _done(kvc)
    assert torch.equal(s["sel"][0, 0, [0, 2]], good["sel"][0, 0, [0, 2]])
    for t, row in enumerate(s["sel"][0, 0, 1].cpu().numpy()):
        own = (500 + t) // 16
        assert (np.diff(row) > 0).all() and row[0] == 0 and row[-1] == own and own - 1 in row


# ------------------------------------------------------------------ invalid and full units
def test_units_out_of_range_are_skipped(kvc):
    """Lengths that are negative, shrink, grow by more than T or pass the table: reported, rows and
    lists left alone; the other units' results as ever."""
    for n, wide in ((1, None), (40, None), (40, WIDE)):
        c = Q8(kvc, [50, 60, 70, 80, 90], [n], H=5, page=16, max_pages=wide)
        c.fill_new()
        s = c.upload()
        good = c.upload()
        c.attn(good)
        s["len"].view(-1)[0] = -1
        s["new"].view(-1)[1] = 59
        s["new"].view(-1)[2] = 70 + n + 1
        s["len"].view(-1)[3], s["new"].view(-1)[3] = 1 << 30, (1 << 30) + n
        c.attn(s)
        _done(kvc, kvc.KVC_EDEVICE)
        c.select(s, 3, 1, 1)
        _done(kvc, kvc.KVC_EDEVICE)
        assert (s["out"][0, 0, :16] == 7.0).all() and (s["lse"][0, 0, :16] == 7.0).all()
        assert torch.equal(s["out"][0, 0, 16:], good["out"][0, 0, 16:])
        assert (s["sel"][0, 0, :4] == -9).all() and (s["sel"][0, 0, 4] != -9).all()


def test_pages_outside_the_extent_are_reported(kvc):
    """A page number out of range: no access outside the cache; the other unit as ever."""
    for n, wide in ((1, None), (40, None), (40, WIDE)):
        c = Q8(kvc, [100, 100], [n], H=2, page=16, max_pages=wide)
        c.fill_new()
        for bad in (-1, c.n_pages, 1 << 30):
            s = c.upload()
            good = c.upload()
            c.attn(good)
            s["c"]._keep[0].view(2, -1)[0, 2] = bad
            c.attn(s)
            _done(kvc, kvc.KVC_EDEVICE)
            assert torch.equal(s["out"][0, 0, 4:], good["out"][0, 0, 4:])
            c.select(s, 4, 1, 1)
            _done(kvc, kvc.KVC_EDEVICE)
            c.select(good, 4, 1, 1)
            _done(kvc)
            assert torch.equal(s["sel"][0, 0, 1], good["sel"][0, 0, 1])


APPEND_BAD = {
    "a length below 0": (lambda s, c: s["len"].view(-1).__setitem__(0, -1), "EDEVICE"),
    "no room": (lambda s, c: s["cap"].view(-1).__setitem__(0, 102), "ECAPACITY"),
    "past the table": (lambda s, c: (s["len"].view(-1).__setitem__(0, 16 * c.table.shape[1]), s["cap"].view(-1).__setitem__(0, 1 << 30)), "EDEVICE"),
    "past table and room": (lambda s, c: s["len"].view(-1).__setitem__(0, 16 * c.table.shape[1]), "ECAPACITY"),
    "a page out of range": (lambda s, c: s["c"]._keep[0].view(3, -1)[0].__setitem__(slice(6, 8), c.n_pages), "EDEVICE"),
    "a page below 0": (lambda s, c: s["c"]._keep[0].view(3, -1)[0].__setitem__(6, -3), "EDEVICE"),
}


@pytest.mark.parametrize("name", list(APPEND_BAD))
@pytest.mark.parametrize("n", [5, 20])
def test_append_skips_bad_and_full_units(kvc, name, n):
    """The unit's pages, scales, bounds and length stay as they were; the others are appended to."""
    c = Q8(kvc, [100, 31, 64], [n], H=3, page=16, reserve=16)
    s = c.upload()
    before = {k: s[k].clone() for k in ("K", "V", "k_scale", "v_scale", "bounds", "logm")}
    spoil, code = APPEND_BAD[name]
    spoil(s, c)
    old = s["len"].clone()
    c.append(s)
    _done(kvc, getattr(kvc, "KVC_" + code))
    assert s["len_out"].view(-1)[0] == old.view(-1)[0]
    c.units = [1, 2]
    q = c.do_append()
    for k in before:
        rows = 16 if before[k].shape[0] == c.n_pages * 16 else 1
        for p in [x for x in c.table[0] if x >= 0]:
            assert torch.equal(s[k][p * rows:(p + 1) * rows].view(torch.uint8), before[k][p * rows:(p + 1) * rows].view(torch.uint8)), (k, p)
    c.check_cache(s, name)
    assert (s["len_out"].view(-1)[1:].cpu() == torch.tensor([31 + n, 64 + n])).all()
    assert torch.equal(s["q_out"][0, 0, 4:].cpu(), q[0, 0, 4:])


@pytest.mark.parametrize("pos", [-0.5, float("nan"), float("inf"), 1e9, None])
def test_positions_outside_the_tables_are_refused_on_the_device(kvc, pos):
    """Nothing of that sequence is appended or rotated; None: the last token's alone is outside."""
    c = Q8(kvc, [10, 20], [3, 2], B=2, page=16)
    s = c.upload()
    s["pos_new"][0] = pos if pos is not None else (c.n_half - 4) / 2
    c.append(s)
    _done(kvc, kvc.KVC_EDEVICE)
    assert (s["q_out"][0] == 5.0).all() and s["len_out"].view(-1).tolist() == [10, 22]
    c.units = [1]
    c.do_append()
    c.check_cache(s)
    s["pos_new"][0] = (c.n_half - 6) / 2                   # the last that fits
    c.append(s)
    _done(kvc)
    assert s["len_out"].view(-1).tolist() == [13, 22]


def test_counts_out_of_range(kvc):
    c = Q8(kvc, [10, 20, 5], [3, 2, 1], B=3, page=16)
    s = c.upload()
    s["c"]._keep[1][0], s["c"]._keep[1][2] = 4, -1
    c.append(s)
    _done(kvc, kvc.KVC_EDEVICE)
    assert s["len_out"].view(-1).tolist() == [10, 22, 5]
    assert (s["q_out"][0] == 5.0).all() and (s["q_out"][2] == 5.0).all()
    c.units = [1]
    c.do_append()
    c.check_cache(s)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 8, 9, 40])
def test_append_without_rotation_queries_or_bounds(kvc, dtype, n):
    c = Q8(kvc, [30, 0, 17], [n], H=3, dtype=dtype, rope=False, bounds=False, logm=False)
    s = c.upload()
    c.append(s, q=False)
    _done(kvc)
    assert (s["q_out"] == 5.0).all()
    c.do_append()
    c.check_cache(s)


@pytest.mark.parametrize("n", [2, 30])
def test_queries_are_rotated_in_place(kvc, n):
    c = Q8(kvc, [30, 64], [n, n - 1], B=2)
    s = c.upload()
    s["q_out"] = s["q"]
    c.append(s)
    _done(kvc)
    want = c.do_append()
    for b, k in enumerate((n, n - 1)):
        assert torch.equal(s["q"][b, :, :, :k].cpu(), want[b, :, :, :k])
    assert torch.isnan(s["q"][1, :, :, n - 1:].float()).all()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_a_page_grows_token_by_token(kvc, page, d):
    """Scales that grow, stay and would shrink; zeros; every step against the oracle."""
    c = Q8(kvc, [0, 5, page - 2], [1], H=3, d=d, page=page, reserve=40, spread=3.0, rope=False)
    c.caps[:] = c.lens + 41
    s = c.upload()
    rng = np.random.default_rng(2)
    for t in range(24):
        size = [0.0, 1.0, 2.0 ** -20, 300.0, 2.0 ** 30][t % 5] if t > 2 else 0.0
        c.k_new = torch.from_numpy((size * rng.standard_normal((1, 1, 3, 1, d))).astype(np.float32)).bfloat16()
        c.v_new = torch.from_numpy((size * rng.standard_normal((1, 1, 3, 1, d))).astype(np.float32)).bfloat16()
        s["k_new"].copy_(c.k_new)
        s["v_new"].copy_(c.v_new)
        c.append(s)
        _done(kvc)
        c.do_append()
        c.check_cache(s, f"step {t}")
        c.lens = c.lens + 1
        s["len"].copy_(s["len_out"])
        assert (s["len"].cpu().view(-1).numpy() == c.lens).all()


def test_values_beyond_the_scales_saturate(kvc):
    c = Q8(kvc, [0], [2], rope=False)
    for x in (c.k_new, c.v_new):
        x.fill_(2.0 ** 60)
        x[..., 1, :] = -2.0 ** 45
    s = c.upload()
    c.append(s)
    _done(kvc)
    c.do_append()
    c.check_cache(s)
    p = int(c.table[0, 0])
    assert s["k_scale"][p] == 2.0 ** 40 and (s["K"].view(torch.float8_e4m3fn)[p * 16].float() == 448).all()


# ------------------------------------------------------------------ pack
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 128), (128, 64)])
def test_pack(kvc, dtype, d, page):
    """A ragged packed cache (any row offsets) into pages; an (l, h) out of range or too long gets
    length 0 and nothing else."""
    c = Q8(kvc, [0, 1, page, page + 1, 300, 77], [0], L=3, H=2, d=d, page=page, dtype=dtype, T=1)
    for n in "KV":
        c.val[n][:], c.exp[n][:] = np.nan, 0
    c.used[:] = False
    c.logm[:] = np.nan
    rng = np.random.default_rng(4)
    off = np.cumsum(c.lens + 3) - c.lens - 1
    rows = int((c.lens + 3).sum()) + 5
    dt = DT[dtype]
    Kp, Vp = (torch.from_numpy((rng.standard_normal((rows, d)) * np.exp2(rng.integers(-3, 4, (rows, 1)))).astype(np.float32)).to(dt)
              for _ in range(2))
    lm = rng.uniform(0, 2, rows).astype(np.float32)
    s = c.upload()
    dev = dict(Kp=Kp.cuda(), Vp=Vp.cuda(), lm=torch.from_numpy(lm).cuda(), off=torch.from_numpy(off).cuda())
    before = {k: s[k].clone() for k in ("K", "V")}
    kvc.kvc_q8_pack(s["p"], s["c"], s["x"], dev["Kp"], dev["Vp"], dev["lm"], s["len"], dev["off"], s["cap"], s["len_out"])
    _done(kvc)
    for u in range(c.U):
        for j in range(-(-int(c.lens[u]) // page)):
            p, k = c.table[u, j], min(page, int(c.lens[u]) - j * page)
            r = off[u] + j * page
            for n, src in (("K", Kp), ("V", Vp)):
                c.val[n][p, :k], c.exp[n][p] = Q.page_append(np.zeros((0, d)), 0, src[r:r + k].float().numpy())
            c.used[p, :k] = True
            c.logm[p * page:p * page + k] = lm[r:r + k]
    c.check_cache(s)
    assert (s["len_out"].cpu().view(-1).numpy() == c.lens).all()
    # what does not fit is left out
    for k in before:
        s[k].copy_(before[k])
    s["cap"].view(-1)[4], dev["off"][3], s["len"].view(-1)[2] = 299, rows, -4
    kvc.kvc_q8_pack(s["p"], s["c"], s["x"], dev["Kp"], dev["Vp"], dev["lm"], s["len"], dev["off"], s["cap"], s["len_out"])
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() in (kvc.KVC_EDEVICE, kvc.KVC_ECAPACITY)
    assert s["len_out"].cpu().view(-1).tolist() == [0, 1, 0, 0, 0, 77]
    for p in c.table[3:5][c.table[3:5] >= 0]:
        assert (s["K"][p * page:(p + 1) * page] == UNUSED).all()


# ------------------------------------------------------------------ streams, graphs, devices
def test_other_streams_and_graphs(kvc):
    """The calls on a stream that is not current, and captured together and replayed with new inputs."""
    c = Q8(kvc, [100, 37, 200, 64], [3, 2], B=2, H=2, page=32)
    ref = c.upload()
    c.append(ref)
    ref["new"].copy_(ref["len_out"])
    c.select(ref, 4, 1, 1, q="q_out")
    c.attn(ref, ref["sel"], q="q_out")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = c.upload()
    s["sel"] = torch.full_like(ref["sel"], -9)
    ws = torch.empty(kvc.kvc_q8_workspace_bytes(s["p"], s["c"], 4), dtype=torch.uint8, device="cuda")

    def calls(stream):
        c.append(s, stream)
        kvc.kvc_q8_select(s["p"], s["c"], s["x"], s["q_out"], s["len"], s["len_out"], 1, 1, s["sel"], stream)
        kvc.kvc_q8_attn(s["p"], s["c"], s["x"], s["q_out"], s["len"], s["len_out"], s["sel"], s["out"], s["lse"], ws, stream)

    def same():
        torch.cuda.synchronize()
        assert kvc.kvc_device_error() == 0
        for k in ("K", "V", "k_scale", "bounds", "q_out", "sel", "out", "lse"):
            assert torch.equal(s[k].view(torch.uint8), ref[k].view(torch.uint8)), k
    torch.cuda.synchronize()
    calls(side)
    same()
    graphs = []
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):                                     # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            calls(side)
        graphs.append(g)
    fresh = c.upload()
    for k in ("K", "V", "k_scale", "v_scale", "bounds", "logm"):
        s[k].copy_(fresh[k])
    for k in ("sel", "out", "lse", "q_out"):
        s[k].zero_()
    s["out"].copy_(fresh["out"]), s["lse"].copy_(fresh["lse"]), s["q_out"].copy_(fresh["q_out"]), s["sel"].fill_(-9)
    graphs[0].replay()
    graphs[1].replay()
    graphs[0].replay()
    same()


def test_tensors_of_other_kinds_are_refused(kvc):
    c = Q8(kvc, [20], [1])
    s = c.upload()
    ws = c.workspace(s)
    with pytest.raises(ValueError):
        kvc.kvc_q8_attn(s["p"], s["c"], s["x"], s["q"].cpu(), s["len"], s["new"], None, s["out"], s["lse"], ws)
    with pytest.raises(ValueError):
        kvc.kvc_q8_attn(s["p"], s["c"], s["x"], s["q"].repeat(1, 1, 1, 1, 2)[..., ::2], s["len"], s["new"], None, s["out"], s["lse"], ws)
    with pytest.raises(ValueError):
        kvc.make_q8(s["K"].t(), s["V"], s["k_scale"], s["v_scale"])
    with pytest.raises(kvc.KvcError):
        kvc.kvc_q8_append(s["p"], s["c"], s["x"], None, None, None, s["k_new"], s["v_new"], None, None, s["len"], s["cap"], s["len"])


# ------------------------------------------------------------------ large
def test_rows_beyond_2_31_elements(kvc):
    """A cache whose pages lie beyond 2^31 bytes and elements: append, choice, attention of few and
    many rows."""
    page, d, pages = 128, 128, 140000                      # 17.9 M rows, 2.3 G codes each of K and V
    c = Q8(kvc, [300, 260], [70, 66], B=2, G=2, page=page, seed=3)
    base = Q8(kvc, [300, 260], [70, 66], B=2, G=2, page=page, seed=3)
    up = pages - c.n_pages
    s = c.upload()
    big = {}
    for k in ("K", "V"):
        big[k] = torch.full((pages * page, d), UNUSED, dtype=torch.uint8, device="cuda")
        big[k][up * page:] = s[k]
    for k, n in (("k_scale", 1), ("v_scale", 1), ("bounds", 1), ("logm", page)):
        big[k] = torch.zeros((pages * n, *s[k].shape[1:]), dtype=s[k].dtype, device="cuda")
        big[k][up * n:] = s[k]
    s["p"] = c.params(packed_rows=pages * page)
    table = torch.from_numpy(np.where(c.table >= 0, c.table + up, c.table).astype(np.int32)).cuda()
    s["c"] = kvc.make_chunk(c.T, 0, 1, page_rows=page, page_table=table, n_new=torch.tensor([70, 66], dtype=torch.int32, device="cuda"))
    s["x"] = kvc.make_q8(*(big[k] for k in ("K", "V", "k_scale", "v_scale", "bounds", "logm")))
    small = base.upload()
    for x in (s, small):
        base.append(x)
        base.select(x, 2, 0, 1, q="q_out")
        base.attn(x, x["sel"], q="q_out")
        x["picked"] = x["out"].clone()
        base.attn(x, q="q_out")
    _done(kvc)
    for k, n in (("K", page), ("V", page), ("k_scale", 1), ("v_scale", 1), ("bounds", 1), ("logm", page)):
        assert torch.equal(big[k][up * n:].view(torch.uint8), small[k].view(torch.uint8)), k
    for k in ("q_out", "sel", "picked", "out", "lse", "len_out"):
        assert torch.equal(s[k].view(torch.uint8), small[k].view(torch.uint8)), k


def test_choice_of_many_pages(kvc):
    """32768 pages a (b, l, h), the most there are; scores that are all equal give the lowest pages."""
    page, R = 16, 32768
    n = R * page - 3
    p = kvc.make_params(B=1, L=1, H=1, G=4, d=64, P=1, W=1, n_max=64, S_max=1, dtype=kvc.KVC_BF16, packed_rows=R * page)
    z = dict(device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    bounds = torch.randint(-112, 113, (R, 2, 64), generator=g, dtype=torch.int8, **z).sort(1).values.contiguous()
    scale = torch.exp2(torch.randint(-2, 3, (R,), generator=g, **z).float())
    K = torch.zeros((R * page, 64), dtype=torch.uint8, **z)
    x = kvc.make_q8(K, K.clone(), scale, scale.clone(), bounds)
    table = torch.randperm(R, generator=g, **z).int().view(1, R)
    for T in (1, 2):
        c = kvc.make_chunk(T, 0, 1, page_rows=page, page_table=table)
        q = torch.randn((1, 1, 4, T, 64), generator=g, **z).bfloat16()
        lens = torch.tensor([n - T], dtype=torch.int32, **z)
        sel = torch.empty((1, 1, 1, T, 500), dtype=torch.int32, **z)
        kvc.kvc_q8_select(p, c, x, q, lens, lens + T, 2, 3, sel)
        _done(kvc)
        t = table[0].long().cpu()
        for k in range(T):
            own = (n - T + k) // page
            want = Q.pick_pages(q[0, 0, :, k].float().cpu().numpy(), bounds.cpu().numpy()[t[:own + 1]], scale.cpu().numpy()[t[:own + 1]],
                                own, 500, 2, 3)
            np.testing.assert_array_equal(sel[0, 0, 0, k].cpu().numpy(), want)
        q.zero_()
        kvc.kvc_q8_select(p, c, x, q, lens, lens + T, 2, 3, sel)
        _done(kvc)
        assert sel[0, 0, 0, 0].tolist() == list(range(497)) + [(n - T) // page - 2 + i for i in range(3)]


# ------------------------------------------------------------------ scores whose steps are large
@pytest.mark.parametrize("n, dtype", [(1, "bf16"), (9, "bf16"), (9, "f32"), (70, "bf16"), (70, "f32")])
@pytest.mark.parametrize("power", [24, 28, 34])
def test_scores_with_steps_far_above_one(kvc, n, dtype, power):
    """Scores around 2^power (in fp32 a step is 1 to 1024 there): the row's one largest still gives 1.
    A score is off by at most d 2^-23 of the sum of its products' magnitudes, so a row whose largest score leads by
    more than twice that and 60 has the output of that entry alone, to the roundings of its numerator and of the result."""
    c = Q8(kvc, [1300, 700, 90, 3000], [n] * 2, B=2, H=2, T=n, dtype=dtype, max_pages=700, logm=False, seed=31 + power)
    c.fill_new()
    c.q *= 2.0 ** power / 4
    s = c.upload()
    c.attn(s)
    torch.cuda.synchronize()
    assert kvc.kvc_device_error() == 0
    c.check_attn(s)
    out, alone = s["out"].double().cpu().numpy(), 0
    rtol = EPS[dtype] + (2.0 ** -22 if dtype == "f32" else 2.0 ** -8 if n == 70 else 2.0 ** -11) + 2.0 ** -21
    for u in c.units:
        b, lr, h, hs, n_b, n0 = c.where(u)
        K, V, lm = c.entries(u)
        q = c.q[b, lr, hs].double().numpy()
        x = Q.q8_scores(q, K, lm, n0, c.page)
        off = c.d * 2.0 ** -23 * (np.abs(q) @ np.abs(K).T / np.sqrt(c.d)).max(-1)
        best, rest = x.argmax(-1), np.sort(x, -1)[..., -2]
        clear = x.max(-1) - rest > 2 * off + 60
        alone += clear.sum()
        np.testing.assert_allclose(out[b, lr, hs][clear], V[best][clear], rtol=rtol, atol=1e-12)
    assert alone > 0
