"""Cases and plain forms of the operators of the 8-bit KV cache.

  append  kvc_q8_append: the queries and keys of n new tokens per sequence are
          rotated by their positions, and every (b, l, h)'s keys and values go
          into its pages as e4m3 codes with a power-of-two scale for each page
  attn    kvc_q8_attn: the new tokens attend over the 8-bit cache
  sparse  kvc_q8_select and kvc_q8_attn: every token of every KV head picks pages
          by a cheap score and attends over these

Units are the (b, l, h) in order; U = B*L*H.  A page holds R entries of one unit.
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634
TOP, LEAST, MOST = 448.0, -40, 40        # largest code; the scales are 2^LEAST .. 2^MOST
UNUSED = 0x7F                            # the code that is not a number


def _case(name, op, B=1, L=1, H=8, G=4, d=128, T=1, lo=256, hi=512, page=64, dtype="bf16",
          logm=False, ragged=False, n_sel=0, first=1, recent=2):
    c = dict(op=op, B=B, L=L, H=H, G=G, d=d, T=T, lo=lo, hi=hi, page=page, dtype=dtype, logm=logm,
             ragged=ragged, n_sel=n_sel, first=first, recent=recent)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one layer: pure latency, as a model that runs layer by layer calls it
        _case("append one token, one layer", "append", lo=200, hi=512),
        # a decode step of a batch of 16, all 32 layers in one call
        _case("append one token, 16 sequences", "append", B=16, L=32, lo=200, hi=700),
        # up to 5 drafted tokens for 16 sequences, fp32, small pages
        _case("append drafts, fp32", "append", B=16, T=5, lo=1000, hi=4096, page=16, dtype="f32",
              ragged=True),
        # a 2048-token chunk of a prompt, one layer
        _case("append 2048-token chunk", "append", T=2048, lo=6001, hi=6001),
        # one token of one layer over a short compressed cache: latency
        _case("attn one token, one layer", "attn", lo=200, hi=512, logm=True),
        # one decode step of all layers over a 16K context compressed to 25%
        _case("attn one token, all layers", "attn", L=32, lo=3200, hi=5000, logm=True),
        # up to 5 drafted tokens verified for 16 sequences
        _case("attn drafts", "attn", B=16, T=5, lo=1000, hi=4096, page=32, ragged=True),
        # the last 2048-token chunk of a 16K prompt, one layer
        _case("attn 2048-token chunk of 16K", "attn", T=2048, lo=14336, hi=14336, page=128),
        # the repository's small fp32 configuration (2 KV / 8 query heads, d 64, context 512)
        _case("attn small fp32", "attn", H=2, d=64, T=33, lo=128, hi=512, page=16, dtype="f32",
              logm=True),
        # a decode step of one layer over a 16K context, 2048 of its entries
        _case("sparse one token, one layer", "sparse", lo=15000, hi=16384, n_sel=32),
        # a decode step of all layers over 32K tokens, 2048 entries each
        _case("sparse one token, all layers", "sparse", L=32, lo=30000, hi=32768, n_sel=32),
        # a 300-token follow-up turn over a 16K context, every token with pages of its own
        _case("sparse follow-up turn", "sparse", T=300, lo=15000, hi=16384, page=32, n_sel=32,
              recent=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("append", "attn", "attn", "sparse"))
        f32 = rng.random() < 0.15
        B, L = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
        H, G = rng.choice((1, 2, 3, 8, 8, 8)), rng.choice((1, 2, 4, 4, 8))
        T = 1 if rng.random() < 0.3 else _log_int(rng, 1, 300 if op == "sparse" else 2048)
        hi = _log_int(rng, 33, 32768 if op == "sparse" else 16384)
        first, recent = rng.choice((0, 1, 2)), rng.choice((1, 2, 4))
        c = _case(None, op, B=B, L=L, H=H, G=G, d=rng.choice((64, 128, 128)), T=T,
                  lo=int(hi * rng.uniform(0.0, 1.0)), hi=hi, page=rng.choice((16, 32, 64, 128)),
                  dtype="f32" if f32 else "bf16", logm=op != "append" and rng.random() < 0.5,
                  ragged=B > 1 and rng.random() < 0.5,
                  n_sel=_log_int(rng, first + recent, 64) if op == "sparse" else 0,
                  first=first, recent=recent)
        units, rows, keys = B * L * H, G * T, hi + T
        if not 2e5 < units * keys * c["d"] < (1.1e9 if op == "sparse" else 1.5e8):
            continue
        if op == "attn" and units * rows * keys > (3e7 if f32 else 1.0e9):
            continue
        if op == "sparse" and units * T * max(c["n_sel"] * c["page"] * c["d"], G * keys / c["page"]) > 4e8:
            continue
        if op == "append" and units * (T + 2 * c["page"]) * c["d"] * (2 + G) > 2.5e8:
            continue
        return c


# ------------------------------------------------------------------ inputs
def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _lengths(case):
    """Cache lengths of the units, evenly spread over [lo, hi] (the seed only orders them)."""
    U = case["B"] * case["L"] * case["H"]
    return torch.linspace(case["lo"], case["hi"], U, dtype=torch.float64).round().to(torch.int64)


def _new_tokens(case):
    """New tokens of each sequence: T, or evenly spread over [1, T] when ragged."""
    B, T = case["B"], case["T"]
    n = torch.full((B,), T, dtype=torch.int64)
    if case["ragged"]:
        n = torch.linspace(1, T, B, dtype=torch.float64).round().to(torch.int64)
    return n


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed) + 1)
    B, L, H, G, d, T, R = (case[k] for k in ("B", "L", "H", "G", "d", "T", "page"))
    U, dt = B * L * H, _dt(case)
    before = _lengths(case)[torch.randperm(U, generator=cpu)]
    n_new = _new_tokens(case)
    caps = before + T
    pages = (caps + R - 1) // R
    n_pages = int(pages.sum()) + 3
    ids = torch.randperm(n_pages, generator=cpu).to(torch.int32)
    table = torch.full((U, int(pages.max())), -1, dtype=torch.int32)
    col = torch.arange(table.shape[1])[None] < pages[:, None]
    table[col] = ids[:int(pages.sum())]                  # pages of a unit in no order
    after = before + n_new.repeat_interleave(L * H)
    s = dict(case=dict(case), U=U, rows=n_pages * R, pages=n_pages, table=table.to(dev),
             len=before.to(dev, torch.int32), after=after.to(dev, torch.int32),
             cap=caps.to(dev, torch.int32), n_new=n_new.to(dev, torch.int32))
    # a few channels of the keys are larger than the others, as in trained models
    chan = torch.exp(0.5 * torch.randn((2, d), generator=gen, device=dev))
    # entries that the cache holds: those before the chunk, and for attention the chunk's too
    held = s["len"] if case["op"] == "append" else s["after"]
    there = torch.zeros(n_pages, dtype=torch.int64, device=dev)     # entries of each page
    j = torch.arange(table.shape[1], device=dev)[None]
    cnt = (held[:, None].long() - j * R).clamp(0, R)
    there[s["table"][cnt > 0].long()] = cnt[cnt > 0]
    fill = torch.arange(R, device=dev)[None] < there[:, None]
    for i, name in enumerate(("K", "V")):
        codes = torch.full((n_pages, R, d), UNUSED, dtype=torch.uint8, device=dev)
        scale = torch.full((n_pages,), float("nan"), device=dev)
        bounds = torch.full((n_pages, 2, d), -1, dtype=torch.int8, device=dev)
        for at in range(0, n_pages, 1 << 14):            # in pieces: the values take four times the room
            p = slice(at, min(n_pages, at + (1 << 14)))
            w = torch.randn((p.stop - at, R, d), generator=gen, device=dev) * chan[i]
            x = _exponent(torch.where(fill[p, :, None], w, 0.0).abs().amax((1, 2)))
            c = _e4m3(w * _pow2(-x)[:, None, None])
            codes[p] = torch.where(fill[p, :, None], c.view(torch.uint8), codes[p])
            scale[p] = torch.where(there[p] > 0, _pow2(x), scale[p])
            b = _bounds(c, fill[p])
            bounds[p] = torch.where(there[p, None, None] > 0, b, bounds[p])
        s[name] = codes.view(n_pages * R, d)
        s["k_scale" if i == 0 else "v_scale"] = scale
        if i == 0:
            s["bounds"] = bounds
    s["logm"] = None
    if case["logm"]:                                     # merged entries carry ln m > 0
        u01 = torch.rand((2, s["rows"]), generator=gen, device=dev)
        lm = torch.where(u01[0] < 0.4, u01[1] * math.log(16.0), 0.0)
        s["logm"] = torch.where(fill.reshape(-1), lm, float("nan"))
    q = 2.0 * torch.randn((B, L, H * G, T, d), generator=gen, device=dev)
    s["q"] = q.to(dt)
    if case["op"] == "append":
        s["k_new"] = (torch.randn((B, L, H, T, d), generator=gen, device=dev) * chan[0]).to(dt)
        s["v_new"] = (torch.randn((B, L, H, T, d), generator=gen, device=dev) * chan[1]).to(dt)
        s["q_out"] = torch.zeros_like(s["q"])
        s["pos_new"] = before.view(B, -1).amax(1).to(dev, torch.float32) * 2 + 0.5
        n_half = 2 * (2 * case["hi"] + T + 2)
        e = torch.arange(n_half, device=dev, dtype=torch.float64)
        ang = 0.5 * e[:, None] * 10000.0 ** (-2.0 * torch.arange(d // 2, device=dev, dtype=torch.float64) / d)
        s["cos"], s["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
        s["len_out"] = torch.zeros(U, dtype=torch.int32, device=dev)
        return s
    s["out"] = torch.zeros((B, L, H * G, T, d), dtype=dt, device=dev)
    s["lse"] = torch.zeros((B, L, H * G, T), device=dev)
    if case["op"] == "sparse":
        s["sel"] = torch.full((B, L, H, T, case["n_sel"]), -1, dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ the 8-bit form
def _pow2(x):
    """2^x as fp32, exactly."""
    return ((x.to(torch.int32) + 127) << 23).view(torch.float32)


def _log2(scale):
    """The exponent of a power of two."""
    return ((scale.view(torch.int32) >> 23) & 255) - 127


def _exponent(a):
    """The least x with a <= 448 * 2^x, held to the scales there are."""
    f, e = torch.frexp(a)
    x = (e - 9 + (f > 0.875)).clamp(LEAST, MOST)
    return torch.where(a > 0, x, LEAST).to(torch.int32)


def _e4m3(v):
    return v.clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _bounds(c, fill):
    """int8 [.., 2, d]: least and largest rint(code / 4) of a page's entries."""
    i8 = torch.round(c.float() * 0.25)
    lo = torch.where(fill[..., None], i8, 127.0).amin(-2)
    hi = torch.where(fill[..., None], i8, -127.0).amax(-2)
    return torch.stack((lo, hi), -2).to(torch.int8)


def _unit_new(s):
    case = s["case"]
    return s["n_new"].repeat_interleave(case["L"] * case["H"])


# ------------------------------------------------------------------ plain forms
def _rotated(s, x):
    """Rows [B, L, heads, T, d] at positions pos_new[b] + t, in 32 bits."""
    h = s["case"]["d"] // 2
    e = (2 * s["pos_new"]).long()[:, None] + 2 * torch.arange(s["case"]["T"], device=x.device)
    cos, sin = s["cos"][e][:, None, None], s["sin"][e][:, None, None]
    a, b = x[..., :h].float(), x[..., h:].float()
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _append_plain(s):
    case = s["case"]
    B, T, R, d, U = case["B"], case["T"], case["page"], case["d"], s["U"]
    dev = s["len"].device
    t = torch.arange(T, device=dev)
    live = t[None] < s["n_new"][:, None]
    q = _rotated(s, s["q"]).to(s["q"].dtype)
    s["q_out"].copy_(torch.where(live[:, None, None, :, None], q, s["q_out"]))
    n, before = _unit_new(s).long(), s["len"].long()
    # the pages that a unit's tokens go into: entries e of [U, P, R]
    P = (T + R - 2) // R + 1
    page_no = (before // R)[:, None] + torch.arange(P, device=dev)
    e = page_no[..., None] * R + torch.arange(R, device=dev)
    fresh = (e >= before[:, None, None]) & (e < (before + n)[:, None, None])
    old = e < before[:, None, None]
    touched = fresh.any(-1)
    page = s["table"].gather(1, page_no.clamp(max=s["table"].shape[1] - 1)).long()
    page = torch.where(touched, page, 0)
    row = page[..., None] * R + torch.arange(R, device=dev)
    at = (e - before[:, None, None]).clamp(0, T - 1).view(U, P * R, 1).expand(-1, -1, d)
    write = touched[..., None] & (fresh | old)
    for name, new in (("K", _rotated(s, s["k_new"])), ("V", s["v_new"].float())):
        scale = s["k_scale" if name == "K" else "v_scale"]
        new = new.reshape(U, T, d).gather(1, at).view(U, P, R, d)
        was = _values(s[name])[row]
        x = _exponent(torch.where(fresh[..., None], new, 0.0).abs().amax((2, 3)))
        had = old.any(-1)
        x_old = torch.where(had, _log2(scale[page]), LEAST)
        x = torch.maximum(x, x_old)
        codes = torch.where(fresh[..., None], _e4m3(new * _pow2(-x)[..., None, None]).view(torch.uint8),
                            _e4m3(was * _pow2(x_old - x)[..., None, None]).view(torch.uint8))
        s[name][row[write]] = codes[write]
        scale[page[touched]] = _pow2(x)[touched]
        if name == "K":
            s["bounds"][page[touched]] = _bounds(_values(codes), fresh | old)[touched]
    s["len_out"].copy_(before + n)


def _select_plain(s):
    case = s["case"]
    G, T, d, R, k, U = case["G"], case["T"], case["d"], case["page"], case["n_sel"], s["U"]
    dev = s["len"].device
    q = s["q"].reshape(U, G, T, d).float()
    a = q.abs().amax(-1, keepdim=True)
    i8 = torch.round(q * torch.where(a > 0, 127.0 / a, 0.0))
    N = s["table"].shape[1]
    page = s["table"].long().clamp(min=0)
    lohi = s["bounds"][page].float()                               # [U, N, 2, d]
    pos, neg = i8.clamp(min=0).view(U, G * T, d), i8.clamp(max=0).view(U, G * T, d)
    D = torch.bmm(pos, lohi[:, :, 1].transpose(1, 2)) + torch.bmm(neg, lohi[:, :, 0].transpose(1, 2))
    score = (D.view(U, G, T, N) * s["k_scale"][page][:, None, None]) * a
    score = score.amax(1)                                          # [U, T, N]
    j = torch.arange(N, device=dev)
    last = (s["len"].long()[:, None] + torch.arange(T, device=dev)) // R      # the token's own page
    always = (j < case["first"]) | (j > (last - case["recent"])[..., None])
    score = torch.where(always, float("inf"), score)
    score = torch.where(j <= last[..., None], score, float("-inf"))
    if N < k:
        score = torch.cat((score, torch.full((U, T, k - N), float("-inf"), device=dev)), -1)
    idx = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    valid = torch.arange(k, device=dev) <= last[..., None]
    none = torch.iinfo(torch.int32).max
    idx = torch.sort(torch.where(valid, idx, none), dim=-1).values
    idx = torch.where(idx == none, -1, idx).to(torch.int32).view(s["sel"].shape)
    live = (torch.arange(T, device=dev)[None] < _unit_new(s)[:, None]).view(s["sel"].shape[:-1])
    s["sel"].copy_(torch.where(live[..., None], idx, s["sel"]))


def _softmax_av(x, v):
    """(out, base-2 lse) of base-2 scores x [.., N] and values v [.., N, d]; -inf: not seen."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp2(x.sub_(torch.where(torch.isinf(m), 0.0, m)))
    tot = p.sum(-1)
    o = torch.matmul(p, v) * torch.where(tot > 0, 1.0 / tot, 0.0)[..., None]
    return o, m[..., 0] + torch.log2(tot)


def _finish(s, o, lse):
    """Rows of tokens that there are; the others stay."""
    T, shape = s["case"]["T"], s["lse"].shape
    live = torch.arange(T, device=o.device)[None] < _unit_new(s)[:, None]           # [U, T]
    live = live[:, None].expand(-1, s["case"]["G"], -1).reshape(shape)
    s["out"].copy_(torch.where(live[..., None], o.reshape(s["out"].shape).to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(live, lse.reshape(shape), s["lse"]))


def _rows(s, e, ok):
    R = s["case"]["page"]
    flat = e.reshape(s["U"], -1)
    col = torch.where(ok.reshape(flat.shape), flat // R, 0)
    page = s["table"].gather(1, col).long()
    return torch.where(ok.reshape(flat.shape), page * R + flat % R, 0).view(e.shape)


def _dequantised(s, name, row, ok):
    scale = s["k_scale" if name == "K" else "v_scale"]
    v = _values(s[name][row]) * scale[torch.div(row, s["case"]["page"], rounding_mode="floor")][..., None]
    return torch.where(ok[..., None], v, 0.0)


def _attn_plain(s):
    case = s["case"]
    U, G, T, d = s["U"], case["G"], case["T"], case["d"]
    dev = s["len"].device
    N = int(case["hi"]) + T
    e = torch.arange(N, device=dev)[None].expand(U, -1)
    ok = e < s["after"][:, None]
    row = _rows(s, e, ok)
    q = s["q"].view(U, G * T, d).float() / math.sqrt(d)
    x = torch.bmm(q, _dequantised(s, "K", row, ok).transpose(1, 2)).view(U, G, T, N)
    if s["logm"] is not None:
        x += torch.where(ok, s["logm"][row], 0.0)[:, None, None]
    see = ok[:, None] & (e[:, None] <= s["len"][:, None, None] + torch.arange(T, device=dev)[:, None])
    x = x.masked_fill_(~see[:, None], float("-inf")).mul_(LOG2E)
    o, lse = _softmax_av(x.view(U, G * T, N), _dequantised(s, "V", row, ok))
    _finish(s, o, lse)


def _sparse_plain(s):
    _select_plain(s)
    case = s["case"]
    U, G, T, d, R, k = s["U"], case["G"], case["T"], case["d"], case["page"], case["n_sel"]
    dev = s["len"].device
    sel = s["sel"].view(U, T, k).long()
    e = (sel[..., None] * R + torch.arange(R, device=dev)).view(U, T, k * R)
    own_e = s["len"].long()[:, None] + torch.arange(T, device=dev)
    ok = (sel >= 0)[..., None].expand(-1, -1, -1, R).reshape(e.shape) & (e <= own_e[..., None]) \
        & (e < s["after"].long()[:, None, None])
    row = _rows(s, e, ok)                                          # [U, T, kR]
    q = s["q"].view(U, G, T, d).transpose(1, 2).float() / math.sqrt(d)
    x = torch.matmul(q, _dequantised(s, "K", row, ok).transpose(2, 3))               # [U, T, G, kR]
    if s["logm"] is not None:
        x += torch.where(ok, s["logm"][row], 0.0)[:, :, None]
    x = x.masked_fill_(~ok[:, :, None], float("-inf")).mul_(LOG2E)
    o, lse = _softmax_av(x, _dequantised(s, "V", row, ok))
    _finish(s, o.transpose(1, 2), lse.transpose(1, 2))


# ------------------------------------------------------------------ the framework's calls
def _plan(s):
    from kv_cache_compression_probe_gb300 import kvc
    c = s["case"]
    p = kvc.make_params(B=c["B"], L=c["L"], H=c["H"], G=c["G"], d=c["d"], P=1, W=1,
                        dtype=kvc.KVC_F32 if c["dtype"] == "f32" else kvc.KVC_BF16, n_max=17,
                        S_max=1, packed_rows=s["rows"])
    ch = kvc.make_chunk(T=c["T"], layer_begin=0, layer_end=c["L"], page_rows=c["page"],
                        page_table=s["table"], n_new=s["n_new"])
    x = kvc.make_q8(s["K"], s["V"], s["k_scale"], s["v_scale"], s["bounds"], s["logm"])
    ws = None
    if c["op"] != "append":
        ws = torch.empty(kvc.kvc_q8_workspace_bytes(p, ch, c["n_sel"]), dtype=torch.uint8, device="cuda")
    return kvc, p, ch, x, ws


def _run_own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    kvc, p, ch, x, ws = s["plan"]
    c = s["case"]
    if c["op"] == "append":
        kvc.kvc_q8_append(p, ch, x, s["cos"], s["sin"], s["q"], s["k_new"], s["v_new"], s["pos_new"],
                          s["q_out"], s["len"], s["cap"], s["len_out"])
        return
    if c["op"] == "sparse":
        kvc.kvc_q8_select(p, ch, x, s["q"], s["len"], s["after"], c["first"], c["recent"], s["sel"])
    kvc.kvc_q8_attn(p, ch, x, s["q"], s["len"], s["after"], s.get("sel"), s["out"], s["lse"], ws)


def run(s):
    op = s["case"]["op"]
    if own:
        _run_own(s)
    else:
        {"append": _append_plain, "attn": _attn_plain, "sparse": _sparse_plain}[op](s)
    if op == "append":                                             # e4m3 codes, in units of the scales
        e4m3 = torch.float8_e4m3fn
        return {"q": s["q_out"], "K": s["K"].view(e4m3), "V": s["V"].view(e4m3), "k_scale": s["k_scale"],
                "v_scale": s["v_scale"], "bounds": s["bounds"], "len": s["len_out"]}
    got = {"out": s["out"], "lse": s["lse"]}
    return dict(got, sel=s["sel"]) if op == "sparse" else got


# ------------------------------------------------------------------ work, exact values
def work(case):
    U, G, d, R = case["B"] * case["L"] * case["H"], case["G"], case["d"], case["page"]
    x = 4 if case["dtype"] == "f32" else 2
    n = [int(v) for v in _new_tokens(case)]
    per, lens = U // case["B"], [int(v) for v in _lengths(case)]
    tokens = sum(n) * per                                          # of all units
    rows = G * tokens
    mean = tokens / U
    if case["op"] == "append":
        pages = sum((v + max(1, round(mean)) - 1) // R - v // R + 1 for v in lens)
        return {"bytes": 2 * rows * d * x + 2 * tokens * d * (x + 1) + sum(n) * d * 4 + pages * (4 * d + 16),
                "flops": 3 * d * (rows + tokens)}
    lm = 4 if case["logm"] else 0
    if case["op"] == "attn":
        keys = sum(lens) + tokens
        pairs = G * mean * (sum(lens) + U * (mean + 1) / 2)
        return {"bytes": keys * (2 * d + lm) + keys / R * 8 + rows * (2 * d * x + 4), "flops": 4 * d * pairs}
    pages = sum((v + mean) / R for v in lens)
    seen = sum(min(case["n_sel"], v // R + 1) for v in lens)       # pages that one token attends over
    read = min(pages, seen * mean)
    return {"bytes": pages * (2 * d + 4) + read * (R * (2 * d + lm) + 4) + rows * (2 * d * x + 4) + tokens * 4 * case["n_sel"],
            "flops": 4 * d * G * mean * seen * R + 4 * d * G * mean * pages}


def exact(case, seed):
    """The definition in 64 bits, one unit (and, where pages are picked, one token) at a time."""
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "sparse": _exact_attn}[case["op"]](s)


def _f64(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float64)


def _exact_append(s):
    """The codes before rounding: the values in units of their page's scale."""
    case = s["case"]
    B, L, H, T, R, d = (case[k] for k in ("B", "L", "H", "T", "page", "d"))
    f64, h = torch.float64, d // 2
    if s["U"] * (T // R + 2) > 20000:
        return None
    got = {n: _f64(s[n]) for n in ("K", "V")}
    scales = {n: s[n].to(f64) for n in ("k_scale", "v_scale")}
    q = s["q_out"].to(f64)
    lens, table, news = s["len"].tolist(), s["table"].tolist(), s["n_new"].tolist()
    for b in range(B):
        n = news[b]
        e = (2 * float(s["pos_new"][b]) + 2 * torch.arange(n, device="cuda")).long()
        c, w = s["cos"][e].to(f64), s["sin"][e].to(f64)

        def turn(v):
            v = v.to(f64)
            return torch.cat([v[..., :h] * c - v[..., h:] * w, v[..., :h] * w + v[..., h:] * c], -1)
        q[b, :, :, :n] = turn(s["q"][b, :, :, :n])
        new_k, new_v = turn(s["k_new"][b, :, :, :n]), s["v_new"][b, :, :, :n].to(f64)
        for lh in range(L * H):
            u = b * L * H + lh
            n0 = lens[u]
            for pg in range(n0 // R, (n0 + n - 1) // R + 1 if n else n0 // R):
                page = table[u][pg]
                t0, t1 = max(0, pg * R - n0), min(n, (pg + 1) * R - n0)
                had = max(0, min(R, n0 - pg * R))
                r0 = page * R
                for name, sc, rows in (("K", "k_scale", new_k), ("V", "v_scale", new_v)):
                    vals = rows[lh // H, lh % H, t0:t1]
                    top = float(vals.abs().max())
                    e2 = max(-40, min(40, math.ceil(math.log2(top / 448.0)))) if top > 0 else -40
                    unit = 2.0 ** e2
                    if had:
                        unit = max(unit, float(scales[sc][page]))
                        got[name][r0:r0 + had] *= float(scales[sc][page]) / unit
                    got[name][r0 + had:r0 + had + t1 - t0] = vals / unit
                    scales[sc][page] = unit
    return {"q": q, "K": got["K"], "V": got["V"], "k_scale": scales["k_scale"],
            "v_scale": scales["v_scale"], "bounds": None, "len": None}


def _pages_of(s, u, t, n0):
    """Page numbers that token t of unit u picks (integers, and the score's two roundings to fp32)."""
    case = s["case"]
    G, T, d, R, k = (case[i] for i in ("G", "T", "d", "page", "n_sel"))
    own_page = (n0 + t) // R
    if own_page < k:
        return list(range(own_page + 1))
    j = torch.arange(own_page + 1, device="cuda")
    page = s["table"][u, :own_page + 1].long()
    q = s["q"].view(-1, G, T, d)[u, :, t].float()
    top = q.abs().max(1).values
    ints = torch.round(q * (127.0 / top)[:, None]).nan_to_num(0.0).to(torch.float64)
    both = s["bounds"][page].to(torch.float64)                     # [N, 2, d]
    D = torch.maximum(ints[:, None] * both[None, :, 0], ints[:, None] * both[None, :, 1]).sum(-1)
    best = ((D.to(torch.float32) * s["k_scale"][page]) * top[:, None]).max(0).values.tolist()
    keep = set(range(case["first"])) | set(range(own_page - case["recent"] + 1, own_page + 1))
    rest = sorted((i for i in j.tolist() if i not in keep), key=lambda i: (-best[i], i))
    return sorted(list(keep) + rest[:k - len(keep)])


def _exact_attn(s):
    case = s["case"]
    f64 = torch.float64
    G, T, d, R = (case[k] for k in ("G", "T", "d", "page"))
    U, sparse = s["U"], case["op"] == "sparse"
    lens, ends = s["len"].tolist(), s["after"].tolist()
    if sparse and U * T > 3000:
        return None
    out, lse = s["out"].to(f64).view(U, G, T, d), s["lse"].to(f64).view(U, G, T)
    for u in range(U):
        n0, N = lens[u], ends[u]
        i = torch.arange(N, device="cuda")
        page = s["table"][u].long()[torch.div(i, R, rounding_mode="floor")]
        row = page * R + i % R
        K = _f64(s["K"][row]) * s["k_scale"][page].to(f64)[:, None]
        V = _f64(s["V"][row]) * s["v_scale"][page].to(f64)[:, None]
        lm = 0.0 if s["logm"] is None else s["logm"][row].to(f64)
        tok = torch.arange(N - n0, device="cuda")
        see = i[None] <= n0 + tok[:, None]
        if sparse:
            for t in range(N - n0):
                picked = torch.zeros(-(-N // R), dtype=torch.bool, device="cuda")
                got = _pages_of(s, u, t, n0)
                picked[torch.tensor(got, device="cuda")] = True
                s["sel"].view(U, T, -1)[u, t, :len(got)] = torch.tensor(got, dtype=torch.int32)
                see[t] &= picked[torch.div(i, R, rounding_mode="floor")]
        for g in range(G):
            z = (s["q"].view(U, G, T, d)[u, g, :N - n0].to(f64) @ K.T) * d ** -0.5 + lm
            z = torch.where(see, z, -math.inf)
            tot = torch.logsumexp(z, 1)
            lse[u, g, :N - n0] = tot / math.log(2.0)
            out[u, g, :N - n0] = torch.exp(z - torch.where(torch.isinf(tot), 0.0, tot)[:, None]) @ V
    got = {"out": out.view(s["out"].shape), "lse": lse.view(s["lse"].shape)}
    return dict(got, sel=s["sel"]) if sparse else got
