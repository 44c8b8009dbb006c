"""Cases and plain forms of the chunk operators over the packed KV cache.

  attn    kvc_chunk_attn: n new tokens per sequence are appended to every
          (b, l, h)'s cache (contiguous rows or pages) and attend over it
  mass    kvc_chunk_mass: the attention weight every entry received from the
          chunk, added to its decayed mass
  evict   kvc_mass_evict: per-(b, l, h) eviction to a target length by mass

Units are the (b, l, h) in order; U = B*L*H, R = G*T query rows per unit.
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634


def _case(name, op, B=1, L=1, H=8, G=4, d=128, T=1, lo=256, hi=512, stretch=1, page=0,
          dtype="bf16", softcap=0.0, window=0.0, slopes=False, ragged=False, decay=1.0,
          keep=0.75, recent=32):
    c = dict(op=op, B=B, L=L, H=H, G=G, d=d, T=T, lo=lo, hi=hi, stretch=stretch, page=page,
             dtype=dtype, softcap=softcap, window=window, slopes=slopes, ragged=ragged,
             decay=decay, keep=keep, recent=recent)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one layer over a short compressed cache: pure latency
        _case("attn one token, one layer", "attn", lo=200, hi=512, stretch=4),
        # one decode step of all layers over a 16K context compressed to 25%
        _case("attn one token, all layers", "attn", L=32, lo=3200, hi=5000, stretch=4),
        # up to 5 drafted tokens verified for 16 sequences over pages, capped scores
        _case("attn drafts, paged, capped", "attn", B=16, T=5, lo=1000, hi=4096, page=64,
              softcap=30.0, ragged=True),
        # a 300-token follow-up turn over the compressed cache, distance bias
        _case("attn follow-up turn, slopes", "attn", B=2, L=4, T=300, lo=3000, hi=5200,
              stretch=4, slopes=True, ragged=True),
        # a 512-token chunk with a 4096-token sliding window over an uncompressed paged cache
        _case("attn chunk, sliding window", "attn", T=512, lo=11000, hi=12000, page=128,
              window=4096.0),
        # the last 2048-token chunk of a 16K prompt, one layer
        _case("attn 2048-token chunk of 16K", "attn", T=2048, lo=14336, hi=14336, page=128),
        # the repository's small fp32 configuration (2 KV / 8 query heads, d 64, context 512)
        _case("attn small fp32", "attn", H=2, d=64, T=33, lo=128, hi=512, stretch=4, dtype="f32"),
        # mass after a decode step of all layers
        _case("mass one token, all layers", "mass", L=32, lo=3200, hi=5000, stretch=4, decay=0.98),
        # mass after a 1024-token chunk of a prompt, one layer, paged
        _case("mass 1024-token chunk", "mass", T=1024, lo=7168, hi=7168, page=64),
        # one layer's cache of a short context back to its budget: latency
        _case("evict one layer, short", "evict", lo=500, hi=600, stretch=4, keep=0.9),
        # all layers of a 16K context at 25%, a little over budget
        _case("evict all layers, few rows", "evict", L=32, lo=3300, hi=5100, stretch=4, keep=0.98),
        # four layers after a prompt chunk, paged, a third of the rows leave
        _case("evict after a chunk, paged", "evict", B=2, L=4, lo=5000, hi=8192, page=64,
              keep=0.66, recent=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("attn", "attn", "mass", "evict"))
        f32 = op != "evict" and rng.random() < 0.12
        B, L = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
        H, G = rng.choice((1, 2, 3, 8, 8, 8)), rng.choice((1, 2, 4, 4, 8))
        T = 1 if rng.random() < 0.25 else _log_int(rng, 1, 2048)
        hi = _log_int(rng, 33, 16384)
        lo = int(hi * rng.uniform(0.0, 1.0))
        bias = rng.choice(("none", "none", "cap", "slopes", "window", "all"))
        c = _case(None, op, B=B, L=L, H=H, G=G, d=rng.choice((64, 128, 128)),
                  T=1 if op == "evict" else T, lo=lo, hi=hi, stretch=rng.choice((1, 4)),
                  page=rng.choice((0, 0, 16, 64, 128)), dtype="f32" if f32 else "bf16",
                  softcap=30.0 if bias in ("cap", "all") else 0.0,
                  window=float(_log_int(rng, 8, 8192)) if bias in ("window", "all") else 0.0,
                  slopes=bias in ("slopes", "all"), ragged=B > 1 and rng.random() < 0.5,
                  decay=rng.choice((1.0, 0.98)), keep=round(rng.uniform(0.1, 1.0), 3),
                  recent=rng.choice((0, 32, 256)))
        units, rows, keys = B * L * H, G * c["T"], hi + c["T"]
        if units * rows * keys > (3e7 if f32 else 1.0e9):
            continue
        if not 2e5 < units * keys * c["d"] < 1.5e8:
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
    B, L, H, G, d, T = (case[k] for k in ("B", "L", "H", "G", "d", "T"))
    U, dt, page = B * L * H, _dt(case), case["page"]
    lens = _lengths(case)[torch.randperm(U, generator=cpu)]
    n_new = _new_tokens(case)
    caps = lens + T
    if page:
        pages = (caps + page - 1) // page
        n_pages = int(pages.sum()) + 3
        ids = torch.randperm(n_pages, generator=cpu).to(torch.int32)
        table = torch.full((U, int(pages.max())), -1, dtype=torch.int32)
        col = torch.arange(table.shape[1])[None] < pages[:, None]
        table[col] = ids[:int(pages.sum())]              # pages of a unit in no order
        rows = n_pages * page
        off = torch.zeros(U, dtype=torch.int64)
    else:
        table = None
        off = torch.cumsum(caps, 0) - caps
        rows = int(caps.sum())
    s = dict(case=dict(case), U=U, rows=rows, N=int(lens.max()) + T,
             len=lens.to(dev, torch.int32), cap=caps.to(dev, torch.int32), off=off.to(dev),
             table=None if table is None else table.to(dev),
             n_new=n_new.to(dev, torch.int32),
             # positions: entry e of a unit stands for tokens around e * stretch
             pos_new=torch.full((B,), 0.0, device=dev))
    ctx = (lens.view(B, -1).amax(1) * case["stretch"]).to(dev, torch.float32)
    s["pos_new"] = ctx.contiguous()
    e, row, valid, old = _entries(s)
    nan = float("nan")
    K = torch.randn((rows, d), generator=gen, device=dev, dtype=torch.float32).to(dt)
    V = torch.randn((rows, d), generator=gen, device=dev, dtype=torch.float32).to(dt)
    meta = torch.full((3, rows), nan, device=dev)        # ln m, position, mass
    taken = torch.zeros(rows, dtype=torch.bool, device=dev)
    taken[row[old]] = True
    K[~taken], V[~taken] = nan, nan                      # rows that hold nothing yet
    r = row[old]
    u01 = torch.rand((2, r.numel()), generator=gen, device=dev)
    if case["stretch"] > 1:                              # merged entries carry ln m > 0
        meta[0, r] = torch.where(u01[0] < 0.4, u01[1] * math.log(16.0), 0.0)
    else:
        meta[0, r] = 0.0
    ub = torch.arange(U, device=dev) // (L * H)
    first = s["pos_new"][ub][:, None] - s["len"][:, None] * float(case["stretch"])
    frac = torch.floor(torch.rand(e.shape, generator=gen, device=dev) * 2 * (case["stretch"] - 1)) / 2
    meta[1, r] = (first + e * float(case["stretch"]) + frac)[old]
    w = torch.rand(r.numel(), generator=gen, device=dev)
    meta[2, r] = 0.05 / (0.01 + w)                       # few heavy hitters, a long tail
    s.update(K=K, V=V, meta=meta, logm=meta[0], pos=meta[1], mass=meta[2])
    if case["op"] == "evict":
        s["meta0"] = meta.clone()
        s["keep"] = (lens.to(torch.float64) * case["keep"]).floor().to(dev, torch.int32)
        s["len_out"] = torch.zeros(U, dtype=torch.int32, device=dev)
        return s
    q = 2.0 * torch.randn((B, L, H * G, T, d), generator=gen, device=dev, dtype=torch.float32)
    s["q"] = q.to(dt)
    s["k_new"] = torch.randn((B, L, H, T, d), generator=gen, device=dev, dtype=torch.float32).to(dt)
    s["v_new"] = torch.randn((B, L, H, T, d), generator=gen, device=dev, dtype=torch.float32).to(dt)
    s["slopes"] = None
    if case["slopes"]:
        i = torch.arange(1, H * G + 1, device=dev, dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * i / (H * G))
    s["out"] = torch.zeros((B, L, H * G, T, d), dtype=dt, device=dev)
    s["lse"] = torch.zeros((B, L, H * G, T), device=dev)
    s["len_out"] = torch.zeros(U, dtype=torch.int32, device=dev)
    if case["op"] == "mass":                             # the chunk has attended already
        _append(s)
        _, lse, live = _softmax(s, _scores(s))
        s["lse"].copy_(torch.where(live.reshape(s["lse"].shape), lse.view(s["lse"].shape), s["lse"]))
    return s


def _entries(s):
    """Entry indices [U, N], their rows, and which are entries after / before the append."""
    page, dev = s["case"]["page"], s["len"].device
    e = torch.arange(s["N"], device=dev)[None].expand(s["U"], -1)
    per_b = s["U"] // s["case"]["B"]
    old = e < s["len"][:, None]
    valid = e < (s["len"] + s["n_new"].repeat_interleave(per_b))[:, None]
    if page:
        col = torch.clamp(e // page, max=s["table"].shape[1] - 1)
        row = s["table"].gather(1, col).long() * page + e % page
    else:
        row = s["off"][:, None] + e
    return e, torch.where(valid, row, 0), valid, old


def _append(s):
    """The chunk's keys and values become entries len .. len + n - 1."""
    _, row, valid, old = _entries(s)
    case = s["case"]
    T, d = case["T"], case["d"]
    t = torch.arange(T, device=row.device)
    at = torch.clamp(s["len"][:, None].long() + t, max=s["N"] - 1)
    live = (t[None] < s["n_new"][:, None]).repeat_interleave(s["U"] // case["B"], 0)
    r = row.gather(1, at)[live]
    s["K"][r] = s["k_new"].view(s["U"], T, d)[live]
    s["V"][r] = s["v_new"].view(s["U"], T, d)[live]
    s["logm"][r] = 0.0
    p = s["pos_new"][:, None] + t
    s["pos"][r] = p.repeat_interleave(s["U"] // case["B"], 0)[live]


# ------------------------------------------------------------------ plain forms
def _scores(s):
    """Base-2 scores [U, G, T, N] in 32 bits, -inf where a row may not look."""
    case = s["case"]
    G, T, d, H, U = case["G"], case["T"], case["d"], case["H"], s["U"]
    e, row, valid, _ = _entries(s)
    k = torch.where(valid[..., None], s["K"][row].float(), 0.0)
    q = s["q"].view(U, G * T, d).float() / math.sqrt(d)
    x = torch.bmm(q, k.transpose(1, 2)).view(U, G, T, -1)
    if case["softcap"] > 0:
        x = torch.tanh_(x.div_(case["softcap"])).mul_(case["softcap"])
    x += torch.where(valid, s["logm"][row], 0.0)[:, None, None]
    t = torch.arange(T, device=e.device)
    see = valid[:, None] & (e[:, None] <= s["len"][:, None, None] + t[:, None])      # [U, T, N]
    if case["slopes"] or case["window"] > 0:
        b = torch.arange(U, device=e.device) // (U // case["B"])
        dist = (s["pos_new"][b][:, None] + t)[..., None] - torch.where(valid, s["pos"][row], 0.0)[:, None]
        if case["slopes"]:
            h = torch.arange(U, device=e.device) % H
            slope = s["slopes"].view(H, G)[h]
            x -= slope[..., None, None] * dist[:, None]
        if case["window"] > 0:
            see &= dist < case["window"]
    return x.masked_fill_(~see[:, None], float("-inf")).mul_(LOG2E)


def _softmax(s, x):
    """Numerators over the row maximum, the base-2 LSE and which rows are tokens of the chunk."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp2(x.sub_(torch.where(torch.isinf(m), 0.0, m)))
    lse = (m + torch.log2(p.sum(-1, keepdim=True)))[..., 0]
    t = torch.arange(s["case"]["T"], device=x.device)
    live = (t[None] < s["n_new"][:, None]).repeat_interleave(s["U"] // s["case"]["B"], 0)
    return p, lse, live[:, None].expand(lse.shape)


def _attn_plain(s):
    case = s["case"]
    _append(s)
    p, lse, live = _softmax(s, _scores(s))
    _, row, valid, _ = _entries(s)
    v = torch.where(valid[..., None], s["V"][row].float(), 0.0)
    l = p.sum(-1)
    o = torch.bmm(p.view(s["U"], -1, p.shape[-1]), v).view(*l.shape, -1)
    o = torch.where(l > 0, 1.0 / l, 0.0)[..., None] * o
    shape, keep = s["out"].shape, live.reshape(s["lse"].shape)
    s["out"].copy_(torch.where(keep[..., None], o.view(shape).to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(keep, lse.view(s["lse"].shape), s["lse"]))
    s["len_out"].copy_(s["len"] + s["n_new"].repeat_interleave(s["U"] // case["B"]))


def _mass_plain(s):
    x = _scores(s)
    lse = s["lse"].view(x.shape[:3])
    t = torch.arange(s["case"]["T"], device=x.device)
    live = (t[None] < s["n_new"][:, None]).repeat_interleave(s["U"] // s["case"]["B"], 0)
    x.sub_(torch.where(torch.isinf(lse), 0.0, lse)[..., None]).masked_fill_(~live[:, None, :, None], float("-inf"))
    got = torch.exp2(x).sum((1, 2))
    _, row, valid, old = _entries(s)
    new = torch.where(old, s["mass"][row], 0.0) * s["case"]["decay"] + got
    s["mass"][row[valid]] = new[valid]


def _evict_plain(s):
    s["meta"].copy_(s["meta0"])              # the pass starts from the same masses every time
    e, row, _, old = _entries(s)
    case = s["case"]
    b = torch.arange(s["U"], device=e.device) // (s["U"] // case["B"])
    safe = old & (s["pos"][row] >= (s["pos_new"][b] - float(case["recent"]))[:, None])
    key = torch.where(safe, float("inf"), torch.where(old, s["mass"][row], float("-inf")))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, e.contiguous())
    B = torch.minimum(torch.maximum(s["keep"].long(), safe.sum(1)), s["len"].long())[:, None]
    kept = old & (rank < B)
    to, frm = row[old & ~kept & (e < B)], row[kept & (e >= B)]
    s["K"][to], s["V"][to] = s["K"][frm], s["V"][frm]
    s["meta"][:, to] = s["meta"][:, frm]
    s["len_out"].copy_(B[:, 0])


# ------------------------------------------------------------------ the framework's calls
def _plan(s):
    from kv_cache_compression_probe_gb300 import kvc
    c = s["case"]
    p = kvc.make_params(B=c["B"], L=c["L"], H=c["H"], G=c["G"], d=c["d"], P=1, W=1,
                        dtype=kvc.KVC_F32 if c["dtype"] == "f32" else kvc.KVC_BF16,
                        n_max=max(s["N"], 17), S_max=1, packed_rows=s["rows"])
    ch = kvc.make_chunk(T=c["T"], layer_begin=0, layer_end=c["L"], page_rows=c["page"],
                        page_table=s["table"], n_new=s["n_new"], softcap=c["softcap"],
                        window=c["window"], slopes=s.get("slopes"))
    if c["op"] == "evict":
        ws = kvc.kvc_mass_evict_workspace_bytes(p, ch, s["N"])
    else:
        ws = kvc.kvc_chunk_workspace_bytes(p, ch)
    return kvc, p, ch, torch.empty(ws, dtype=torch.uint8, device="cuda")


def _run_own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    kvc, p, ch, ws = s["plan"]
    c = s["case"]
    if c["op"] == "attn":
        kvc.kvc_chunk_attn(p, ch, s["q"], s["k_new"], s["v_new"], s["pos_new"], s["K"], s["V"],
                           s["logm"], s["pos"], s["len"], s["cap"], s["off"], s["out"], s["lse"],
                           s["len_out"], ws)
    elif c["op"] == "mass":
        kvc.kvc_chunk_mass(p, ch, s["q"], s["K"], s["logm"], s["pos"], s["pos_new"], s["len"],
                           s["off"], s["lse"], c["decay"], s["mass"], ws)
    else:
        s["meta"].copy_(s["meta0"])
        kvc.kvc_mass_evict(p, ch, s["mass"], s["keep"], c["recent"], s["pos_new"], s["K"], s["V"],
                           s["logm"], s["pos"], s["len"], s["off"], s["len_out"], s["N"], ws)


def run(s):
    if own:
        _run_own(s)
    else:
        {"attn": _attn_plain, "mass": _mass_plain, "evict": _evict_plain}[s["case"]["op"]](s)
    if s["case"]["op"] == "mass":
        return {"mass": s["mass"]}
    got = {"K": s["K"], "V": s["V"], "logm": s["logm"], "pos": s["pos"], "len": s["len_out"]}
    if s["case"]["op"] == "evict":
        return dict(got, mass=s["mass"])
    return dict(got, out=s["out"], lse=s["lse"])


# ------------------------------------------------------------------ work, exact values
def work(case):
    U, G, d = case["B"] * case["L"] * case["H"], case["G"], case["d"]
    x = 4 if case["dtype"] == "f32" else 2
    lens = [int(v) for v in _lengths(case)]
    n = [int(v) for v in _new_tokens(case)]
    per = U // case["B"]
    mean_n = sum(n) * per / U
    total = sum(lens)
    if case["op"] == "evict":
        gone = sum(v - int(v * case["keep"]) for v in lens)
        moved = gone * case["keep"]          # evicted rows below the cut, for masses in no order
        return {"bytes": total * 8 + 2 * moved * (2 * d * x + 12), "flops": 0}
    look = total                             # cache entries that some row may see
    if case["window"] > 0:
        look = sum(min(v, case["window"] / case["stretch"] + mean_n) for v in lens)
    seen = total                             # of these, what one row sees
    if case["window"] > 0:
        seen = sum(min(v, case["window"] / case["stretch"]) for v in lens)
    wide = 4 if case["slopes"] or case["window"] > 0 else 0
    keys = look + mean_n * U
    rows = G * mean_n
    own_keys = (mean_n + 1) / 2 if case["window"] <= 0 else min((mean_n + 1) / 2, case["window"])
    pairs = rows * (seen + own_keys * U)
    if case["op"] == "mass":
        return {"bytes": keys * (d * x + 8 + wide + 4) + U * rows * (d * x + 4),
                "flops": 2 * d * pairs}
    return {"bytes": keys * (2 * d * x + 4 + wide) + U * rows * (2 * d * x + 4)
            + U * mean_n * (2 * d * x + 8), "flops": 4 * d * pairs}


def exact(case, seed):
    """The definition in 64 bits, one (b, l, h) at a time.  The rows that the append or the
    eviction copies have no computed value: their place holds None (evict: all of them)."""
    if case["op"] == "evict":
        return None
    s = prepare(case, seed)
    if case["op"] == "attn":
        _append(s)
    f64 = torch.float64
    G, T, d, H, B = (case[k] for k in ("G", "T", "d", "H", "B"))
    U = s["U"]
    out = s["out"].double().view(U, G, T, d)
    lse = s["lse"].double().view(U, G, T)
    mass = s["mass"].double()
    lens, news, offs = s["len"].tolist(), s["n_new"].tolist(), s["off"].tolist()
    for u in range(U):
        b, h = u // (U // B), u % H
        n0, n = lens[u], news[b]
        N = n0 + n
        i = torch.arange(N, device="cuda")
        if case["page"]:
            rows = s["table"][u].long()[torch.div(i, case["page"], rounding_mode="floor")] * case["page"] + i % case["page"]
        else:
            rows = offs[u] + i
        K, V = s["K"][rows].to(f64), s["V"][rows].to(f64)
        lm, pos = s["logm"][rows].to(f64), s["pos"][rows].to(f64)
        got = torch.zeros(N, dtype=f64, device="cuda")
        tq = torch.arange(n, device="cuda")
        pq = s["pos_new"][b].to(f64) + tq
        for g in range(G):
            z = (s["q"].view(U, G, T, d)[u, g, :n].to(f64) @ K.T) * d ** -0.5
            if case["softcap"] > 0:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            z = z + lm
            gap = pq[:, None] - pos[None]
            if case["slopes"]:
                z = z - s["slopes"][h * G + g].to(f64) * gap
            hide = i[None] > n0 + tq[:, None]
            if case["window"] > 0:
                hide = hide | (gap >= case["window"])
            z[hide] = -math.inf
            if case["op"] == "mass":
                ref = s["lse"].view(U, G, T)[u, g, :n].to(f64) * math.log(2.0)
                ref = torch.where(torch.isinf(ref), 0.0, ref)
                got += torch.exp(z - ref[:, None]).sum(0)
            else:
                tot = torch.logsumexp(z, 1)
                lse[u, g, :n] = tot / math.log(2.0)
                out[u, g, :n] = torch.exp(z - torch.where(torch.isinf(tot), 0.0, tot)[:, None]) @ V
        if case["op"] == "mass":
            was = torch.where(i < n0, mass[rows], 0.0)
            mass[rows] = case["decay"] * was + got
    if case["op"] == "mass":
        return {"mass": mass}
    return {"K": None, "V": None, "logm": None, "pos": None, "len": None,
            "out": out.view(s["out"].shape), "lse": lse.view(s["lse"].shape)}
