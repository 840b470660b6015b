"""Cases that time and check the paged-cache operators: append with rotation,
decode attention over pages, decode with a shared prefix, and decode over the
pages that a cheap score selects.

Each case is a dict of plain values.  `prepare` makes what a serving program
has in hand (page pool, tables, lengths, new rows, queries), `run` makes one
pass: the plain torch form, or with `own` the calls of the library.  The page
layout that both read is the one `include/kvq.h` describes.
"""

import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def _append(name, fmt="q8_0/q5_1", dtype="bf16", page=64, Hq=32, Hkv=8, D=128, n=1, t=(1, 1), ctx=(0, 0),
            rope=128, inter=False):
    return dict(name=name, op="append", fmt=fmt, dtype=dtype, page=page, Hq=Hq, Hkv=Hkv, D=D, n=n, t_lo=t[0], t_hi=t[1],
                ctx_lo=ctx[0], ctx_hi=ctx[1], rope=rope, inter=inter)


def _decode(name, fmt="q8_0/q5_1", dtype="bf16", page=64, Hq=32, Hkv=8, D=128, n=1, T=1, length=(512, 512), window=0,
            sinks=False, softcap=0.0):
    return dict(name=name, op="decode", fmt=fmt, dtype=dtype, page=page, Hq=Hq, Hkv=Hkv, D=D, n=n, T=T, len_lo=length[0],
                len_hi=length[1], window=window, sinks=sinks, softcap=softcap)


def _shared(name, groups=1, prefix=8192, suffix=(1, 1024), **kw):
    c = _decode(name, length=suffix, **kw)
    c.update(op="shared", groups=groups, prefix=prefix)
    return c


def _sparse(name, keep=64, **kw):
    c = _decode(name, **kw)
    c.update(op="sparse", keep=keep)
    return c


def listed():
    return [
        # one decode step of a batch: a row for each sequence, keys and queries rotated (latency)
        _append("append step, 64 sequences", n=64, ctx=(1023, 16383)),
        # prompts of different lengths in one packed batch
        _append("append prompts, 8k rows", n=6, t=(200, 2600)),
        # three draft rows of a few sequences, small pages, half of each head rotated in interleaved pairs
        _append("append drafts e4m3 f32", fmt="e4m3", dtype="f32", page=16, Hq=16, Hkv=4, D=256, n=5, t=(3, 3), ctx=(0, 700),
                rope=128, inter=True),
        # the smallest decode: one short sequence (latency)
        _decode("decode 512", Hq=8, Hkv=2),
        # one long sequence
        _decode("decode 32k", length=(32768, 32768)),
        # a serving batch of different lengths
        _decode("decode batch 64", n=64, length=(1024, 16384)),
        # verifying eight draft rows, f32 queries and outputs
        _decode("decode verify f32", dtype="f32", Hq=16, Hkv=4, D=256, T=8, length=(16384, 16384)),
        # a sliding window with sinks over E4M3 rows
        _decode("decode window e4m3", fmt="e4m3", Hq=64, Hkv=8, D=64, page=32, n=7, length=(1000, 65536), window=4096,
                sinks=True),
        # a system prompt that a whole batch shares
        _shared("shared batch 64", n=64, prefix=8192, suffix=(1, 1024)),
        # three groups of odd sizes, a prefix that ends inside a page
        _shared("shared 3 groups e4m3", fmt="e4m3", Hq=64, Hkv=8, D=64, page=16, n=25, groups=3, prefix=2007,
                suffix=(3, 300), sinks=True),
        # one step at a very long context: append a row, select pages, attend to them
        _sparse("sparse 128k", Hq=64, Hkv=8, D=64, page=32, length=(131072, 131072), keep=128),
        # the same for a batch
        _sparse("sparse batch 16", n=16, page=32, length=(2048, 32768), keep=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "shared", "sparse"])
    Hkv = rng.choice([1, 2, 4, 8])
    kw = dict(fmt=rng.choice(["q8_0/q5_1", "q8_0/q5_1", "e4m3"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
              page=rng.choice([16, 32, 64, 128]), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), D=rng.choice([64, 128, 256]))
    if op == "append":
        n = _log(rng, 1, 128)
        row = (2 * kw["Hq"] + 2 * kw["Hkv"]) * kw["D"] * (4 if kw["dtype"] == "f32" else 2)
        hi = _log(rng, 1, max(1, min(8192, 250_000_000 // row) // n))
        lo = hi if rng.random() < 0.5 else rng.randint(0, hi)
        ctx = _log(rng, 1, 16384)
        c = _append("", n=n, t=(lo, hi), ctx=(rng.randint(0, ctx), ctx),
                    rope=rng.choice([0, kw["D"], kw["D"], kw["D"] // 2, 32]), inter=rng.random() < 0.4, **kw)
    else:
        n = _log(rng, 1, 96)
        T = rng.choice([1, 1, 1, 2, 3, 5, 8])
        row = kw["Hkv"] * kw["D"]
        most = max(64, min(65536, 300_000_000 // (n * row * (2 if kw["dtype"] == "f32" else 1))))
        hi = _log(rng, T + 8, most)
        lo = rng.randint(T, hi)
        kw.update(n=n, T=T, sinks=rng.random() < 0.3)
        if op == "decode":
            c = _decode("", length=(lo, hi), window=rng.choice([0, 0, _log(rng, 1, hi)]),
                        softcap=rng.choice([0.0, 0.0, 0.0, 20.0]), **kw)
        elif op == "shared":
            prefix = _log(rng, 16, most)
            c = _shared("", groups=rng.randint(1, min(4, n)), prefix=prefix, suffix=(T, _log(rng, T + 1, 1024)), **kw)
        else:
            kw["T"] = min(T, 4)
            c = _sparse("", length=(lo, hi), keep=_log(rng, 3, 128), **kw)
    del c["name"]
    return c


# ------------------------------------------------- sizes that a case stands for

def _spread(lo, hi, n):
    """n whole numbers spread over [lo, hi], both ends among them (hi alone for one)."""
    if n == 1:
        return [hi]
    xs = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0) + 0.5) for i in range(n)]
    xs[0], xs[-1] = lo, hi
    return xs


def _rows(c):
    """Rows appended to each entry, and the lengths after that."""
    if c["op"] == "append":
        t = _spread(c["t_lo"], c["t_hi"], c["n"])
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["n"])
        return t, [a + b for a, b in zip(t, ctx)]
    lens = _spread(c["len_lo"], c["len_hi"], c["n"])
    if c["op"] == "shared":
        lens = [c["prefix"] + x for x in lens]
    return [c["T"]] * c["n"], lens


def _group_starts(c):
    n, g = c["n"], c["groups"]
    cuts = [i * n // g for i in range(g + 1)]
    return [x + (1 if 0 < i < g and x + 1 < cuts[i + 1] else 0) for i, x in enumerate(cuts)]


def _row_bytes(c):
    nb = c["D"] // 32
    return c["Hkv"] * nb * (58 if c["fmt"] != "e4m3" else 64)


def work(c):
    t, lens = _rows(c)
    esz = 4 if c["dtype"] == "f32" else 2
    rb = _row_bytes(c)
    if c["op"] == "append":
        rows = sum(t)
        # new rows and queries in, rotated queries and packed rows out, and the rows read back as bf16 values
        return {"bytes": rows * ((2 * c["Hq"] + 2 * c["Hkv"]) * c["D"] * esz + 2 * rb + 2 * c["Hkv"] * c["D"] * 2),
                "flops": rows * c["D"] * 10 * (c["Hq"] + 2 * c["Hkv"])}
    T, n = c["T"], c["n"]
    qo = 2 * n * T * c["Hq"] * c["D"] * esz
    per_row = 4 * c["Hq"] * c["D"]
    if c["op"] == "decode":
        vis = [min(x, c["window"] + T - 1) if c["window"] else x for x in lens]
        one = [min(x, c["window"]) if c["window"] else x for x in lens]
        return {"bytes": sum(vis) * rb + qo, "flops": sum(one) * T * per_row}
    if c["op"] == "shared":
        alone = sum(x - c["prefix"] for x in lens)
        return {"bytes": (alone + c["groups"] * c["prefix"]) * rb + qo, "flops": sum(lens) * T * per_row}
    pages = [-(-x // c["page"]) for x in lens]
    kept = sum(min(p, c["keep"]) for p in pages) * T
    bounds = sum(pages) * c["Hkv"] * (c["D"] // 32) * 68
    return {"bytes": bounds + kept * c["page"] * rb + qo + n * T * (2 * c["Hkv"] * c["D"] * esz + rb),
            "flops": kept * c["page"] * per_row + sum(pages) * T * 4 * c["Hq"] * c["D"]}


# -------------------------------------------------------------- the page pool

def _cell_bytes(c):
    return (c["D"] // 32) * (928 if c["fmt"] != "e4m3" else 1024)


def _pack_cells(c, k, v):
    """Quantise k, v [N, 16, D] (f32) into N cells of 16 rows of one head."""
    N, D = k.shape[0], c["D"]
    NB = D // 32
    if c["fmt"] == "e4m3":
        kb = k.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        vb = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        # V: token = 8 h + 2 j + s, dim = 32 b + 4 g + r -> [h][b][g][j] entries of 8 bytes, pairs of entries in 16
        vb = vb.view(N, 2, 4, 2, NB, 8, 4).permute(0, 1, 4, 5, 2, 6, 3)          # N h b g j r s
        vb = vb.reshape(N, NB, 2, 32, 8).permute(0, 1, 3, 2, 4).reshape(N, -1)    # chunk, entry -> lane, entry
        parts = [_k_order(kb, NB), vb]
    else:
        x = k.view(N, 16, NB, 32)
        d = (x.abs().amax(-1) / 127).half()
        q = torch.where(d[..., None] > 0, x / d.float()[..., None], torch.zeros_like(x)).round().clamp(-127, 127)
        kb = (q + 128).to(torch.uint8).view(N, 16, D)
        y = v.view(N, 16, NB, 32)
        lo, hi = y.amin(-1), y.amax(-1)
        dv, mv = ((hi - lo) / 31).half(), lo.half()
        u = torch.where(dv[..., None] > 0, (y - mv.float()[..., None]) / dv.float()[..., None], torch.zeros_like(y))
        u = u.round().clamp(0, 31).to(torch.int32).view(N, 2, 4, 2, NB, 8, 4)      # h j s b g r
        unit = u[..., 0] | (u[..., 1] << 5) | (u[..., 2] << 10) | ((u[..., 3] >> 4) << 15)   # N h j s b g
        unit = unit.permute(0, 1, 4, 5, 2, 3).reshape(N, 2 * NB, 32, 2)            # (h b) lane s
        unit = unit.view(N, NB // 2, 4, 32, 2).permute(0, 1, 3, 2, 4).contiguous() # chunk lane word s
        unit = torch.where(unit >= 32768, unit - 65536, unit).to(torch.int16).view(torch.uint8).view(N, -1)
        nib = (u[..., 3] & 15).permute(0, 1, 4, 5, 2, 3).reshape(N, NB // 2, 4, 32, 2)  # word, nibble, lane, s
        nib = nib.permute(0, 1, 3, 4, 2)                                           # word lane s nibble
        nib = (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8).reshape(N, -1)
        h16 = lambda a: a.view(N, 2, 4, 2, NB).permute(0, 2, 4, 1, 3).reshape(N, 4, NB, 4)  # [j][b][h s]
        dm = torch.stack([h16(dv), h16(mv)], 3).contiguous().view(torch.uint8).view(N, -1)
        ks = h16(d).contiguous().view(torch.uint8).view(N, -1)
        parts = [_k_order(kb, NB), ks, unit, nib, dm]
    return torch.cat([p.reshape(N, -1) for p in parts], 1)


def _k_order(kb, NB):
    """[N, 16, D] bytes -> [N, NB/2, 16, 4, 2, 8]: 8-dim pieces of a block pair side by side."""
    N = kb.shape[0]
    return kb.view(N, 16, NB // 2, 2, 4, 8).permute(0, 2, 1, 4, 3, 5).reshape(N, -1)


def _unpack_cells(c, cells):
    """The f32 values K, V [N, 16, D] of N cells."""
    N, D = cells.shape[0], c["D"]
    NB = D // 32
    kb = cells[:, :512 * NB].reshape(N, NB // 2, 16, 4, 2, 8).permute(0, 2, 1, 4, 3, 5).reshape(N, 16, D)
    if c["fmt"] == "e4m3":
        k = kb.contiguous().view(torch.float8_e4m3fn).float()
        vb = cells[:, 512 * NB:].reshape(N, NB, 32, 2, 8).permute(0, 1, 3, 2, 4).reshape(N, 2, NB, 8, 4, 4, 2)
        vb = vb.permute(0, 1, 4, 6, 2, 3, 5).reshape(N, 16, D)
        return k, vb.contiguous().view(torch.float8_e4m3fn).float()
    h16 = lambda a: a.view(N, 4, NB, 2, 2).permute(0, 3, 1, 4, 2).reshape(N, 16, NB)
    part = lambda lo, hi: cells[:, lo * NB:hi * NB].contiguous()
    ks = h16(part(512, 544).view(torch.float16))
    unit = part(544, 800).view(torch.int16).view(N, NB // 2, 32, 4, 2).permute(0, 1, 3, 2, 4).to(torch.int32)
    unit = unit.reshape(N, 2, NB, 8, 4, 2)                                          # h b g j s
    nib = part(800, 864).view(N, NB // 2, 32, 2, 2)
    nib = torch.stack([nib & 15, nib >> 4], -1).reshape(N, NB // 2, 32, 2, 4).permute(0, 1, 4, 2, 3)
    nib = nib.reshape(N, 2, NB, 8, 4, 2).to(torch.int32)
    u = torch.stack([unit & 31, (unit >> 5) & 31, (unit >> 10) & 31, ((unit >> 15) & 1) * 16 + nib], -1)
    u = u.permute(0, 1, 4, 5, 2, 3, 6).reshape(N, 16, NB, 32)
    dm = part(864, 928).view(torch.float16).view(N, 4, NB, 2, 4)
    dv, mv = h16(dm[:, :, :, 0].contiguous()), h16(dm[:, :, :, 1].contiguous())
    k = ((kb.to(torch.float32) - 128).view(N, 16, NB, 32) * ks.float()[..., None]).view(N, 16, D)
    v = (u.float() * dv.float()[..., None] + mv.float()[..., None]).view(N, 16, D)
    return k, v


def _bounds_of(k):
    """Key bounds of pages: k [P, Hkv, rows, D] f32 with NaN for rows that hold nothing yet -> codes [P, Hkv, NB, 2, 32] int8, scales."""
    P, H, R, D = k.shape
    x = k.view(P, H, R, D // 32, 32)
    none = torch.isnan(x)
    mn = torch.where(none, math.inf, x).amin(2)
    mx = torch.where(none, -math.inf, x).amax(2)
    empty = none.all(2)
    mn, mx = mn.masked_fill(empty, 0.0), mx.masked_fill(empty, 0.0)
    ds = torch.maximum(mn.abs().amax(-1), mx.abs().amax(-1)) / 127
    safe = torch.where(ds > 0, ds, torch.ones_like(ds))[..., None]
    lo = torch.where(ds[..., None] > 0, mn / safe, torch.zeros_like(mn)).floor().clamp(-127, 127)
    hi = torch.where(ds[..., None] > 0, mx / safe, torch.zeros_like(mx)).ceil().clamp(-127, 127)
    return torch.stack([lo, hi], 3).to(torch.int8), ds


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt, D, Hkv, Hq, page, n = DT[c["dtype"]], c["D"], c["Hkv"], c["Hq"], c["page"], c["n"]
    t, lens = _rows(c)
    cpp = page // 16
    need = [max(1, -(-x // page)) for x in lens]
    shared = [0] * n
    first = list(range(n))
    if c["op"] == "shared":
        st = _group_starts(c)
        for i in range(c["groups"]):
            for b in range(st[i] + 1, st[i + 1]):
                shared[b], first[b] = c["prefix"] // page, st[i]
    total = sum(need) - sum(shared)
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=g, device=DEV)[:total].to(torch.int32).cpu()
    width = max(need)
    tables = torch.zeros(n, width, dtype=torch.int32)
    at = 0
    for b in range(n):
        if shared[b]:
            tables[b, :shared[b]] = tables[first[b], :shared[b]]
        m = need[b] - shared[b]
        tables[b, shared[b]:need[b]] = order[at:at + m]
        at += m
    tables = tables.to(DEV)
    cb = _cell_bytes(c)
    pool = torch.empty(n_pages * Hkv * cpp, cb, dtype=torch.uint8, device=DEV)
    chan = torch.exp(0.3 * torch.randn(D, generator=g, device=DEV))             # channels of unlike size, as keys have
    step = max(1, (1 << 26) // (16 * D))
    for lo in range(0, pool.shape[0], step):
        m = min(step, pool.shape[0] - lo)
        k = torch.randn(m, 16, D, generator=g, device=DEV) * chan
        v = torch.randn(m, 16, D, generator=g, device=DEV)
        pool[lo:lo + m] = _pack_cells(c, k, v)
    if c["op"] == "shared" and c["prefix"] % page:
        # the page in which the prefix ends is each sequence's own copy of its group's
        slot = c["prefix"] // page
        whole = pool.view(n_pages, -1)
        whole[tables[:, slot].long()] = whole[tables[first, slot].long()]
    s = dict(c=c, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), t=t, pool=pool.view(-1), dt=dt)
    draw_ = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(dt)
    if c["op"] == "append":
        rows = sum(t)
        shape = (rows,) if c["t_lo"] != c["t_hi"] else (n, t[0])
        s["k"], s["v"], s["q"] = draw_(*shape, Hkv, D), draw_(*shape, Hkv, D), draw_(*shape, Hq, D)
        s["starts"] = None
        if len(shape) == 1:
            s["starts"] = torch.tensor([sum(t[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
        out = lambda H, d: torch.empty(*shape, H, D, dtype=d, device=DEV)
        s["q_out"], s["k_out"], s["v_out"] = out(Hq, dt), out(Hkv, torch.bfloat16), out(Hkv, torch.bfloat16)
        s["most"] = max(t)
    else:
        s["q"] = draw_(n, c["T"], Hq, D)
        s["sinks"] = torch.randn(Hq, generator=g, device=DEV) if c["sinks"] else None
    if c["op"] == "shared":
        s["group_start"] = torch.tensor(_group_starts(c), dtype=torch.int32, device=DEV)
        s["prefix"] = torch.full((c["groups"],), c["prefix"], dtype=torch.int32, device=DEV)
    if c["op"] == "sparse":
        s["k"], s["v"] = draw_(n, c["T"], Hkv, D) * chan.to(dt), draw_(n, c["T"], Hkv, D)
        s["bounds"] = _page_bounds(s, torch.tensor([x - c["T"] for x in lens], dtype=torch.int32, device=DEV))
    s["maxlen"] = max(lens)
    if own:
        from quantized_kv_cache_08_gb300.cache import PagedKVCache
        s["cache"] = PagedKVCache(n_pages, page, Hkv, D, Hq, max_seqs=n, max_pages=width, max_t=c.get("T", 1), fmt=c["fmt"],
                                  rope_dim=c.get("rope", 0), rope_interleaved=c.get("inter", False),
                                  bounds=c["op"] == "sparse", pool=s["pool"],
                                  bounds_buf=s["bounds"] if c["op"] == "sparse" else None)
    return s


def _page_bounds(s, lens):
    """The bounds buffer of every page: codes of all (page, KV head), then their f32 scales."""
    c = s["c"]
    Hkv, page, D = c["Hkv"], c["page"], c["D"]
    n_pages = s["pool"].numel() // (Hkv * (page // 16) * _cell_bytes(c))
    codes = torch.empty(n_pages, Hkv, D // 32, 2, 32, dtype=torch.int8, device=DEV)
    scales = torch.empty(n_pages, Hkv, D // 32, dtype=torch.float32, device=DEV)
    valid = torch.full((n_pages,), page, dtype=torch.int64, device=DEV)
    slot = torch.arange(s["tables"].shape[1], device=DEV)[None]
    used = slot * page < lens[:, None]
    last = torch.clamp(lens[:, None] - slot * page, max=page)
    valid[s["tables"].long()[used]] = last[used].long()
    row = torch.arange(page, device=DEV)
    step = max(1, (1 << 26) // (Hkv * page * D))
    cells = s["pool"].view(n_pages, -1, _cell_bytes(c))
    for lo in range(0, n_pages, step):
        m = min(step, n_pages - lo)
        k = _unpack_cells(c, cells[lo:lo + m].reshape(-1, _cell_bytes(c)))[0].view(m, Hkv, page, D)
        k = torch.where((row < valid[lo:lo + m, None])[:, None, :, None], k, math.nan)
        codes[lo:lo + m], scales[lo:lo + m] = _bounds_of(k)
    return torch.cat([codes.view(-1).view(torch.uint8), scales.view(-1).view(torch.uint8)])


# ------------------------------------------------------------------ the plain form

def _half(x):
    """float64 -> float16, nearest with ties to even, in one rounding."""
    h = x.float().half().view(torch.int16).to(torch.int32)
    cand = torch.stack([h, h - 1, h + 1])
    val = cand.to(torch.int16).view(torch.float16)
    err = (val.double() - x).abs()
    ok = torch.isfinite(val) & ((cand & 0x7fff) <= 0x7c00)
    err = torch.where(ok, err, math.inf) * 2
    best = err.amin(0)
    odd = (cand & 1).double()
    pick = torch.where(err == best, odd, 2.0).argmin(0)
    return torch.gather(val.view(torch.int16), 0, pick[None])[0].view(torch.float16)


def _away(x):
    return torch.sign(x) * torch.floor(x.abs() + 0.5)


def _token_places(s):
    """Entry and position of each new row."""
    t = torch.tensor(s["t"], device=DEV)
    entry = torch.repeat_interleave(torch.arange(len(s["t"]), device=DEV), t)
    start = torch.cumsum(t, 0) - t
    r = torch.arange(entry.numel(), device=DEV) - start[entry]
    return entry, s["lens"].long()[entry] - t[entry] + r


def _rotate(c, x, pos):
    """x [rows, H, D] f32, turned by its positions (angles in 64 bits)."""
    rot = c.get("rope", 0)
    if not rot:
        return x
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = pos.double()[:, None] * f
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    y = x.clone()
    if c["inter"]:
        p, q = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = p * cos - q * sin, p * sin + q * cos
    else:
        p, q = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = p * cos - q * sin, p * sin + q * cos
    return y


def _write_rows(s, k, v, entry, pos):
    """Quantise rows k, v [rows, Hkv, D] f32 into their pages (codes decided in 64 bits)."""
    c = s["c"]
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    NB, cb = D // 32, _cell_bytes(c)
    rows = k.shape[0]
    pg = s["tables"].long()[entry, pos // page]
    cell = (pg[:, None] * Hkv + torch.arange(Hkv, device=DEV)) * (page // 16) + (pos % page // 16)[:, None]
    t = (pos % 16)[:, None, None]
    e = torch.arange(D, device=DEV)
    b, i = e // 32, e % 32
    base = (cell * cb)[..., None]
    pool = s["pool"]
    koff = base + (b // 2) * 1024 + t * 64 + (i // 8) * 16 + (b % 2) * 8 + i % 8
    h, j, sl = t // 8, t % 8 // 2, t % 2
    g, r = i // 4, i % 4
    n = h * NB + b
    if c["fmt"] == "e4m3":
        pool[koff] = k.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[base + 512 * NB + n // 2 * 512 + (4 * g + j) * 16 + n % 2 * 8 + r * 2 + sl] = \
            v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return
    x = k.double().view(rows, Hkv, NB, 32)
    d = _half(x.abs().amax(-1) / 127)
    dd = d.double()[..., None]
    q = torch.where(dd > 0, _away(x / dd), torch.zeros_like(x)).clamp(-127, 127)
    pool[koff] = (q + 128).to(torch.uint8).view(rows, Hkv, D)
    y = v.double().view(rows, Hkv, NB, 32)
    lo, hi = y.amin(-1), y.amax(-1)
    dv, mv = _half((hi - lo) / 31), lo.half()
    dd = dv.double()[..., None]
    u = torch.where(dd > 0, _away((y - mv.double()[..., None]) / dd), torch.zeros_like(y)).clamp(0, 31).to(torch.int32)
    u = u.view(rows, Hkv, NB, 8, 4)
    half = pool.view(torch.int16)
    bb = torch.arange(NB, device=DEV)
    nn, i4 = h * NB + bb, 2 * h + sl
    half[(base + 512 * NB + (j * NB + bb) * 8 + i4 * 2) // 2] = d.view(torch.int16)
    off = base + 864 * NB + (j * NB + bb) * 16 + i4 * 2
    half[off // 2] = dv.view(torch.int16)
    half[off // 2 + 4] = mv.view(torch.int16)
    unit = u[..., 0] | (u[..., 1] << 5) | (u[..., 2] << 10) | (u[..., 3] >> 4 << 15)
    unit = torch.where(unit >= 32768, unit - 65536, unit).to(torch.int16)
    gg = torch.arange(8, device=DEV)
    lane = 4 * gg + j[..., None]
    n3 = nn[..., None]
    half[(base[..., None] + 544 * NB + n3 // 4 * 512 + lane * 16 + n3 % 4 * 4 + sl[..., None] * 2) // 2] = unit
    nib = u[..., 3] & 15
    nib = (nib[:, :, 0::2] | (nib[:, :, 1::2] << 4)).to(torch.uint8)
    n2 = n3[:, :, 0::2]
    pool[base[..., None] + 800 * NB + n2 // 4 * 128 + lane * 4 + sl[..., None] * 2 + n2 % 4 // 2] = nib


def _gather_cells(s, cell_pages, cell_in_page):
    """Cells [..., Hkv] of page numbers and cells inside them, unpacked: K, V [..., Hkv, 16, D] f32."""
    c = s["c"]
    Hkv, cb, cpp = c["Hkv"], _cell_bytes(c), c["page"] // 16
    idx = (cell_pages[..., None] * Hkv + torch.arange(Hkv, device=DEV)) * cpp + cell_in_page[..., None]
    k, v = _unpack_cells(c, s["pool"].view(-1, cb)[idx.reshape(-1)])
    shape = tuple(idx.shape) + (16, c["D"])
    return k.view(shape), v.view(shape)


def _plain_append(s):
    c = s["c"]
    entry, pos = _token_places(s)
    flat = lambda x: x.float().reshape(-1, x.shape[-2], c["D"])
    q = _rotate(c, flat(s["q"]), pos)
    _write_rows(s, _rotate(c, flat(s["k"]), pos), flat(s["v"]), entry, pos)
    k, v = _gather_cells(s, s["tables"].long()[entry, pos // c["page"]], pos % c["page"] // 16)
    r = torch.arange(pos.numel(), device=DEV)
    k, v = k[r, :, pos % 16], v[r, :, pos % 16]
    return {"q": q.to(s["dt"]).view(s["q"].shape), "k": k.bfloat16().view(s["k"].shape), "v": v.bfloat16().view(s["v"].shape)}


def _attend(c, q, k, v, see, sinks):
    """q [n, T, Hkv, hpk, D], k and v [n, (T,) Hkv, L, D], see [n, T, (Hkv,) L] -> [n, T, Hkv, hpk, D]."""
    if k.dim() == 4:
        s = torch.einsum("nthqd,nhld->nthql", q, k)
    else:
        s = torch.einsum("nthqd,nthld->nthql", q, k)
    s = s / math.sqrt(c["D"])
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    see = see[:, :, None, None] if see.dim() == 3 else see[:, :, :, None]
    s = s.masked_fill(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    if sinks is not None:
        z = sinks.view(1, 1, c["Hkv"], -1, 1)
        m = torch.maximum(m, z)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(s - m)
    den = p.sum(-1, keepdim=True)
    if sinks is not None:
        den = den + torch.exp(z - m)
    o = torch.einsum("nthql,nhld->nthqd" if v.dim() == 4 else "nthql,nthld->nthqd", p, v)
    return torch.where(den > 0, o / den, torch.zeros_like(o))


def _plain_dense(s):
    """Every sequence over its own rows, a few sequences at a time so that the unpacked rows fit."""
    c = s["c"]
    n, T, D, Hkv, page = c["n"], c["T"], c["D"], c["Hkv"], c["page"]
    cells = -(-s["maxlen"] // 16)
    most = max(1, (1 << 31) // (cells * 16 * Hkv * D))
    ci = torch.arange(cells, device=DEV)
    rows = torch.arange(cells * 16, device=DEV)
    out = []
    for lo in range(0, n, most):
        ids = slice(lo, min(n, lo + most))
        lens = s["lens"][ids].long()
        m = lens.numel()
        pages = s["tables"][ids].long()[:, ci * 16 // page]
        k, v = _gather_cells(s, pages, (ci * 16 % page // 16).expand(m, -1))
        k, v = (x.permute(0, 2, 1, 3, 4).reshape(m, Hkv, cells * 16, D) for x in (k, v))
        pos = lens[:, None] - T + torch.arange(T, device=DEV)
        see = rows <= pos[..., None]
        if c["window"]:
            see = see & (rows > pos[..., None] - c["window"])
        q = s["q"][ids].float().view(m, T, Hkv, -1, D)
        out.append(_attend(c, q, k, v, see, s["sinks"]).reshape(m, T, -1, D))
    return torch.cat(out).to(s["dt"])


def _plain_select(s):
    c = s["c"]
    n, T, D, Hkv, page = c["n"], c["T"], c["D"], c["Hkv"], c["page"]
    NB, width = D // 32, s["tables"].shape[1]
    x = s["q"].float().view(n, T, Hkv, -1, NB, 32)
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, 127 / amax, torch.zeros_like(amax))
    code = torch.round(x * inv[..., None])
    dq = amax / 127
    n_pages = s["pool"].numel() // (Hkv * (page // 16) * _cell_bytes(c))
    cut = n_pages * Hkv * NB * 64
    codes = s["bounds"][:cut].view(torch.int8).view(n_pages, Hkv, NB, 2, 32)
    scales = s["bounds"][cut:].view(torch.float32).view(n_pages, Hkv, NB)
    tab = s["tables"].long()
    f, ds = codes[tab].float(), scales[tab]                                # [n, width, Hkv, NB, 2, 32]
    dot = torch.einsum("nthqbi,nphbi->nthqpb", code.clamp(min=0), f[:, :, :, :, 1]) + \
        torch.einsum("nthqbi,nphbi->nthqpb", code.clamp(max=0), f[:, :, :, :, 0])   # whole numbers below 2^24
    part = dq[:, :, :, :, None] * ds.permute(0, 2, 1, 3)[:, None, :, None] * dot
    score = torch.zeros_like(part[..., 0])
    for b in range(NB):                                                    # the order of this sum is the operator's
        score = score + part[..., b]
    score = score.amax(3)                                                  # [n, T, Hkv, width]
    pos = s["lens"].long()[:, None] - T + torch.arange(T, device=DEV)
    count = torch.div(pos + page, page, rounding_mode="floor")             # pages with a visible row
    slot = torch.arange(width, device=DEV)
    there = slot < count[..., None]
    kept = (slot < 1) | (slot >= count[..., None] - 1)
    score = score.masked_fill(kept[:, :, None], math.inf).masked_fill(~there[:, :, None], -math.inf)
    keep = c["keep"]
    top = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :keep]
    if keep > width:
        top = torch.nn.functional.pad(top, (0, keep - width), value=width)
    top = torch.where(torch.arange(keep, device=DEV) < count[:, :, None, None], top, width + 1)
    top = torch.sort(top, dim=-1)[0]
    return torch.where(top < width, top, -1).to(torch.int32)


def _plain_sparse(s):
    c = s["c"]
    n, T, D, Hkv, page = c["n"], c["T"], c["D"], c["Hkv"], c["page"]
    entry, pos = _token_places(s)
    _write_rows(s, s["k"].float().view(-1, Hkv, D), s["v"].float().view(-1, Hkv, D), entry, pos)
    # bounds of the pages that got rows
    first = (s["lens"].long() - T).clamp(min=0) // page
    last = (s["lens"].long() - 1) // page
    slots = (first[:, None] + torch.arange((T + page - 2) // page + 1, device=DEV)).clamp(max=last[:, None])
    pg = torch.gather(s["tables"].long(), 1, slots)
    cpp = page // 16
    cells = torch.arange(cpp, device=DEV)
    k, _ = _gather_cells(s, pg[..., None].expand(-1, -1, cpp), cells.expand(*pg.shape, -1))
    k = k.permute(0, 1, 3, 2, 4, 5).reshape(-1, Hkv, page, D)
    valid = (s["lens"].long()[:, None] - slots * page).clamp(max=page).reshape(-1, 1)
    k = torch.where((torch.arange(page, device=DEV) < valid)[:, None, :, None], k, math.nan)
    codes, ds = _bounds_of(k)
    n_pages = s["pool"].numel() // (Hkv * cpp * _cell_bytes(c))
    cut = n_pages * Hkv * (D // 32) * 64
    s["bounds"][:cut].view(torch.int8).view(n_pages, Hkv, D // 32, 2, 32)[pg.reshape(-1)] = codes
    s["bounds"][cut:].view(torch.float32).view(n_pages, Hkv, D // 32)[pg.reshape(-1)] = ds
    top = _plain_select(s)
    keep = c["keep"]
    got = top >= 0
    slot = top.long().clamp(min=0)
    tab = s["tables"].long()[:, None, None].expand(-1, T, Hkv, -1)
    pages = torch.gather(tab, 3, slot)
    head = torch.arange(Hkv, device=DEV)[:, None, None]
    idx = (pages[..., None] * Hkv + head) * cpp + cells
    k, v = _unpack_cells(c, s["pool"].view(-1, _cell_bytes(c))[idx.reshape(-1)])
    k, v = (x.view(n, T, Hkv, keep * page, D) for x in (k, v))
    at = (slot[..., None] * page + torch.arange(page, device=DEV)).view(n, T, Hkv, -1)
    pos = s["lens"].long()[:, None] - T + torch.arange(T, device=DEV)
    see = (at <= pos[:, :, None, None]) & got[..., None].expand(-1, -1, -1, -1, page).reshape(n, T, Hkv, -1)
    q = s["q"].float().view(n, T, Hkv, -1, D)
    return {"pages": top, "out": _attend(c, q, k, v, see, s["sinks"]).reshape(n, T, -1, D).to(s["dt"])}


def run(s):
    c = s["c"]
    if not own:
        if c["op"] == "append":
            return _plain_append(s)
        if c["op"] == "sparse":
            return _plain_sparse(s)
        return _plain_dense(s)
    kv = s["cache"]
    if c["op"] == "append":
        kv.append(s["k"], s["v"], s["tables"], s["lens"], starts=s["starts"], q=s["q"], q_out=s["q_out"])
        kv.read(s["tables"], s["lens"], s["k_out"], s["v_out"], starts=s["starts"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "decode":
        return kv.decode(s["q"], s["tables"], s["lens"], sinks=s["sinks"], window=c["window"], softcap=c["softcap"])
    if c["op"] == "shared":
        return kv.decode_shared(s["q"], s["tables"], s["lens"], s["group_start"], s["prefix"], sinks=s["sinks"])
    kv.append(s["k"], s["v"], s["tables"], s["lens"])
    pages = kv.select(s["q"], s["tables"], s["lens"], c["keep"], n_first=1, n_last=1)
    return {"pages": pages, "out": kv.decode_sparse(s["q"], s["tables"], s["lens"], pages, sinks=s["sinks"])}


# ------------------------------------------------------------ from the definition, in 64 bits

def _exact_rows(c, pool, cell_bases):
    """K, V (float64) [N, 16, D] of the cells that start at the given bytes, each byte found by its own address."""
    D = c["D"]
    NB = D // 32
    t = torch.arange(16, device=DEV)[:, None]
    e = torch.arange(D, device=DEV)[None]
    b, i = e // 32, e % 32
    g, r, h, j, s = i // 4, i % 4, t // 8, (t // 2) % 4, t % 2
    entry = h * NB + b
    byte = lambda off: pool[cell_bases[:, None, None] + off].long()
    word = lambda off: byte(off) + 256 * byte(off + 1)

    def f16(bits):
        sign, ex, fr = bits >> 15, (bits >> 10) & 31, (bits & 1023).double()
        mag = torch.where(ex == 0, fr * 2.0 ** -24, (1 + fr / 1024) * torch.exp2((ex - 15).double()))
        return torch.where(sign == 1, -mag, mag)

    def e4m3(x):
        sign, ex, fr = x >> 7, (x >> 3) & 15, (x & 7).double()
        mag = torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * torch.exp2((ex - 7).double()))
        return torch.where(sign == 1, -mag, mag)

    kc = byte((b // 2) * 1024 + t * 64 + (i // 8) * 16 + (b % 2) * 8 + i % 8)
    lane = 4 * g + j
    if c["fmt"] == "e4m3":
        return e4m3(kc), e4m3(byte(512 * NB + (entry // 2) * 512 + lane * 16 + (entry % 2) * 8 + 2 * r + s))
    four = 2 * h + s
    kd = f16(word(512 * NB + (j * NB + b) * 8 + 2 * four))
    w = word(544 * NB + (entry // 4) * 512 + lane * 16 + (entry % 4) * 4 + 2 * s)
    nib = (byte(800 * NB + (entry // 4) * 128 + lane * 4 + 2 * s + (entry % 4) // 2) >> (4 * (entry % 2))) & 15
    code = torch.where(r == 3, nib + 16 * (w >> 15), (w >> (5 * r.clamp(max=2))) & 31)
    at = 864 * NB + (j * NB + b) * 16 + 2 * four
    return (kc - 128).double() * kd, code.double() * f16(word(at)) + f16(word(at + 8))


def exact(c, seed):
    s = prepare(c, seed)
    D, Hkv, Hq, page = c["D"], c["Hkv"], c["Hq"], c["page"]
    hpk, cb = Hq // Hkv, _cell_bytes(c)
    t, lens = _rows(c)
    if c["op"] == "append":
        rot = c["rope"]
        places = torch.tensor([x - m + r for m, x in zip(t, lens) for r in range(m)], dtype=torch.float64, device=DEV)

        def turned(x):
            x = x.double().reshape(-1, x.shape[-2], D).clone()
            for i in range(rot // 2):
                one, two = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)
                a = places * math.exp(-math.log(10000.0) * 2 * i / rot)
                z = torch.complex(x[..., one], x[..., two]) * torch.polar(torch.ones_like(a), a)[:, None]
                x[..., one], x[..., two] = z.real, z.imag
            return x

        def stored(x, bits):
            if c["fmt"] == "e4m3":
                mag = x.abs().clamp(max=448)
                q = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
                return torch.sign(x) * torch.round(mag / q) * q
            y = x.reshape(*x.shape[:-1], D // 32, 32)
            if bits == 8:
                d = _half(y.abs().amax(-1) / 127).double()[..., None]
                z = torch.clamp(torch.trunc(y / d.clamp(min=1e-30) + 0.5 * torch.sign(y)), -127, 127) * d
            else:
                m = _half(y.amin(-1)).double()[..., None]
                d = _half((y.amax(-1) - y.amin(-1)) / 31).double()[..., None]
                z = torch.clamp(torch.floor((y - m) / d.clamp(min=1e-30) + 0.5), 0, 31) * d + m
            return z.reshape(x.shape)

        k, v = stored(turned(s["k"]), 8), stored(s["v"].double().reshape(-1, Hkv, D), 5)
        return {"q": turned(s["q"]).view(s["q"].shape), "k": k.view(s["k"].shape), "v": v.view(s["v"].shape)}
    if sum(lens) * Hkv * D > 1_500_000_000:
        return None
    T, cpp = c["T"], page // 16
    pages = None
    if c["op"] == "sparse":
        pages = _plain_sparse(s)["pages"]          # writes the new rows; which pages are kept is decided in whole numbers
    out = torch.zeros(c["n"], T, Hq, D, dtype=torch.float64, device=DEV)
    for b in range(c["n"]):
        cells = -(-lens[b] // 16)
        ci = torch.arange(cells, device=DEV)
        pg = s["tables"][b].long()[ci * 16 // page]
        at = torch.arange(cells * 16, device=DEV)
        for g in range(Hkv):
            k, v = _exact_rows(c, s["pool"], ((pg * Hkv + g) * cpp + ci % cpp) * cb)
            k, v = k.reshape(-1, D), v.reshape(-1, D)
            for r in range(T):
                p = lens[b] - T + r
                lo = max(0, p + 1 - c["window"]) if c["window"] else 0
                see = (at >= lo) & (at <= p)
                if pages is not None:
                    see &= torch.isin(at // page, pages[b, r, g].long())
                x = s["q"][b, r, g * hpk:(g + 1) * hpk].double() @ k[see].T * D ** -0.5
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                top = x.amax(1, keepdim=True)
                w = torch.exp(x - top)
                den = w.sum(1, keepdim=True)
                if s["sinks"] is not None:
                    den = den + torch.exp(s["sinks"][g * hpk:(g + 1) * hpk, None].double() - top)
                out[b, r, g * hpk:(g + 1) * hpk] = w @ v[see] / den
    return {"pages": None, "out": out} if c["op"] == "sparse" else out
