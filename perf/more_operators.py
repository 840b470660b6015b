"""Cases that time and check the operators around a cache's rows: appends at
positions that the caller gives (one axis or several), decodes that accumulate
attention weights, eviction by those weights, and the verification of drafted
tokens.

Each case is a dict of plain values.  `prepare` makes what a serving program
has in hand (page pool, tables, lengths, rows, positions, probabilities),
`run` makes one pass: the plain torch form, or with `own` the calls of the
library.  The page layout that both read is the one `include/kvq.h` describes.
"""

import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def _kv(name, op, fmt="q8_0/q5_1", dtype="bf16", page=64, Hq=32, Hkv=8, D=128, n=1):
    return dict(name=name, op=op, fmt=fmt, dtype=dtype, page=page, Hq=Hq, Hkv=Hkv, D=D, n=n)


def _place(name, axes=3, t=(1, 1), ctx=(0, 0), rope=128, inter=False, cycle=False, **kw):
    return dict(_kv(name, "place", **kw), axes=axes, t_lo=t[0], t_hi=t[1], ctx_lo=ctx[0], ctx_hi=ctx[1], rope=rope,
                inter=inter, cycle=cycle)


def _scored(name, T=1, length=(512, 512), window=0, sinks=False, softcap=0.0, decay=1.0, **kw):
    return dict(_kv(name, "scored", **kw), T=T, len_lo=length[0], len_hi=length[1], window=window, sinks=sinks,
                softcap=softcap, decay=decay)


def _evict(name, keep, length=(512, 512), first=4, last=32, **kw):
    return dict(_kv(name, "evict", **kw), len_lo=length[0], len_hi=length[1], keep=keep, first=first, last=last)


def _verify(name, n=1, T=5, V=32000, dtype="f32", point=False, short=False, pad=0):
    return dict(name=name, op="verify", n=n, T=T, V=V, dtype=dtype, point=point, short=short, pad=pad)


def listed():
    return [
        # one decode step of a batch whose sequences were evicted: a row each, at positions beyond its index (latency)
        _place("place step, 64 sequences", axes=1, n=64, ctx=(1023, 16383)),
        # prompts of text, images and video in one packed batch: time, height and width
        _place("place prompts, 8k rows", n=6, t=(200, 2600)),
        # clips of odd lengths, half of each head rotated in interleaved pairs, axes in turn
        _place("place clips e4m3 f32", fmt="e4m3", dtype="f32", page=16, Hq=16, Hkv=4, D=256, n=5, t=(77, 611),
               ctx=(0, 700), rope=128, inter=True, cycle=True),
        # the smallest scored decode: one short sequence (latency)
        _scored("scored 512", Hq=8, Hkv=2),
        # a serving batch of different lengths, weights added up step by step
        _scored("scored batch 64", n=64, length=(1024, 16384)),
        # the last eight rows of four prompts, f32, old weights fading; a window and sinks over E4M3 rows
        _scored("scored last 8 e4m3 f32", fmt="e4m3", dtype="f32", page=32, Hq=64, Hkv=8, D=64, n=4, T=8,
                length=(3000, 40001), window=16384, sinks=True, decay=0.875),
        # one sequence over its budget by a chunk
        _evict("evict 4608 to 4096", keep=4096, length=(4608, 4608)),
        # one long context cut to an eighth
        _evict("evict 128k e4m3", fmt="e4m3", page=32, Hq=64, Hkv=8, D=64, keep=16384, length=(131072, 131072), last=1024),
        # a batch of different lengths, some of them under the budget
        _evict("evict batch 32", n=32, keep=2000, length=(900, 16384), last=333),
        # four drafts of one sequence (latency)
        _verify("verify 1 x 4, 32000"),
        # a batch with seven drafts each, a large vocabulary
        _verify("verify 64 x 7, 131072", n=64, T=8, V=131072),
        # drafts without a distribution (looked up), of different counts, over bf16 rows of an odd vocabulary
        _verify("verify 37 x 3 lookups bf16", n=37, T=4, V=50021, dtype="bf16", point=True, short=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["place", "scored", "evict", "verify"])
    if op == "verify":
        n, T = _log(rng, 1, 64), rng.randint(1, 9)
        return {k: v for k, v in _verify("", n=n, T=T, V=min(_log(rng, 1000, 131072), 67_000_000 // (n * T)),
                                         dtype=rng.choice(["f32", "f32", "bf16"]), point=rng.random() < 0.3,
                                         short=rng.random() < 0.3, pad=rng.choice([0, 0, 8, 3])).items() if k != "name"}
    Hkv = rng.choice([1, 2, 4, 8])
    kw = dict(fmt=rng.choice(["q8_0/q5_1", "q8_0/q5_1", "e4m3"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
              page=rng.choice([16, 32, 64, 128]), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), D=rng.choice([64, 128, 256]))
    row = Hkv * kw["D"]
    if op == "place":
        n = _log(rng, 1, 128)
        wide = (2 * kw["Hq"] + 2 * Hkv) * kw["D"] * (4 if kw["dtype"] == "f32" else 2)
        hi = _log(rng, 1, max(1, min(8192, 250_000_000 // wide) // n))
        lo = hi if rng.random() < 0.5 else rng.randint(0, hi)
        ctx = _log(rng, 1, 16384)
        c = _place("", n=n, axes=rng.choice([1, 2, 3, 3]), t=(lo, hi), ctx=(rng.randint(0, ctx), ctx),
                   rope=rng.choice([kw["D"], kw["D"], kw["D"] // 2, 32]), inter=rng.random() < 0.4,
                   cycle=rng.random() < 0.4, **kw)
    elif op == "scored":
        n, T = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 3, 5, 8])
        most = max(64, min(65536, 300_000_000 // (n * row * (2 if kw["dtype"] == "f32" else 1))))
        hi = _log(rng, T + 8, most)
        c = _scored("", n=n, T=T, length=(rng.randint(T, hi), hi), window=rng.choice([0, 0, _log(rng, 1, hi)]),
                    sinks=rng.random() < 0.3, softcap=rng.choice([0.0, 0.0, 0.0, 20.0]),
                    decay=rng.choice([1.0, 1.0, 0.0, 0.9375]), **kw)
    else:
        n = _log(rng, 1, 64)
        most = max(64, min(131072, 250_000_000 // (n * row)))
        hi = _log(rng, 48, most)
        keep = _log(rng, 8, max(9, min(hi, 60_000_000 // (n * row))))
        first = rng.randint(0, min(keep, 8))
        c = _evict("", keep, n=n, length=(rng.randint(1, hi), hi), first=first, last=rng.randint(0, (keep - first) // 2), **kw)
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
    """Rows that each entry brings, and the lengths after that."""
    if c["op"] == "place":
        t = _spread(c["t_lo"], c["t_hi"], c["n"])
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["n"])
        return t, [a + b for a, b in zip(t, ctx)]
    return [c.get("T", 0)] * c["n"], _spread(c["len_lo"], c["len_hi"], c["n"])


def _row_bytes(c):
    return c["Hkv"] * (c["D"] // 32) * (58 if c["fmt"] != "e4m3" else 64)


def work(c):
    esz = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "verify":
        # of each sequence one row of probabilities (and of the draft's), and what the drafts ask for
        return {"bytes": c["n"] * (c["V"] * esz * (1 if c["point"] else 2) + c["T"] * (8 + 2 * esz) + 8),
                "flops": c["n"] * c["V"] * 4}
    t, lens = _rows(c)
    rb, n = _row_bytes(c), c["n"]
    if c["op"] == "place":
        rows = sum(t)
        # new rows, queries and positions in, rotated queries and packed rows out, and the rows read back as bf16 values
        return {"bytes": rows * ((2 * c["Hq"] + 2 * c["Hkv"]) * c["D"] * esz + 2 * rb + 2 * c["Hkv"] * c["D"] * 2 + 4 * c["axes"]),
                "flops": rows * c["D"] * 10 * (c["Hq"] + 2 * c["Hkv"])}
    if c["op"] == "scored":
        T = c["T"]
        vis = [min(x, c["window"] + T - 1) if c["window"] else x for x in lens]
        one = [min(x, c["window"]) if c["window"] else x for x in lens]
        # rows and queries once, outputs, and the scores read (where they are) and written
        scored = sum(vis) if c["decay"] == 1.0 else sum(lens)
        return {"bytes": sum(vis) * rb + 2 * n * T * c["Hq"] * c["D"] * esz + scored * c["Hkv"] * (8 if c["decay"] else 4),
                "flops": sum(one) * T * 4 * c["Hq"] * c["D"]}
    kept = sum(min(x, c["keep"]) for x in lens)
    over = sum(x for x in lens if x > c["keep"])
    # scores of what competes; kept rows and their scores moved, listed, and read back as bf16 values
    return {"bytes": over * c["Hkv"] * 4 + kept * (3 * rb + c["Hkv"] * (8 + 4 + 2 * c["D"] * 2)),
            "flops": over * c["Hkv"]}


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


def _axes_of(c):
    """Axis of each rotated pair: shares of 1/4, 3/8, 3/8 (halves for two) side by side, or in turn."""
    half, a = c["rope"] // 2, c["axes"]
    if c["cycle"]:
        return [i % a for i in range(half)]
    cuts = {1: [half], 2: [half // 2, half], 3: [half // 4, half // 4 + (half * 3) // 8, half]}[a]
    return [next(x for x, hi in enumerate(cuts) if i < hi) for i in range(half)]


def _positions(c, t, lens, g):
    """Positions [rows, axes] of the new rows: a quarter of each entry is text, behind it pictures of a square grid
    one after the other; entries start beyond their row's index, as after evictions."""
    t_, lens_ = torch.tensor(t, device=DEV), torch.tensor(lens, device=DEV)
    entry = torch.repeat_interleave(torch.arange(c["n"], device=DEV), t_)
    r = torch.arange(entry.numel(), device=DEV) - (torch.cumsum(t_, 0) - t_)[entry]
    base = (lens_ - t_ + torch.randint(0, 100000, (c["n"],), generator=g, device=DEV))[entry]
    text = t_[entry] // 4
    side = torch.clamp((t_[entry].double() / 3).sqrt().long(), min=1)
    p = (r - text).clamp(min=0)
    grid = torch.stack([p // (side * side), p // side % side, p % side], -1)
    pos = torch.where((r < text)[:, None], (base + r)[:, None], (base + text)[:, None] + grid)
    return (pos if c["axes"] == 3 else pos[:, -c["axes"]:] if c["axes"] == 2 else (base + r)[:, None]).to(torch.int32).contiguous()


def _probabilities(c, g):
    n, T, V, dt = c["n"], c["T"], c["V"], DT[c["dtype"]]
    target = torch.empty(n, T, V + c["pad"], dtype=dt, device=DEV)[..., :V]
    draft = None if c["point"] or T == 1 else torch.empty(n, T - 1, V + c["pad"], dtype=dt, device=DEV)[..., :V]
    tokens = torch.empty(n, T - 1, dtype=torch.int32, device=DEV)
    for t in range(T):
        # one likely token over a long tail, as a model's; the draft's are near the target's
        z = 2.5 * torch.randn(n, V, generator=g, device=DEV)
        likely = torch.randint(0, V, (n, 1), generator=g, device=DEV)
        z.scatter_(1, likely, torch.logsumexp(z, 1, keepdim=True) + 1.5 * torch.randn(n, 1, generator=g, device=DEV))
        target[:, t] = torch.softmax(z, -1)
        if t == T - 1:
            break
        if draft is None:
            tokens[:, t] = likely[:, 0]
        else:
            q = torch.softmax(z + 0.5 * torch.randn(n, V, generator=g, device=DEV), -1)
            draft[:, t] = q
            tokens[:, t] = torch.multinomial(q, 1, generator=g)[:, 0]
    if c["short"] and T > 1:
        count = torch.randint(0, T, (n, 1), generator=g, device=DEV)
        tokens = torch.where(torch.arange(T - 1, device=DEV) < count, tokens, -1)
    u = torch.rand(n, T, generator=g, device=DEV)
    return dict(c=c, target=target, draft=draft, tokens=tokens.contiguous(), u=u,
                lens=torch.randint(T, 5000, (n,), generator=g, device=DEV).to(torch.int32))


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if c["op"] == "verify":
        return _probabilities(c, g)
    dt, D, Hkv, Hq, page, n = DT[c["dtype"]], c["D"], c["Hkv"], c["Hq"], c["page"], c["n"]
    t, lens = _rows(c)
    cpp = page // 16
    need = [max(1, -(-x // page)) for x in lens]
    into = [-(-min(x, c["keep"]) // page) for x in lens] if c["op"] == "evict" else [0] * n
    width, total = max(need), sum(need) + sum(into)
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=g, device=DEV)[:total].to(torch.int32)

    def table(counts, at):
        k = torch.tensor(counts, device=DEV)
        slot = torch.arange(width, device=DEV)
        idx = at + (torch.cumsum(k, 0) - k)[:, None] + slot
        return torch.where(slot < k[:, None], order[idx.clamp(max=total - 1)], torch.zeros_like(order[:1]))

    tables = table(need, 0)
    cb = _cell_bytes(c)
    pool = torch.empty(n_pages * Hkv * cpp, cb, dtype=torch.uint8, device=DEV)
    chan = torch.exp(0.3 * torch.randn(D, generator=g, device=DEV))             # channels of unlike size, as keys have
    step = max(1, (1 << 26) // (16 * D))
    for lo in range(0, pool.shape[0], step):
        m = min(step, pool.shape[0] - lo)
        k = torch.randn(m, 16, D, generator=g, device=DEV) * chan
        v = torch.randn(m, 16, D, generator=g, device=DEV)
        pool[lo:lo + m] = _pack_cells(c, k, v)
    s = dict(c=c, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), t=t, pool=pool.view(-1), dt=dt,
             maxlen=max(lens))
    draw_ = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(dt)
    kw = {}
    if c["op"] == "place":
        rows = sum(t)
        shape = (rows,) if c["t_lo"] != c["t_hi"] else (n, t[0])
        s["k"], s["v"], s["q"] = draw_(*shape, Hkv, D), draw_(*shape, Hkv, D), draw_(*shape, Hq, D)
        s["starts"] = None
        if len(shape) == 1:
            s["starts"] = torch.tensor([sum(t[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
        out = lambda H, d: torch.empty(*shape, H, D, dtype=d, device=DEV)
        s["q_out"], s["k_out"], s["v_out"] = out(Hq, dt), out(Hkv, torch.bfloat16), out(Hkv, torch.bfloat16)
        s["pos"] = _positions(c, t, lens, g).view(*shape, c["axes"])
        kw = dict(rope_dim=c["rope"], rope_interleaved=c["inter"], rope_axes=_axes_of(c))
    else:
        # weights as steps leave them: most rows little, some much, some none
        x = torch.exp(2 * torch.randn(n_pages, Hkv, page, generator=g, device=DEV)) / max(lens)
        s["scores"] = x * (torch.rand(n_pages, Hkv, page, generator=g, device=DEV) > 0.02)
        kw = dict(scores_buf=s["scores"])
    if c["op"] == "scored":
        s["q"] = draw_(n, c["T"], Hq, D)
        s["sinks"] = torch.randn(Hq, generator=g, device=DEV) if c["sinks"] else None
    if c["op"] == "evict":
        s["into"] = table(into, sum(need))
        s["k_out"], s["v_out"] = (torch.empty(n, c["keep"], Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    if own:
        from quantized_kv_cache_08_gb300.cache import PagedKVCache
        s["cache"] = PagedKVCache(n_pages, page, Hkv, D, Hq, max_seqs=n, max_pages=width, max_t=c.get("T", 1), fmt=c["fmt"],
                                  pool=s["pool"], **kw)
    return s


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
    """x [rows, H, D] f32, its pairs turned by the positions [rows, axes] of their axes (angles in 64 bits)."""
    rot = c["rope"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = pos.double()[:, _axes_of(c)] * f
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


def _plain_place(s):
    c = s["c"]
    entry, at = _token_places(s)
    flat = lambda x: x.float().reshape(-1, x.shape[-2], c["D"])
    pos = s["pos"].view(-1, c["axes"])
    q = _rotate(c, flat(s["q"]), pos)
    _write_rows(s, _rotate(c, flat(s["k"]), pos), flat(s["v"]), entry, at)
    k, v = _gather_cells(s, s["tables"].long()[entry, at // c["page"]], at % c["page"] // 16)
    r = torch.arange(at.numel(), device=DEV)
    k, v = k[r, :, at % 16], v[r, :, at % 16]
    return {"q": q.to(s["dt"]).view(s["q"].shape), "k": k.bfloat16().view(s["k"].shape), "v": v.bfloat16().view(s["v"].shape)}


def _plain_scored(s):
    """Attention and the weights' sums, a few sequences at a time so that the unpacked rows fit."""
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
        x = torch.einsum("nthqd,nhld->nthql", s["q"][ids].float().view(m, T, Hkv, -1, D), k) / math.sqrt(D)
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        x = x.masked_fill(~see[:, :, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        if s["sinks"] is not None:
            z = s["sinks"].view(1, 1, Hkv, -1, 1)
            top = torch.maximum(top, z)
        p = torch.exp(x - top)
        den = p.sum(-1, keepdim=True)
        if s["sinks"] is not None:
            den = den + torch.exp(z - top)
        p = p / den
        out.append(torch.einsum("nthql,nhld->nthqd", p, v).reshape(m, T, -1, D))
        b, r = torch.nonzero(rows < lens[:, None], as_tuple=True)      # every row of every sequence
        at = (s["tables"][ids].long()[b, r // page], slice(None), r % page)
        w = p.sum((1, 3))[b, :, r]                                     # [rows, Hkv]
        s["scores"][at] = w if c["decay"] == 0.0 else c["decay"] * s["scores"][at] + w
    return {"out": torch.cat(out).to(s["dt"]), "scores": s["scores"]}


def _row_bytes_of(c, t):
    """Where the bytes of row t [...] of a cell lie: [..., bytes of a row]."""
    D = c["D"]
    NB = D // 32
    t = t[..., None]
    h, j, sl = t // 8, t % 8 // 2, t % 2
    e = torch.arange(D, device=DEV)
    b, i = e // 32, e % 32
    g, r = i // 4, i % 4
    n = h * NB + b
    k = (b // 2) * 1024 + t * 64 + (i // 8) * 16 + (b % 2) * 8 + i % 8
    if c["fmt"] == "e4m3":
        return torch.cat([k, 512 * NB + n // 2 * 512 + (4 * g + j) * 16 + n % 2 * 8 + r * 2 + sl], -1)
    bb, i4 = torch.arange(NB, device=DEV), 2 * h + sl
    two = lambda x: torch.cat([x, x + 1], -1)
    n4, g4 = n[..., ::4], g[::4]                                       # every four elements: a unit
    n8, g8 = n4.reshape(*n4.shape[:-1], NB, 8)[..., ::2, :].reshape(*n4.shape[:-1], -1), g4.view(NB, 8)[::2].reshape(-1)
    return torch.cat([k, two(512 * NB + (j * NB + bb) * 8 + i4 * 2), two(864 * NB + (j * NB + bb) * 16 + i4 * 2),
                      two(864 * NB + (j * NB + bb) * 16 + i4 * 2 + 8),
                      two(544 * NB + n4 // 4 * 512 + (4 * g4 + j) * 16 + n4 % 4 * 4 + sl * 2),
                      800 * NB + n8 // 4 * 128 + (4 * g8 + j) * 4 + sl * 2 + n8 % 4 // 2], -1)


def _plain_evict(s):
    c = s["c"]
    n, D, Hkv, page, keep = c["n"], c["D"], c["Hkv"], c["page"], c["keep"]
    lens, tab, into = s["lens"].long(), s["tables"].long(), s["into"].long()
    L, cpp, cb = s["maxlen"], page // 16, _cell_bytes(c)
    r = torch.arange(L, device=DEV)
    x = s["scores"][tab[:, r // page], :, r % page].permute(0, 2, 1)   # [n, Hkv, L]
    there = r < lens[:, None]
    kept = (r < c["first"]) | (r >= lens[:, None] - c["last"])
    x = x.masked_fill(kept[:, None], math.inf).masked_fill(~there[:, None], -math.inf)
    new = lens.clamp(max=keep)
    top = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :keep]
    if keep > L:
        top = torch.nn.functional.pad(top, (0, keep - L))
    d = torch.arange(keep, device=DEV)
    live = d < new[:, None]                                            # [n, keep]
    top = torch.where(live[:, None], top, L)
    top = torch.sort(top, dim=-1)[0]
    # move the rows' bytes and scores, some at a time
    b, to = torch.nonzero(live, as_tuple=True)
    src = top[b, :, to]                                                # [rows, Hkv]
    head = torch.arange(Hkv, device=DEV)
    cell = lambda pg, at: (pg * Hkv + head) * cpp + at % page // 16
    sp, dp = tab[b[:, None], src // page], into[b, to // page][:, None]
    s["scores"][dp, head, (to % page)[:, None]] = s["scores"][sp, head, src % page]
    by_cell = s["pool"].view(-1, cb)
    step = max(1, (1 << 27) // (Hkv * D))
    for lo in range(0, b.numel(), step):
        m = slice(lo, lo + step)
        by_cell[cell(dp[m], to[m, None])[..., None], _row_bytes_of(c, (to[m] % 16)[:, None])] = \
            by_cell[cell(sp[m], src[m])[..., None], _row_bytes_of(c, src[m] % 16)]
    # the rows as values: each entry's last `keep`, nothing before its first
    k_out, v_out = torch.zeros_like(s["k_out"]), torch.zeros_like(s["v_out"])
    at = new[:, None] - keep + d
    b, i = torch.nonzero(at >= 0, as_tuple=True)
    for lo in range(0, b.numel(), step // 16 + 1):
        m = slice(lo, lo + step // 16 + 1)
        row = at[b[m], i[m]]
        k, v = _gather_cells(s, into[b[m], row // page], row % page // 16)
        z = torch.arange(row.numel(), device=DEV)
        k_out[b[m], i[m]], v_out[b[m], i[m]] = k[z, :, row % 16].bfloat16(), v[z, :, row % 16].bfloat16()
    return {"rows": torch.where(top < L, top, -1).to(torch.int32), "lens": new.to(torch.int32), "scores": s["scores"],
            "k": k_out, "v": v_out}


def _plain_verify(s):
    c = s["c"]
    n, T, V = c["n"], c["T"], c["V"]
    p, q, d, u = s["target"], s["draft"], s["tokens"].long(), s["u"]
    whole = lambda x: (x.double().clamp(0, 1) * 2.0 ** 52).floor().long()
    there = (d >= 0) & (d < V)
    at = d.clamp(0, V - 1)[..., None]
    pd = torch.gather(p[:, :T - 1], 2, at)[..., 0].double()
    qd = torch.ones_like(pd) if q is None else torch.gather(q, 2, at)[..., 0].double()
    ok = there & (u[:, :T - 1].double() * qd < pd)
    a = torch.cumprod(ok.long(), 1).sum(1)                             # accepted drafts
    b = torch.arange(n, device=DEV)
    P = whole(p[b, a])
    W = P
    if T > 1:
        last = a.clamp(max=T - 2)
        rejected = (a < T - 1) & there[b, last]                        # a draft stood here
        if q is None:
            Q = torch.zeros_like(P).scatter_(1, at[b, last], 1 << 52)
        else:
            Q = whole(q[b, last])
        left = (P - Q).clamp(min=0)
        W = torch.where((rejected & (left.sum(1) > 0))[:, None], left, P)
    run_ = torch.cumsum(W, 1)
    S = run_[:, -1]
    U = (u[:, T - 1].double() * 2.0 ** 31).floor().long()
    x = (S >> 31) * U + (((S & ((1 << 31) - 1)) * U) >> 31)            # floor(S U / 2^31)
    token = torch.where(S > 0, (run_ <= x[:, None]).sum(1), -1)
    return {"accept": (a + 1).to(torch.int32), "next": token.to(torch.int32), "lens": s["lens"] - (T - 1 - a).to(torch.int32)}


def run(s):
    c = s["c"]
    if not own:
        return {"place": _plain_place, "scored": _plain_scored, "evict": _plain_evict, "verify": _plain_verify}[c["op"]](s)
    if c["op"] == "verify":
        from quantized_kv_cache_08_gb300.cache import verify
        lens = s["lens"].clone()
        accept, token = verify(s["target"], s["draft"], s["tokens"], s["u"], lens=lens)
        return {"accept": accept, "next": token, "lens": lens}
    kv = s["cache"]
    if c["op"] == "place":
        kv.append(s["k"], s["v"], s["tables"], s["lens"], starts=s["starts"], q=s["q"], q_out=s["q_out"], positions=s["pos"])
        kv.read(s["tables"], s["lens"], s["k_out"], s["v_out"], starts=s["starts"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "scored":
        out = kv.decode_scored(s["q"], s["tables"], s["lens"], decay=c["decay"], sinks=s["sinks"], window=c["window"],
                               softcap=c["softcap"])
        return {"out": out, "scores": s["scores"]}
    rows = kv.select_rows(s["tables"], s["lens"], c["keep"], n_first=c["first"], n_last=c["last"])
    new = kv.compact(s["tables"], s["lens"], rows, tables_out=s["into"])
    kv.read(s["into"], new, s["k_out"], s["v_out"])
    return {"rows": rows, "lens": new, "scores": s["scores"], "k": s["k_out"], "v": s["v_out"]}


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


def _exact_verify(c, s):
    import numpy as np
    out = {"accept": [], "next": [], "lens": s["lens"].tolist()}
    u, d = s["u"].cpu().double().numpy(), s["tokens"].cpu().numpy()
    for b in range(c["n"]):
        a, held = 0, False
        while a < c["T"] - 1 and 0 <= d[b, a] < c["V"]:
            held = True
            qd = 1.0 if s["draft"] is None else float(s["draft"][b, a, d[b, a]])
            if not u[b, a] * qd < float(s["target"][b, a, d[b, a]]):
                break
            a, held = a + 1, False
        units = lambda x: np.floor(np.ldexp(x.double().cpu().numpy(), 52)).astype(np.uint64).astype(object)
        p = units(s["target"][b, a])
        w = p
        if held:
            if s["draft"] is None:
                q = np.zeros_like(p)
                q[d[b, a]] = 2 ** 52
            else:
                q = units(s["draft"][b, a])
            w = np.maximum(p - q, 0)
            if w.sum() == 0:
                w = p
        x = w.sum() * int(u[b, -1] * 2 ** 31) >> 31
        total, token = 0, -1
        for i, y in enumerate(w):
            total += y
            if total > x:
                token = i
                break
        out["accept"].append(a + 1)
        out["next"].append(token)
        out["lens"][b] -= c["T"] - 1 - a
    return {k: torch.tensor(v, dtype=torch.int32) for k, v in out.items()}


def _exact_place(c, s):
    D, Hkv, rot = c["D"], c["Hkv"], c["rope"]
    axis, pos = _axes_of(c), s["pos"].view(-1, c["axes"]).double()

    def turned(x):
        x = x.double().reshape(-1, x.shape[-2], D).clone()
        for i in range(rot // 2):
            one, two = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)
            a = pos[:, axis[i]] * math.exp(-math.log(10000.0) * 2 * i / rot)
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


def _exact_scored(c, s, lens):
    D, Hkv, Hq, page, T = c["D"], c["Hkv"], c["Hq"], c["page"], c["T"]
    hpk, cb, cpp = Hq // Hkv, _cell_bytes(c), page // 16
    out = torch.zeros(c["n"], T, Hq, D, dtype=torch.float64, device=DEV)
    score = s["scores"].double()
    for b in range(c["n"]):
        cells = -(-lens[b] // 16)
        ci = torch.arange(cells, device=DEV)
        pg = s["tables"][b].long()[ci * 16 // page]
        at = torch.arange(lens[b], device=DEV)
        for g in range(Hkv):
            k, v = _exact_rows(c, s["pool"], ((pg * Hkv + g) * cpp + ci % cpp) * cb)
            k, v = k.reshape(-1, D)[:lens[b]], v.reshape(-1, D)[:lens[b]]
            gain = torch.zeros(lens[b], dtype=torch.float64, device=DEV)
            for r in range(T):
                p = lens[b] - T + r
                lo = max(0, p + 1 - c["window"]) if c["window"] else 0
                x = s["q"][b, r, g * hpk:(g + 1) * hpk].double() @ k[lo:p + 1].T * D ** -0.5
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                den = torch.logsumexp(x, 1)
                if s["sinks"] is not None:
                    den = torch.logaddexp(den, s["sinks"][g * hpk:(g + 1) * hpk].double())
                w = torch.exp(x - den[:, None])
                gain[lo:p + 1] += w.sum(0)
                out[b, r, g * hpk:(g + 1) * hpk] = w @ v[lo:p + 1]
            where = (s["tables"][b].long()[at // page], torch.full_like(at, g), at % page)
            score[where] = (score[where] * c["decay"] if c["decay"] else 0.0) + gain
    return {"out": out, "scores": score}


def _exact_evict(c, s, lens):
    D, Hkv, page, keep = c["D"], c["Hkv"], c["page"], c["keep"]
    cb, cpp = _cell_bytes(c), page // 16
    rows = torch.full((c["n"], Hkv, keep), -1, dtype=torch.int32, device=DEV)
    k = torch.zeros(c["n"], keep, Hkv, D, dtype=torch.float64, device=DEV)
    v, score = torch.zeros_like(k), s["scores"].double()
    for b in range(c["n"]):
        m = min(lens[b], keep)
        at = torch.arange(lens[b], device=DEV)
        pg = s["tables"][b].long()[at // page]
        for g in range(Hkv):
            free = at[c["first"]:lens[b] - c["last"]] if lens[b] > keep else at[:0]
            best = free[torch.argsort(-s["scores"].double()[pg[free], g, free % page], stable=True)][:m - c["first"] - c["last"]]
            pick = at if lens[b] <= keep else torch.sort(torch.cat([at[:c["first"]], best, at[lens[b] - c["last"]:]]))[0]
            rows[b, g, :m] = pick
            kk, vv = _exact_rows(c, s["pool"], ((pg[pick] * Hkv + g) * cpp + pick % page // 16) * cb)
            i = torch.arange(m, device=DEV)
            k[b, keep - m:, g], v[b, keep - m:, g] = kk[i, pick % 16], vv[i, pick % 16]
            score[s["into"][b].long()[i // page], g, i % page] = s["scores"].double()[pg[pick], g, pick % page]
    return {"rows": rows, "lens": torch.tensor([min(x, keep) for x in lens], dtype=torch.int32), "scores": score, "k": k, "v": v}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "verify":
        return _exact_verify(c, s)
    lens = _rows(c)[1]
    if c["op"] == "place":
        return _exact_place(c, s)
    if c["op"] == "scored":
        return None if sum(lens) * c["Hkv"] * c["D"] > 1_500_000_000 else _exact_scored(c, s, lens)
    return _exact_evict(c, s, lens)
