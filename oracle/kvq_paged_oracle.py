"""fp64 oracle of the paged cache (numpy): the position rotation, the cell
layout byte by byte, attention over any set of visible rows, key bounds and
page selection.  Test infrastructure; shares no code with the CUDA path."""

from __future__ import annotations

import numpy as np

from oracle import kvq_oracle as O


def rotate(x, pos, rope_dim, interleaved=False, base=10000.0, freq=None):
    """x float64 [rows, H, D] turned by pos [rows]: pair i by pos * freq[i]."""
    x = np.array(x, dtype=np.float64)
    if rope_dim == 0:
        return x
    half = rope_dim // 2
    f = np.asarray(freq, np.float64) if freq is not None else float(base) ** (-2.0 * np.arange(half) / rope_dim)
    a = np.asarray(pos, np.float64)[:, None] * f
    w = (np.cos(a) + 1j * np.sin(a))[:, None, :]
    one, two = (slice(0, rope_dim, 2), slice(1, rope_dim, 2)) if interleaved else (slice(0, half), slice(half, rope_dim))
    z = (x[..., one] + 1j * x[..., two]) * w
    x[..., one], x[..., two] = z.real, z.imag
    return x


def blocks(x, fmt, which):
    """Block bytes of rows [rows, H, D]: uint8 [rows, H, NB, 34 | 24 | 32]; which: "k" or "v"."""
    x = np.asarray(x, np.float32)
    rows, H, D = x.shape
    y = x.reshape(rows, H, D // 32, 32)
    if fmt == "e4m3":
        return O.e4m3_bits(y.astype(np.float64))
    return O.q8_0_quantize(y) if which == "k" else O.q5_1_quantize(y)


def values(blk, fmt, which):
    """Block bytes -> float64 rows [rows, H, D]."""
    v = O.e4m3_value(blk) if fmt == "e4m3" else O.q8_0_dequantize(blk) if which == "k" else O.q5_1_dequantize(blk)
    return v.reshape(v.shape[0], v.shape[1], -1)


def cell_bytes(D, fmt):
    return D // 32 * (1024 if fmt == "e4m3" else 928)


def put_row(cell, t, kblk, vblk, fmt):
    """Write row t (block bytes [NB, ..] of one head) into a cell (uint8 view)."""
    NB = kblk.shape[0]
    h, j, s = t // 8, (t % 8) // 2, t % 2
    for b in range(NB):
        n, four = h * NB + b, 2 * h + s
        if fmt == "e4m3":
            kc, vc = kblk[b], vblk[b]
        else:
            kc = (kblk[b][2:].view(np.int8).astype(np.int64) + 128).astype(np.uint8)
            _, _, u = O.q5_1_fields(vblk[b])
            at = 512 * NB + (j * NB + b) * 8 + four * 2
            cell[at:at + 2] = kblk[b][:2]
            at = 864 * NB + (j * NB + b) * 16 + four * 2
            cell[at:at + 2] = vblk[b][0:2]
            cell[at + 8:at + 10] = vblk[b][2:4]
        for i in range(32):
            g, r = i // 4, i % 4
            lane = 4 * g + j
            cell[(b // 2) * 1024 + t * 64 + (i // 8) * 16 + (b % 2) * 8 + i % 8] = kc[i]
            if fmt == "e4m3":
                cell[512 * NB + (n // 2) * 512 + lane * 16 + (n % 2) * 8 + r * 2 + s] = vc[i]
        if fmt != "e4m3":
            for g in range(8):
                lane = 4 * g + j
                c = [int(x) for x in u[4 * g:4 * g + 4]]
                unit = c[0] | c[1] << 5 | c[2] << 10 | (c[3] >> 4) << 15
                at = 544 * NB + (n // 4) * 512 + lane * 16 + (n % 4) * 4 + s * 2
                cell[at], cell[at + 1] = unit & 255, unit >> 8
                at = 800 * NB + (n // 4) * 128 + lane * 4 + s * 2 + (n % 4) // 2
                keep = 0xF0 if n % 2 == 0 else 0x0F
                cell[at] = (int(cell[at]) & keep) | ((c[3] & 15) << (4 * (n % 2)))


def attend(q, k, v, see, scale=None, softcap=0.0, sink=None):
    """One query q [D] over rows k, v [L, D] where see [L] (counts: a row seen
    twice counts twice).  Returns the output and sum p |v| of the same p."""
    D = q.shape[0]
    scale = 1.0 / np.sqrt(D) if not scale or scale <= 0 else scale
    idx = np.flatnonzero(see)
    if len(idx) == 0:
        return np.zeros(D), np.zeros(D)
    s = k[idx] @ q * scale
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    m = s.max() if sink is None else max(s.max(), sink)
    p = np.exp(s - m) * np.asarray(see, np.float64)[idx]
    den = p.sum() + (0.0 if sink is None else np.exp(sink - m))
    p = p / den
    return p @ v[idx], p @ np.abs(v[idx])


def bounds(k):
    """Key bounds of one page's rows k [rows, D] (values): codes int8 [NB, 2, 32], scales f32 [NB]."""
    f = np.float32
    x = k.astype(f).reshape(k.shape[0], -1, 32)
    mn, mx = x.min(0), x.max(0)
    ds = (np.maximum(np.abs(mn).max(-1), np.abs(mx).max(-1)) * (f(1) / f(127))).astype(f)
    safe = np.where(ds > 0, ds, f(1))[:, None]
    lo = np.where(ds[:, None] > 0, np.clip(np.floor(mn / safe), -127, 127), 0)
    hi = np.where(ds[:, None] > 0, np.clip(np.ceil(mx / safe), -127, 127), 0)
    return np.stack([lo, hi], 1).astype(np.int8), ds


def scores(q, codes, ds):
    """f32 scores of pages for one KV head: q [hpk, D] (f32), codes [P, NB, 2, 32], ds [P, NB] -> [P]."""
    f = np.float32
    x = q.astype(f).reshape(q.shape[0], -1, 32)
    am = np.abs(x).max(-1)
    with np.errstate(divide="ignore"):
        inv = np.where(am > 0, (f(1) / am) * f(127), f(0)).astype(f)
    c = np.rint((x * inv[..., None]).astype(f)).astype(np.int64)
    dq = (am * (f(1) / f(127))).astype(f)
    w = codes.astype(np.int64)
    dot = np.maximum(c, 0)[:, None] * w[None, :, :, 1] + np.minimum(c, 0)[:, None] * w[None, :, :, 0]
    dot = dot.sum(-1).astype(f)
    s = np.zeros(dot.shape[:2], f)
    for b in range(dot.shape[2]):
        part = ((dq[:, None, b] * ds[None, :, b]).astype(f) * dot[..., b]).astype(f)
        s = (s + part).astype(f)
    return s.max(0)


def select(score, keep, n_first, n_last):
    """Kept page indexes of scores [P], ascending."""
    P = len(score)
    forced = [p for p in range(P) if p < n_first or p >= P - n_last]
    rest = sorted((p for p in range(P) if p not in set(forced)), key=lambda p: (-score[p], p))
    order = forced + rest
    return sorted(order[:keep])
