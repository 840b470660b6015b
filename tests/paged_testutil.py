"""A device paged cache beside an oracle that keeps every sequence's rows as
fp64 values, fed with the same host arrays."""

import numpy as np
import torch

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300.cache import PagedKVCache
from tests.kvq_testutil import need_gpu

GARBAGE = 0xFF     # NaN scales and codes: bytes that nothing may read as values


class PagedPair:
    def __init__(self, n, Hkv, D, Hq, page=16, max_pages=8, fmt="q8_0/q5_1", max_t=4, seed=0, **kw):
        need_gpu()
        self.n, self.Hkv, self.D, self.Hq, self.page, self.max_pages, self.fmt = n, Hkv, D, Hq, page, max_pages, fmt
        self.rng = np.random.default_rng(seed)
        self.n_pages = n * max_pages + 3
        order = self.rng.permutation(self.n_pages)[:n * max_pages]
        self.tab = order.reshape(n, max_pages).astype(np.int32)
        self.dev = PagedKVCache(self.n_pages, page, Hkv, D, Hq, max_seqs=max(n, 2), max_pages=max_pages, max_t=max_t,
                                fmt=fmt, **kw)
        self.dev.pool.fill_(GARBAGE)
        self.tables = torch.from_numpy(self.tab).cuda()
        self.k = [np.zeros((0, Hkv, D)) for _ in range(n)]        # values as stored
        self.v = [np.zeros((0, Hkv, D)) for _ in range(n)]
        self.kb = [[] for _ in range(n)]                          # block bytes of each row
        self.vb = [[] for _ in range(n)]

    def lens(self):
        return torch.tensor([len(x) for x in self.k], dtype=torch.int32, device="cuda")

    def randn(self, *shape, dtype=torch.float32):
        return torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).to(dtype)

    def note(self, b, k, v):
        """Oracle side of appending rows k, v [T, Hkv, D] (float32 values, already rotated)."""
        if len(k) == 0:
            return
        kb, vb = P.blocks(k, self.fmt, "k"), P.blocks(v, self.fmt, "v")
        self.kb[b] += list(kb)
        self.vb[b] += list(vb)
        self.k[b] = np.concatenate([self.k[b], P.values(kb, self.fmt, "k")])
        self.v[b] = np.concatenate([self.v[b], P.values(vb, self.fmt, "v")])

    def append(self, counts, dtype=torch.float32, scale=1.0):
        """Packed append of counts[b] random rows to each sequence (no rotation)."""
        rows = int(sum(counts))
        k, v = self.randn(rows, self.Hkv, self.D) * scale, self.randn(rows, self.Hkv, self.D) * scale
        k, v = k.to(dtype), v.to(dtype)
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        for b in range(self.n):
            s = slice(starts[b], starts[b + 1])
            self.note(b, k[s].float().numpy(), v[s].float().numpy())
        self.dev.append(k.cuda(), v.cuda(), self.tables, self.lens(), starts=torch.from_numpy(starts).cuda())

    def expected_pool(self):
        cb, cpp = P.cell_bytes(self.D, self.fmt), self.page // 16
        pool = np.full((self.n_pages, self.Hkv, cpp, cb), GARBAGE, np.uint8)
        for b in range(self.n):
            for r in range(len(self.kb[b])):
                pg = pool[self.tab[b, r // self.page]]
                for h in range(self.Hkv):
                    P.put_row(pg[h, r % self.page // 16], r % 16, self.kb[b][r][h], self.vb[b][r][h], self.fmt)
        return pool.reshape(-1)

    def want(self, q, window=0, sinks=None, softcap=0.0, scale=0.0, pages=None):
        """Outputs and sum p |v| (float64) of queries q [n, T, Hq, D] (host tensor)."""
        qf = q.double().numpy()
        n, T, Hq, D = qf.shape
        hpk = Hq // self.Hkv
        out, mag = np.zeros(qf.shape), np.zeros(qf.shape)
        for b in range(n):
            L = len(self.k[b])
            at = np.arange(L)
            for t in range(T):
                p = L - T + t
                base = (at <= p) & (at > p - window if window else True)
                for h in range(Hq):
                    see = base.astype(np.int64)
                    if pages is not None:
                        listed = [x for x in pages[b, t, h // hpk] if x >= 0]
                        see = see * np.array([listed.count(x // self.page) for x in at], np.int64)
                    o, m = P.attend(qf[b, t, h], self.k[b][:, h // hpk], self.v[b][:, h // hpk], see, scale, softcap,
                                    None if sinks is None else float(sinks[h]))
                    out[b, t, h], mag[b, t, h] = o, m
        return out, mag

    def spread(self):
        """Largest q5_1 block range of the stored values: what 32 code steps can span."""
        m = 0.0
        for v in self.v:
            if len(v):
                y = v.reshape(len(v), self.Hkv, -1, 32)
                m = max(m, float((y.max(-1) - y.min(-1)).max()))
        return m


def assert_attention(pair, got, want, mag, what="output"):
    """Elementwise bounds.  bf16: the output's rounding (2^-8 of it), and inside
    the roundings of p and of v to fp16 (2^-11 each of every p |v|), with as
    much again for the f32 sums.  f32: q in two fp16 parts and p d in two bf16
    parts leave 2^-22 of a score's products and 2^-16 of p d |u - 16|, at most
    2^-16 * (range * 16/31); scores here stay below 2^5 in sum |q k| scale, so
    2^-16 of mag covers them with the f32 sums."""
    assert got.shape == tuple(want.shape)
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: non-finite"
    err = np.abs(g - want)
    if got.dtype == torch.bfloat16:
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag + 1e-30
    else:
        tol = 2.0 ** -16 * (mag + pair.spread()) + 1e-30
    bad = err > tol
    assert not bad.any(), f"{what}: {bad.sum()} beyond the bound, worst ratio {np.max(err / tol):.2f}"
