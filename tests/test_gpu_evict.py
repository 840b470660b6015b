"""Row scores, the rows that stay and their move, on the GPU against the oracle:
weights within what the decode's arithmetic leaves, choices and bytes exactly."""

import re
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300.cache import PagedKVCache, verify
from tests.kvq_testutil import need_gpu
from tests.paged_testutil import PagedPair, assert_attention

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
Q8, F8 = "q8_0/q5_1", "e4m3"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def scores_of(p, b, dev=None):
    """Scores of sequence b's rows, float32 [L, Hkv]."""
    s = (p.dev.scores if dev is None else dev).cpu().numpy()
    r = np.arange(len(p.k[b]))
    return s[p.tab[b, r // p.page], :, r % p.page]


def gains(p, q, **kw):
    """What a decode of q [n, T, Hq, D] adds to each row: a list of float64 [L, Hkv]."""
    qf, window = q.double().numpy(), kw.pop("window", 0)
    sinks = kw.pop("sinks", None)
    n, T, Hq, D = qf.shape
    out = []
    for b in range(n):
        L = len(p.k[b])
        at, w = np.arange(L), np.zeros((L, p.Hkv))
        for t in range(T):
            pos = L - T + t
            see = (at <= pos) & (at > pos - window if window else True)
            for h in range(Hq):
                g = h // (Hq // p.Hkv)
                w[:, g] += P.weights(qf[b, t, h], p.k[b][:, g], see, sink=None if sinks is None else float(sinks[h]), **kw)
        out.append(w)
    return out


def near(got, old, gain, decay):
    """A score's two factors of 2^(s - m) and the sum of weights come from scores s
    that are off by 2^-22 of sum |q k| scale < 2^5 and by f32 sums: 2^-16 of the
    gain; then one product and one sum in f32 on what was there."""
    want = decay * old.astype(np.float64) + gain
    tol = 2.0 ** -16 * gain + 2.0 ** -23 * (np.abs(want) + np.abs(old)) + 1e-30
    bad = np.abs(got.astype(np.float64) - want) > tol
    assert not bad.any(), f"{bad.sum()} scores off, worst {np.max(np.abs(got - want) / tol):.2f}"


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,Hkv,hpk,T,page,lens,kw", [
    (64, 2, 4, 1, 16, [1, 0, 33, 96], {}),
    (64, 1, 8, 1, 16, [50, 16], {}),
    (128, 2, 2, 4, 32, [3, 1100, 700], dict(window=90)),             # pages of many fragments, a window's front
    (128, 1, 1, 1, 32, [5, 190, 64], {}),
    (128, 3, 5, 3, 16, [2, 80, 3], dict(window=7)),                  # a sequence with positions below 0
    (256, 1, 8, 2, 64, [130, 17], dict(softcap=5.0)),
    (64, 1, 16, 8, 16, [8, 77], dict(window=20)),
    (128, 2, 16, 8, 128, [300, 9], {}),                              # several tiles of queries
    (256, 1, 16, 8, 16, [100], dict(window=33)),                     # several passes of them
    (128, 1, 33, 4, 16, [90, 5], {}),
])
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.5])
@pytest.mark.parametrize("scratch", [True, False])
def test_scored_decode(fmt, dtype, D, Hkv, hpk, T, page, lens, kw, decay, scratch):
    if scratch and hpk * T > 8:
        pytest.skip("no scratch for so many queries")
    n, mp = len(lens), max(2, -(-max(lens) // page))
    p = PagedPair(n, Hkv, D, Hkv * hpk, page=page, max_pages=mp, fmt=fmt, max_t=T, seed=D + T, scores=True, score_scratch=scratch)
    assert (p.dev.scratch is not None) == scratch
    p.append(lens)
    for step, sink in enumerate((False, True)):
        before = torch.rand(p.dev.scores.shape, device="cuda")
        p.dev.scores.copy_(before)
        if decay == 0.0:
            p.dev.scores[p.dev.scores > 0.5] = float("nan")          # not read
            before = p.dev.scores.clone()
        q = p.randn(n, T, Hkv * hpk, D, dtype=dtype)
        sinks = p.randn(Hkv * hpk) if sink else None
        out = p.dev.decode_scored(q.cuda(), p.tables, p.lens(), decay=decay, sinks=None if sinks is None else sinks.cuda(), **kw)
        same = p.dev.decode(q.cuda(), p.tables, p.lens(), sinks=None if sinks is None else sinks.cuda(), **kw)
        assert torch.equal(out, same)
        assert_attention(p, out, *p.want(q, sinks=None if sinks is None else sinks.numpy(), **kw))
        gain = gains(p, q, sinks=None if sinks is None else sinks.numpy(), **kw)
        left = torch.ones(before.shape, dtype=torch.bool)
        for b in range(n):
            old = scores_of(p, b, before)
            near(scores_of(p, b), np.nan_to_num(old) if decay == 0.0 else old, gain[b], decay)
            r = np.arange(lens[b])
            left[p.tab[b, r // page], :, r % page] = False
        a, c = before.cpu()[left], p.dev.scores.cpu()[left]
        assert torch.equal(torch.nan_to_num(a, nan=-1.0), torch.nan_to_num(c, nan=-1.0))     # all other rows as they were
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("scratch", [True, False])
def test_weights_add_up_and_repeat(scratch):
    """Many sequences of very different lengths over all blocks: a query's weights sum to 1; two runs give the same bits."""
    need_gpu()
    n, Hkv, D, page, mp = 33, 4, 64, 64, 64
    lens = [1 + (i * 997) % 4096 for i in range(n)]
    c = PagedKVCache(n * mp, page, Hkv, D, 4 * Hkv, max_seqs=n, max_pages=mp, scores=True, score_scratch=scratch)
    tab = torch.randperm(n * mp, generator=torch.Generator().manual_seed(1)).view(n, mp).int().cuda()
    starts = i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    k = torch.randn(sum(lens), Hkv, D, device="cuda", dtype=BF)
    c.append(k, k, tab, i32(lens), starts=starts)
    q = torch.randn(n, 1, 4 * Hkv, D, device="cuda", dtype=BF)
    got = []
    for _ in range(2):
        c.scores.zero_()
        c.decode_scored(q, tab, i32(lens))
        got.append(c.scores.clone())
    assert torch.equal(*got)
    s = got[0][tab.long()].permute(0, 2, 1, 3).reshape(n, Hkv, -1).double()
    assert (s.sum(-1) - 4).abs().max() <= 4 * 2.0 ** -15
    c.decode_scored(q, tab, i32(lens))
    assert ((c.scores - 2 * got[0]).abs() <= 2.0 ** -23 * c.scores).all()


@pytest.mark.parametrize("bounds", [False, True])
@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 0, 23]])
def test_appended_rows_start_at_zero(fmt, counts, bounds):
    p = PagedPair(3, 2, 128, 4, page=16, max_pages=4, fmt=fmt, scores=True, bounds=bounds)
    p.append([5, 7, 0])
    p.dev.scores.fill_(3.0)
    old = [len(x) for x in p.k]
    if counts[0] == 1:                                  # a row each, without starts
        k = p.randn(3, 1, 2, 128)
        for b in range(3):
            p.note(b, k[b].numpy(), k[b].numpy())
        p.dev.append(k.cuda(), k.cuda(), p.tables, p.lens())
    else:
        p.append(counts)
    want = torch.full(p.dev.scores.shape, 3.0)
    for b in range(3):
        for r in range(old[b], len(p.k[b])):
            want[p.tab[b, r // 16], :, r % 16] = 0.0
    assert torch.equal(p.dev.scores.cpu(), want)
    assert np.array_equal(p.dev.pool.cpu().numpy(), p.expected_pool())


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", [1e2, 1e4, 1e6, 1e12])
@pytest.mark.parametrize("scratch", [True, False])
def test_weights_of_large_scores_add_up(fmt, dtype, scale, scratch):
    """Scores of thousands and more: their steps in f32 are no small change of a weight any more, but weights are
    worked out from the same numbers as the softmax's sum, so that they add up to 1 a query: 2^-21 for the sum of 300 f32
    numbers either way, as much again for the product."""
    p = PagedPair(2, 2, 128, 8, page=16, max_pages=20, fmt=fmt, max_t=1, scores=True, score_scratch=scratch)
    assert (p.dev.scratch is not None) == scratch
    p.append([300, 33])
    out = p.dev.decode_scored(p.randn(2, 1, 8, 128, dtype=dtype).cuda(), p.tables, p.lens(), scale=scale)
    assert torch.isfinite(out).all()
    for b in range(2):
        assert np.abs(scores_of(p, b).astype(np.float64).sum(0) - 4).max() <= 4 * 2.0 ** -19


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scratch", [True, False])
def test_queries_that_are_not_finite_add_nothing(dtype, scratch):
    p = PagedPair(2, 1, 64, 4, page=16, max_pages=3, max_t=1, scores=True, score_scratch=scratch)
    p.append([40, 20])
    q = p.randn(2, 1, 4, 64, dtype=dtype)
    bad = q.clone()
    bad[0, 0, 1, 3], bad[0, 0, 2, 60], bad[1, 0, :, 0] = float("nan"), float("inf"), float("-inf")
    out = p.dev.decode_scored(bad.cuda(), p.tables, p.lens())
    assert torch.isnan(out[0, 0, 1:3]).all() and torch.isnan(out[1]).all() and torch.isfinite(out[0, 0, 0::3]).all()
    only = q.clone()
    w = sum(P.weights(q[0, 0, h].double().numpy(), p.k[0][:, 0], np.ones(40)) for h in (0, 3))
    near(scores_of(p, 0), np.zeros((40, 1)), w[:, None], 1.0)
    assert (scores_of(p, 1) == 0).all()
    # scores beyond f32: the query's output is NaN, and it adds nothing
    p.dev.scores.zero_()
    big = only * 1e30 if dtype == BF else only * 1e36
    out = p.dev.decode_scored(big.cuda(), p.tables, p.lens(), scale=1e20)
    s = p.dev.scores.cpu()
    assert torch.isfinite(s).all()
    seen = torch.isfinite(out).all(-1).sum(-1).sum(-1)
    for b in range(2):
        assert abs(float(scores_of(p, b).sum()) - int(seen[b])) <= 1e-4


def test_rows_of_garbage_behind_the_length_do_no_harm():
    """Bytes behind the length inside its cell are NaN scales and codes (the pool is filled with them)."""
    p = PagedPair(3, 2, 128, 8, page=16, max_pages=2, max_t=1, scores=True)
    p.dev.scratch.fill_(float("nan"))
    p.append([1, 17, 31])
    p.dev.scores.fill_(1.0)
    p.dev.decode_scored(p.randn(3, 1, 8, 128).cuda(), p.tables, p.lens())
    assert torch.isfinite(p.dev.scores).all()


# ------------------------------------------------------------------ choice

def chosen(score, keep, first, last):
    rank = np.unique(np.where(np.isnan(score), 0.0, score), return_inverse=True)[1]
    return P.select(np.where(np.isnan(score), -1, rank), keep, first, last)     # (a NaN below -inf)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "zeros", "odd"])
@pytest.mark.parametrize("lens,keep,first,last,page", [
    ([100, 16, 17, 0, 33], 16, 2, 3, 16), ([1000, 4096, 999, 1], 1000, 4, 32, 64), ([50, 5], 1, 0, 0, 16),
    ([70, 64], 5, 5, 0, 32), ([70, 64], 5, 0, 5, 32), ([300], 7, 3, 4, 256), ([20000, 12345], 4097, 1, 600, 128), ([40], 64, 1, 1, 16),
])
def test_selected_rows(kind, lens, keep, first, last, page):
    n, Hkv, mp = len(lens), 3, max(1, -(-max(lens) // page))
    p = PagedPair(n, Hkv, 64, Hkv, page=page, max_pages=mp, scores=True, seed=keep)
    g = torch.Generator().manual_seed(len(lens) + keep)
    s = torch.randn(p.dev.scores.shape, generator=g).exp() ** 3
    if kind == "ties":
        s = (s * 4).round() / 4
    if kind == "equal":
        s = torch.full_like(s, 0.125)
    if kind == "zeros":
        s = torch.where(torch.rand(s.shape, generator=g) < 0.9, torch.where(torch.rand(s.shape, generator=g) < 0.5, 0.0, -0.0), s)
    if kind == "odd":
        odd = torch.tensor([float("nan"), float("inf"), float("-inf"), -1.0, 1e-42, -1e-42, 3.4e38])
        s = torch.where(torch.rand(s.shape, generator=g) < 0.5, odd[torch.randint(0, 7, s.shape, generator=g)], s)
    p.dev.scores.copy_(s)
    rows = p.dev.select_rows(p.tables, i32(lens), keep, n_first=first, n_last=last).cpu().numpy()
    sc = s.numpy()
    for b, L in enumerate(lens):
        r = np.arange(L)
        mine = sc[p.tab[b, r // page], :, r % page]
        for h in range(Hkv):
            want = list(range(L)) if L <= keep else chosen(mine[:, h], keep, first, last)
            assert rows[b, h].tolist() == want + [-1] * (keep - len(want)), (b, h)
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("n,rows", [(1, 700000), (40, 3000), (200, 100)])
def test_selected_rows_of_many_blocks_and_few(n, rows):
    """One long sequence (more scores than a block's shared memory holds) and many short ones."""
    need_gpu()
    page, Hkv, keep = 256, 1, rows // 3
    mp = -(-rows // page)
    c = PagedKVCache(n * mp, page, Hkv, 64, 1, max_seqs=n, max_pages=mp, pool=torch.empty(n * mp * page * 2 * 58, dtype=torch.uint8, device="cuda"), scores=True)
    tab = torch.randperm(n * mp, generator=torch.Generator().manual_seed(n)).view(n, mp).int().cuda()
    c.scores.copy_((torch.randn(c.scores.shape, device="cuda") * 50).round())
    got = c.select_rows(tab, i32([rows] * n), keep, n_first=3, n_last=5)
    s = c.scores[tab.long(), 0].reshape(n, -1)[:, :rows].clone()
    s[:, :3] = s[:, rows - 5:] = float("inf")
    want = torch.sort(torch.sort(s, dim=-1, descending=True, stable=True)[1][:, :keep], dim=-1)[0].int()
    assert torch.equal(got[:, 0], want)


# ------------------------------------------------------------------ move

def moved(p, pool, rows, lens, into):
    """The pool's bytes after rows[b][h] moved to the front of into[b]."""
    cb, cpp = P.cell_bytes(p.D, p.fmt), p.page // 16
    out = pool.reshape(p.n_pages, p.Hkv, cpp, cb).copy()
    for b, L in enumerate(lens):
        for h in range(p.Hkv):
            for i, r in enumerate(x for x in rows[b, h] if x >= 0):
                P.put_row(out[into[b, i // p.page], h, i % p.page // 16], i % 16, p.kb[b][r][h], p.vb[b][r][h], p.fmt)
    return out.reshape(-1)


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("D,Hkv,page,lens,keep", [
    (64, 2, 16, [60, 3, 33, 0], 20), (128, 1, 32, [90, 96, 31], 32), (256, 2, 16, [48, 17], 16), (128, 3, 64, [200, 64], 50),
    (64, 1, 256, [700], 333), (128, 1, 16, [40], 1), (256, 1, 32, [65, 64], 64),
])
def test_moved_rows_are_the_same_bytes(fmt, in_place, D, Hkv, page, lens, keep):
    n, mp = len(lens), -(-max(lens) // page)
    p = PagedPair(2 * n, Hkv, D, Hkv, page=page, max_pages=mp, fmt=fmt, seed=keep + D, scores=True, bounds=True)
    p.append(lens + [0] * n)
    p.dev.scores.copy_(torch.rand(p.dev.scores.shape))
    pool, old = p.dev.pool.cpu().numpy().copy(), p.dev.scores.cpu().clone()
    codes = p.dev.bounds.clone()
    tables, ld = p.tables[:n], p.lens()[:n].clone()
    rows = p.dev.select_rows(tables, ld, keep, n_first=1 if keep > 1 else 0, n_last=min(2, keep - 1))
    into = p.tab[:n] if in_place else p.tab[n:]
    new = p.dev.compact(tables, ld, rows, lens_out=ld if in_place else None, tables_out=None if in_place else p.tables[n:].contiguous())
    assert (new.data_ptr() == ld.data_ptr()) == in_place
    assert new.tolist() == [min(x, keep) for x in lens]
    r = rows.cpu().numpy()
    got, want = p.dev.pool.cpu().numpy(), moved(p, pool, r, lens, into)
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    for b in range(n):
        for h in range(Hkv):
            for i, x in enumerate(y for y in r[b, h] if y >= 0):
                old_row = old[p.tab[b, x // page], h, x % page]
                assert p.dev.scores[into[b, i // page], h, i % page] == old_row
    # bounds of the pages that now hold rows: as of pages filled anew
    fresh = p.dev.bounds.clone()
    p.dev.bounds.copy_(codes)
    p.dev.update_bounds(torch.from_numpy(into).cuda().contiguous(), new, keep)
    assert torch.equal(p.dev.bounds, fresh)
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("fmt", [Q8, F8])
def test_many_windows(in_place, fmt):
    """Long sequences: many windows of a cluster in place, many blocks else; rows chosen near the front, the back and anywhere."""
    need_gpu()
    n, Hkv, D, page, L, keep = 3, 2, 64, 32, 9001, 6007
    mp = -(-L // page)
    c = PagedKVCache(2 * n * mp, page, Hkv, D, Hkv, max_seqs=n, max_pages=mp, fmt=fmt, scores=True)
    g = torch.Generator().manual_seed(8)
    tab = torch.randperm(2 * n * mp, generator=g).view(2 * n, mp).int().cuda()
    k, v = (torch.randn(n, L, Hkv, D, generator=g).cuda() for _ in range(2))
    lens = i32([L, L - 7, keep + 1])
    starts = i32([0, L, 2 * L - 7, 2 * L - 7 + keep + 1])
    flat = lambda x: torch.cat([x[0], x[1, :L - 7], x[2, :keep + 1]])
    c.append(flat(k), flat(v), tab[:n], lens, starts=starts)
    r = torch.arange(L, device="cuda").float()
    c.scores[tab[:n].long()] = torch.rand(n, mp, Hkv, page, device="cuda")
    c.scores[tab[1].long()] += (torch.arange(mp * page, device="cuda") / 9001).view(mp, 1, page)
    ko, vo = (torch.empty(n, L, Hkv, D, device="cuda") for _ in range(2))
    c.read(tab[:n], lens, ko, vo)
    ko, vo = (torch.stack([x[b, L - int(lens[b]):].new_zeros(L, Hkv, D).index_copy(0, torch.arange(int(lens[b]), device="cuda"), x[b, L - int(lens[b]):]) for b in range(n)]) for x in (ko, vo))
    rows = c.select_rows(tab[:n], lens, keep, n_first=4, n_last=100)
    into = tab[:n] if in_place else tab[n:].contiguous()
    new = c.compact(tab[:n], lens, rows, tables_out=None if in_place else into)
    assert new.tolist() == [keep] * 3
    k2, v2 = (torch.empty(n, keep, Hkv, D, device="cuda") for _ in range(2))
    c.read(into, new, k2, v2)
    idx = rows.long().permute(0, 2, 1)[..., None].expand(n, keep, Hkv, D)
    assert torch.equal(k2, torch.gather(ko, 1, idx)) and torch.equal(v2, torch.gather(vo, 1, idx))
    assert c.device_error() == 0


def test_lists_that_are_wrong_leave_their_rows():
    """Entries out of range or order: the error word, and nothing but the named rows moves."""
    p = PagedPair(2, 1, 64, 1, page=16, max_pages=3, scores=True)
    p.append([40, 40])
    for bad in ([3, 3], [5, 4], [2, 40], [2, -1], [1 << 30, 7], [-5, 1]):
        pool = p.dev.pool.clone()
        rows = i32([[[1, 3, 6, 9] + bad], [[0, 1, 2, 3, 4, 5]]])
        keep = rows.shape[-1]
        p.dev.compact(p.tables, i32([40, 40]), rows)
        assert p.dev.device_error() == 1
        got = p.dev.pool.cpu().numpy()
        one = rows.cpu().numpy().copy()
        want = pool.cpu().numpy()
        good, prev = [], -1
        for i, r in enumerate(one[0, 0]):
            if r > prev and i <= r < 40:
                good.append((i, r))
            prev = r
        cells = want.reshape(p.n_pages, 1, 1, -1)
        for i, r in good:
            P.put_row(cells[p.tab[0, 0], 0, 0], i, p.kb[0][r][0], p.vb[0][r][0], Q8)
        assert np.array_equal(got, cells.reshape(-1)), bad
        p.dev.pool.copy_(pool)
        assert keep == 6


def test_bad_lengths_and_pages():
    p = PagedPair(4, 2, 64, 4, page=16, max_pages=3, scores=True)
    p.append([40, 40, 40, 40])
    tables = p.tables.clone()
    tables[2, 1] = p.n_pages
    tables[3, 0] = -1
    pool = p.dev.pool.clone()
    lens = i32([-1, 49, 40, 40])
    q = p.randn(4, 1, 4, 64).cuda()
    p.dev.scores.fill_(0.5)
    p.dev.decode_scored(q, tables, lens)
    assert p.dev.device_error() == 1
    s = p.dev.scores.cpu()
    for b in range(4):
        for j in range(3):
            ok = b >= 2 and 0 <= tables[b, j] < p.n_pages and p.tab[b, j] == int(tables[b, j])
            changed = (s[p.tab[b, j]] != 0.5).any()
            assert bool(changed) == ok, (b, j)
    rows = p.dev.select_rows(tables, lens, 20, n_first=1, n_last=1)
    assert p.dev.device_error() == 1
    assert (rows[:2] == -1).all() and (rows[2:] >= 0).all()
    new = p.dev.compact(tables, lens, rows)
    assert p.dev.device_error() == 1
    assert new.tolist() == [-1, 49, 20, 20]
    same = p.dev.pool.view(p.n_pages, -1) == pool.view(p.n_pages, -1)
    mine = {int(x) for b in (2, 3) for x in p.tab[b]}
    for pg in range(p.n_pages):
        if pg not in mine:
            assert same[pg].all(), pg


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", [Q8, F8])
def test_a_servers_steps(fmt):
    """Prompt, scored draft steps with their verification, eviction when the budget is passed, appends at positions
    that go on counting: every step against the oracle, which keeps each head's rows for itself."""
    need_gpu()
    n, Hkv, Hq, D, page, T, V, budget = 2, 2, 4, 64, 16, 3, 50, 40
    mp = 8
    c = PagedKVCache(n * mp, page, Hkv, D, Hq, max_seqs=n, max_pages=mp, max_t=8, fmt=fmt, rope_dim=D, scores=True)
    r = np.random.default_rng(3)
    rnd = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))
    tab = torch.arange(n * mp).view(n, mp).int().cuda()
    lens, pos = i32([0] * n), np.zeros(n, np.int64)
    K = [[np.zeros((0, D)) for _ in range(Hkv)] for _ in range(n)]
    Vv = [[np.zeros((0, D)) for _ in range(Hkv)] for _ in range(n)]
    S = [[np.zeros(0, np.float32) for _ in range(Hkv)] for _ in range(n)]

    def append(t):
        k, v, q = rnd(n, t, Hkv, D), rnd(n, t, Hkv, D), rnd(n, t, Hq, D)
        at = pos[:, None] + np.arange(t)
        lens.add_(t)
        qr = c.append(k.cuda(), v.cuda(), tab, lens, q=q.cuda(), positions=i32(at.tolist()))
        ko, vo = torch.empty(n, t, Hkv, D, device="cuda"), torch.empty(n, t, Hkv, D, device="cuda")
        c.read(tab, lens, ko, vo)
        for b in range(n):
            turned = P.rotate(q[b].double().numpy(), at[b], D)
            assert np.abs(turned - qr[b].double().cpu().numpy()).max() <= 2.0 ** -19 * 6
            for h in range(Hkv):                       # the rows as stored (bytes are tested elsewhere)
                K[b][h] = np.concatenate([K[b][h], ko[b, :, h].double().cpu().numpy()])
                Vv[b][h] = np.concatenate([Vv[b][h], vo[b, :, h].double().cpu().numpy()])
                S[b][h] = np.concatenate([S[b][h], np.zeros(t, np.float32)])
        return qr

    def decode(q, t, decay):
        out = c.decode_scored(q, tab, lens, decay=decay)
        qd, mag = q.double().cpu().numpy(), 0.0
        s = c.scores.cpu().numpy()
        for b in range(n):
            L = len(K[b][0])
            gain = np.zeros((L, Hkv))
            for i in range(t):
                see = np.arange(L) <= L - t + i
                for h in range(Hq):
                    g = h // (Hq // Hkv)
                    o, m = P.attend(qd[b, i, h], K[b][g], Vv[b][g], see)
                    err = np.abs(out[b, i, h].double().cpu().numpy() - o)
                    assert (err <= 2.0 ** -16 * (m + 10.0)).all()
                    gain[:, g] += P.weights(qd[b, i, h], K[b][g], see)
            at = np.arange(L)
            mine = s[tab[b].cpu().numpy()[at // page], :, at % page]
            near(mine, np.stack(S[b], 1), gain, decay)
            for h in range(Hkv):
                S[b][h] = mine[:, h].copy()

    append(30)
    pos += 30
    decode(torch.from_numpy(r.standard_normal((n, 8, Hq, D)).astype(np.float32)).cuda(), 8, 0.0)
    evictions = 0
    for step in range(14):
        q = append(T)
        decode(q, T, 1.0)
        z = rnd(n, T, V)
        t, d = torch.softmax(z, -1), torch.softmax(z[:, :T - 1] + 0.3 * rnd(n, T - 1, V), -1)
        tok = torch.multinomial(d.reshape(-1, V), 1, generator=torch.Generator().manual_seed(step)).view(n, T - 1).int()
        u = torch.from_numpy(r.random((n, T)).astype(np.float32))
        accept, token = verify(t.cuda(), d.cuda(), tok.cuda(), u.cuda(), lens=lens)
        for b in range(n):
            a, x = P.verify(t[b].double().numpy(), d[b].double().numpy(), tok[b].numpy(), u[b].double().numpy())
            assert (accept[b].item(), token[b].item()) == (a, x)
            cut = len(K[b][0]) - (T - a)
            for h in range(Hkv):
                K[b][h], Vv[b][h], S[b][h] = K[b][h][:cut], Vv[b][h][:cut], S[b][h][:cut]
            pos[b] += a
        assert lens.tolist() == [len(K[b][0]) for b in range(n)]
        if max(lens.tolist()) > budget:
            rows = c.select_rows(tab, lens, 24, n_first=2, n_last=6)
            c.compact(tab, lens, rows, lens_out=lens)
            evictions += 1
            for b in range(n):
                for h in range(Hkv):
                    L = len(K[b][h])
                    w = list(range(L)) if L <= 24 else chosen(S[b][h], 24, 2, 6)
                    assert rows[b, h].tolist() == w + [-1] * (24 - len(w))
                    K[b][h], Vv[b][h], S[b][h] = K[b][h][w], Vv[b][h][w], S[b][h][w]
    assert evictions >= 1 and c.device_error() == 0


def test_captured_steps_follow_the_lengths():
    """append at positions, scored decode, choice and move in one graph: replays give what eager calls give."""
    need_gpu()
    n, Hkv, D, page, mp, keep = 3, 2, 128, 16, 6, 48

    def make():
        c = PagedKVCache(n * mp, page, Hkv, D, 8, max_seqs=n, max_pages=mp, rope_dim=D, scores=True)
        c.pool.zero_()
        return c

    g = torch.Generator().manual_seed(4)
    tab = torch.randperm(n * mp, generator=g).view(n, mp).int().cuda()
    k0, q0 = torch.randn(n, 47, Hkv, D, generator=g).cuda(), torch.randn(n, 1, 8, D, generator=g).cuda()
    steps = [torch.randn(n, 1, Hkv, D, generator=g).cuda() for _ in range(5)]
    start = i32([47, 20, 46])
    got = []
    for captured in (False, True):
        c, lens, pos = make(), start.clone(), i32([[1000], [20], [77]])
        c.append(k0, k0, tab, i32([47] * 3))
        k, out = steps[0].clone(), torch.empty_like(q0)

        def step():
            lens.add_(1)
            q = c.append(k, k, tab, lens, q=q0, positions=pos)
            c.decode_scored(q, tab, lens, out=out)
            rows = c.select_rows(tab, lens, keep, n_first=1, n_last=8)
            c.compact(tab, lens, rows, lens_out=lens)
            pos.add_(1)

        if captured:
            graph = torch.cuda.CUDAGraph()
            state = [x.clone() for x in (lens, pos, c.pool, c.scores)]
            with torch.cuda.graph(graph):
                step()
            for x, y in zip((lens, pos, c.pool, c.scores), state):
                x.copy_(y)
        seen = []
        for x in steps:
            k.copy_(x)
            graph.replay() if captured else step()
            seen.append((lens.tolist(), out.clone()))
        got.append((seen, c.pool.clone(), c.scores.clone()))
        assert c.device_error() == 0
    (a, pa, sa), (b, pb, sb) = got
    assert [x[0] for x in a] == [x[0] for x in b] and all(torch.equal(x[1], y[1]) for x, y in zip(a, b))
    assert torch.equal(pa, pb) and torch.equal(sa, sb) and a[-1][0][0] == keep


def test_the_documented_round():
    need_gpu()
    text = (Path(__file__).resolve().parents[1] / "README.md").read_text()
    code = next(x for x in re.findall(r"```python\n(.*?)```", text, re.S) if "decode_scored" in x)
    names = {"torch": torch}
    exec(code, names)
    assert names["out"].shape == (2, 4, 32, 128) and torch.isfinite(names["out"]).all()
    assert names["lens"].tolist() == [512, 512] and names["c"].device_error() == 0
    assert all(1 <= x <= 4 for x in names["accept"].tolist()) and all(0 <= x < 1000 for x in names["token"].tolist())


def test_two_caches_on_two_streams():
    """Whole steps of two caches at once on streams of their own give what they give one after the other."""
    need_gpu()
    n, Hkv, D, page, mp, keep = 4, 2, 64, 16, 32, 200

    def make(seed):
        g = torch.Generator().manual_seed(seed)
        c = PagedKVCache(n * mp, page, Hkv, D, 8, max_seqs=n, max_pages=mp, rope_dim=D, scores=True)
        c.pool.zero_()
        tab = torch.randperm(n * mp, generator=g).view(n, mp).int().cuda()
        k, q = torch.randn(n, 400, Hkv, D, generator=g).cuda(), torch.randn(n, 1, 8, D, generator=g).cuda()
        p = torch.softmax(torch.randn(n, 3, 5000, generator=g), -1).cuda()
        tok = torch.randint(0, 5000, (n, 2), generator=g).int().cuda()
        return c, tab, k, q, p, tok, torch.rand(n, 3, generator=g).cuda(), torch.arange(400).int().cuda().expand(n, 400).contiguous()

    def step(s, stream):
        c, tab, k, q, p, tok, u, at = s
        lens = i32([400] * n)
        stream.wait_stream(torch.cuda.current_stream())
        c.append(k, k, tab, lens, positions=at, stream=stream)
        for _ in range(8):
            out = c.decode_scored(q, tab, lens, stream=stream)
            verify(p, p[:, :2], tok, u, stream=stream)
        rows = c.select_rows(tab, lens, keep, n_first=2, n_last=20, stream=stream)
        new = c.compact(tab, lens, rows, stream=stream)
        a, t = verify(p, p[:, :2], tok, u, lens=new, stream=stream)
        return out, rows, new, a, t, lens

    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    ref = []
    for seed in (1, 2):
        s = make(seed)
        r = step(s, one)
        torch.cuda.synchronize()
        ref.append([x.clone() for x in r] + [s[0].pool.clone(), s[0].scores.clone()])
    both = [make(1), make(2)]
    torch.cuda.synchronize()
    got = [step(both[0], one), step(both[1], two)]
    torch.cuda.synchronize()
    for s, r, w in zip(both, got, ref):
        for x, y in zip(list(r) + [s[0].pool, s[0].scores], w):
            assert torch.equal(x, y)


@pytest.mark.parametrize("scratch", [True, False])
@pytest.mark.parametrize("fmt", [Q8, F8])
def test_pages_beyond_four_gigabytes(fmt, scratch):
    """Pages at the end of a pool of more than 2^32 bytes give what pages at the front of a small one give."""
    need_gpu()
    n, Hkv, Hq, D, page, mp, keep = 2, 8, 8, 256, 256, 3, 300
    g = torch.Generator().manual_seed(3)
    k, v, q = (torch.randn(n, 700, Hkv, D, generator=g).cuda() for _ in range(3))
    at = torch.arange(700).int().cuda().expand(n, 700).contiguous()
    got = []
    for n_pages in (8, 5000):
        c = PagedKVCache(n_pages, page, Hkv, D, Hq, max_seqs=n, max_pages=mp, max_t=1, fmt=fmt, rope_dim=D, scores=True, score_scratch=scratch)
        assert n_pages == 8 or c.pool.numel() > 1 << 32
        last = (torch.arange(n * mp).view(n, mp).flip(0) + n_pages - 7).int().cuda()
        lens = i32([700, 513])
        c.append(k, v, last, i32([700, 700]), positions=at)
        out = c.decode_scored(q[:, :1].contiguous(), last, lens)
        scores = c.scores[last.long()].clone()
        rows = c.select_rows(last, lens, keep, n_first=2, n_last=30)
        new = c.compact(last, lens, rows)
        ko, vo = torch.empty(n, keep, Hkv, D, device="cuda"), torch.empty(n, keep, Hkv, D, device="cuda")
        c.read(last, new, ko, vo)
        got.append((out, scores, rows, new, ko, vo))
        assert c.device_error() == 0
        del c
    assert all(torch.equal(x, y) for x, y in zip(*got)) and got[0][3].tolist() == [keep, keep]


def test_on_another_stream():
    p = PagedPair(2, 2, 64, 4, page=16, max_pages=4, scores=True)
    p.append([60, 35])
    q, lens = p.randn(2, 1, 4, 64).cuda(), p.lens()
    ref = p.dev.decode_scored(q, p.tables, lens)
    want = p.dev.scores.clone()
    p.dev.scores.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = p.dev.decode_scored(q, p.tables, lens, stream=s)
    rows = p.dev.select_rows(p.tables, lens, 20, stream=s)
    new = p.dev.compact(p.tables, lens, rows, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and new.tolist() == [20, 20]
    r = rows.cpu().numpy()
    for b in range(2):
        for h in range(2):
            i = np.arange(20)
            old = want.cpu().numpy()[p.tab[b, r[b, h] // 16], h, r[b, h] % 16]
            assert np.array_equal(p.dev.scores.cpu().numpy()[p.tab[b, i // 16], h, i % 16], old)


def test_refusals():
    p = PagedPair(2, 2, 64, 4, page=16, max_pages=4)
    p.append([20, 20])
    q, lens = p.randn(2, 1, 4, 64).cuda(), p.lens()
    for call in (lambda: p.dev.decode_scored(q, p.tables, lens), lambda: p.dev.select_rows(p.tables, lens, 4)):
        with pytest.raises(B.KvqError) as e:                            # no score buffer
            call()
        assert e.value.status == B.KVQ_EINVAL
    rows = i32([[[0, 1], [2, 3]], [[4, 5], [6, 7]]])
    with pytest.raises(B.KvqError):
        B.kvq_paged_compact(p.dev.handle, p.tables.data_ptr(), lens.data_ptr(), 2, rows.data_ptr(), 2, p.tables.data_ptr(), lens.data_ptr())
    with pytest.raises(B.KvqError):
        B.kvq_paged_compact(p.dev.handle, p.tables.data_ptr(), lens.data_ptr(), 2, rows.data_ptr(), 2, None, None)
    buf = torch.zeros(p.n_pages, 2, 16, device="cuda")
    with pytest.raises(B.KvqError):
        B.kvq_paged_set_scores(p.dev.handle, buf.data_ptr() + 4)
    for off in ((2, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 2, 0, 0), (0, 0, 0, 3, 0), (0, 0, 0, 0, 2)):      # not on their elements
        at = [x.data_ptr() + o for x, o in zip((p.tables, lens, rows, p.tables.clone(), lens.clone()), off)]
        with pytest.raises(B.KvqError):
            B.kvq_paged_compact(p.dev.handle, at[0], at[1], 2, at[2], 2, at[3], at[4])
    B.kvq_paged_set_scores(p.dev.handle, buf.data_ptr())
    for at, queries in ((4, 1), (0, 0), (0, 9), (0, -1)):
        with pytest.raises(B.KvqError):
            B.kvq_paged_set_score_scratch(p.dev.handle, buf.data_ptr() + at, queries)
    for bad in (dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")), dict(out=q), dict(softcap=-1.0), dict(window=-1)):
        with pytest.raises((ValueError, B.KvqError)):
            p.dev.decode_scored(q, p.tables, lens, **bad)
    for bad in (dict(keep=0), dict(keep=4, n_first=-1), dict(keep=4, n_last=-1), dict(keep=4, n_first=3, n_last=2)):
        with pytest.raises((ValueError, RuntimeError, B.KvqError)):
            p.dev.select_rows(p.tables, lens, **bad)
    for bad in (dict(rows=rows.long()), dict(rows=rows[:1]), dict(lens_out=i32([0])), dict(tables_out=p.tables[:, :2])):
        with pytest.raises(ValueError):
            p.dev.compact(p.tables, lens, **dict(dict(rows=rows), **bad))
    assert (buf == 0).all() and p.dev.device_error() == 0
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 2, 64, 4, max_seqs=1, max_pages=2, scores_buf=torch.zeros(4, 2, 8, device="cuda"))
