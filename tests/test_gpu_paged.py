"""Paged cache on the GPU against the fp64 oracle: bytes of the append, the
rotation, decode, shared prefixes, key bounds, selection, listed pages."""

import re
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300.cache import PagedKVCache
from tests.kvq_testutil import need_gpu
from tests.paged_testutil import PagedPair, assert_attention

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
Q8, F8 = "q8_0/q5_1", "e4m3"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("D,page,Hkv", [(64, 16, 3), (128, 32, 2), (256, 64, 1), (128, 128, 5)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_append_writes_the_oracles_bytes_and_nothing_else(fmt, D, page, Hkv, dtype):
    p = PagedPair(4, Hkv, D, Hkv, page=page, max_pages=2, fmt=fmt, seed=D + page)
    for counts in ([1, 0, 17, 5], [0, 3, 1, 0], [13, 1, 0, 2]):
        counts = [min(c, 2 * page - len(p.k[b])) for b, c in enumerate(counts)]
        p.append(counts, dtype=dtype)
    got = p.dev.pool.cpu().numpy()
    want = p.expected_pool()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    assert p.dev.device_error() == 0


def test_append_ties_and_constant_blocks():
    """Scales and codes on rounding borders, zero and constant blocks."""
    p = PagedPair(1, 1, 64, 1, page=32, max_pages=1)
    rows = []
    for i in range(12):
        d = 2.0 ** (i - 20)
        x = np.zeros(64, np.float32)
        x[0] = 127 * d
        x[1:30] = (np.arange(29) - 14 + 0.5) * d                 # halves of a step
        x[32:] = {0: 0.0, 1: -3.25}.get(i % 3, d * 31 * (np.arange(32) / 62))
        rows.append(x)
    k = torch.from_numpy(np.stack(rows)[:, None])
    v = k.flip(-1).contiguous()
    p.note(0, k.numpy(), v.numpy())
    p.dev.append(k[None].cuda(), v[None].cuda(), p.tables, i32([12]))
    assert np.array_equal(p.dev.pool.cpu().numpy(), p.expected_pool())


@pytest.mark.parametrize("fmt,D,rot,inter,dtype", [
    (Q8, 128, 128, False, BF), (Q8, 128, 64, True, F32), (F8, 64, 16, False, F32), (Q8, 256, 256, False, F32),
    (F8, 256, 32, True, BF), (Q8, 64, 64, True, BF), (Q8, 64, 32, False, F32),
])
def test_rotation_against_the_definition(fmt, D, rot, inter, dtype):
    n, Hkv, Hq, page = 3, 2, 6, 64
    p = PagedPair(n, Hkv, D, Hq, page=page, max_pages=3, fmt=fmt, rope_dim=rot, rope_interleaved=inter)
    ctx, T = [0, 100, 183], 9
    k, v, q = (p.randn(n, T, H, D).to(dtype) for H in (Hkv, Hkv, Hq))
    lens = i32([c + T for c in ctx])
    q_out = p.dev.append(k.cuda(), v.cuda(), p.tables, lens, q=q.cuda())
    pos = np.concatenate([np.arange(c, c + T) for c in ctx])
    flat = lambda x: x.double().numpy().reshape(n * T, -1, D)
    qr, kr = P.rotate(flat(q), pos, rot, inter), P.rotate(flat(k), pos, rot, inter)
    size = np.abs(flat(q)).max()
    # q: angles good to 2^-24 of a turn (2^-21 radians), f32 products, the output's rounding
    tol = 2.0 ** -19 * size + (2.0 ** -8 if dtype == BF else 2.0 ** -24) * np.abs(qr)
    assert (np.abs(flat(q_out.cpu()) - qr) <= tol).all()
    ko, vo = torch.empty(n, T, Hkv, D, device="cuda"), torch.empty(n, T, Hkv, D, device="cuda")
    p.dev.read(p.tables, lens, ko, vo)
    got = flat(ko.cpu())
    if fmt == F8:
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(kr), 2.0 ** -6)))) * 2.0 ** -4      # half a step
    else:
        am = np.abs(kr).reshape(n * T, Hkv, -1, 32).max(-1, keepdims=True)
        step = np.broadcast_to(am / 127 * (0.5 + 0.0 * am) * (1 + 2.0 ** -9) + am * 2.0 ** -11, (*am.shape[:3], 32)).reshape(kr.shape)
    assert (np.abs(got - kr) <= step * (1 + 1e-6) + 2.0 ** -19 * size).all()
    assert np.array_equal(flat(vo.cpu()), P.values(P.blocks(flat(v), fmt, "v"), fmt, "v").astype(np.float32))


def test_rotation_at_far_positions_and_given_frequencies():
    """Positions near 2^24, frequencies of the caller's own."""
    need_gpu()
    D, page, far = 64, 256, (1 << 24) - 5
    freq = [1.0, 0.75, 0.1, 0.033] + [0.001 * i for i in range(12)]
    c = PagedKVCache(2, page, 1, D, 2, max_seqs=1, max_pages=1 << 16, rope_dim=32, rope_freq=freq)
    tab = torch.zeros(1, 1 << 16, dtype=torch.int32, device="cuda")
    k = torch.randn(1, 3, 1, D, generator=torch.Generator().manual_seed(1))
    q = c.append(k.cuda(), k.cuda(), tab, i32([far]), q=k.cuda())
    want = P.rotate(k.double().numpy().reshape(3, 1, D), far - 3 + np.arange(3), 32, freq=freq)
    assert np.abs(q.cpu().double().numpy().reshape(3, 1, D) - want).max() <= 2.0 ** -19 * 4
    assert c.device_error() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
def test_fused_projection_slices_and_rotation_in_place(dtype):
    """k, v, q as slices of one projection; q rotated in place; the rest of the buffers untouched."""
    Hkv, Hq, D, n, T = 2, 4, 128, 2, 5
    p = PagedPair(n, Hkv, D, Hq, page=16, max_pages=2, rope_dim=128)
    qkv = p.randn(n, T, (Hq + 2 * Hkv) * D + 8).to(dtype).cuda()
    before = qkv.clone()
    cut = lambda lo, H: qkv[..., lo:lo + H * D].unflatten(-1, (H, D))
    q, k, v = cut(0, Hq), cut(Hq * D, Hkv), cut((Hq + Hkv) * D, Hkv)
    lens = i32([T, T + 3])
    one = p.dev.append(k, v, p.tables, lens, q=q)
    pool = p.dev.pool.clone()
    assert torch.equal(qkv, before)
    dense = q.contiguous()
    two = p.dev.append(k.contiguous(), v.contiguous(), p.tables, lens, q=dense, q_out=dense)
    assert two.data_ptr() == dense.data_ptr() and torch.equal(one, two) and torch.equal(pool, p.dev.pool)
    with pytest.raises(B.KvqError):
        B.kvq_paged_append(p.dev.handle, k.data_ptr(), k.stride(1), v.data_ptr(), v.stride(1), q.data_ptr(),
                           q.stride(1), q.data_ptr(), Hq, 1 if dtype == BF else 0, p.tables.data_ptr(),
                           lens.data_ptr(), n, T, None, n * T)


def test_packed_rows_outside_the_starts_are_left_alone():
    p = PagedPair(3, 1, 64, 2, page=16, max_pages=2, rope_dim=64)
    k, q = p.randn(20, 1, 64).cuda(), p.randn(20, 2, 64).cuda()
    q_out = torch.full_like(q, 7.0)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    starts, lens = i32([2, 9, 9, 16]), i32([7, 4, 11])
    p.dev.append(k, k, p.tables, lens, starts=starts, q=q, q_out=q_out)
    p.dev.read(p.tables, lens, ko, vo, starts=starts)
    for x in (q_out, ko, vo):
        assert (x[:2] == 7).all() and (x[16:] == 7).all() and (x[2:16] != 7).any(-1).all()
    p.dev.append(k[:0], k[:0], p.tables, lens, starts=i32([0, 0, 0, 0]))
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,Hkv,page,rot,inter", [(64, 3, 16, 64, False), (128, 2, 32, 96, False), (256, 1, 64, 256, False),
                                                  (64, 1, 128, 32, True), (128, 5, 16, 0, False), (256, 2, 32, 48, True)])
@pytest.mark.parametrize("ctx,counts", [([3, 5, 0, 8, 16, 15], [37, 0, 1, 8, 64, 9]), ([0, 7, 1, 2, 30, 0, 3, 9], [70, 1, 1, 2, 0, 3, 1, 2]),
                                        ([0], [16]), ([9, 24], [7, 40])])
def test_many_rows_a_sequence_write_what_single_steps_write(fmt, dtype, D, Hkv, page, rot, inter, ctx, counts):
    n, Hq = len(ctx), 3 * Hkv
    kw = dict(page=page, max_pages=-(-96 // page), fmt=fmt, rope_dim=rot, rope_interleaved=inter)
    a, b = (PagedPair(n, Hkv, D, Hq, seed=3, **kw) for _ in range(2))
    front, rows = 2, sum(counts)
    k, v, q = (a.randn(front + rows + 3, H, D).to(dtype).cuda() for H in (Hkv, Hkv, Hq))
    starts = front + np.concatenate([[0], np.cumsum(counts)])
    lens = np.array(ctx) + np.array(counts)
    out = torch.full_like(q, 7.0)
    a.dev.append(k, v, a.tables, i32(lens.tolist()), starts=i32(starts.tolist()), q=q, q_out=out)
    want = torch.full_like(q, 7.0)
    for i in range(n):
        for r in range(counts[i]):
            at = slice(int(starts[i]) + r, int(starts[i]) + r + 1)
            want[at] = b.dev.append(k[at][None], v[at][None], b.tables[i:i + 1], i32([ctx[i] + r + 1]), q=q[at][None])[0]
    assert torch.equal(a.dev.pool, b.dev.pool) and torch.equal(out, want)
    assert a.dev.device_error() == 0 and b.dev.device_error() == 0


# ------------------------------------------------------------------ decode

LENS = [0, 1, 15, 16, 17, 40, 63]


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,Hkv,Hq,page,T,kw", [
    (128, 2, 8, 16, 1, {}),
    (64, 1, 7, 32, 1, dict(sinks=True)),
    (64, 2, 2, 16, 3, dict(window=5)),
    (128, 1, 5, 64, 4, dict(sinks=True, window=20)),
    (256, 1, 4, 16, 8, dict(softcap=3.0)),
    (256, 2, 2, 32, 1, dict(scale=0.3)),
    (128, 1, 40, 16, 1, {}),
    (64, 3, 9, 16, 2, dict(window=1, sinks=True)),
])
def test_decode(fmt, dtype, D, Hkv, Hq, page, T, kw):
    p = PagedPair(len(LENS), Hkv, D, Hq, page=page, max_pages=-(-64 // page), fmt=fmt, max_t=8, seed=D + T)
    p.append(LENS)
    q = p.randn(p.n, T, Hq, D).to(dtype)
    kw = dict(kw)
    sinks = p.randn(Hq) if kw.pop("sinks", False) else None
    want, mag = p.want(q, sinks=sinks, **kw)
    got = p.dev.decode(q.cuda(), p.tables, p.lens(), sinks=None if sinks is None else sinks.cuda(), **kw)
    assert_attention(p, got, want, mag)
    assert p.dev.device_error() == 0
    again = p.dev.decode(q.cuda(), p.tables, p.lens(), sinks=None if sinks is None else sinks.cuda(), **kw)
    assert torch.equal(got, again)


@pytest.mark.parametrize("fmt,dtype", [(Q8, BF), (Q8, F32), (F8, BF), (F8, F32)])
def test_decode_long_rows_cut_among_all_cta(fmt, dtype):
    """Enough rows that every CTA has several cells, of sequences of unlike lengths."""
    p = PagedPair(3, 2, 64, 8, page=64, max_pages=64, fmt=fmt, seed=5)
    p.append([4096, 33, 1500])
    q = p.randn(3, 1, 8, 64).to(dtype)
    want, mag = p.want(q)
    assert_attention(p, p.dev.decode(q.cuda(), p.tables, p.lens()), want, mag)


def test_decode_of_unlike_magnitudes():
    """Scores far apart (one row takes all), values from 1e-3 to 1e3, tiny and huge queries."""
    for seed, (ks, vs, qs) in enumerate([(1, 1e-3, 1), (30, 1, 30), (1e-4, 1e3, 1e4), (1, 1, 0.0)]):
        for dtype in (BF, F32):
            p = PagedPair(1, 1, 128, 4, page=16, max_pages=8, seed=seed)
            k, v = p.randn(100, 1, 128) * ks, p.randn(100, 1, 128) * vs
            p.note(0, k.numpy(), v.numpy())
            p.dev.append(k[None].cuda(), v[None].cuda(), p.tables, i32([100]))
            q = (p.randn(1, 1, 4, 128) * qs).to(dtype)
            want, mag = p.want(q, scale=1e-2 if ks * qs > 100 else 0.0)
            got = p.dev.decode(q.cuda(), p.tables, p.lens(), scale=1e-2 if ks * qs > 100 else 0.0)
            g = got.double().cpu().numpy()
            # scores up to 2^6 here: f32 parts leave 2^-22 * 2^9 of p; bf16 as ever
            tol = (2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag) if dtype == BF else 2.0 ** -13 * (mag + p.spread())
            assert (np.abs(g - want) <= tol + 1e-30).all(), (seed, dtype)


def test_shared_pages_of_two_tables_and_rollback():
    """Two tables over the same pages; a smaller length is a rollback."""
    p = PagedPair(1, 2, 128, 8, page=32, max_pages=4)
    p.append([90])
    tabs = p.tables.repeat(2, 1).contiguous()
    q = p.randn(2, 1, 8, 128).to(BF)
    got = p.dev.decode(q.cuda(), tabs, i32([90, 41]))
    want, mag = p.want(q[:1])
    assert_attention(p, got[:1], want, mag)
    p.k[0], p.v[0] = p.k[0][:41], p.v[0][:41]
    want, mag = p.want(q[1:])
    assert_attention(p, got[1:], want, mag)


# ------------------------------------------------------------------ shared prefix

def shared_case(sizes, prefix, suffix, fmt=Q8, D=64, Hkv=2, Hq=4, page=16, outside=0, T=1, seed=0):
    """Groups of len(sizes) sharing prefix[i] rows, then `outside` sequences without one."""
    n = sum(sizes) + outside
    longest = max(list(prefix) + [0]) + max(suffix)
    p = PagedPair(n, Hkv, D, Hq, page=page, max_pages=-(-longest // page) + 1, fmt=fmt, max_t=max(T, 1), seed=seed)
    b = 0
    for m, rows in zip(sizes, prefix):
        k, v = p.randn(rows, Hkv, D), p.randn(rows, Hkv, D)
        for i in range(m):
            if i:
                full = rows // page
                p.tab[b + i, :full] = p.tab[b, :full]
        p.tables = torch.from_numpy(p.tab).cuda()
        for i in range(m):
            p.note(b + i, k.numpy(), v.numpy())
        if rows and m:
            kk, vv = (x[None].expand(m, -1, -1, -1).contiguous().cuda() for x in (k, v))
            p.dev.append(kk, vv, p.tables[b:b + m].contiguous(), i32([rows] * m))
        b += m
    p.append([suffix[i % len(suffix)] for i in range(n)])
    starts = i32(np.concatenate([[0], np.cumsum(sizes)]).tolist())
    return p, starts, i32(list(prefix))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [
    dict(sizes=[5], prefix=[64], suffix=[3, 20]),
    dict(sizes=[3, 1, 6], prefix=[70, 33, 16], suffix=[1, 9, 30], outside=2),
    dict(sizes=[0, 4, 0], prefix=[0, 100, 20], suffix=[2], fmt=F8, T=2),
    dict(sizes=[20], prefix=[130], suffix=[1, 5], Hkv=1, Hq=8, D=128),
    dict(sizes=[9], prefix=[7], suffix=[1, 2, 40], D=256, Hkv=1, Hq=3),
])
@pytest.mark.parametrize("att", [{}, dict(window=25), dict(sinks=True, softcap=4.0)])
def test_decode_shared(dtype, kw, att):
    p, starts, prefix = shared_case(**kw)
    T = kw.get("T", 1)
    q = p.randn(p.n, T, p.Hq, p.D).to(dtype)
    att = dict(att)
    sinks = p.randn(p.Hq) if att.pop("sinks", False) else None
    want, mag = p.want(q, sinks=sinks, **att)
    sk = None if sinks is None else sinks.cuda()
    got = p.dev.decode_shared(q.cuda(), p.tables, p.lens(), starts, prefix, sinks=sk, **att)
    assert_attention(p, got, want, mag)
    assert torch.equal(got, p.dev.decode_shared(q.cuda(), p.tables, p.lens(), starts, prefix, sinks=sk, **att))
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("fmt,D,Hq,page", [(Q8, 128, 8, 64), (F8, 128, 8, 16), (Q8, 64, 16, 32), (F8, 64, 2, 128),
                                           (Q8, 256, 4, 64)])
def test_decode_shared_long_prefix_many_queries(fmt, D, Hq, page):
    """Prefixes of thousands of rows for more queries than one tile holds."""
    p, starts, prefix = shared_case(sizes=[37, 11], prefix=[1111, 2048], suffix=[1, 17, 40], fmt=fmt, D=D, Hkv=2, Hq=Hq,
                                    page=page)
    q = p.randn(p.n, 1, Hq, D).to(BF)
    want, mag = p.want(q)
    assert_attention(p, p.dev.decode_shared(q.cuda(), p.tables, p.lens(), starts, prefix), want, mag)


def test_members_shorter_than_their_prefix():
    """A member rolled back into the prefix, one of length 0, rows before position 0."""
    p, starts, prefix = shared_case(sizes=[4], prefix=[48], suffix=[6], T=3)
    lens = [54, 20, 0, 2]
    for b, L in enumerate(lens):
        p.k[b], p.v[b] = p.k[b][:L], p.v[b][:L]
    for dtype in (BF, F32):
        q = p.randn(4, 3, p.Hq, p.D).to(dtype)
        want, mag = p.want(q)
        assert_attention(p, p.dev.decode_shared(q.cuda(), p.tables, i32(lens), starts, prefix), want, mag)


# ------------------------------------------------------------------ bounds, selection, listed pages

def sparse_pair(fmt=Q8, D=64, Hkv=2, Hq=6, page=16, lens=(300, 17, 1, 0, 161), seed=3):
    p = PagedPair(len(lens), Hkv, D, Hq, page=page, max_pages=-(-max(lens) // page) + 1, fmt=fmt, max_t=3, seed=seed,
                  bounds=True)
    p.append([max(0, x - 2) for x in lens])
    p.append([min(x, 2) for x in lens], dtype=BF)
    return p


def host_bounds(p):
    NB = p.D // 32
    cut = p.n_pages * p.Hkv * NB * 64
    raw = p.dev.bounds.cpu().numpy()
    return (raw[:cut].view(np.int8).reshape(p.n_pages, p.Hkv, NB, 2, 32),
            raw[cut:cut + p.n_pages * p.Hkv * NB * 4].view(np.float32).reshape(p.n_pages, p.Hkv, NB))


@pytest.mark.parametrize("fmt,D,page", [(Q8, 64, 16), (Q8, 128, 32), (F8, 128, 64), (F8, 256, 16)])
def test_bounds_and_selection_match_the_oracle(fmt, D, page):
    p = sparse_pair(fmt, D, page=page)
    codes, ds = host_bounds(p)
    for b in range(p.n):
        for s in range(-(-len(p.k[b]) // page)):
            for h in range(p.Hkv):
                c, d = P.bounds(p.k[b][s * page:(s + 1) * page, h])
                pg = p.tab[b, s]
                assert np.array_equal(codes[pg, h], c) and np.array_equal(ds[pg, h], d), (b, s, h)
    for dtype, T, keep, first, last in [(BF, 1, 6, 1, 1), (F32, 3, 4, 0, 2), (BF, 2, 1, 1, 0), (F32, 1, 40, 2, 3),
                                        (BF, 1, 3, 0, 0)]:
        q = p.randn(p.n, T, p.Hq, D).to(dtype)
        got = p.dev.select(q.cuda(), p.tables, p.lens(), keep, n_first=first, n_last=last).cpu().numpy()
        hpk = p.Hq // p.Hkv
        for b in range(p.n):
            for t in range(T):
                np_ = max(0, -(-(len(p.k[b]) - T + t + 1) // page))
                for h in range(p.Hkv):
                    pages = p.tab[b, :np_]
                    sc = P.scores(q[b, t, h * hpk:(h + 1) * hpk].float().numpy(), codes[pages, h], ds[pages, h])
                    want = P.select(sc, keep, first, last)
                    assert got[b, t, h].tolist() == want + [-1] * (keep - len(want)), (dtype, b, t, h)
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("fmt,D,Hkv,page,dtype", [(Q8, 64, 3, 16, BF), (Q8, 128, 2, 32, F32), (F8, 256, 1, 64, BF),
                                                  (Q8, 256, 2, 16, F32), (F8, 64, 5, 32, F32)])
def test_bounds_of_single_row_appends(fmt, D, Hkv, page, dtype):
    """Steps of one row over a page's end leave what going over the pages again gives."""
    p = PagedPair(4, Hkv, D, Hkv, page=page, max_pages=4, fmt=fmt, bounds=True, rope_dim=32, seed=D + page)
    k, v = (p.randn(4, page, Hkv, D).to(dtype).cuda() for _ in range(2))
    lens = np.array([page - 3, 5, 0, 2 * page - 1])
    p.dev.append(k[:, :1].repeat(1, 2 * page, 1, 1), v[:, :1].repeat(1, 2 * page, 1, 1), p.tables, i32([2 * page] * 4))
    for step in range(page):
        lens += 1
        kk = (k[:, step:step + 1] * (1 + step % 5)).contiguous()
        p.dev.append(kk, v[:, step:step + 1].contiguous(), p.tables, i32(lens.tolist()))
        got = p.dev.bounds.clone()
        p.dev.update_bounds(p.tables, i32(lens.tolist()), 1)
        assert torch.equal(got, p.dev.bounds), step
    # a length of 0 and a bad page write nothing
    p.dev.append(kk, v[:, :1].contiguous(), p.tables, i32([0] * 4))
    assert p.dev.device_error() == 1
    p.dev.append(kk, v[:, :1].contiguous(), torch.full_like(p.tables, -1), i32([1] * 4))
    assert p.dev.device_error() == 1 and torch.equal(got, p.dev.bounds)


def test_scores_bound_the_coded_products_and_ties_go_low():
    p = sparse_pair()
    codes, ds = host_bounds(p)
    x = p.randn(1, p.D).numpy()
    for s in range(3):
        sc = P.scores(x, codes[p.tab[0, s]][None, 0], ds[p.tab[0, s]][None, 0])
        am = np.abs(x.reshape(-1, 32)).max(-1, keepdims=True)
        c = np.rint(x.reshape(-1, 32) / am * 127) * am / 127
        assert (p.k[0][s * 16:(s + 1) * 16, 0] @ c.reshape(-1) <= sc + 1e-4).all()
    # equal pages: every score ties
    q = torch.zeros(p.n, 1, p.Hq, p.D, device="cuda")
    got = p.dev.select(q, p.tables, p.lens(), 5, n_first=0, n_last=1).cpu().numpy()
    assert got[0, 0, 0].tolist() == [0, 1, 2, 3, 18]


def test_selection_over_many_pages():
    """More pages than threads of the pick, many equal scores."""
    p = PagedPair(1, 1, 64, 2, page=16, max_pages=1500, bounds=True, seed=8)
    rows = 1500 * 16 - 3
    k = torch.from_numpy(np.repeat(p.rng.integers(-2, 3, (1500, 1, 64)).astype(np.float32), 16, 0)[:rows])
    p.dev.append(k[None].cuda(), k[None].cuda(), p.tables, i32([rows]))
    codes, ds = host_bounds(p)
    q = torch.zeros(1, 1, 2, 64)
    q[..., 0] = 1.0
    for keep in (2, 700, 1499, 1500, 1600):
        got = p.dev.select(q.cuda(), p.tables, i32([rows]), keep).cpu().numpy()[0, 0, 0].tolist()
        want = P.select(P.scores(q[0, 0].numpy(), codes[p.tab[0], 0], ds[p.tab[0], 0]), keep, 1, 1)
        assert got == want + [-1] * (keep - len(want))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt,D,page,T", [(Q8, 64, 16, 1), (Q8, 128, 32, 3), (F8, 256, 64, 1), (F8, 64, 16, 2)])
def test_decode_over_selected_and_given_pages(dtype, fmt, D, page, T):
    p = sparse_pair(fmt, D, page=page)
    q = p.randn(p.n, T, p.Hq, D).to(dtype)
    sinks = p.randn(p.Hq)
    pages = p.dev.select(q.cuda(), p.tables, p.lens(), 4)
    want, mag = p.want(q, pages=pages.cpu().numpy(), sinks=sinks, softcap=6.0)
    got = p.dev.decode_sparse(q.cuda(), p.tables, p.lens(), pages, sinks=sinks.cuda(), softcap=6.0)
    assert_attention(p, got, want, mag)
    # a list of the caller's own: out of order, holes, one page twice, pages behind the length, nothing at all
    own = torch.full((p.n, T, p.Hkv, 6), -1, dtype=torch.int32)
    own[0, ..., 0], own[0, ..., 2], own[0, ..., 3], own[0, ..., 5] = 3, 0, 3, p.max_pages - 1
    own[1, ..., 4] = 0
    want, mag = p.want(q, pages=own.numpy())
    assert_attention(p, p.dev.decode_sparse(q.cuda(), p.tables, p.lens(), own.cuda()), want, mag)
    assert p.dev.device_error() == 0


# ------------------------------------------------------------------ bad arrays, streams, graphs, a whole run

def test_bad_pages_and_lengths_are_reported_and_contained():
    p = PagedPair(3, 1, 64, 2, page=16, max_pages=3, bounds=True)
    p.append([20, 40, 33])
    q = p.randn(3, 1, 2, 64).to(BF)
    good = p.dev.decode(q.cuda(), p.tables, p.lens())
    assert p.dev.device_error() == 0
    for bad_page in (-1, p.n_pages, 1 << 30):
        tab = p.tables.clone()
        tab[1, 1] = bad_page
        got = p.dev.decode(q.cuda(), tab, p.lens())
        assert p.dev.device_error() == 1 and p.dev.device_error() == 0
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2]) and torch.isfinite(got).all()
    for bad_len in (-1, 49, 1 << 30):
        lens = i32([20, bad_len, 33])
        got = p.dev.decode(q.cuda(), p.tables, lens)
        assert p.dev.device_error() == 1
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2]) and (got[1] == 0).all()
        before = p.dev.pool.clone()
        p.dev.append(p.randn(3, 1, 1, 64).cuda(), p.randn(3, 1, 1, 64).cuda(), p.tables, i32([1, bad_len, 1]),)
        assert p.dev.device_error() == 1
        p.dev.pool.copy_(before)
        p.dev.select(q.cuda(), p.tables, lens, 2)
        assert p.dev.device_error() == 1
    pages = torch.zeros(3, 1, 1, 2, dtype=torch.int32, device="cuda")
    pages[1, 0, 0, 1] = 3
    p.dev.decode_sparse(q.cuda(), p.tables, p.lens(), pages)
    assert p.dev.device_error() == 1
    for starts, prefix in (([0, 4], [16]), ([2, 1], [16]), ([-1, 2], [16]), ([0, 2], [999]), ([0, 2], [-5])):
        got = p.dev.decode_shared(q.cuda(), p.tables, p.lens(), i32(starts), i32(prefix))
        assert p.dev.device_error() == 1 and torch.isfinite(got).all()


def test_graph_replays_follow_lengths_tables_and_inputs():
    p = PagedPair(2, 2, 128, 8, page=16, max_pages=8, bounds=True, rope_dim=0, seed=12)
    p.append([30, 64])
    k, v = torch.zeros(2, 1, 2, 128, device="cuda"), torch.zeros(2, 1, 2, 128, device="cuda")
    q = torch.zeros(2, 1, 8, 128, device="cuda", dtype=BF)
    lens, gs, pre = p.lens(), i32([0, 2]), i32([0])

    def step():
        p.dev.append(k, v, p.tables, lens)
        pages = p.dev.select(q, p.tables, lens, 3)
        return (p.dev.decode(q, p.tables, lens), p.dev.decode_sparse(q, p.tables, lens, pages), pages,
                p.dev.decode_shared(q, p.tables, lens, gs, pre))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens.add_(1)
    with torch.cuda.stream(side):
        step()                      # also the first calls of every kernel
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(6):
        kn, vn, qn = p.randn(2, 1, 2, 128), p.randn(2, 1, 2, 128), p.randn(2, 1, 8, 128).to(BF)
        for b in range(2):
            p.note(b, kn[b].numpy(), vn[b].numpy())
        k.copy_(kn), v.copy_(vn), q.copy_(qn), lens.copy_(p.lens())
        g.replay()
        want, mag = p.want(qn)
        assert_attention(p, outs[0], want, mag, f"dense {i}")
        assert_attention(p, outs[3], want, mag, f"shared {i}")
        want, mag = p.want(qn, pages=outs[2].cpu().numpy())
        assert_attention(p, outs[1], want, mag, f"sparse {i}")
    assert p.dev.device_error() == 0


def test_captured_steps_over_a_shared_prefix():
    """Append, shared decode and dense decode in one graph, with more queries a group than a
    slice holds: each replay sees its own step's rows and queries."""
    p, starts, prefix = shared_case(sizes=[9, 7], prefix=[200, 64], suffix=[1, 9, 30], Hkv=2, Hq=8, D=64)
    n, steps = p.n, 12
    k, v = torch.zeros(n, 1, 2, 64, device="cuda", dtype=BF), torch.zeros(n, 1, 2, 64, device="cuda", dtype=BF)
    q, lens = torch.zeros(n, 1, 8, 64, device="cuda", dtype=BF), p.lens()
    data = [(p.randn(n, 1, 2, 64).to(BF).cuda(), p.randn(n, 1, 2, 64).to(BF).cuda(), p.randn(n, 1, 8, 64).to(BF).cuda())
            for _ in range(steps)]
    pool, first = p.dev.pool.clone(), lens.clone()

    def step():
        r = p.dev.append(k, v, p.tables, lens, q=q)
        return p.dev.decode_shared(r, p.tables, lens, starts, prefix), p.dev.decode(r, p.tables, lens)

    eager = []
    for a, b, c in data:
        k.copy_(a), v.copy_(b), q.copy_(c), lens.add_(1)
        torch.cuda.synchronize()
        eager.append([x.clone() for x in step()])
        torch.cuda.synchronize()
    # two steps a graph, so that kernels of one follow those of the other with nothing between
    ins = [[torch.zeros_like(x) for x in (k, v, q)] + [torch.zeros_like(lens)] for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = []
        for a, b, c, m in ins:
            r = p.dev.append(a, b, p.tables, m, q=c)
            outs.append((p.dev.decode_shared(r, p.tables, m, starts, prefix), p.dev.decode(r, p.tables, m)))
    p.dev.pool.copy_(pool)
    for i in range(0, steps, 2):
        for u in range(2):
            for dst, src in zip(ins[u], (*data[i + u], first + (i + u + 1))):
                dst.copy_(src)
        g.replay()
        for u in range(2):
            assert torch.equal(outs[u][0], eager[i + u][0]) and torch.equal(outs[u][1], eager[i + u][1]), i + u
    for got, want in zip(eager[-1], eager[-1][::-1]):
        assert (got.float() - want.float()).abs().max() < 0.1
    assert p.dev.device_error() == 0


def test_two_caches_on_two_streams():
    a, b = PagedPair(2, 1, 64, 4, page=16, max_pages=4, seed=1), PagedPair(3, 2, 128, 4, page=32, max_pages=4, seed=2)
    for p in (a, b):
        p.append([50, 9, 64][:p.n])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    q = [p.randn(p.n, 1, p.Hq, p.D).to(BF).cuda() for p in (a, b)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, p in enumerate((a, b)):
            outs[i].append(p.dev.decode(q[i], p.tables, p.lens(), stream=s[i]))
            torch.cuda.synchronize() if _ == 0 else None
    torch.cuda.synchronize()
    for i, p in enumerate((a, b)):
        want, mag = p.want(q[i].cpu())
        for o in outs[i]:
            assert_attention(p, o, want, mag)


def test_shared_decodes_on_two_streams():
    """Both kernels of a shared decode of two caches at once, with appends between."""
    cases = [shared_case(sizes=[12], prefix=[300], suffix=[1, 40], Hkv=2, Hq=8, D=64, seed=1),
             shared_case(sizes=[5, 9], prefix=[130, 64], suffix=[9, 2], Hkv=1, Hq=4, D=128, fmt=F8, seed=2)]
    q = [p.randn(p.n, 1, p.Hq, p.D).to(BF).cuda() for p, _, _ in cases]
    lens = [p.lens() for p, _, _ in cases]
    again = [[torch.zeros(p.n, 1, p.Hkv, p.D, device="cuda") for _ in range(2)] for p, _, _ in cases]
    for (p, _, _), n, (k, v) in zip(cases, lens, again):
        p.dev.read(p.tables, n, k, v)                # the last rows, to be written over themselves
    want = [p.dev.decode_shared(x, p.tables, n, st, pre) for (p, st, pre), x, n in zip(cases, q, lens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(30):
        for i, (p, st, pre) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                if i == 1:                           # E4M3 rows give their bytes back
                    p.dev.append(*again[i], p.tables, lens[i])
                outs[i].append(p.dev.decode_shared(q[i], p.tables, lens[i], st, pre))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
        assert cases[i][0].dev.device_error() == 0


@pytest.mark.parametrize("fmt", [Q8, F8])
def test_a_serving_run(fmt):
    """A shared prompt, its sequences' own prompts, decode steps with rotation, a rollback, sparse and shared decodes."""
    n, Hkv, Hq, D, page, rot = 3, 2, 8, 64, 16, 64
    p = PagedPair(n, Hkv, D, Hq, page=page, max_pages=12, fmt=fmt, bounds=True, rope_dim=rot, max_t=4, seed=21)
    p.tab[1:, :2] = p.tab[0, :2]
    p.tables = torch.from_numpy(p.tab).cuda()
    lens = np.zeros(n, np.int64)

    def feed(counts, which=None):
        """Append counts rows; the oracle notes what the device stored (its codes of rotated keys are
        checked against the definition elsewhere)."""
        nonlocal lens
        lens = lens + counts
        T = int(counts[0])
        k, v, q = p.randn(n, T, Hkv, D).to(BF), p.randn(n, T, Hkv, D).to(BF), p.randn(n, T, Hq, D).to(BF)
        if which == "same":
            k, v = k[:1].expand(n, -1, -1, -1).contiguous(), v[:1].expand(n, -1, -1, -1).contiguous()
        dl = i32(lens.tolist())
        q = p.dev.append(k.cuda(), v.cuda(), p.tables, dl, q=q.cuda())
        ko, vo = torch.empty(n, T, Hkv, D, device="cuda"), torch.empty(n, T, Hkv, D, device="cuda")
        p.dev.read(p.tables, dl, ko, vo)
        for b in range(n):
            p.k[b] = np.concatenate([p.k[b], ko[b].double().cpu().numpy()])
            p.v[b] = np.concatenate([p.v[b], vo[b].double().cpu().numpy()])
        return q, dl

    feed([32] * n, "same")
    feed([21] * n)
    for step in range(5):
        q, dl = feed([1] * n if step != 2 else [4] * n)
        want, mag = p.want(q.cpu())
        assert_attention(p, p.dev.decode(q, p.tables, dl), want, mag, f"dense {step}")
        assert_attention(p, p.dev.decode_shared(q, p.tables, dl, i32([0, n]), i32([32])), want, mag, f"shared {step}")
        pages = p.dev.select(q, p.tables, dl, 3)
        want, mag = p.want(q.cpu(), pages=pages.cpu().numpy())
        assert_attention(p, p.dev.decode_sparse(q, p.tables, dl, pages), want, mag, f"sparse {step}")
        if step == 2:                                  # reject some of the draft rows
            for b, cut in enumerate((3, 0, 2)):
                lens[b] -= cut
                p.k[b], p.v[b] = p.k[b][:lens[b]], p.v[b][:lens[b]]
    assert p.dev.device_error() == 0


# ------------------------------------------------------------------ sizes and calls at the ends of the ranges

@pytest.mark.parametrize("fmt,D,Hq,dtype", [(F8, 256, 16, BF), (F8, 256, 2, F32), (Q8, 128, 12, BF), (F8, 64, 3, BF)])
def test_as_many_sequences_as_a_call_takes(fmt, D, Hq, dtype):
    """1024 sequences, then 1024 groups of one over them, then 2048 listed rows."""
    n = 1024
    p = PagedPair(n, 1, D, Hq, page=16, max_pages=2, fmt=fmt, max_t=2, bounds=True, seed=D + Hq)
    p.append([int(x) for x in p.rng.integers(0, 33, n)])
    q = p.randn(n, 1, Hq, D).to(dtype)
    want, mag = p.want(q)
    got = p.dev.decode(q.cuda(), p.tables, p.lens())
    assert p.dev.device_error() == 0
    assert_attention(p, got, want, mag)
    got = p.dev.decode_shared(q.cuda(), p.tables, p.lens(), i32(list(range(n + 1))), i32([16] * n))
    assert p.dev.device_error() == 0
    assert_attention(p, got, want, mag, "groups of one")
    q = p.randn(n, 2, Hq, D).to(dtype)
    pages = p.dev.select(q.cuda(), p.tables, p.lens(), 2)
    want, mag = p.want(q)
    got = p.dev.decode_sparse(q.cuda(), p.tables, p.lens(), pages)
    assert p.dev.device_error() == 0
    assert_attention(p, got, want, mag, "every page listed")


@pytest.mark.parametrize("fmt", [Q8, F8])
def test_a_pool_beyond_32_bits(fmt):
    """The same rows in a small pool and at both ends of one of more than 2^32 bytes."""
    torch.manual_seed(1)
    cfg = dict(page_rows=256, n_kv_heads=8, head_dim=256, max_q_heads=16, max_seqs=2, max_pages=2, fmt=fmt, bounds=True,
               rope_dim=64)
    small, big = PagedKVCache(4, **cfg), PagedKVCache(5200, **cfg)
    assert big.sizes.pool > 2 ** 32
    k, v = (torch.randn(2, 500, 8, 256, device="cuda").to(BF) for _ in range(2))
    q, lens = torch.randn(2, 1, 16, 256, device="cuda").to(BF), i32([500, 500])
    outs = []
    for c, tab in ((small, [[0, 1], [2, 3]]), (big, [[5199, 0], [2600, 5198]])):
        tab = i32(tab)
        c.append(k, v, tab, lens)
        ko, vo = torch.empty(2, 3, 8, 256, device="cuda"), torch.empty(2, 3, 8, 256, device="cuda")
        c.read(tab, lens, ko, vo)
        pages = c.select(q, tab, lens, 1, n_first=0, n_last=0)
        outs.append([c.decode(q, tab, lens), c.decode_sparse(q, tab, lens, pages), pages, ko, vo,
                     c.decode_shared(q, tab[:1].expand(2, -1).contiguous(), lens, i32([0, 2]), i32([256]))])
        assert c.device_error() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_one_row_through_long_ones():
    """Every length around a cell, a page and the pages that one lookup takes."""
    lens = [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 511, 512, 513, 527, 1023, 1025]
    p = PagedPair(len(lens), 1, 64, 4, page=32, max_pages=33, seed=8)
    p.append(lens)
    for dtype in (BF, F32):
        q = p.randn(p.n, 1, 4, 64).to(dtype)
        want, mag = p.want(q)
        assert_attention(p, p.dev.decode(q.cuda(), p.tables, p.lens()), want, mag)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sinks_of_no_weight_and_of_all(dtype):
    """A sink of -inf is none, also where no row is visible; a huge one takes everything."""
    p = PagedPair(3, 1, 64, 4, page=16, max_pages=4, max_t=2)
    p.append([40, 0, 1])
    q = p.randn(3, 2, 4, 64).to(dtype)
    plain, mag = p.want(q)
    sinks = torch.tensor([-float("inf"), 0.5, 1e4, -1e4])
    got = p.dev.decode(q.cuda(), p.tables, p.lens(), sinks=sinks.cuda())
    want, _ = p.want(q, sinks=torch.tensor([-1e9, 0.5, 1e4, -1e9]))
    assert_attention(p, got, want, mag)
    assert (got[1] == 0).all() and (got[:, :, 2] == 0).all()
    shared = p.dev.decode_shared(q.cuda(), p.tables, p.lens(), i32([0, 1]), i32([32]), sinks=sinks.cuda())
    assert_attention(p, shared, want, mag, "shared")


def test_a_query_that_is_not_a_number_stays_alone():
    """NaN and inf in one query head leave every other output as it was."""
    p = PagedPair(2, 1, 128, 8, page=16, max_pages=8, max_t=2, bounds=True)
    p.append([100, 128])
    for dtype in (BF, F32):
        q = p.randn(2, 2, 8, 128).to(dtype).cuda()
        bad = q.clone()
        bad[0, 1, 3, 5], bad[0, 1, 6, 0] = float("nan"), float("inf")
        args = (p.tables, p.lens())
        for call in (lambda x: p.dev.decode(x, *args),
                     lambda x: p.dev.decode_shared(x, *args, i32([0, 2]), i32([0]))):
            a, b = call(q), call(bad)
            a[0, 1, 3], b[0, 1, 3], a[0, 1, 6], b[0, 1, 6] = 0, 0, 0, 0
            assert torch.equal(a, b)
        pages = p.dev.select(bad, *args, 3)
        assert torch.equal(pages[1], p.dev.select(q, *args, 3)[1])
        assert ((pages >= 0) & (pages < 8)).all()
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_rows_that_are_not_finite_stay_with_the_queries_that_see_them(fmt, dtype, bad):
    """Draft rows and rows before a window: queries that do not see them give the same bits."""
    Hkv, Hq, D, T = 1, 4, 64, 4
    p = PagedPair(5, Hkv, D, Hq, page=16, max_pages=6, fmt=fmt, max_t=24, seed=13)
    lens = i32([40, 17, 80, 33, 64])
    rows = 20
    k, v = p.randn(5, rows, Hkv, D).to(dtype).cuda(), p.randn(5, rows, Hkv, D).to(dtype).cuda()
    fill_k, fill_v = p.randn(5, 96, Hkv, D).cuda(), p.randn(5, 96, Hkv, D).cuda()
    q = p.randn(5, T, Hq, D).to(dtype).cuda()
    outs = []
    for x in (0.5, bad):
        for b, L in enumerate(lens.tolist()):
            p.dev.append(fill_k[b:b + 1, :L].contiguous(), fill_v[b:b + 1, :L].contiguous(), p.tables[b:b + 1], i32([L]))
        kk, vv = k[:, -4:].clone(), v[:, -4:].clone()
        kk[:, -1], vv[:, -1] = x, x                  # the newest row: only the last query row sees it
        vv[:, -2, :, 5] = x                          # one value of the row before
        p.dev.append(kk.contiguous(), vv.contiguous(), p.tables, lens)
        outs.append([p.dev.decode(q, p.tables, lens), p.dev.decode(q, p.tables, lens, window=9),
                     p.dev.decode_shared(q, p.tables, lens, i32([0, 5]), i32([16]))])
    for a, b in zip(*outs):
        assert torch.equal(a[:, :2], b[:, :2])
        assert torch.isfinite(b[:, :3]).all()
    # a prefix whose row 8 is seen by some members only (window 8, lengths 9 .. 24)
    lens = i32([16, 24, 17, 20, 16])
    tab = p.tables.clone()
    tab[:, 0] = tab[0, 0]
    outs = []
    for x in (0.5, bad):
        kk, vv = fill_k[:1, :16].to(dtype), fill_v[:1, :16].to(dtype)
        kk[:, 8], vv[:, 8] = x, x
        p.dev.append(kk.contiguous(), vv.contiguous(), tab[:1], i32([16]))
        outs.append(p.dev.decode_shared(q, tab, lens, i32([0, 5]), i32([16]), window=8))
    see = torch.tensor([[0 <= p_ - 8 < 8 for p_ in range(L - T, L)] for L in lens.tolist()], device="cuda")
    assert see.any() and not see.all()
    assert torch.equal(outs[0][~see], outs[1][~see])


def test_output_over_the_queries():
    p = PagedPair(3, 2, 128, 8, page=16, max_pages=64, bounds=True, seed=4)
    p.append([1000, 3, 700])
    q = p.randn(3, 1, 8, 128).to(BF).cuda()
    pages = p.dev.select(q, p.tables, p.lens(), 8)
    args = (p.tables, p.lens())
    for call, more in ((p.dev.decode, ()), (p.dev.decode_sparse, (pages,)),
                       (p.dev.decode_shared, (i32([0, 1]), i32([512])))):
        own = q.clone()
        assert torch.equal(call(own, *args, *more, out=own), call(q, *args, *more))


def test_two_graphs_share_one_cache():
    """Graphs captured on the same workspace, replayed in turn, with eager calls between."""
    p = PagedPair(2, 1, 128, 20, page=16, max_pages=32, bounds=True, seed=6)
    p.append([400, 77])
    lens, gs, pre = p.lens(), i32([0, 2]), i32([0])
    q = [p.randn(2, 1, 20, 128).to(BF).cuda() for _ in range(2)]
    want = [p.dev.decode(x, p.tables, lens) for x in q]
    shared = [p.dev.decode_shared(x, p.tables, lens, gs, pre) for x in q]
    graphs, outs = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((p.dev.decode(x, p.tables, lens), p.dev.decode_shared(x, p.tables, lens, gs, pre)))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        for o in outs[i]:
            o.zero_()
        graphs[i].replay()
        p.dev.decode(q[1 - i], p.tables, lens)
        assert torch.equal(outs[i][0], want[i]) and torch.equal(outs[i][1], shared[i])


def test_calls_of_another_stream_and_its_capture():
    p = PagedPair(2, 1, 64, 4, page=16, max_pages=4, bounds=True, seed=9)
    p.append([33, 50])
    q, lens = p.randn(2, 1, 4, 64).to(BF).cuda(), p.lens()
    want = p.dev.decode(q, p.tables, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = p.dev.decode(q, p.tables, lens, stream=s)
    pages = p.dev.select(q, p.tables, lens, 4, stream=s)
    sparse = p.dev.decode_sparse(q, p.tables, lens, pages, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert_attention(p, sparse, *p.want(q.cpu()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = p.dev.decode(q, p.tables, lens)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("fmt,dtype,D,Hkv,Hq,T,n", [(Q8, BF, 64, 1, 16, 64, 1), (F8, F32, 128, 1, 8, 33, 2), (Q8, F32, 64, 2, 32, 17, 1),
                                                    (Q8, BF, 64, 128, 128, 1, 2), (F8, BF, 64, 1, 128, 1, 2)])
def test_many_query_rows_and_many_heads(fmt, dtype, D, Hkv, Hq, T, n):
    p = PagedPair(n, Hkv, D, Hq, page=32, max_pages=4, max_t=64, fmt=fmt, seed=T)
    p.append([90, 41][:n])
    q = p.randn(n, T, Hq, D).to(dtype)
    want, mag = p.want(q)
    assert_attention(p, p.dev.decode(q.cuda(), p.tables, p.lens()), want, mag)
    shared = p.dev.decode_shared(q.cuda(), p.tables, p.lens(), i32([0, 1]), i32([32]))
    assert_attention(p, shared, want, mag, "shared")
    assert p.dev.device_error() == 0


def test_table_entries_behind_a_length_are_not_read():
    """Unused entries may hold anything."""
    p, starts, prefix = shared_case(sizes=[9], prefix=[40], suffix=[3, 30], Hkv=1, Hq=4)
    b = PagedKVCache(p.n_pages, 16, 1, 64, 4, max_seqs=9, max_pages=p.max_pages, max_t=1, bounds=True, pool=p.dev.pool)
    lens = p.lens()
    tab = p.tables.clone()
    for i, x in enumerate(lens.tolist()):
        tab[i, -(-x // 16):] = (-1, 1 << 30)[i % 2]
    b.update_bounds(tab, lens, max(lens.tolist()))
    q = p.randn(9, 1, 4, 64).to(BF).cuda()
    pages = b.select(q, tab, lens, 2)
    b.decode_sparse(q, tab, lens, pages)
    want, mag = p.want(q.cpu())
    assert_attention(p, b.decode(q, tab, lens), want, mag)
    assert_attention(p, b.decode_shared(q, tab, lens, starts, prefix), want, mag, "shared")
    assert b.device_error() == 0


def test_the_documented_example():
    need_gpu()
    text = (Path(__file__).resolve().parents[1] / "README.md").read_text()
    code = next(x for x in re.findall(r"```python\n(.*?)```", text, re.S) if "PagedKVCache(" in x)
    names = {"torch": torch}
    exec(code, names)
    assert names["out"].shape == (2, 1, 32, 128) and torch.isfinite(names["out"]).all()
    assert names["c"].device_error() == 0


# ------------------------------------------------------------------ refusals

def test_refusals_of_the_calls():
    p = PagedPair(2, 2, 64, 8, page=16, max_pages=4, max_t=2, bounds=True)
    p.append([20, 40])
    c, tab, lens = p.dev, p.tables, p.lens()
    before = c.pool.clone()
    q = torch.zeros(2, 1, 8, 64, device="cuda", dtype=BF)
    kv = torch.zeros(2, 1, 2, 64, device="cuda", dtype=BF)
    pages = torch.zeros(2, 1, 2, 3, device="cuda", dtype=torch.int32)

    def refused(fn, *a, error=(ValueError, B.KvqError), **kw):
        with pytest.raises(error):
            fn(*a, **kw)

    # queries
    for bad in (q[:1], q[..., :32], q.half(), q[0], q.cpu(), q.transpose(1, 2), q[:, :, :3].contiguous(),
                q[:, :, :, :].expand(2, 1, 8, 64)[:, :0], torch.zeros(2, 3, 8, 64, device="cuda", dtype=BF),
                torch.zeros(2, 1, 16, 64, device="cuda", dtype=BF)):
        refused(c.decode, bad, tab, lens)
        refused(c.decode_shared, bad, tab, lens, i32([0, 2]), i32([16]))
        refused(c.select, bad, tab, lens, 3)
        refused(c.decode_sparse, bad, tab, lens, pages)
    shifted = torch.zeros(2 * 8 * 64 + 1, device="cuda", dtype=BF)[1:].view(2, 1, 8, 64)
    refused(c.decode, shifted, tab, lens)
    refused(c.decode, q, tab, lens, out=shifted)
    refused(c.decode, q, tab, lens, out=q.float())
    # tables and lengths
    for t, n in ((tab.long(), lens), (tab[:, :3], lens), (tab[:, :3].contiguous(), lens), (tab, lens.float()),
                 (tab, lens[:1]), (tab.cpu(), lens), (tab, lens.cpu()), (tab[:1], lens)):
        refused(c.decode, q, t, n)
        refused(c.append, kv, kv, t, n)
    many = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    refused(c.decode, torch.zeros(3, 1, 8, 64, device="cuda", dtype=BF), many, i32([0, 0, 0]))
    # numbers
    for kw in (dict(window=-1), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
               dict(softcap=1e-35), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-35),
               dict(sinks=torch.zeros(7, device="cuda")), dict(sinks=torch.zeros(8)),
               dict(sinks=torch.zeros(8, device="cuda", dtype=BF))):
        refused(c.decode, q, tab, lens, **kw)
    # groups
    refused(c.decode_shared, q, tab, lens, i32([0]), i32([]))
    refused(c.decode_shared, q, tab, lens, i32([0, 1, 2, 2]), i32([0, 0, 0]))
    refused(c.decode_shared, q, tab, lens, i32([0, 2]).long(), i32([0]))
    refused(c.decode_shared, q, tab, lens, i32([0, 1, 2]), i32([0]))
    # selection and lists
    for kw in (dict(keep=0), dict(keep=1), dict(keep=3, n_first=2, n_last=2), dict(keep=3, n_first=-1),
               dict(keep=3, n_last=-1)):
        refused(c.select, q, tab, lens, **kw, error=(ValueError, B.KvqError, RuntimeError))
    refused(c.select, q, tab, lens, 3, pages=pages.long())
    refused(c.select, q, tab, lens, 2, pages=pages)
    refused(c.decode_sparse, q, tab, lens, pages.long())
    refused(c.decode_sparse, q, tab, lens, pages[:, :, :1].contiguous())
    plain = PagedKVCache(4, 16, 2, 64, 8, max_seqs=2, max_pages=4)
    refused(plain.select, q, tab, lens, 3)
    refused(plain.update_bounds, tab, lens, 1)
    # rows
    for k, v, kw in ((kv, kv.float(), {}), (kv.half(), kv.half(), {}), (kv[:, :, :1], kv[:, :, :1], {}),
                     (kv[:1], kv[:1], {}), (kv[:, :0], kv[:, :0], {}), (kv[0], kv[0], {}), (kv, kv[:1], {}),
                     (kv, kv, dict(starts=i32([0, 1, 2]))), (kv[:, 0], kv[:, 0], dict(starts=i32([0, 2]))),
                     (kv[:, 0], kv[:, 0], dict(starts=i32([0, 1, 2]).long())), (kv.cpu(), kv.cpu(), {}),
                     (kv, kv, dict(q=q.float())), (kv, kv, dict(q=q[:1])), (kv, kv, dict(q_out=q)),
                     (kv, kv, dict(q=q, q_out=q.float())), (kv, kv, dict(q=torch.zeros(2, 1, 9, 64, device="cuda", dtype=BF))),
                     (kv.transpose(2, 3), kv, {}), (kv.expand(2, 1, 2, 64)[..., ::2], kv[..., ::2], {})):
        refused(c.append, k, v, tab, lens, **kw)
    odd = torch.zeros(2, 1, 2 * 64 + 4, device="cuda", dtype=BF)[..., :128].unflatten(-1, (2, 64))
    refused(c.append, odd, kv, tab, lens)
    refused(c.read, tab, lens, kv, kv.float())
    refused(c.read, tab, lens, kv.half(), kv.half())
    refused(c.read, tab, lens, kv.transpose(2, 3), kv)
    for bad in (torch.zeros(8, dtype=torch.uint8, device="cuda"), c.pool.view(torch.int8), c.pool.cpu()):
        refused(PagedKVCache, p.n_pages, 16, 2, 64, 8, max_seqs=2, max_pages=4, pool=bad, device="cuda:0")
    refused(PagedKVCache, 4, 16, 2, 64, 8, max_seqs=2, max_pages=4, fmt="q4")
    refused(PagedKVCache, 4, 16, 2, 64, 8, max_seqs=2, max_pages=4, rope_dim=16, rope_freq=[1.0])
    assert c.device_error() == 0 and torch.equal(c.pool, before)
