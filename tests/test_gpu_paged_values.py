"""Paged cache on the GPU: values at the ends of their ranges (keys and values
far from 1, numbers that are not finite, extreme scales and windows), against
the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300.cache import PagedKVCache
from tests.kvq_testutil import need_gpu
from tests.paged_testutil import PagedPair

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
Q8, F8 = "q8_0/q5_1", "e4m3"
NAN, INF = float("nan"), float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prefix_pair(n, rows, suffix, D=128, Hkv=1, Hq=4, page=16, ks=1.0, vs=1.0, fmt=Q8, seed=0, **kw):
    """n sequences whose first `rows` rows (whole pages) are the same pages."""
    p = PagedPair(n, Hkv, D, Hq, page=page, max_pages=-(-(rows + suffix) // page), fmt=fmt, seed=seed, **kw)
    assert rows % page == 0
    p.tab[1:, :rows // page] = p.tab[0, :rows // page]
    p.tables = torch.from_numpy(p.tab).cuda()
    k, v = p.randn(rows, Hkv, D) * ks, p.randn(rows, Hkv, D) * vs
    for b in range(n):
        p.note(b, k.numpy(), v.numpy())
    p.dev.append(k[None].cuda(), v[None].cuda(), p.tables[:1], i32([rows]))
    k, v = p.randn(n, suffix, Hkv, D) * ks, p.randn(n, suffix, Hkv, D) * vs
    for b in range(n):
        p.note(b, k[b].numpy(), v[b].numpy())
    p.dev.append(k.cuda(), v.cuda(), p.tables, p.lens())
    return p


def assert_bf16(p, q, got, want, mag, scale):
    """The output's rounding (2^-8), fp16 roundings of p and v (2^-11 each of p |v|) with as much again for
    sums and records, and keys as fp16: each off by 2^-11 of itself at most, a score so by d = 2^-11 of
    sum |q k| scale, and an output by at most 2 d sum p |v|."""
    qf, hpk = q.double().numpy(), p.Hq // p.Hkv
    a = np.zeros(want.shape[:3] + (1,))
    for b in range(p.n):
        for h in range(p.Hq):
            a[b, :, h, 0] = (np.abs(qf[b, :, h]) @ np.abs(p.k[b][:, h // hpk]).T).max(-1)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -10 * a * scale) * mag + 1e-30
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst ratio {np.nanmax(err / tol):.2f}"


@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("ks", [1e4, 30.0, 1.0, 1e-2, 1e-4, 1e-5, 1e-6])
def test_shared_prefix_of_keys_far_from_one(D, Hq, ks):
    """Keys of any size that the format holds, scores of the same size all the same."""
    p = prefix_pair(10, 160, 3, D=D, Hq=Hq, ks=ks, seed=D)
    q = p.randn(10, 1, Hq, D).to(BF)
    scale = 1.5 / (ks * D ** 0.5)
    want, mag = p.want(q, scale=scale)
    args = (q.cuda(), p.tables, p.lens())
    assert_bf16(p, q, p.dev.decode(*args, scale=scale), want, mag, scale)
    assert_bf16(p, q, p.dev.decode_shared(*args, i32([0, 10]), i32([160]), scale=scale), want, mag, scale)


def test_shared_prefix_of_keys_unlike_each_other():
    """Rows 32 and more apart, and blocks of a row, from 1e-5 to 1e3 in one prefix."""
    D, rows = 128, 256
    p = prefix_pair(10, rows, 3, D=D, seed=5)
    size = 10.0 ** torch.linspace(-5, 3, 8)
    k = p.randn(rows, 1, D) * size.repeat_interleave(32)[:, None, None]
    k[:, :, :32] *= 1e-3                                 # (one block of each row)
    v = p.randn(rows, 1, D)
    kb, vb = P.blocks(k.numpy(), Q8, "k"), P.blocks(v.numpy(), Q8, "v")
    for b in range(p.n):
        p.k[b][:rows], p.v[b][:rows] = P.values(kb, Q8, "k"), P.values(vb, Q8, "v")
    p.dev.append(k[None].cuda(), v[None].cuda(), p.tables[:1], i32([rows]))
    q = p.randn(10, 1, 4, D).to(BF)
    args = (p.tables, p.lens(), i32([0, 10]), i32([rows]))
    for only in range(8):
        # the other rows are not seen: a window over one stretch of 32, by sequences that end there
        lens = i32([32 * only + 32] * 10)
        scale = 1.5 / (float(size[only]) * D ** 0.5)
        want, mag = np.zeros((10, 1, 4, D)), np.zeros((10, 1, 4, D))
        at = slice(32 * only, 32 * only + 32)
        a = 0.0
        for b in range(10):
            for h in range(4):
                x = q[b, 0, h].double().numpy()
                want[b, 0, h], mag[b, 0, h] = P.attend(x, p.k[b][at, 0], p.v[b][at, 0], np.ones(32, np.int64), scale)
                a = max(a, float((np.abs(x) @ np.abs(p.k[b][at, 0]).T).max()) * scale)
        got = p.dev.decode_shared(q.cuda(), p.tables, lens, *args[2:], scale=scale, window=32)
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -10 * a) * mag
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all(), only


@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("vs", [1e4, 1.0, 1e-4, 1e-5, 1e-6])
def test_shared_prefix_of_values_far_from_one(D, Hq, vs):
    """A query of zeros takes the mean of the values: no key's rounding is in it."""
    p = prefix_pair(10, 160, 3, D=D, Hq=Hq, vs=vs, seed=D)
    q = torch.zeros(10, 1, Hq, D, dtype=BF)
    want, mag = p.want(q)
    args = (q.cuda(), p.tables, p.lens())
    assert_bf16(p, q, p.dev.decode(*args), want, mag, 1.0)
    assert_bf16(p, q, p.dev.decode_shared(*args, i32([0, 10]), i32([160])), want, mag, 1.0)


# ------------------------------------------------------------------ numbers that are not finite

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("rows", [16, 1600])
def test_a_query_of_nan_gives_nan_however_the_work_is_cut(dtype, fmt, rows):
    """One range a key, many ranges, listed pages, a shared prefix: NaN for that head, numbers for the others."""
    p = prefix_pair(3, rows, 5, D=64, Hkv=1, Hq=12, fmt=fmt, bounds=True, seed=rows)
    q = p.randn(3, 1, 12, 64).to(dtype).cuda()
    q[1, 0, 7, 3] = NAN
    lens = p.lens()
    pages = i32(np.tile(np.arange(p.max_pages), (3, 1, 1, 1)).tolist())
    outs = [p.dev.decode(q, p.tables, lens), p.dev.decode_sparse(q, p.tables, lens, pages),
            p.dev.decode(q, p.tables, lens, sinks=torch.zeros(12, device="cuda")),
            p.dev.decode_shared(q, p.tables, lens, i32([0, 3]), i32([rows])),
            p.dev.decode_shared(q, p.tables, lens, i32([0, 3]), i32([rows]), softcap=5.0)]
    for i, o in enumerate(outs):
        assert torch.isnan(o[1, 0, 7]).all(), i
        o[1, 0, 7] = 0
        assert torch.isfinite(o).all(), i


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("rows", [16, 1600])
def test_a_score_that_overflows_gives_nan_however_the_work_is_cut(dtype, fmt, rows):
    """The largest queries over keys of one sign: in the prefix alone, among a sequence's own rows alone."""
    for where in ("prefix", "own"):
        p = PagedPair(2, 1, 64, 12, page=16, max_pages=rows // 16 + 1, fmt=fmt, bounds=True, seed=rows)
        p.tab[1:, :rows // 16] = p.tab[0, :rows // 16]
        p.tables = torch.from_numpy(p.tab).cuda()
        k, v = p.randn(2, rows + 5, 1, 64), p.randn(2, rows + 5, 1, 64)
        k[1], v[1, :rows] = k[0], v[0, :rows]
        k[:, slice(3, 4) if where == "prefix" else slice(rows + 2, rows + 3)] = 400.0
        k[:, rows + 3] = 0.0
        p.dev.append(k.cuda(), v.cuda(), p.tables, i32([rows + 5] * 2))
        q = p.randn(2, 1, 12, 64)
        q[1, 0, 7] = 3e38
        q, lens = q.to(dtype).cuda(), i32([rows + 5] * 2)
        pages = i32(np.tile(np.arange(p.max_pages), (2, 1, 1, 1)).tolist())
        for i, o in enumerate((p.dev.decode(q, p.tables, lens), p.dev.decode_sparse(q, p.tables, lens, pages),
                               p.dev.decode_shared(q, p.tables, lens, i32([0, 2]), i32([rows])))):
            assert torch.isnan(o[1, 0, 7]).all(), (where, i)
            o[1, 0, 7] = 0
            assert torch.isfinite(o).all(), (where, i)


def test_a_query_that_is_not_finite_and_sees_no_row_gives_zeros():
    p = prefix_pair(3, 16, 2, D=64, Hq=12, max_t=4)
    q = p.randn(3, 4, 12, 64)
    q[0, 0], q[0, 3] = NAN, INF
    for dtype in (BF, F32):
        x, lens = q.to(dtype).cuda(), i32([2, 18, 18])
        for o in (p.dev.decode(x, p.tables, lens), p.dev.decode_shared(x, p.tables, lens, i32([0, 3]), i32([16]))):
            assert (o[0, :2] == 0).all() and torch.isfinite(o[0, 2]).all() and torch.isnan(o[0, 3]).all()
            assert torch.isfinite(o[1:]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("bad", [NAN, INF, -INF, 1e30, -1e7])
@pytest.mark.parametrize("many", [1, 9])
def test_keys_that_are_not_finite_are_stored_as_the_header_says(dtype, fmt, bad, many):
    """One element, a block, a row; few rows and many: what is read back is finite, NaN as zero and the rest at the
    format's end, and the rows that see them attend to that."""
    D, n, page = 64, 3, 16
    p = PagedPair(n, 1, D, 4, page=page, max_pages=3, fmt=fmt, bounds=True, seed=many)
    k, v = p.randn(n, many, 1, D).to(dtype), p.randn(n, many, 1, D).to(dtype)
    for b, cut in enumerate((slice(37, 38), slice(32, 64), slice(0, 64))):
        k[b, -1, :, cut] = bad
    end = 448.0 if fmt == F8 else 65504.0 * 127
    clean = torch.nan_to_num(k.float(), nan=0.0, posinf=end, neginf=-end).clamp(-end, end)
    for b in range(n):
        p.note(b, clean[b].numpy(), v[b].float().numpy())
    p.dev.append(k.cuda(), v.cuda(), p.tables, p.lens())
    assert np.array_equal(p.dev.pool.cpu().numpy(), p.expected_pool())
    bounds = p.dev.bounds.clone()
    p.dev.update_bounds(p.tables, p.lens(), many)
    assert torch.equal(p.dev.bounds, bounds)
    q = (p.randn(n, 1, 4, D) * 1e-3).to(dtype)
    want, mag = p.want(q, scale=1e-4)
    for o in (p.dev.decode(q.cuda(), p.tables, p.lens(), scale=1e-4),
              p.dev.decode_shared(q.cuda(), p.tables, p.lens(), i32([0, 1, 2, 3]), i32([0, 0, 0]), scale=1e-4)):
        assert_bf16(p, q, o, want, mag, 1e-4)
    assert p.dev.device_error() == 0


# ------------------------------------------------------------------ ends of the arguments' ranges

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("att", [{}, dict(softcap=2.0)])
def test_scales_and_queries_at_the_ends_of_their_ranges(dtype, att):
    """Scores that vanish, masked rows among them, are zeros: the mean of the visible values.  So are scores of
    zero keys under the largest factors."""
    p = prefix_pair(10, 144, 3, D=128, Hq=4)
    q = p.randn(10, 1, 4, 128)
    args = (p.tables, p.lens(), i32([0, 10]), i32([144]))
    want, mag = p.want(torch.zeros_like(q))
    calls = [(1e-30, (q * 1e-15).to(dtype)), (1e-30, (q * 1e-30).to(dtype)), (1e-30, torch.zeros_like(q).to(dtype))]
    z = prefix_pair(10, 144, 3, D=128, Hq=4, ks=0.0)
    for scale, x in calls:
        for got in (p.dev.decode(x.cuda(), *args[:2], scale=scale, **att), p.dev.decode_shared(x.cuda(), *args, scale=scale, **att)):
            assert_bf16(p, torch.zeros_like(q), got, want, mag, 1.0)
    want, mag = z.want(torch.zeros_like(q))
    x = (q * 1e36).clamp(-3e38, 3e38).to(dtype)
    for got in (z.dev.decode(x.cuda(), z.tables, z.lens(), scale=1e30, **att),
                z.dev.decode_shared(x.cuda(), z.tables, z.lens(), *args[2:], scale=1e30, **att)):
        assert_bf16(z, torch.zeros_like(q), got, want, mag, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,ks,qs,scale", [(128, 1e4, 1e4, 0.0), (64, 3e3, 1e6, 1.0), (256, 1e6, 1e25, 1.0), (128, 1e-6, 1e38, 4096.0)])
def test_scores_far_apart_leave_the_largest_alone(D, ks, qs, scale, dtype):
    """Scores of 1e8 to 1e37: the row of the largest takes all, where the next one is further from it than the
    keys' roundings to fp16 can be (2^-11 of sum |q k| each)."""
    p = prefix_pair(10, 144, 3, D=D, Hq=4, ks=ks, seed=D)
    q = (p.randn(10, 1, 4, D) * qs).clamp(-3e38, 3e38).to(dtype)
    more = (i32([0, 10]), i32([144]))
    outs = (p.dev.decode(q.cuda(), p.tables, p.lens(), scale=scale),
            p.dev.decode_shared(q.cuda(), p.tables, p.lens(), *more, scale=scale))
    n = 0
    for b in range(10):
        for h in range(4):
            x = q[b, 0, h].double().numpy()
            s = p.k[b][:, 0] @ x
            top, next_ = np.sort(s)[-1], np.sort(s)[-2]
            if top - next_ < 2.0 ** -10 * (np.abs(p.k[b][:, 0]) @ np.abs(x)).max():
                continue
            n += 1
            want = p.v[b][int(s.argmax()), 0]
            for i, o in enumerate(outs):
                assert (np.abs(o[b, 0, h].double().cpu().numpy() - want) <=
                        2.0 ** -7 * np.abs(want) + 2.0 ** -18 * p.spread()).all(), (i, b, h)
    assert n >= 10                                       # (19 of 40 at the least: it depends on the inputs alone)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_below_any_reference_still_count(dtype):
    """Rows whose scores are all far below -1e30: the largest takes all."""
    p = prefix_pair(10, 48, 1, D=64, Hq=4, seed=7)
    q = p.randn(10, 1, 4, 64).abs().to(dtype)
    for b in range(10):
        p.k[b] = np.zeros_like(p.k[b])
    k = -torch.arange(1, 50, dtype=torch.float32)[:, None, None].expand(49, 1, 64) * 64
    v = p.randn(49, 1, 64)
    for b in range(10):
        p.v[b] = P.values(P.blocks(v.numpy(), Q8, "v"), Q8, "v")
        p.dev.append(k[None].contiguous().cuda(), v[None].cuda(), p.tables[b:b + 1], i32([49]))
    want = np.stack([np.repeat(p.v[b][None, 0], 4, 1) for b in range(10)])[:, None].reshape(10, 1, 4, 64)   # row 0 has the largest score
    args = (q.cuda(), p.tables, p.lens())
    # (capped at 1e30, all scores are the same)
    mean = np.stack([np.repeat(p.v[b][None].mean(1)[None], 4, 2) for b in range(10)]).reshape(want.shape)
    for att, w in (({}, want), (dict(softcap=1e30), mean)):
        for got in (p.dev.decode(*args, scale=1e30, **att), p.dev.decode_shared(*args, i32([0, 10]), i32([48]), scale=1e30, **att)):
            # the output's rounding, and fp16 roundings of p and v: 2^-9 of the largest value
            tol = 2.0 ** -8 * np.abs(w) + 2.0 ** -9 * np.abs(p.v[0]).max()
            assert (np.abs(got.double().cpu().numpy() - w) <= tol).all(), att


@pytest.mark.parametrize("dtype", [BF, F32])
def test_windows_of_any_size(dtype):
    """A window beyond every length is none, for sequences shorter than the rows of queries too."""
    p = prefix_pair(10, 32, 7, D=64, Hq=4, max_t=8)
    lens = i32([1, 2, 5, 8, 33, 39, 39, 39, 39, 3])
    q = p.randn(10, 8, 4, 64).to(dtype).cuda()
    more = (i32([0, 10]), i32([32]))
    dense, shared = p.dev.decode(q, p.tables, lens), p.dev.decode_shared(q, p.tables, lens, *more)
    for w in (39, 1 << 24, (1 << 24) + 1, 2 ** 31 - 1):
        assert torch.equal(p.dev.decode(q, p.tables, lens, window=w), dense), w
        assert torch.equal(p.dev.decode_shared(q, p.tables, lens, *more, window=w), shared), w
    for w in (2 ** 31, 2 ** 32 + 5, -1, -2 ** 32 + 5):
        with pytest.raises(Exception):
            p.dev.decode(q, p.tables, lens, window=w)


def test_errors_of_calls_behind_a_read_error_are_kept():
    """On a stream that does not wait for the default one: each bad call is reported, none is cleared away."""
    p = PagedPair(1, 1, 64, 2, page=16, max_pages=2)
    p.append([20])
    q = p.randn(1, 1, 2, 64).to(BF).cuda()
    bad, s = torch.full_like(p.tables, -1), torch.cuda.Stream()
    lens = p.lens()
    torch.cuda.synchronize()
    for _ in range(300):
        p.dev.decode(q, bad, lens, stream=s)
        assert p.dev.device_error(stream=s) == 1
    assert p.dev.device_error(stream=s) == 0


def test_rotation_by_more_than_half_a_turn_a_position():
    """Frequencies up to the 64 radians that a call takes, at the farthest positions."""
    need_gpu()
    D, page, far = 64, 256, 1 << 24
    freq = [64.0, -63.7, 50.3, 33.3, 20.123, 12.9, 6.5, 6.2, 4.0, 3.2] + [1.0, 0.3, -0.2, 0.1, 0.01, 0.001]
    c = PagedKVCache(2, page, 1, D, 2, max_seqs=1, max_pages=1 << 16, rope_dim=32, rope_freq=freq)
    tab = torch.zeros(1, 1 << 16, dtype=torch.int32, device="cuda")
    k = torch.randn(1, 64, 1, D, generator=torch.Generator().manual_seed(1))
    for end in (far, far - 1234567, 1 << 20):
        q = c.append(k.cuda(), k.cuda(), tab, i32([end]), q=k.cuda())
        want = P.rotate(k.double().numpy().reshape(64, 1, D), end - 64 + np.arange(64), 32, freq=freq)
        # 2^-24 of a turn are 2^-21.3 radians; twice that for the fp64 product of position and frequency and f32 arithmetic
        assert np.abs(q.cpu().double().numpy().reshape(64, 1, D) - want).max() <= 2.0 ** -20 * 4
    assert c.device_error() == 0


# ------------------------------------------------------------------ accuracy of f32 queries

@pytest.mark.parametrize("D,Hq", [(64, 4), (64, 16), (128, 8), (128, 16), (256, 4), (256, 16)])
def test_f32_outputs_keep_all_24_bits_of_p_d(D, Hq):
    """Scores without a rounding of their own: each key has one element that is not zero, 127 d of a d with few
    bits, and each query one power of two, so that a score is off by its factors' roundings alone.  Row 0 has
    the largest score and values of zero, row 1 values d (u - 16).  p_1 is then off by its exponent's roundings,
    at most 2^-22 for each of factor, product and sum (the sum is below 8), ln 2 of that, and 2^-22 of ex2: less
    than 2^-20 together; as much again covers the sum of weights, its reciprocal, the final product and the
    three parts of p d (2^-24).  Two rounded parts of 8 bits would leave up to 2^-18: the case tells them apart."""
    n = 64
    p = PagedPair(n, 1, D, Hq, page=16, max_pages=1, seed=D + Hq)
    rng = np.random.default_rng(D)
    k, v = np.zeros((n, 2, 1, D), np.float32), np.zeros((n, 2, 1, D), np.float32)
    k[:, 0, 0, 0] = 127 * 2.0 ** -10
    d = rng.integers(1024, 2047, n) * 2.0 ** -17                   # eleven bits
    k[:, 1, 0, 0] = -127 * rng.integers(1024, 2047, n) * 2.0 ** -17
    u = rng.integers(0, 32, (n, D))
    u[:, 0::32], u[:, 1::32] = 0, 31
    v[:, 1, 0] = (u - 16) * d[:, None]
    for b in range(n):
        p.note(b, k[b], v[b])
        assert np.array_equal(p.k[b], k[b]) and np.array_equal(p.v[b], v[b])
    p.dev.append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), p.tables, p.lens())
    q = torch.zeros(n, 1, Hq, D)
    q[..., 0] = 2.0 ** torch.randint(0, 3, (n, 1, Hq), generator=torch.Generator().manual_seed(1)).float()
    scale = 0.11
    want, mag = p.want(q, scale=scale)
    got = p.dev.decode(q.cuda(), p.tables, p.lens(), scale=scale).double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -19 * np.abs(want)).all(), (np.abs(got - want)[want != 0] / np.abs(want)[want != 0]).max()
    # what two parts would have given, on the host
    s = q[:, 0, :, 0].double().numpy() * (k[:, 1, 0, 0].astype(np.float64) - float(k[0, 0, 0, 0]))[:, None] * scale
    x = np.float32(64 * np.exp(s) * d[:, None])
    bf = lambda y: torch.from_numpy(y).bfloat16().float().numpy()
    rest = x - bf(x)
    assert (np.abs(rest - bf(rest)) / x).max() > 1.5 * 2.0 ** -19


# ------------------------------------------------------------------ selection over more pages than the pick holds

@pytest.mark.parametrize("np_", [8191, 8192, 8193, 20001])
def test_selection_around_and_beyond_8192_pages(np_):
    """Two KV heads whose rows of scores share cache lines, scores with many ties."""
    need_gpu()
    D, page, Hkv, Hq, NB = 64, 16, 2, 6, 2
    g = np.random.default_rng(np_)
    n_pages, width = 20011, 20001
    c = PagedKVCache(n_pages, page, Hkv, D, Hq, max_seqs=2, max_pages=width, max_t=2, bounds=True)
    lo, hi = g.integers(-3, 1, (n_pages, Hkv, NB, 32)), g.integers(0, 4, (n_pages, Hkv, NB, 32))
    codes = np.stack([lo, hi], 3).astype(np.int8)
    ds = g.choice([0.5, 1.0], (n_pages, Hkv, NB)).astype(np.float32)
    raw = np.concatenate([codes.reshape(-1).view(np.uint8), ds.reshape(-1).view(np.uint8)])
    c.bounds[:raw.size].copy_(torch.from_numpy(raw))
    tab = np.stack([g.permutation(n_pages)[:width] for _ in range(2)]).astype(np.int32)
    q = torch.from_numpy(g.choice([-1.0, 0.0, 0.0, 1.0], (2, 2, Hq, D)).astype(np.float32))
    lens = np.array([np_ * page - 3, width * page])
    for keep in (1, 64, 300, 5000):
        got = c.select(q.cuda(), torch.from_numpy(tab).cuda(), i32(lens.tolist()), keep, n_first=min(1, keep), n_last=0).cpu().numpy()
        for b in range(2):
            for t in range(2):
                m = -(-(int(lens[b]) - 2 + t + 1) // page)
                for h in range(Hkv):
                    sc = P.scores(q[b, t, 3 * h:3 * h + 3].numpy(), codes[tab[b, :m], h], ds[tab[b, :m], h])
                    # (ties to the lower index, as the oracle's select, which is slow at this size)
                    order = [0] + [int(i) + 1 for i in np.argsort(-sc[1:], kind="stable")]
                    assert got[b, t, h].tolist() == sorted(order[:keep]), (keep, b, t, h)
    assert c.device_error() == 0
