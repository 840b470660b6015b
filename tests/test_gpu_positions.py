"""Appends at given positions on the GPU: one axis or several, against the
oracle's rotation, and against the append by index where both apply."""

import numpy as np
import pytest
import torch

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300.cache import PagedKVCache
from tests.kvq_testutil import need_gpu
from tests.paged_testutil import PagedPair

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
Q8, F8 = "q8_0/q5_1", "e4m3"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def axes_of(rot, n, cycle):
    half = rot // 2
    return [i % n for i in range(half)] if cycle else [min(n - 1, i * n // half) for i in range(half)]


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("D,rot,inter,n_axes,cycle,T,dtype", [
    (128, 128, False, 3, False, 1, BF), (128, 128, False, 3, False, 40, F32), (64, 32, True, 2, True, 9, F32),
    (256, 128, True, 4, True, 17, BF), (64, 64, False, 1, False, 33, BF), (256, 256, False, 3, True, 3, F32),
])
def test_against_the_definition(fmt, D, rot, inter, n_axes, cycle, T, dtype):
    n, Hkv, Hq, page = 3, 2, 6, 32
    axes = axes_of(rot, n_axes, cycle)
    p = PagedPair(n, Hkv, D, Hq, page=page, max_pages=8, fmt=fmt, rope_dim=rot, rope_interleaved=inter, rope_axes=axes, seed=T)
    assert p.dev.n_axes == n_axes
    ctx = [0, 100, 183]
    k, v, q = (p.randn(n, T, H, D).to(dtype) for H in (Hkv, Hkv, Hq))
    pos = p.rng.integers(0, 1 << 17, (n, T, n_axes))
    pos[0, 0], pos[1, T - 1] = 0, (1 << 24) - 1
    lens = i32([c + T for c in ctx])
    q_out = p.dev.append(k.cuda(), v.cuda(), p.tables, lens, q=q.cuda(), positions=i32(pos.tolist()))
    flat = lambda x: x.double().numpy().reshape(n * T, -1, D)
    at = pos.reshape(n * T, n_axes)
    qr, kr = P.rotate(flat(q), at, rot, inter, axes=axes), P.rotate(flat(k), at, rot, inter, axes=axes)
    size = np.abs(flat(q)).max()
    # angles good to 2^-24 of a turn (2^-21 radians), f32 products, the output's rounding
    tol = 2.0 ** -19 * size + (2.0 ** -8 if dtype == BF else 2.0 ** -24) * np.abs(qr)
    assert (np.abs(flat(q_out.cpu()) - qr) <= tol).all()
    ko, vo = torch.empty(n, T, Hkv, D, device="cuda"), torch.empty(n, T, Hkv, D, device="cuda")
    p.dev.read(p.tables, lens, ko, vo)
    got = flat(ko.cpu())
    if fmt == F8:
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(kr), 2.0 ** -6)))) * 2.0 ** -4      # half a step
    else:
        # half a code of d, d the fp16 of amax / 127 (2^-11 off), and a code's end that d rounded down leaves out
        am = np.abs(kr).reshape(n * T, Hkv, -1, 32).max(-1, keepdims=True)
        step = np.broadcast_to(am / 127 * 0.5 * (1 + 2.0 ** -9) + am * 2.0 ** -11, (*am.shape[:3], 32)).reshape(kr.shape)
    assert (np.abs(got - kr) <= step * (1 + 1e-6) + 2.0 ** -19 * size).all()
    assert np.array_equal(flat(vo.cpu()), P.values(P.blocks(flat(v), fmt, "v"), fmt, "v").astype(np.float32))
    assert p.dev.device_error() == 0


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("counts", [[1, 1, 1], [50, 3, 21], [0, 1, 300]])
@pytest.mark.parametrize("n_axes", [1, 3])
def test_a_rows_own_index_places_rows_as_the_append_by_index(fmt, counts, n_axes):
    """The same rows, values and bounds but for what an angle's last bits (2^-24 of a turn by index) move over a border."""
    n, Hkv, Hq, D = 3, 2, 4, 128
    kw = dict(page=16, max_pages=24, fmt=fmt, rope_dim=64, bounds=True, rope_axes=axes_of(64, n_axes, True))
    a, b = (PagedPair(n, Hkv, D, Hq, seed=7, **kw) for _ in range(2))
    rows = sum(counts)
    ctx = [5, 0, 17]
    k, v, q = a.randn(rows, Hkv, D).cuda(), a.randn(rows, Hkv, D).cuda(), a.randn(rows, Hq, D).cuda()
    lens = i32([x + y for x, y in zip(ctx, counts)])
    starts = i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
    pos = np.concatenate([np.arange(x, x + y) for x, y in zip(ctx, counts)])
    given = i32(np.repeat(pos[:, None], n_axes, 1).tolist())
    for p in (a, b):
        p.dev.pool.zero_()
        p.dev.bounds.zero_()
    forms = [starts] if counts != [1, 1, 1] else [starts, None]
    for st in forms:
        shape = (lambda x: x) if st is not None else (lambda x: x.unsqueeze(1))
        qa = a.dev.append(shape(k), shape(v), a.tables, lens, starts=st, q=shape(q))
        qb = b.dev.append(shape(k), shape(v), b.tables, lens, starts=st, q=shape(q), positions=shape(given))
        assert (qa - qb).abs().max() <= 2.0 ** -20 * q.abs().max() and torch.equal(qa[..., 64:], qb[..., 64:])
        differ = (a.dev.pool != b.dev.pool).sum().item()
        # an angle off by 2^-21 radians moves an element by 2^-21 of its pair, a code's border lies
        # 2^-8 (E4M3: 2^-4 of the element) away on average: fewer than one in a thousand
        assert differ <= 1e-3 * rows * Hkv * D + 2, differ
        out = [torch.empty(rows, Hkv, D, device="cuda") for _ in range(4)]
        a.dev.read(a.tables, lens, out[0], out[1], starts=starts)
        b.dev.read(b.tables, lens, out[2], out[3], starts=starts)
        assert torch.equal(out[1], out[3])
        am = out[0].abs().view(rows, Hkv, -1, 32).amax(-1, keepdim=True).expand(-1, -1, -1, 32).reshape(out[0].shape)
        step = am / 127 * (1 + 2.0 ** -9) + am * 2.0 ** -10 if fmt == Q8 else torch.maximum(out[0].abs(), out[2].abs()) * 2.0 ** -3 + 2.0 ** -9
        assert ((out[0] - out[2]).abs() <= step).all()
        assert (a.dev.bounds != b.dev.bounds).sum().item() <= 2e-2 * a.dev.bounds.numel()
    if n_axes == 1:                                     # the last dimension may be left out
        qc = b.dev.append(k, v, b.tables, lens, starts=starts, q=q, positions=given[:, 0].contiguous())
        assert torch.equal(qc, qb.view_as(qc))


@pytest.mark.parametrize("inter", [False, True])
def test_angles_of_given_positions_to_the_last_bits(inter):
    """f32 queries at positions up to 2^24 - 1: cos and sin 0.65 of a last bit (2^-24 of them at most), the angle what two floats
    of frequency leave (2^-50 a position: 2^-23.3 radians at the end), and the two products' and the sum's roundings."""
    need_gpu()
    D, n = 128, 4096
    axes = [i % 3 for i in range(D // 2)]
    c = PagedKVCache(n // 16, 16, 1, D, 1, max_seqs=1, max_pages=n // 16, rope_dim=D, rope_interleaved=inter, rope_axes=axes)
    r = np.random.default_rng(4)
    pos = np.exp(r.uniform(0, np.log(2.0 ** 24), (n, 3))).astype(np.int64).clip(0, (1 << 24) - 1)
    pos[0], pos[1], pos[2:40] = 0, (1 << 24) - 1, np.arange(38)[:, None]
    x = torch.randn(1, n, 1, D, generator=torch.Generator().manual_seed(6))
    tab = torch.arange(n // 16).view(1, -1).int().cuda()
    got = c.append(x.cuda(), x.cuda(), tab, i32([n]), q=x.cuda(), positions=i32(pos[None].tolist())).cpu().double().numpy()[0]
    xd = x[0].double().numpy()
    want = P.rotate(xd, pos, D, inter, axes=axes)
    one, two = (slice(0, D, 2), slice(1, D, 2)) if inter else (slice(0, D // 2), slice(D // 2, D))
    size = np.abs(xd[..., one]) + np.abs(xd[..., two])
    tol = np.empty_like(xd)
    tol[..., one] = tol[..., two] = (0.65 + 1 + 1) * 2.0 ** -24 * size
    far = pos[:, axes][:, None, :] * 2.0 ** -50 * 2 * np.pi * size
    tol[..., one] += far
    tol[..., two] += far
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert c.device_error() == 0


@pytest.mark.parametrize("fmt", [Q8, F8])
@pytest.mark.parametrize("T", [1, 2, 40])
def test_bad_positions_skip_their_rows_alone(fmt, T):
    """Positions below 0 or from 2^24 on: the row and its query are left as they were, all others written."""
    n, Hkv, Hq, D = 4, 2, 2, 64
    p = PagedPair(n, Hkv, D, Hq, page=16, max_pages=4, fmt=fmt, rope_dim=64, rope_axes=axes_of(64, 2, False), scores=True)
    k, q = p.randn(n, T, Hkv, D).cuda(), p.randn(n, T, Hq, D).cuda()
    lens = i32([T + 3] * n)
    pos = torch.zeros(n, T, 2, dtype=torch.int32)
    bad = [(0, 0, 0, -1), (1, T - 1, 1, 1 << 24), (2, T // 2, 1, -2147483648)]
    good_q = p.dev.append(k, k, p.tables, lens, q=q, positions=pos.cuda())
    good = p.dev.pool.clone()
    assert p.dev.device_error() == 0
    for b, t, x, v in bad:
        pos[b, t, x] = v
    p.dev.pool.fill_(0x55)
    p.dev.scores.fill_(2.0)
    out = torch.full_like(q, 9.0)
    p.dev.append(k, k, p.tables, lens, q=q, q_out=out, positions=pos.cuda())
    assert p.dev.device_error() == 1
    ok = torch.ones(n, T, dtype=torch.bool)
    for b, t, _, _ in bad:
        ok[b, t] = False
    assert torch.equal(out[ok], good_q[ok]) and (out[~ok] == 9.0).all()
    ko, vo, kg, vg = (torch.empty(n, T, Hkv, D, device="cuda") for _ in range(4))
    p.dev.read(p.tables, lens, ko, vo)
    after, s = p.dev.pool.clone(), p.dev.scores.cpu()
    p.dev.pool.copy_(good)
    p.dev.read(p.tables, lens, kg, vg)
    assert torch.equal(ko[ok], kg[ok]) and torch.equal(vo[ok], vg[ok])
    p.dev.pool.fill_(0x55)
    p.dev.read(p.tables, lens, kg, vg)
    assert torch.equal(torch.nan_to_num(ko[~ok]), torch.nan_to_num(kg[~ok]))
    for b in range(n):
        for t in range(T):
            r = 3 + t
            assert (s[p.tab[b, r // 16], :, r % 16] == (0.0 if ok[b, t] else 2.0)).all()
    assert after.numel() == good.numel()


def test_refusals():
    need_gpu()
    mk = lambda **kw: PagedKVCache(4, 16, 1, 64, 1, max_seqs=1, max_pages=2, **kw)
    k, tab, lens = torch.zeros(1, 2, 1, 64, device="cuda"), i32([[0, 1]]), i32([2])
    with pytest.raises(B.KvqError):
        mk().append(k, k, tab, lens, positions=i32([[0, 1]]))                  # nothing is rotated
    with pytest.raises(B.KvqError):
        mk(rope_axes=[])
    for axes in ([0] * 15 + [4], [0] * 15 + [-1]):
        with pytest.raises(B.KvqError):
            mk(rope_dim=32, rope_axes=axes)
    with pytest.raises(ValueError):
        mk(rope_dim=32, rope_axes=[0] * 15)
    c = mk(rope_dim=32, rope_axes=[0, 1] * 8)
    for pos in (i32([[0, 1]]), i32([[[0], [1]]]), torch.zeros(1, 2, 2, device="cuda"), torch.zeros(1, 2, 2, dtype=torch.int32),
                torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")[..., ::2]):
        with pytest.raises(ValueError):
            c.append(k, k, tab, lens, positions=pos)
    with pytest.raises(B.KvqError):
        B.kvq_paged_append_at(c.handle, k.data_ptr(), 64, k.data_ptr(), 64, None, 0, None, 0, 0, tab.data_ptr(), lens.data_ptr(), 1, 2,
                              None, 2, None)
    with pytest.raises(B.KvqError):                                            # not on its elements
        B.kvq_paged_append_at(c.handle, k.data_ptr(), 64, k.data_ptr(), 64, None, 0, None, 0, 0, tab.data_ptr(), lens.data_ptr(), 1, 2,
                              None, 2, tab.data_ptr() + 2)
    for axis, n in (([0] * 16, 0), ([0] * 16, 5), (None, 1), ([2] * 16, 2)):
        with pytest.raises(B.KvqError):
            B.kvq_paged_set_axes(c.handle, axis, n)
    assert c.device_error() == 0
