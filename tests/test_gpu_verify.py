"""Draft verification on the GPU against the oracle's whole numbers: every
result is equal, not near."""

import numpy as np
import pytest
import torch

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300.cache import KVCache, verify
from tests.kvq_testutil import need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def draw(n, T, V, dtype, seed, point=False, near=0.5, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    z = sharp * torch.randn(n, T, V, generator=g)
    target = torch.softmax(z, -1).to(dtype)
    draft = torch.softmax(z[:, :T - 1] + near * torch.randn(n, T - 1, V, generator=g), -1).to(dtype)
    src = target[:, :T - 1] if point else draft
    tokens = torch.multinomial(src.reshape(-1, V).float(), 1, generator=g).view(n, T - 1).int() if T > 1 else torch.zeros(n, 0, dtype=torch.int32)
    u = torch.rand(n, T, generator=g)
    return target, None if point else draft, tokens, u


def want(target, draft, tokens, u):
    t, q = target.double().numpy(), None if draft is None else draft.double().numpy()
    r = [P.verify(t[b], None if q is None else q[b], tokens[b].numpy(), u[b].double().numpy()) for b in range(len(t))]
    return [x[0] for x in r], [x[1] for x in r]


def check(target, draft, tokens, u, dev=None):
    """dev: the device tensors, where they are not plain copies."""
    need_gpu()
    lens = torch.arange(len(target), dtype=torch.int32, device="cuda") + 1000
    d = dev or [None if x is None else x.cuda() for x in (target, draft, tokens, u)]
    accept, token = verify(*d, lens=lens)
    a, n = want(target, draft, tokens, u)
    assert accept.tolist() == a and token.tolist() == n
    T = target.shape[1]
    assert (lens.cpu() - 1000 - torch.arange(len(target))).tolist() == [x - T for x in a]
    return a, n


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,T,V", [(1, 1, 1), (1, 2, 2), (3, 1, 33), (5, 4, 97), (2, 9, 1000), (40, 3, 257), (1, 5, 32000), (2, 3, 50021),
                                   (170, 2, 4096), (1, 2, 262144), (700, 2, 64), (3, 65, 31), (1, 512, 40)])
def test_against_the_oracle(n, T, V, dtype):
    check(*draw(n, T, V, dtype, n * 1000 + V))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,V", [(2, 65), (4, 3000), (5, 131072)])
def test_drafts_that_were_looked_up(T, V, dtype):
    t, _, k, u = draw(9, T, V, dtype, V, point=True, sharp=6.0)
    a, _ = check(t, None, k, u)
    assert 1 < sum(a) < 9 * T


@pytest.mark.parametrize("dtype", [F32, BF])
def test_every_count_of_accepted_drafts(dtype):
    """The same tokens with uniforms that let 0, 1 .. T - 1 of them stand; sequences with fewer drafts."""
    T, V = 6, 517
    t, q, k, u = draw(2 * T, T, V, dtype, 3)
    u[:, :-1] = 0.0                                  # 0 * q < p: a draft stands where p > 0
    for b in range(T):
        if b < T - 1:
            t[b, b, k[b, b]] = 0.0                   # p = 0: falls at b
            k[T + b, b] = [-1, V, -7, 1 << 30, -2147483648][b]
    a, _ = check(t, q, k, u)
    assert a == [1, 2, 3, 4, 5, 6, 1, 2, 3, 4, 5, 6]


def test_borders_of_the_test_and_of_the_draw():
    """u q = p falls, the next float below stands; u at both ends, beyond them and NaN."""
    V = 64
    p, q = torch.full((8, 2, V), 1 / 64), torch.full((8, 1, V), 1 / 32)
    k = torch.full((8, 1), 5, dtype=torch.int32)
    u = torch.zeros(8, 2)
    u[0, 0], u[1, 0] = 0.5, 0.5 - 2.0 ** -25
    u[:, 1] = torch.tensor([0.0, 0.25, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan"), float("inf")])
    a, n = check(p, q, k, u)
    assert a[:2] == [1, 2] and n[0] == 0 and n[1] == 16 and n[2] == n[3] == n[4] == n[7] == 63 and n[5] == n[6] == 0


def test_rows_with_nothing_in_them():
    """p = q leaves p itself; all zeros, NaN, negative and infinite entries."""
    V, n = 300, 6
    t, q, k, u = draw(n, 2, V, F32, 11)
    u[:, 0] = 1 - 2.0 ** -24
    q[:] = t[:, :1]
    t[0, 0, k[0, 0]] = q[0, 0, k[0, 0]] = 0.25       # u q < p with u < 1: stands
    q[1] = 1.0                                        # q above p everywhere: nothing is left
    t[2] = 0.0
    t[3, 0] = float("nan")
    t[4, 0, ::3], t[4, 0, 1::3], t[4, 0, 2] = -1.0, float("nan"), float("inf")
    q[4] = 0.0
    q[5, 0, ::2] = float("nan")
    a, nx = check(t, q, k, u)
    assert a[0] == 2 and a[2] == 1 and nx[2] == -1 and nx[3] == -1


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_apart_and_rows_at_odd_addresses(dtype):
    t, q, k, u = draw(4, 4, 1003, dtype, 21)
    wide = torch.full((4, 5, 1040), float("nan"), dtype=dtype, device="cuda")
    narrow = torch.full((4, 4, 1009), float("nan"), dtype=dtype, device="cuda")
    wide[:, :4, 7:1010], narrow[:, :3, 2:1005] = t.cuda(), q.cuda()
    check(t, q, k, u, [wide[:, :4, 7:1010], narrow[:, :3, 2:1005], k.cuda(), u.cuda()])
    one = t[:1, :1].expand(4, 4, 1003)               # one row for all (strides of 0)
    check(one.contiguous(), q, k, u, [t[:1, :1].cuda().expand(4, 4, 1003), q.cuda(), k.cuda(), u.cuda()])


def test_sums_that_pass_their_range_stay_in_range():
    """Rows that are no probabilities: any token, or -1, but no other."""
    V = 131072
    t = torch.ones(3, 1, V, device="cuda")
    _, token = verify(t, None, torch.zeros(3, 0, dtype=torch.int32, device="cuda"), torch.rand(3, 1, device="cuda"))
    assert ((token >= -1) & (token < V)).all()


def test_on_a_stream_and_captured():
    t, q, k, u = (x.cuda() for x in draw(5, 4, 2000, F32, 31))
    ref = verify(t, q, k, u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = verify(t, q, k, u, stream=s)
    s.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    acc, nxt, lens = (torch.zeros(5, dtype=torch.int32, device="cuda") for _ in range(3))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        verify(t, q, k, u, lens=lens, accept=acc, next_tokens=nxt)
    for seed in (32, 33):
        new = draw(5, 4, 2000, F32, seed)
        for x, y in zip((t, q, k, u), new):
            x.copy_(y)
        lens.fill_(50)
        g.replay()
        a, n = want(*new)
        assert acc.tolist() == a and nxt.tolist() == n and lens.tolist() == [46 + x for x in a]


def test_the_flat_caches_draft_round():
    """append T, decode T, verify, truncate by its counts, without a host wait."""
    n, Hkv, D, T, V = 3, 2, 64, 4, 500
    c = KVCache(n, Hkv, D, Hkv, max_t=T, max_rows=64)
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    c.append(rnd(n, T, Hkv, D), rnd(n, T, Hkv, D))
    total = [T] * n
    for r in range(4):
        c.append(rnd(n, T, Hkv, D), rnd(n, T, Hkv, D))
        c.decode(rnd(n, T, Hkv, D))
        t, q, k, u = draw(n, T, V, F32, 40 + r)
        accept, token = verify(t.cuda(), q.cuda(), k.cuda(), u.cuda())
        c.truncate_device(accept, T)
        a, nx = want(t, q, k, u)
        assert token.tolist() == nx
        total = [x + y for x, y in zip(total, a)]
    c.sync_len()
    assert c.lens() == total and c.device_error() == 0


def test_refusals_of_the_wrapper():
    need_gpu()
    t, q, k, u = (x.cuda() for x in draw(2, 3, 40, F32, 1))
    for bad in (lambda: verify(t.half(), q, k, u), lambda: verify(t.cpu(), q, k, u), lambda: verify(t[0], q, k, u),
                lambda: verify(t, q.bfloat16(), k, u), lambda: verify(t, q[:, :1], k, u), lambda: verify(t, q, k.long(), u),
                lambda: verify(t, q, k[:, :1], u), lambda: verify(t, q, k, u.double()), lambda: verify(t, q, k, u[:, :2]),
                lambda: verify(t.transpose(1, 2), None, k, u), lambda: verify(t, q, k, u, lens=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: verify(t, q, k, u, accept=torch.zeros(2, device="cuda")), lambda: verify(t, q.cpu(), k, u)):
        with pytest.raises((ValueError, B.KvqError)):
            bad()
