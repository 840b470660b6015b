"""What the header promises of row scores, eviction and draft verification at the
edges of its ranges, on the GPU."""

import numpy as np
import pytest
import torch

from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300.cache import PagedKVCache, verify
from tests.kvq_testutil import need_gpu
from tests.paged_testutil import PagedPair
from tests.test_gpu_evict import gains, i32, near, scores_of
from tests.test_rows_contract_host import ODD, odd_rows

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
Q8, F8 = "q8_0/q5_1", "e4m3"


# ------------------------------------------------------------------ verification

@pytest.mark.parametrize("dtype", [F32, BF])
def test_probabilities_of_a_draft_that_are_none(dtype):
    """A drafted token's own p and q: NaN and what is not above 0 are 0, what is above 1 is 1."""
    need_gpu()
    rows = [odd_rows(*c[:3]) for c in ODD]
    t, q, k, u = (torch.from_numpy(np.stack([r[i] for r in rows])) for i in range(4))
    accept, token = verify(t.to(dtype).cuda(), q.to(dtype).cuda(), k.cuda(), u.float().cuda())
    assert accept.tolist() == [2 if c[3] else 1 for c in ODD]
    assert token.tolist() == [6 if c[3] else 4 for c in ODD]


# ------------------------------------------------------------------ room for kept scores

@pytest.mark.parametrize("fmt,D,hpk,max_t,queries", [
    (Q8, 128, 4, 1, 4), (Q8, 128, 4, 4, 8), (F8, 128, 2, 64, 8), (Q8, 64, 8, 1, 8), (F8, 256, 16, 1, 8),
    (F8, 64, 8, 1, 7),                                   # (8 scores are as many bytes as a row's keys)
    (F8, 64, 4, 4, 7),
])
def test_room_for_scores_is_what_a_call_can_use(fmt, D, hpk, max_t, queries):
    """Room for 8 queries a KV head, or as many as a call can have, and a cache made for drafts keeps
    the scores of its steps of few rows; calls of more leave the room as it is.  Scores are right either way."""
    p = PagedPair(2, 2, D, 2 * hpk, page=16, max_pages=4, fmt=fmt, max_t=max_t, scores=True, seed=D)
    assert p.dev.scratch.numel() == p.n_pages * 2 * 16 * queries
    p.append([50, 7])
    key = D * (32 if fmt == F8 else 34) // 32
    for T in (1, 2, 3, 5):
        if T > max_t:
            break
        p.dev.scratch.fill_(float("nan"))
        p.dev.scores.zero_()
        q = p.randn(2, T, 2 * hpk, D)
        p.dev.decode_scored(q.cuda(), p.tables, p.lens())
        kept = hpk * T <= 8 and 8 * hpk * T < key
        assert bool((~torch.isnan(p.dev.scratch)).any()) == kept, T
        gain = gains(p, q)
        for b in range(2):
            near(scores_of(p, b), np.zeros(gain[b].shape), gain[b], 1.0)
    assert p.dev.device_error() == 0


def test_caches_of_one_stream_share_the_room():
    """Two caches with one buffer for kept scores, their calls by turns: scores as with one each."""
    need_gpu()
    n, Hkv, D, page, mp, T = 5, 2, 128, 16, 80, 2
    g = torch.Generator().manual_seed(11)
    tab = torch.randperm(n * mp, generator=g).view(n, mp).int().cuda()
    lens = i32([1280, 1, 700, 16, 999])
    k = [torch.randn(n, 1280, Hkv, D, generator=g).cuda() for _ in range(2)]
    q = [torch.randn(n, T, 4 * Hkv, D, generator=g).cuda() for _ in range(2)]
    got = []
    for shared in (False, True):
        c = [PagedKVCache(n * mp, page, Hkv, D, 4 * Hkv, max_seqs=n, max_pages=mp, max_t=T, scores=True, score_scratch=not shared) for _ in range(2)]
        room = torch.empty(n * mp * page * Hkv * 4 * T, device="cuda")
        for x, y in zip(c, k):
            x.append(y, y, tab, i32([1280] * n))
            if shared:
                B.kvq_paged_set_score_scratch(x.handle, room.data_ptr(), 4 * T)
        torch.cuda.synchronize()
        for _ in range(20):
            for x, y in zip(c, q):
                x.decode_scored(y, tab, lens)
        got.append([x.scores.clone() for x in c])
        assert all(x.device_error() == 0 for x in c)
    assert all(torch.equal(x, y) for x, y in zip(*got))


# ------------------------------------------------------------------ eviction

def test_a_move_of_many_rows_renews_its_bounds():
    """n * keep * KV heads beyond 2^31: a list of a table's full length, sequences of 300 rows."""
    need_gpu()
    n, Hkv, D, page, mp, L = 17, 8, 64, 256, 65536, 300
    keep = page * mp
    assert n * keep * Hkv > 1 << 31
    c = PagedKVCache(4 * n, page, Hkv, D, Hkv, max_seqs=n, max_pages=mp, bounds=True)
    c.pool.zero_()
    tables, into = (torch.zeros(n, mp, dtype=torch.int32, device="cuda") for _ in range(2))
    tables[:, :2] = torch.arange(2 * n, dtype=torch.int32, device="cuda").view(n, 2)
    into[:, :2] = torch.arange(2 * n, 4 * n, dtype=torch.int32, device="cuda").view(n, 2)
    g = torch.Generator().manual_seed(7)
    k = torch.randn(n, L, Hkv, D, generator=g).cuda()
    lens = i32([L] * n)
    c.append(k, k, tables, lens)
    rows = torch.empty(n, Hkv, keep, dtype=torch.int32, device="cuda")     # (all of a list but its first rows is not read)
    rows[:, :, :L] = torch.arange(L, dtype=torch.int32, device="cuda")
    c.bounds.fill_(77)
    want = c.bounds.clone()
    new = c.compact(tables, lens, rows, tables_out=into)
    assert new.tolist() == [L] * n
    got = c.bounds.clone()
    c.bounds.copy_(want)
    c.update_bounds(into, new, L)
    assert torch.equal(got, c.bounds) and not torch.equal(got, want)
    ko, vo = (torch.empty(n, L, Hkv, D, device="cuda") for _ in range(2))
    kn, vn = torch.empty_like(ko), torch.empty_like(vo)
    c.read(tables, lens, ko, vo)
    c.read(into, new, kn, vn)
    assert torch.equal(ko, kn) and torch.equal(vo, vn) and c.device_error() == 0
