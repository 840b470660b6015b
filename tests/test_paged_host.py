"""Paged cache, host side (no GPU): configuration checks, sizes, refusals of
every call, and pins of the oracle."""

import ctypes

import numpy as np
import pytest

from oracle import kvq_oracle as O
from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300 import build as kbuild


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return B.lib()


BASE = dict(n_pages=10, page_rows=16, n_kv_heads=2, head_dim=128, max_q_heads=8, max_seqs=4, max_pages=6)


def test_sizes(L):
    s = B.kvq_paged_required_bytes(B.make_paged_config(**BASE))
    assert s.cell_bytes == 928 * 4 and s.page_bytes == 2 * s.cell_bytes and s.pool == 10 * s.page_bytes
    assert s.bounds == 0 and s.workspace > 0
    s = B.kvq_paged_required_bytes(B.make_paged_config(**dict(BASE, page_rows=64), bounds=1, k_fmt=B.KVQ_FP8_E4M3,
                                                       v_fmt=B.KVQ_FP8_E4M3))
    assert s.cell_bytes == 1024 * 4 and s.page_bytes == 2 * 4 * s.cell_bytes and s.bounds >= 10 * 2 * 4 * 68


@pytest.mark.parametrize("kw,status", [
    (dict(n_pages=0), B.KVQ_EINVAL), (dict(page_rows=8), B.KVQ_EINVAL), (dict(page_rows=48), B.KVQ_EINVAL),
    (dict(page_rows=512), B.KVQ_EINVAL), (dict(n_kv_heads=0), B.KVQ_EINVAL), (dict(n_kv_heads=129), B.KVQ_EINVAL),
    (dict(head_dim=96), B.KVQ_EUNSUPPORTED), (dict(head_dim=32), B.KVQ_EUNSUPPORTED), (dict(max_q_heads=7), B.KVQ_EINVAL),
    (dict(max_q_heads=0), B.KVQ_EINVAL), (dict(max_q_heads=2 * 129), B.KVQ_EINVAL), (dict(max_seqs=0), B.KVQ_EINVAL),
    (dict(max_seqs=1025), B.KVQ_EINVAL), (dict(max_pages=0), B.KVQ_EINVAL), (dict(max_pages=(1 << 20) + 1), B.KVQ_EINVAL),
    (dict(max_t=0), B.KVQ_EINVAL), (dict(max_t=65), B.KVQ_EINVAL), (dict(rope_dim=8), B.KVQ_EINVAL),
    (dict(rope_dim=144), B.KVQ_EINVAL), (dict(rope_dim=-16), B.KVQ_EINVAL),
    (dict(k_fmt=B.KVQ_Q5_1), B.KVQ_EUNSUPPORTED), (dict(v_fmt=B.KVQ_FP8_E4M3), B.KVQ_EUNSUPPORTED),
])
def test_bad_configurations(L, kw, status):
    cfg = B.make_paged_config(**dict(BASE, **kw))
    for call in (lambda: B.kvq_paged_required_bytes(cfg), lambda: B.kvq_paged_alloc(cfg, 16, 16, 16)):
        with pytest.raises(B.KvqError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("kw,args", [
    ({}, (None, None, 16)), ({}, (16, None, None)), (dict(bounds=1), (16, None, 16)), ({}, (8, None, 16)),
    ({}, (16, None, 24)), (dict(bounds=1), (16, 17, 16)), (dict(rope_dim=16, rope_base=0.0), (16, None, 16)),
    (dict(rope_dim=16, rope_base=float("nan")), (16, None, 16)),
])
def test_alloc_refusals(L, kw, args):
    with pytest.raises(B.KvqError) as e:
        B.kvq_paged_alloc(B.make_paged_config(**dict(BASE, **kw)), *args)
    assert e.value.status == B.KVQ_EINVAL


def test_alloc_refuses_frequencies(L):
    for bad in (65.0, float("inf"), float("nan")):
        with pytest.raises(B.KvqError) as e:
            B.kvq_paged_alloc(B.make_paged_config(**BASE, rope_dim=16), 16, None, 16, [0.1] * 7 + [bad])
        assert e.value.status == B.KVQ_EINVAL


def test_null_handles(L):
    q = B.kvq_paged_query()
    for call in (
            lambda: B.kvq_paged_append(None, 16, 256, 16, 256, None, 0, None, 0, 0, 16, 16, 1, 1, None, 1),
            lambda: B.kvq_paged_read(None, 16, 16, 0, 16, 16, 1, 1, None, 1),
            lambda: B.kvq_paged_bounds(None, 16, 16, 1, 1, None, 1),
            lambda: B.kvq_paged_decode(None, q), lambda: B.kvq_paged_decode_shared(None, q, 16, 16, 1),
            lambda: B.kvq_paged_select(None, q, 16, 1, 0, 0), lambda: B.kvq_paged_decode_sparse(None, q, 16, 1),
            lambda: B.kvq_paged_read_error(None)):
        with pytest.raises(B.KvqError) as e:
            call()
        assert e.value.status == B.KVQ_EINVAL
    L.kvq_paged_free(None)


# ------------------------------------------------------------------ pins of the oracle

def test_oracle_rotation():
    x = np.random.default_rng(0).standard_normal((5, 2, 64))
    pos = np.array([0, 1, 7, 1000, 131071])
    for inter in (False, True):
        y = P.rotate(x, pos, 32, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
        i = 3
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 16)
        ang = 7 * 10000.0 ** (-2 * i / 32)
        assert np.allclose(y[2, :, a], x[2, :, a] * np.cos(ang) - x[2, :, b] * np.sin(ang))
        assert np.allclose(y[2, :, b], x[2, :, a] * np.sin(ang) + x[2, :, b] * np.cos(ang))
        # products depend on the distance alone
        u, w = P.rotate(x, pos + 13, 32, inter), P.rotate(x[::-1], pos[::-1] + 13, 32, inter)
        assert np.allclose((u * w).sum(-1), (y * P.rotate(x[::-1], pos[::-1], 32, inter)).sum(-1))


def test_oracle_cell_places_every_byte_once():
    for fmt in ("q8_0/q5_1", "e4m3"):
        NB = 4
        cell = np.zeros(P.cell_bytes(32 * NB, fmt), np.uint8)
        full = np.full(32, 0xFF, np.uint8)
        one = (full, full) if fmt == "e4m3" else (np.concatenate([[255, 255], np.full(32, 127)]).astype(np.uint8),
                                                  np.full(24, 255, np.uint8))
        seen = np.zeros_like(cell, dtype=np.int64)
        for t in range(16):
            cell[:] = 0
            P.put_row(cell, t, np.stack([one[0]] * NB), np.stack([one[1]] * NB), fmt)
            seen += np.unpackbits(cell.reshape(-1, 1), axis=1).sum(1).astype(np.int64)
        assert (seen == 8).all()


def test_oracle_attention_is_softmax():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal(32), r.standard_normal((9, 32)), r.standard_normal((9, 32))
    s = k @ q / np.sqrt(32)
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(P.attend(q, k, v, np.ones(9))[0], w @ v)
    assert np.allclose(P.attend(q, k, v, np.ones(9))[0], O.attend(q[None, None], k[:, None], v[:, None])[0, 0])
    twice = np.ones(9)
    twice[4] = 2
    assert np.allclose(P.attend(q, k, v, twice)[0], P.attend(q, np.vstack([k, k[4:5]]), np.vstack([v, v[4:5]]), np.ones(10))[0])
    assert (P.attend(q, k, v, np.zeros(9), sink=1.0)[0] == 0).all()


def test_oracle_bounds_and_selection():
    r = np.random.default_rng(2)
    k = P.values(P.blocks(r.standard_normal((16, 1, 64)), "q8_0/q5_1", "k"), "q8_0/q5_1", "k")[:, 0]
    c, d = P.bounds(k)
    lo, hi = c[:, 0] * d[:, None].astype(np.float64), c[:, 1] * d[:, None].astype(np.float64)
    y = k.reshape(16, 2, 32)
    slack = d[:, None] * 1e-5
    assert (lo <= y.min(0) + slack).all() and (hi >= y.max(0) - slack).all()
    assert (P.bounds(np.zeros((3, 64)))[0] == 0).all()
    assert P.select(np.array([1.0, 5, 5, 2, 9]), 3, 0, 0) == [1, 2, 4]
    assert P.select(np.array([1.0, 5, 5, 2, 9]), 3, 1, 1) == [0, 1, 4]
    assert P.select(np.array([0.0, 0, 0, 0]), 2, 0, 1) == [0, 3]
