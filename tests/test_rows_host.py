"""Row positions, row scores, eviction and draft verification, host side (no
GPU): refusals that come before anything is enqueued, and pins of the oracle."""

import ctypes

import numpy as np
import pytest

from oracle import kvq_paged_oracle as P
from quantized_kv_cache_08_gb300 import _binding as B
from quantized_kv_cache_08_gb300 import build as kbuild


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return B.lib()


def args(**kw):
    d = dict(target=16, draft=16, tokens=16, uniform=16, dtype=B.KVQ_F32, n_seq=2, T=3, vocab=10, target_seq=30,
             target_row=10, draft_seq=20, draft_row=10, accept=16, next=16, lens=16)
    d.update(kw)
    return B.kvq_verify_args(**d)


@pytest.mark.parametrize("kw", [
    dict(target=None), dict(uniform=None), dict(accept=None), dict(next=None), dict(tokens=None), dict(dtype=2),
    dict(dtype=-1), dict(n_seq=0), dict(n_seq=65537), dict(T=0), dict(T=513), dict(vocab=0), dict(vocab=(1 << 24) + 1),
    dict(target=18), dict(draft=18), dict(tokens=18), dict(uniform=17), dict(accept=18), dict(next=17), dict(lens=18),
    dict(target=17, dtype=B.KVQ_BF16), dict(target_seq=-1), dict(target_row=-1), dict(draft_seq=-1), dict(draft_row=-1),
])
def test_verify_refusals(L, kw):
    with pytest.raises(B.KvqError) as e:
        B.kvq_verify(args(**kw))
    assert e.value.status == B.KVQ_EINVAL and str(e.value)


def test_null_arguments(L):
    q = B.kvq_paged_query()
    assert L.kvq_verify(None, None) == B.KVQ_EINVAL
    for call in (
            lambda: B.kvq_paged_append_at(None, 16, 256, 16, 256, None, 0, None, 0, 0, 16, 16, 1, 1, None, 1, 16),
            lambda: B.kvq_paged_set_axes(None, [0], 1), lambda: B.kvq_paged_set_scores(None, 16),
            lambda: B.kvq_paged_set_score_scratch(None, 16, 1),
            lambda: B.kvq_paged_decode_scored(None, q, 1.0), lambda: B.kvq_paged_select_rows(None, 16, 16, 1, 4, 0, 0, 16),
            lambda: B.kvq_paged_compact(None, 16, 16, 1, 16, 4, None, 16)):
        with pytest.raises(B.KvqError) as e:
            call()
        assert e.value.status == B.KVQ_EINVAL


def test_verify_struct_matches_the_header():
    # 4 pointers, 4 ints, 4 strides, 3 pointers
    assert ctypes.sizeof(B.kvq_verify_args) == 4 * 8 + 4 * 4 + 4 * 8 + 3 * 8


# ------------------------------------------------------------------ pins of the oracle

def test_oracle_rotation_on_axes():
    r = np.random.default_rng(0)
    x = r.standard_normal((4, 2, 32))
    pos = r.integers(0, 500, (4, 3))
    axes = [0, 1, 2, 1, 0, 2, 2, 1]
    one = P.rotate(x, pos[:, 1], 16)
    assert np.array_equal(P.rotate(x, np.repeat(pos[:, 1:2], 3, 1), 16, axes=axes), one)
    y = P.rotate(x, pos, 16, axes=axes)
    a = pos[:, 2] * 10000.0 ** (-2 * 5 / 16)
    assert np.allclose(y[:, 0, 5], x[:, 0, 5] * np.cos(a) - x[:, 0, 13] * np.sin(a))


def test_oracle_weights_give_its_attention():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal(32), r.standard_normal((9, 32)), r.standard_normal((9, 32))
    see = np.array([0, 1, 1, 0, 1, 1, 1, 1, 0])
    for kw in (dict(), dict(sink=0.3), dict(softcap=2.0)):
        assert np.allclose(P.weights(q, k, see, **kw) @ v, P.attend(q, k, v, see, **kw)[0])
    assert (P.weights(q, k, np.zeros(9)) == 0).all()


def test_oracle_verify_keeps_the_targets_distribution():
    """Over all uniforms, accepted drafts and draws together follow the target."""
    r = np.random.default_rng(2)
    V, N = 4, 200
    p, q = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    grid = (np.arange(N) + 0.5) / N
    mass = np.zeros(V)
    for d in range(V):
        for u in grid:
            a, n = P.verify(np.stack([p, p]), q[None], [d], np.array([u, 0.0]))
            if a == 2:
                mass[d] += q[d] / N
            else:
                for v in grid:
                    mass[P.verify(np.stack([p, p]), q[None], [d], np.array([u, v]))[1]] += q[d] / N / N
    assert np.abs(mass - p).max() <= 2.0 / N + 1e-9       # each grid is off by at most a step
