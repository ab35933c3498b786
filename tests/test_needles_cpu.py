"""The bound of the needle rows tells a kernel's errors from its roundings."""
import numpy as np
import pytest

from tests import helpers as H
from tests import serving_helpers as S
from tests import serving_needles as D


def rows_of(mode, n, rows, seed):
    rec = H.random_cache(mode, 1, 1, (n + 15) // 16 * 16, seed)
    K, V = S.kv_of(mode, rec, 0, 0, n)
    rng = np.random.default_rng(seed)
    pairs = [sorted(rng.choice(n, 2, replace=False)) for _ in range(rows)]
    q = np.array([D.needle_query(K, a, b) for a, b in pairs])
    return K, V, pairs, q, np.ones((rows, n), bool)


def attend(q_rot, K, V, seen):
    s = np.where(seen, q_rot @ D.rot(K).T * D.SCALE, -np.inf)
    w = np.exp(s - s.max(1, keepdims=True))
    return (w / w.sum(1, keepdims=True)) @ V


@pytest.mark.parametrize("mode", ["turbo3", "turbo4", "turbo4k_3v"])
def test_the_bound_tells_the_low_half_of_the_query(mode):
    K, V, _, q, seen = rows_of(mode, 517, 96, 5)
    want, bound = D.needle_rows(q, K, V, seen, True)
    full = D.rot(q)
    hi = full.astype(np.float16).astype(np.float64)
    both = hi + (full - hi).astype(np.float16)
    err = lambda x: np.linalg.norm(attend(x, K, V, seen) - want, axis=1)  # noqa: E731
    assert np.all(err(both) < 0.2 * bound)
    assert np.mean(err(hi) > bound) > 0.3        # (any row past its bound fails a test)


@pytest.mark.parametrize("mode", ["turbo3", "turbo4_asym", "turbo3_table"])
def test_the_bound_tells_a_token_too_few_or_too_many(mode):
    K, V, pairs, q, seen = rows_of(mode, 300, 48, 7)
    want, bound = D.needle_rows(q, K, V, seen, mode != "turbo4_asym")
    for r, (a, b) in enumerate(pairs):
        less = seen[r:r + 1].copy()
        less[0, b] = False
        one, one_bound = D.needle_rows(q[r:r + 1], K, V, less, mode != "turbo4_asym")
        far = np.linalg.norm(one[0] - want[r])
        assert far > 20 * bound[r] and far > 20 * one_bound[0]
