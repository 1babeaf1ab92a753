"""Pins of the scored-decode and eviction oracles."""

import numpy as np
import pytest

from oracle.attention import paged_decode
from oracle.cache import PagedKVCache
from oracle.evict import evict, kept_positions, scored_decode


def test_scored_decode_is_decode_and_its_weights_sum_to_one():
    rng = np.random.default_rng(1)
    cache = PagedKVCache(4, 2, 8, 16, "f32")
    k, v = (rng.standard_normal((20, 2, 8)).astype(np.float32) for _ in range(2))
    tables = np.array([[3, 1], [-1, -1]])
    cache.write([int(tables[0, t // 16]) * 16 + t % 16 for t in range(20)], k, v)
    kc, vc = np.stack([cache.k_page(b) for b in range(4)]), np.stack([cache.v_page(b) for b in range(4)])
    q = rng.standard_normal((2, 4, 8)).astype(np.float32)
    out, mag, acc, add = scored_decode(q, kc, vc, tables, [20, 0], 0.4, np.ones((2, 2, 32)))
    assert np.abs(out - paged_decode(q, cache, tables, np.array([20, 0]), 0.4)).max() < 1e-12
    assert np.abs(add[0].sum(axis=1) - 2).max() < 1e-12 and (add[1] == 0).all()
    assert (acc == add + 1).all() and (mag >= np.abs(out) - 1e-12).all()
    one, _, _, add1 = scored_decode(q[:1, 2:3], kc[:, 1:], vc[:, 1:], tables[:1], [20], 0.4, np.zeros((1, 1, 32)))
    z = 0.4 * (k[:, 1].astype(np.float64) @ q[0, 2])
    assert np.abs(add1[0, 0, :20] - np.exp(z) / np.exp(z).sum()).max() < 1e-12


@pytest.mark.parametrize("score,keep,sink,recent,want", [
    ([5, 1, 4, 2, 3], 2, 0, 0, [0, 2]),
    ([1, 1, 1, 1], 2, 0, 0, [0, 1]),               # ties: the lower positions
    ([0, 9, 9, 0, 0], 3, 1, 1, [0, 1, 4]),
    ([3, 2, 1], 5, 1, 1, [0, 1, 2]),               # within the budget
    ([0, 9, 0, 0], 2, 4, 1, [0, 3]),               # the newest first, then the sinks
    ([9, 9, 0, 0], 2, 4, 7, [2, 3]),
    ([1, 2, 3], 0, 1, 1, []),
    ([np.nan, -np.inf, 1, -1], 3, 0, 0, [0, 2, 3]),  # NaN ranks with -infinity
    ([0.0, -0.0, 0.0], 1, 0, 0, [0]),
])
def test_kept_positions(score, keep, sink, recent, want):
    assert kept_positions(score, keep, sink, recent) == want


def test_evict_moves_each_heads_own_tokens():
    kc = np.arange(3 * 2 * 16 * 1).reshape(3, 2, 16, 1)
    s = np.zeros((1, 2, 16))
    s[0, 0, 3] = s[0, 1, 5] = 1
    k2, v2, so, ko = evict(kc, -kc, [[0]], [16], s, [[2]], [2], 0, 1, np.full((1, 2, 3), 7.0), np.full((1, 2, 2), 7))
    assert ko.tolist() == [[[3, 15], [5, 15]]] and so.tolist() == [[[1, 0, 0], [1, 0, 0]]]
    assert k2[2, 0, :2, 0].tolist() == kc[0, 0, [3, 15], 0].tolist()
    assert v2[2, 1, :2, 0].tolist() == (-kc)[0, 1, [5, 15], 0].tolist()
    assert np.array_equal(k2[:2], kc[:2]) and np.array_equal(k2[2, :, 2:], kc[2, :, 2:])
