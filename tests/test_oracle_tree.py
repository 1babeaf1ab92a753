"""Pins of the tree-attention oracle: a chain equals the causal (prefill)
oracle, a star of single tokens equals the decode oracle with one extra
token, and the commit of a path equals writing its tokens one by one."""

import math

import numpy as np
import pytest

from oracle.attention import paged_decode
from oracle.cache import PagedKVCache
from oracle.prefill import paged_prefill
from oracle.tree import ancestors, pack_mask, token, tree_attention, tree_commit


def state(seed, pairs, hk, D):
    rng = np.random.default_rng(seed)
    ctx = np.array([a + b for a, b in pairs])
    nbs = [-(-int(c) // 16) for c in ctx]
    NB = sum(nbs) + 2
    perm = rng.permutation(NB)
    tables = np.full((len(pairs), max(nbs) + 1), -1)
    cache = PagedKVCache(NB, hk, D, 16, "f32")
    kc, vc = np.full((NB, hk, 16, D), np.nan), np.full((NB, hk, 16, D), np.nan)
    off = 0
    for i, n in enumerate(nbs):
        tables[i, :n] = perm[off:off + n]
        off += n
        k = rng.standard_normal((ctx[i], hk, D)).astype(np.float32)
        v = rng.standard_normal((ctx[i], hk, D)).astype(np.float32)
        slots = [int(tables[i, t // 16]) * 16 + t % 16 for t in range(ctx[i])]
        cache.write(slots, k, v)
        for t in range(ctx[i]):
            token(kc, tables[i], t)[...] = k[t]
            token(vc, tables[i], t)[...] = v[t]
    T = sum(b for _, b in pairs)
    return rng, cache, kc, vc, tables, ctx, T


def test_chain_is_causal_attention():
    pairs = [(20, 5), (0, 9), (16, 1)]
    rng, cache, kc, vc, tables, ctx, T = state(1, pairs, 2, 8)
    q = rng.standard_normal((T, 4, 8)).astype(np.float32)
    sees = [ancestors(list(range(-1, n - 1))) for _, n in pairs]
    out, mag = tree_attention(q, kc, vc, tables, ctx, sees, 0.3)
    qs = np.concatenate([[0], np.cumsum([n for _, n in pairs])])
    assert np.abs(out - paged_prefill(q, cache, tables, ctx, qs, 0.3)).max() < 1e-12
    assert (mag >= np.abs(out) - 1e-12).all()


def test_star_is_a_decode_of_each_token():
    """Siblings do not see each other: row j is a decode over the context and token j."""
    rng, cache, kc, vc, tables, ctx, T = state(2, [(20, 4)], 2, 8)
    q = rng.standard_normal((T, 4, 8)).astype(np.float32)
    out, _ = tree_attention(q, kc, vc, tables, ctx, [ancestors([-1] * 4)], 0.3)
    for j in range(4):
        one = PagedKVCache(cache.num_blocks, 2, 8, 16, "f32")
        slots = [int(tables[0, t // 16]) * 16 + t % 16 for t in range(21)]
        src = list(range(20)) + [20 + j]
        rows = [cache.read_token(int(tables[0, t // 16]) * 16 + t % 16) for t in src]
        one.write(slots, np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows]))
        want = paged_decode(q[j:j + 1], one, tables, np.array([21]), 0.3)
        assert np.abs(out[j] - want[0]).max() < 1e-12


def test_ancestors_and_packing():
    s = ancestors([-1, 0, 0, 2, -1])
    assert s.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0],
                                      [0, 0, 0, 0, 1]]
    long = ancestors(list(range(-1, 39)))
    m = pack_mask([s, long], 46, 2).view(np.uint32)
    assert m[3, 0] == 0b1101 and m[5 + 39, 0] == 0xFFFFFFFF and m[5 + 39, 1] == 0xFF and m[45].tolist() == [0, 0]


def test_row_without_keys_is_zero():
    rng, _, kc, vc, tables, ctx, T = state(3, [(0, 3)], 1, 8)
    out, _ = tree_attention(rng.standard_normal((3, 1, 8)), kc, vc, tables, ctx, [np.zeros((3, 3), bool)], 1.0)
    assert (out == 0).all()


@pytest.mark.parametrize("path", [[], [0], [1, 3], [0, 1, 2, 3, 4, 5], [5]])
def test_commit_equals_appending_the_path(path):
    _, _, kc, _, tables, ctx, _ = state(4, [(14, 6)], 2, 4)
    got = tree_commit(kc, tables, ctx, [6], [path])
    want = kc.copy()
    for k, u in enumerate(path):
        want[tables[0, (14 + k) // 16], :, (14 + k) % 16] = kc[tables[0, (14 + u) // 16], :, (14 + u) % 16]
    assert np.array_equal(got, want, equal_nan=True)
    assert math.isnan(kc[tables[0, 1], 0, 15, 0])
