"""Oracle of speculative decoding over a paged cache (test infrastructure; see
the package header): attention of a tree of drafted tokens, and the move of
the accepted path's K/V.

The caches are plain arrays [num_blocks, H_kv, block_size, D]; everything is
fp64, one row and one token at a time.  Definitions:

    sequence i has n_i = query_start[i+1] - query_start[i] drafted tokens at
    positions c_i + u (c_i = context_lens[i] - n_i); row j of it sees the
    positions t < c_i, and c_i + u wherever sees[i][j][u] is true;
    out[r, h] = sum_seen softmax(scale * <q[r,h], K[t, h // G]>)_t V[t, h // G],
    and zero if it sees nothing.
"""

from __future__ import annotations

from typing import List, Sequence, Tuple

import numpy as np


def token(cache: np.ndarray, table: Sequence[int], t: int) -> np.ndarray:
    """Row t of the sequence that a block table names: [H_kv, D]."""
    bs = cache.shape[2]
    return cache[int(table[t // bs]), :, t % bs, :]


def ancestors(parents: Sequence[int]) -> np.ndarray:
    """sees[j, u]: u is j itself or an ancestor of it (parent -1: the context)."""
    n = len(parents)
    sees = np.zeros((n, n), bool)
    for j in range(n):
        u = j
        while u >= 0:
            sees[j, u] = True
            u = parents[u]
    return sees


def pack_mask(sees: Sequence[np.ndarray], rows: int, words: int) -> np.ndarray:
    """int32 [rows, words] of the sequences' sees matrices, one after another."""
    out = np.zeros((rows, words), np.uint32)
    r = 0
    for s in sees:
        for j in range(s.shape[0]):
            for u in np.nonzero(s[j])[0]:
                out[r, u // 32] |= np.uint32(1 << (int(u) % 32))
            r += 1
    return out.view(np.int32)


def tree_attention(q: np.ndarray, kc: np.ndarray, vc: np.ndarray, tables, context_lens, sees: List[np.ndarray],
                   scale: float) -> Tuple[np.ndarray, np.ndarray]:
    """(out, mag), both [sum n_i, H, D] fp64; mag = sum_t p_t |V_t|, the size
    of what the output sums, which rounding errors are proportional to."""
    H, D = q.shape[1:]
    G = H // kc.shape[1]
    out = np.zeros(q.shape, np.float64)
    mag = np.zeros(q.shape, np.float64)
    r = 0
    for i, s in enumerate(sees):
        n, c = s.shape[0], int(context_lens[i]) - s.shape[0]
        for j in range(n):
            pos = list(range(c)) + [c + u for u in range(n) if s[j, u]]
            if pos:
                k = np.stack([token(kc, tables[i], t) for t in pos]).astype(np.float64)
                v = np.stack([token(vc, tables[i], t) for t in pos]).astype(np.float64)
                for h in range(H):
                    z = scale * (k[:, h // G] @ q[r, h].astype(np.float64))
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[r, h] = p @ v[:, h // G]
                    mag[r, h] = p @ np.abs(v[:, h // G])
            r += 1
    return out, mag


def tree_commit(cache: np.ndarray, tables, context_lens, drafts, paths) -> np.ndarray:
    """The cache after every sequence's accepted path moved to the positions
    right after its context (a copy; the argument is left alone)."""
    out = cache.copy()
    for i, path in enumerate(paths):
        c = int(context_lens[i]) - int(drafts[i])
        rows = [token(cache, tables[i], c + u).copy() for u in path]
        for k, row in enumerate(rows):
            token(out, tables[i], c + k)[...] = row
    return out
