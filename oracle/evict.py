"""Oracle of bounding a paged cache by accumulated attention weight (test
infrastructure; see the package header): the decode that accumulates, and
the choice and move of the tokens that stay.  Plain arrays, fp64, one token
at a time."""

from __future__ import annotations

from typing import List, Sequence, Tuple

import numpy as np

from .tree import token


def scored_decode(q: np.ndarray, kc: np.ndarray, vc: np.ndarray, tables, context_lens, scale: float,
                  scores: np.ndarray) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """(out, mag, scores after, weight added): pa_decode's output, sum_t p_t
    |V_t|, and scores[i, g, t] + sum over the heads of group g of p_t."""
    B, H, D = q.shape
    hk = kc.shape[1]
    G = H // hk
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    add = np.zeros(scores.shape)
    for i in range(B):
        n = int(context_lens[i])
        if n == 0:
            continue
        k = np.stack([token(kc, tables[i], t) for t in range(n)]).astype(np.float64)
        v = np.stack([token(vc, tables[i], t) for t in range(n)]).astype(np.float64)
        for h in range(H):
            z = scale * (k[:, h // G] @ q[i, h].astype(np.float64))
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h] = p @ v[:, h // G]
            mag[i, h] = p @ np.abs(v[:, h // G])
            m = min(n, scores.shape[2])
            add[i, h // G, :m] += p[:m]
    return out, mag, scores.astype(np.float64) + add, add


def kept_positions(score: Sequence[float], keep: int, num_sink: int, num_recent: int) -> List[int]:
    """Ascending positions that stay of len(score) tokens."""
    n = len(score)
    k = min(keep, n)
    recent = min(num_recent, k)
    sink = min(num_sink, k - recent)
    if k == n:
        return list(range(n))
    middle = list(range(sink, n - recent))
    rank = {t: (-np.inf if np.isnan(score[t]) else float(score[t])) for t in middle}
    best = sorted(middle, key=lambda t: (-rank[t], t))[: k - sink - recent]
    return sorted(list(range(sink)) + best + list(range(n - recent, n)))


def evict(kc: np.ndarray, vc: np.ndarray, tables, context_lens, scores, dst_tables, keep_lens, num_sink, num_recent,
          scores_out, kept_out):
    """Copies of (kc, vc, scores_out, kept_out) after the eviction."""
    k2, v2, so, ko = kc.copy(), vc.copy(), scores_out.copy(), kept_out.copy()
    for i in range(len(context_lens)):
        n = int(context_lens[i])
        for g in range(kc.shape[1]):
            pos = kept_positions(scores[i, g, :n], int(keep_lens[i]), num_sink, num_recent)
            so[i, g], ko[i, g] = 0, -1
            for j, t in enumerate(pos):
                ko[i, g, j] = t
                so[i, g, j] = scores[i, g, t]
                token(k2, dst_tables[i], j)[g] = token(kc, tables[i], t)[g]
                token(v2, dst_tables[i], j)[g] = token(vc, tables[i], t)[g]
    return k2, v2, so, ko
