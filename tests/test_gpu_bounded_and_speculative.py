"""The new operators together, as a serving loop uses them through
PagedKVCacheGPU: speculative decoding that must give what token-by-token
decoding gives, and generation under a token budget, against a plain model
that keeps lists of tokens in fp64."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_351_b200 as pa
from gpu_harness import check_status_clean
from oracle.evict import kept_positions
from oracle.tree import ancestors, pack_mask
from paged_kv_cache_351_b200.runtime import PagedKVCacheGPU

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, HK, D, VOCAB = 4, 2, 64, 37
SCALE = 1.0 / math.sqrt(D)


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)


class Model:
    """One attention layer whose queries, keys and values are looked up by
    token; the next token is the argmax of a projection of its output."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.k = torch.randn(VOCAB, HK, D, generator=g).to(DEV)
        self.v = torch.randn(VOCAB, HK, D, generator=g).to(DEV)
        self.q = (2 * torch.randn(VOCAB, H, D, generator=g)).to(DEV)
        self.w = torch.randn(H * D, VOCAB, generator=g).to(DEV)

    def write(self, cache, slots, tokens, pairs=None):
        t = torch.as_tensor(tokens, device=DEV, dtype=torch.long)
        pr = None if pairs is None else torch.as_tensor(np.asarray(pairs, np.int64).reshape(-1, 2)).to(DEV)
        cache.write(torch.as_tensor(np.asarray(slots, np.int64)).to(DEV), self.k[t], self.v[t], pairs=pr)

    def next(self, out):
        return (out.reshape(-1, H * D).double() @ self.w.double()).argmax(dim=1).tolist()

    def decode(self, cache, seqs, last):
        """Next token of each sequence whose newest cached token is last[k]."""
        bt, cl = cache.block_tables(seqs, 32)
        out = torch.empty(len(seqs), H, D, device=DEV)
        q = self.q[torch.as_tensor(last, device=DEV)]
        return self.next(cache.decode(out, q, i32(bt), i32(cl), SCALE))


def test_speculative_decoding_equals_token_by_token():
    """Three prompts, drafts that mix right and wrong branches; the accepted
    tokens and the cache are those of plain decoding, and the rejected slots
    come back."""
    m = Model()
    prompts = [[5, 9, 1], list(range(30)), [7] * 16]
    plain, spec = PagedKVCacheGPU(200, HK, D, "f32"), PagedKVCacheGPU(200, HK, D, "f32")
    for cache in (plain, spec):
        for s, p in enumerate(prompts):
            cache.add(s)
            slots, _ = cache.append([s], [len(p)])
            m.write(cache, slots, p)
    seqs = [0, 1, 2]
    want = [list(p) for p in prompts]
    for _ in range(90):  # more than any sequence can be ahead of the slowest
        nxt = m.decode(plain, seqs, [w[-1] for w in want])
        slots, pairs = plain.append(seqs, [1] * 3)
        m.write(plain, slots, nxt, pairs)
        for w, t in zip(want, nxt):
            w.append(t)

    rng = np.random.default_rng(1)
    have = [list(p) for p in prompts]
    steps = 0
    while min(len(h) - len(p) for h, p in zip(have, prompts)) < 20:
        steps += 1
        # the newest token of `have` is cached; its successor comes from the target itself
        first = m.decode(spec, seqs, [h[-1] for h in have])
        drafts, parents = [], []
        for s in seqs:
            at = len(have[s])
            right = want[s][at:at + 4]
            assert right[0] == first[s]
            # a root that the target gave, wrong siblings, and a branch that is right for a while
            tok, par = [first[s]], [-1]
            for depth in range(1, len(right)):
                parent = max(i for i in range(len(tok)) if i == 0 or par[i] >= 0 and tok[i] == right[depth - 1])
                tok += [(right[depth] + 1 + int(rng.integers(0, VOCAB - 1))) % VOCAB, right[depth]]
                if rng.random() < 0.3:
                    tok[-1] = (tok[-1] + 1) % VOCAB  # the draft errs
                par += [parent, parent]
            drafts.append(tok)
            parents.append(par)
        counts = [len(t) for t in drafts]
        base = [spec.alloc.length(s) for s in seqs]
        free = spec.alloc.num_free()
        slots, pairs = spec.append(seqs, counts)
        m.write(spec, slots, sum(drafts, []), pairs)
        bt, cl = spec.block_tables(seqs, 32)
        qs = i32(np.concatenate([[0], np.cumsum(counts)]))
        T, n = sum(counts), max(counts)
        mask = torch.from_numpy(pack_mask([ancestors(p) for p in parents], T, 1)).to(DEV)
        out = torch.empty(T, H, D, device=DEV)
        q = m.q[torch.as_tensor(sum(drafts, []), device=DEV)]
        spec.tree_attention(out, q, i32(bt), i32(cl), qs, mask, n, SCALE)
        target = m.next(out)
        acc = np.zeros((3, 8), np.int32)
        cnt = []
        off = 0
        for s in seqs:
            path = [0]
            while True:
                ahead = [i for i in range(len(drafts[s])) if parents[s][i] == path[-1] and
                         drafts[s][i] == target[off + path[-1]]]
                if not ahead:
                    break
                path.append(ahead[0])
            acc[s, :len(path)] = path
            cnt.append(len(path))
            have[s] += [drafts[s][i] for i in path]
            off += counts[s]
        spec.tree_commit(i32(bt), i32(cl), qs, i32(acc), i32(cnt))
        for s in seqs:
            spec.truncate(s, base[s] + cnt[s])
            assert spec.alloc.length(s) == len(have[s])
        assert free - spec.alloc.num_free() == sum(-(-(b + c) // 16) - -(-b // 16) for b, c in zip(base, cnt))
    check_status_clean()
    assert steps < 20  # some drafts were accepted
    for s in seqs:
        assert have[s] == want[s][:len(have[s])]
        for cache_t, table_t in ((spec.k_cache, m.k), (spec.v_cache, m.v)):
            tab = spec.alloc.block_table(s)
            rows = torch.stack([cache_t[tab[t // 16], :, t % 16] for t in range(len(have[s]))])
            assert torch.equal(rows, table_t[torch.as_tensor(have[s], device=DEV)])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_generation_under_a_budget(dtype):
    """Scored decode, and an eviction whenever a sequence holds more than its
    budget; a fork of one sequence keeps its own blocks.  Scores, choices and
    outputs follow a plain fp64 model of per-head token lists."""
    d = 128 if dtype == "fp8" else D
    g = torch.Generator().manual_seed(3)
    kw = {}
    if dtype == "fp8":
        kw = dict(k_scale=torch.full((HK,), 0.02), v_scale=torch.full((HK,), 0.02))
    cache = PagedKVCacheGPU(64, HK, d, dtype, **kw)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}[dtype]
    B, cap, budget, sink, recent = 2, 96, 40, 2, 8
    start = [50, 20]
    rows = [[[] for _ in range(HK)] for _ in range(B)]  # per head: [k, v, score]

    def add(s, n):
        slots, pairs = cache.append([s], [n])
        k = torch.randn(n, HK, d, generator=g).to(dt)
        v = torch.randn(n, HK, d, generator=g).to(dt)
        cache.write(torch.from_numpy(slots).to(DEV), k.to(DEV), v.to(DEV), torch.from_numpy(pairs).to(DEV))
        if dtype == "fp8":
            code = lambda x: (x.float() / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).double() * float(  # noqa: E731
                np.float32(0.02))
            k, v = code(k), code(v)
        for t in range(n):
            for h in range(HK):
                rows[s][h].append([k[t, h].double().numpy(), v[t, h].double().numpy(), 0.0])

    for s in range(B):
        cache.add(s)
        add(s, start[s])
    scores = [torch.zeros(B, HK, cap, device=DEV), torch.full((B, HK, cap), 9.0, device=DEV)]
    scale = 1.0 / math.sqrt(d)
    tol = 1e-4 if dtype == "f32" else 2.0 ** -6
    forked = None
    for step in range(60):
        for s in range(B):
            add(s, 1)
        bt, cl = cache.block_tables([0, 1], 8)
        q = torch.randn(B, H, d, generator=g).to(dt)
        out = torch.empty(B, H, d, dtype=dt, device=DEV)
        cache.decode_scored(out, scores[0], q.to(DEV), i32(bt), i32(cl), scale)
        got = out.double().cpu().numpy()
        for s in range(B):
            for h in range(HK):
                k, v = (np.stack([r[x] for r in rows[s][h]]) for x in (0, 1))
                for j in range(h * (H // HK), (h + 1) * (H // HK)):
                    z = scale * (k @ q[s, j].double().numpy())
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    assert np.abs(got[s, j] - p @ v).max() <= tol
                    for r, w in zip(rows[s][h], p):
                        r[2] += w
        dev = scores[0].double().cpu().numpy()
        over = [s for s in range(B) if len(rows[s][0]) > budget + 10]
        for s in range(B):
            n = len(rows[s][0])
            for h in range(HK):
                assert np.abs(dev[s, h, :n] - [r[2] for r in rows[s][h]]).max() <= 1e-3
                for r, x in zip(rows[s][h], dev[s, h]):
                    r[2] = float(x)  # the device's sums decide, so that near ties do too
        if over and forked is None:
            cache.fork(over[0], 77)
            forked = ([[list(r) for r in rows[over[0]][h]] for h in range(HK)], cache.alloc.block_table(77))
            held = cache.k_cache[torch.as_tensor(forked[1], device=DEV)].view(torch.uint8).clone()
        if over:
            keep = [budget if s in over else len(rows[s][0]) for s in range(B)]
            kept = cache.evict([0, 1], keep, scores[0], scores[1], num_sink=sink, num_recent=recent).cpu().numpy()
            scores.reverse()
            for s in range(B):
                for h in range(HK):
                    pos = kept_positions([r[2] for r in rows[s][h]], keep[s], sink, recent)
                    assert kept[s, h, :len(pos)].tolist() == pos
                    rows[s][h] = [rows[s][h][t] for t in pos]
                assert cache.alloc.length(s) == len(rows[s][0]) == keep[s]
    check_status_clean()
    assert forked is not None and cache.alloc.block_table(77) == forked[1]
    assert torch.equal(cache.k_cache[torch.as_tensor(forked[1], device=DEV)].view(torch.uint8), held)


def test_evict_out_of_blocks_changes_nothing():
    cache = PagedKVCacheGPU(8, HK, D, "f32")
    cache.add(0)
    cache.append([0], [100])  # 7 of 8 blocks
    before = cache.alloc.block_table(0)
    s = torch.zeros(1, HK, 128, device=DEV)
    with pytest.raises(pa.OutOfBlocksError):
        cache.evict([0], [60], s, torch.zeros_like(s))
    assert cache.alloc.block_table(0) == before and cache.alloc.length(0) == 100
    with pytest.raises(ValueError):
        cache.evict([0], [10], s, s)
    with pytest.raises(ValueError):
        cache.evict([0], [10], s[:, :, :90], torch.zeros_like(s))
    assert cache.alloc.length(0) == 100
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = cache.evict([0], [10], s, torch.ones_like(s), num_recent=3, stream=side)
    side.synchronize()
    assert kept.tolist() == [[[0, 1, 2, 3, 4, 5, 6, 97, 98, 99]] * HK] and cache.alloc.length(0) == 10
    check_status_clean()
