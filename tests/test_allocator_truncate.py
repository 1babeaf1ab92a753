"""pa_seq_truncate and pa_seq_compact: the library's allocator against the
oracle's on random sessions, and what the rules promise, on a store model in
which every slot remembers the token written to it."""

import random
import subprocess
import sys
from pathlib import Path

import pytest

import paged_kv_cache_351_b200 as pa
from oracle.allocator import AllocatorError, BlockAllocator, OutOfBlocks

ROOT = Path(__file__).resolve().parent.parent


def same(c, o):
    assert c.num_free() == o.num_free()
    assert [c.refcount(b) for b in range(o.num_blocks)] == [o.refcount(b) for b in range(o.num_blocks)]
    for s in o.sequences():
        assert c.block_table(s) == o.block_table(s) and c.length(s) == o.length(s)
    assert c.evictable() == list(o._evictable) and c.stats()["num_cached"] == o.num_cached()
    assert c.stats()["waste_slots"] == o.waste_slots()


@pytest.mark.parametrize("seed", range(10))
def test_random_sessions_match_and_keep_contents(seed):
    """Prefix hits, forks, appends, truncations and compactions: the states
    agree, and a sequence whose token ids are known reads them back from the
    slots, whoever wrote those slots (no registered block is overwritten)."""
    rnd = random.Random(700 + seed)
    nb, bs = 40, 4
    order = list(range(nb))
    rnd.shuffle(order)
    c, o = pa.Allocator(nb, bs, order), BlockAllocator(nb, bs, order)
    store, want = {}, {}  # slot -> token, sequence -> tokens
    nxt = 0
    for step in range(600):
        r = rnd.random()
        live = list(want)
        if r < 0.2 or not live:
            prompt = [rnd.randrange(2) for _ in range(rnd.randrange(1, 16))]
            hit = o.add_prefix(nxt, prompt)
            assert c.add_prefix(nxt, prompt) == hit
            want[nxt] = prompt[:hit]
            nxt += 1
        elif r < 0.3:
            p = rnd.choice(live)
            c.fork(p, nxt), o.fork(p, nxt)
            want[nxt] = list(want[p])
            nxt += 1
        elif r < 0.4:
            s = rnd.choice(live)
            c.free(s), o.free(s)
            del want[s]
        elif r < 0.55:
            s = rnd.choice(live)
            n = rnd.randrange(0, o.length(s) + 1)
            c.truncate(s, n), o.truncate(s, n)
            want[s] = want[s][:n]
        elif r < 0.65:
            ss = rnd.sample(live, rnd.randrange(1, min(3, len(live)) + 1))
            kept = [sorted(rnd.sample(range(o.length(s)), rnd.randrange(0, o.length(s) + 1))) for s in ss]
            lens = [len(k) for k in kept]
            src = [[o.slot(s, t) for t in k] for s, k in zip(ss, kept)]
            old = {b for s in ss for b in o.block_table(s)}
            try:
                fresh = o.compact(ss, lens)
            except OutOfBlocks:
                with pytest.raises(pa.OutOfBlocksError):
                    c.compact(ss, lens, 20)
            else:
                got = c.compact(ss, lens, 20)
                assert [[b for b in row if b >= 0] for row in got.tolist()] == fresh
                assert not old & {b for row in fresh for b in row}  # moves in any order are safe
                for s, k, xs in zip(ss, kept, src):
                    for t, x in enumerate(xs):
                        store[o.slot(s, t)] = store[x]
                    want[s] = [want[s][t] for t in k]
        else:
            s = rnd.choice(live)
            known = o._tokens.get(s) is not None and rnd.random() < 0.8
            toks = [rnd.randrange(2) for _ in range(rnd.choice([1, 2, 3, 5, 9]))]
            call = (lambda a: a.append_tokens(s, toks)) if known else (lambda a: a.append(s, len(toks)))
            try:
                slots, cow = call(o)
            except OutOfBlocks:
                with pytest.raises(pa.OutOfBlocksError):
                    call(c)
            else:
                cs, cc = call(c)
                assert cs.tolist() == slots and cc == cow
                for a, b in cow:
                    for k in range(bs):
                        if a * bs + k in store:
                            store[b * bs + k] = store[a * bs + k]
                for x, t in zip(slots, toks):
                    store[x] = t
                want[s] = want[s] + toks
        same(c, o)
        for s, toks in want.items():
            assert [store[o.slot(s, t)] for t in range(len(toks))] == toks, (step, s)


def test_truncated_registered_block_loses_its_key_when_written():
    a = pa.Allocator(8, 4)
    a.add(0)
    a.append_tokens(0, [1, 2, 3, 4, 5, 6, 7, 8])
    assert a.stats()["num_cached"] == 2
    a.truncate(0, 6)
    assert a.stats()["num_cached"] == 2  # intact so far: another request may still use it
    assert a.add_prefix(1, [1, 2, 3, 4, 5, 6, 7, 8, 9]) == 8
    slots, cow = a.append_tokens(0, [9])
    assert len(cow) == 1  # shared now: copied
    a.free(1)
    a.truncate(0, 3)
    slots, cow = a.append_tokens(0, [9])
    assert cow == [] and slots[0] == a.block_table(0)[0] * 4 + 3
    # the old key [1, 2, 3, 4] is gone; the block is registered again under [1, 2, 3, 9]
    assert a.add_prefix(2, [1, 2, 3, 4, 5]) == 0
    assert a.add_prefix(3, [1, 2, 3, 9, 5]) == 4


def test_refusals():
    a = pa.Allocator(8, 4)
    a.set_host_pool(4)
    a.add(0)
    a.append(0, 9)
    one = lambda seq, n: a.compact([seq], [n], 4)  # noqa: E731
    for fn in (a.truncate, one):
        for seq, n in ((0, 10), (0, -1), (1, 0)):
            with pytest.raises(pa.PagedAttentionError) as e:
                fn(seq, n)
            assert e.value.status == 1
    table, free = a.block_table(0), a.num_free()
    a.add(1)
    a.append(1, 4 * (free - 2))
    for args, status in ((([0], [9], 4), 3), (([0, 1], [4, 8], 4), 3), (([0], [9], 2), 1), (([0, 0], [1, 1], 4), 1)):
        with pytest.raises(pa.PagedAttentionError) as e:
            a.compact(*args)  # 2 blocks are free
        assert e.value.status == status
        assert a.block_table(0) == table and a.length(0) == 9
    fresh = a.compact([0], [5], 3).tolist()[0]
    assert fresh[2] == -1 and not set(fresh[:2]) & set(table) and a.num_free() == 3
    a.swap_out(0)
    for fn in (a.truncate, one):
        with pytest.raises(pa.PagedAttentionError):
            fn(0, 1)
    assert a.compact([], [], 3).shape == (0, 3)
    o = BlockAllocator(8, 4)
    o.add(0)
    with pytest.raises(AllocatorError):
        o.truncate(0, 1)


def test_compact_without_host_memory_changes_nothing():
    """A child process with no room for the second sequence's table: the call
    is refused with PA_ERR_HOST_ALLOC and the first keeps its blocks."""
    code = (
        "import ctypes, resource\n"
        "import numpy as np\n"
        "import paged_kv_cache_351_b200 as pa\n"
        "n = 2 << 20\n"
        "a = pa.Allocator(2 * n + 40, 1)\n"
        "for s, k in ((0, 10), (1, n)):\n"
        "    a.add(s)\n"
        "    a.append(s, k)\n"
        "before = a.num_free(), a.block_table(0)\n"
        "out, ids, lens = np.zeros((2, n), np.int32), np.array([0, 1]), np.array([10, n], np.int32)\n"
        "out[:] = 0\n"
        "libc = ctypes.CDLL(None)\n"
        "libc.malloc.restype = ctypes.c_void_p\n"
        "resource.setrlimit(resource.RLIMIT_AS, (1 << 20, resource.RLIM_INFINITY))\n"
        "while libc.malloc(1 << 20):\n"
        "    pass\n"
        "try:\n"
        "    pa._check(pa.library().pa_seq_compact(a._h, pa._i64p(ids), pa._i32p(lens), 2, "
        "pa._i32p(out), n), 'pa_seq_compact')\n"
        "    status = 0\n"
        "except pa.PagedAttentionError as e:\n"
        "    status = e.status\n"
        "resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))\n"
        "print(status, before == (a.num_free(), a.block_table(0)))\n"
    )
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120, cwd=ROOT)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.split() == ["8", "True"]
