"""Host-side argument checking of tree attention, the accepted path's commit,
the scored decode, eviction and their workspace sizes, fuzzed on CPU: valid
descriptors with zero to two fields changed at random, odd scalars and
options.  Every call must return a documented status without crashing, in a
child process that sees no CUDA device (nothing can be launched on the fake
addresses)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, random, sys
import paged_kv_cache_351_b200 as pa
from paged_kv_cache_351_b200._lib import PaTensor, PaOpts

lib = pa.library()
VALS = [-1, 0, 1, 2, 3, 4, 8, 15, 16, 17, 32, 64, 127, 128, 129, 256, 65535, 65536, 1 << 20,
        2**31 - 1, 2**31, 2**32, 2**40, 2**62]
ADDR = 1 << 30  # never dereferenced: no device is visible


def tensor(shape, dtype, at=ADDR):
    t = PaTensor()
    t.data, t.dtype, t.ndim = at, dtype, len(shape)
    acc = 1
    for k in reversed(range(len(shape))):
        t.shape[k], t.stride[k] = shape[k], acc
        acc *= max(shape[k], 1)
    return t


def mutate(r, ts):
    t = r.choice(ts)
    f = r.randrange(5)
    if f == 0:
        t.data = r.choice([0, ADDR + 8, ADDR + 2, ADDR + 256])
    elif f == 1:
        t.dtype = r.choice([-1, 0, 1, 2, 3, 4, 5])
    elif f == 2:
        t.ndim = r.choice([-1, 0, 1, 2, 3, 4, 5, 6])
    elif f == 3:
        t.shape[r.randrange(5)] = r.choice(VALS)
    else:
        t.stride[r.randrange(5)] = r.choice(VALS + [-8])


def options(r):
    if r.random() < 0.1:
        return None
    o = PaOpts()
    o.stream = None
    o.workspace = r.choice([None, ADDR * 4, ADDR * 4 + 64])
    o.workspace_bytes = r.choice([0, 1 << 20, 1 << 40])
    o.partition_tokens = r.choice([-2, -1, 0, 0, 0, 16, 512])
    o.timeout_ms = r.choice([-5, 0, 5])
    return ctypes.byref(o)


def call(r):
    B, Hkv, G = r.choice([0, 1, 3, 64]), r.choice([1, 2, 8]), r.choice([1, 2, 3, 4, 8])
    H, D, NB = Hkv * G, r.choice([64, 128]), r.choice([1, 10, 1000])
    max_nb, T, W = r.choice([0, 1, 5, 128]), r.choice([0, 1, 7, 300, 2000]), r.choice([0, 1, 10, 63])
    dt = r.choice([0, 1, 4])
    qdt = 1 if dt == 4 else dt
    cache = [tensor((NB, Hkv, 16, D), dt), tensor((NB, Hkv, 16, D), dt)]
    seqs = [tensor((B, max_nb), 2), tensor((B,), 2)]
    heads = r.choice([Hkv, Hkv, Hkv + 1, 0, -1])
    scale = r.choice([1.0, 1.0, 0.0, -1.0, float("nan"), float("inf")])
    n = ctypes.c_size_t(0)
    which = r.randrange(6)
    if which == 0:
        ts = [tensor((T, H, D), qdt), tensor((T, H, D), qdt), *cache, *seqs, tensor((B + 1,), 2), tensor((T, W), 2)]
    elif which == 1:
        ts = [*cache, *seqs, tensor((B + 1,), 2), tensor((B, W), 2), tensor((B,), 2)]
    elif which == 2:
        ts = [tensor((B, H, D), qdt), tensor((B, Hkv, 16 * W), 0), tensor((B, H, D), qdt), *cache, *seqs,
              tensor((Hkv,), 0), tensor((Hkv,), 0)]
    elif which == 3:
        ts = [*cache, *seqs, tensor((B, Hkv, 16 * W), 0), tensor((B, r.choice([0, 1, 9])), 2), tensor((B,), 2),
              tensor((B, Hkv, 16 * W), 0, r.choice([ADDR, ADDR * 2])), tensor((B, Hkv, W), 2)]
    elif which == 4:
        a = [r.choice(VALS[:19] + [-5]) for _ in range(6)]
        return lib.pa_decode_scored_workspace_bytes(*a, ctypes.byref(n) if r.random() > 0.03 else None)
    else:
        a = [r.choice(VALS[:19] + [-5]) for _ in range(4)]
        return lib.pa_tree_attention_workspace_bytes(*a, ctypes.byref(n) if r.random() > 0.03 else None)
    for _ in range(r.randrange(3)):
        mutate(r, ts)
    p = [ctypes.byref(t) if r.random() > 0.03 else None for t in ts]
    o = options(r)
    if which == 0:
        return lib.pa_tree_attention(*p, r.choice([-1, 0, 1, T, T, T + 1]), scale, heads, o)
    if which == 1:
        return lib.pa_tree_commit(*p, o)
    if which == 2:
        if dt != 4 and r.random() < 0.9:
            p[7] = p[8] = None
        return lib.pa_decode_scored(*p[:7], scale, heads, p[7], p[8], o)
    return lib.pa_evict(*p[:7], r.choice([-1, 0, 4, 2**31 - 1]), r.choice([-1, 0, 4, 2**31 - 1]), p[7], p[8], o)


r = random.Random(int(sys.argv[1]))
seen = set()
for _ in range(int(sys.argv[2])):
    st = call(r)
    assert 0 <= st <= 8, st
    seen.add(st)
print(" ".join(str(s) for s in sorted(seen)))
'''


def test_new_entry_points_survive_mutated_descriptors():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    res = subprocess.run([sys.executable, "-c", CHILD, "352", "30000"], capture_output=True, text=True,
                         timeout=600, cwd=ROOT, env=env)
    assert res.returncode == 0, res.stderr[-3000:]
    # empty calls, argument errors, unsupported shapes, and calls that pass
    # every check and stop at the missing device
    assert {0, 1, 2, 4} <= set(int(s) for s in res.stdout.split()), res.stdout
