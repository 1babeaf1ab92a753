"""The workspaces that PagedKVCacheGPU keeps: zeroed on the stream that uses
them, one per stream, and never handed to another stream while a call may
still use them.

Each test fills freed memory with ones first, so that merge counters which
start from anything but the call's own zeroing show in the outputs; the
reference is the same call with a workspace zeroed beforehand, which equals
it to the last bit."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_351_b200 as pa
from gpu_harness import check_status_clean
from oracle.tree import ancestors, pack_mask
from paged_kv_cache_351_b200.runtime import PagedKVCacheGPU

pytestmark = pytest.mark.gpu
DEV = "cuda"
HK, D = 8, 128
SCALE = 1.0 / math.sqrt(D)
BEHIND = 40_000_000  # clock cycles of a kernel that holds a stream back: about 20 ms


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)


class Call:
    """One kind of call over a cache of its own: sequences whose pages are cut
    between CTAs, so that the merge counters decide who merges."""

    def __init__(self, kind, B, tokens, H):
        g = torch.Generator(device=DEV).manual_seed(B * tokens + H)
        self.kind, self.B, self.H, self.n = kind, B, H, 9 if kind == "tree_attention" else 1
        nb = -(-tokens // 16) * B + 8
        self.kv = kv = PagedKVCacheGPU(nb, HK, D)
        for pool in (kv.k_cache, kv.v_cache):
            pool.normal_(generator=g)
        seqs = list(range(B))
        for s in seqs:
            kv.add(s)
        kv.append(seqs, [tokens - 7 * s for s in seqs])
        bt, cl = kv.block_tables(seqs, -(-tokens // 16))
        self.bt, self.cl = i32(bt), i32(cl)
        rows = B * self.n
        self.q = torch.randn(rows, H, D, generator=g, device=DEV).to(torch.bfloat16)
        self.scores = torch.rand(B, HK, bt.shape[1] * 16, generator=g, device=DEV)
        self.qs = i32(np.arange(B + 1) * self.n)
        self.mask = torch.from_numpy(pack_mask([ancestors(list(range(-1, self.n - 1)))] * B, rows, 1)).to(DEV)
        self.groups = i32(np.arange(B + 1)), i32(np.zeros(B))
        self.bytes = {"tree_attention": lambda: pa.pa_tree_attention_workspace_bytes(H, HK, D, self.n),
                      "decode_scored": lambda: pa.pa_decode_scored_workspace_bytes(B, H, HK, D, bt.shape[1]),
                      "decode_shared": lambda: pa.pa_decode_cascade_workspace_bytes(B, H, HK, D, 1),
                      }.get(kind, lambda: pa.pa_decode_workspace_bytes(B, H, HK, D, bt.shape[1]))()
        torch.cuda.synchronize()

    def outputs(self):
        return torch.full_like(self.q, 7.0), self.scores.clone()

    def __call__(self, out, scores, **kw):
        if self.kind == "tree_attention":
            self.kv.tree_attention(out, self.q, self.bt, self.cl, self.qs, self.mask, self.n, SCALE, **kw)
        elif self.kind == "decode_scored":
            self.kv.decode_scored(out, scores, self.q, self.bt, self.cl, SCALE, **kw)
        elif self.kind == "decode":
            self.kv.decode(out, self.q, self.bt, self.cl, SCALE, **kw)
        elif self.kind == "decode_shared":
            self.kv.decode_shared(out, self.q, self.bt, self.cl, *self.groups, 1, SCALE, **kw)
        else:  # a prepared step that appends nothing
            row, slots = self.q[:0, :HK], torch.empty(0, dtype=torch.int64, device=DEV)
            self.kv.prepare_step(slots, row, row, out, self.q, self.bt, self.cl, SCALE,
                                 groups=(*self.groups, 1) if self.kind == "shared step" else None, **kw)()

    def want(self):
        o = self.outputs()
        self(*o, workspace=torch.zeros(self.bytes, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        return o


def dirty(nbytes, *streams):
    """Freed memory of every stream holds ones."""
    for s in streams:
        with torch.cuda.stream(s):
            t = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (nbytes, nbytes)]
            del t
    torch.cuda.synchronize()


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


KINDS = ["tree_attention", "decode_scored", "decode", "decode_shared", "step", "shared step"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("raw", [False, True])
def test_first_call_on_another_stream(kind, raw):
    """The current stream is busy: a workspace zeroed there would come too late."""
    c = Call(kind, 12, 900, 32)
    want, got = c.want(), c.outputs()
    side = torch.cuda.Stream()
    dirty(c.bytes, torch.cuda.current_stream(), side)
    torch.cuda._sleep(BEHIND)
    c(*got, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert same(got, want)
    check_status_clean()


@pytest.mark.parametrize("kind", KINDS[1:])  # (tree attention's size follows from the head size alone)
def test_growth_while_the_smaller_call_waits(kind):
    """The outgrown workspace is not handed to the current stream."""
    small, large = Call(kind, 12, 900, 8), Call(kind, 12, 900, 64)
    large.kv, large.bt = small.kv, small.bt  # one cache, more query heads
    assert large.bytes > small.bytes
    want = small.want(), large.want()
    got = small.outputs(), large.outputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BEHIND)
    small(*got[0], stream=side)
    large(*got[1], stream=side)
    t = [torch.full((small.bytes,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1]) and len(t) == 3
    check_status_clean()


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    """Calls on two streams (one of them the current one) overlap and share nothing."""
    c = Call(kind, 12, 900, 32)
    want = c.want()
    side = torch.cuda.Stream()
    got = [[c.outputs() for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(*got):
        c(*a)
        c(*b, stream=side)
    torch.cuda.synchronize()
    assert all(same(o, want) for o in got[0] + got[1])
    check_status_clean()


@pytest.mark.parametrize("kind", KINDS)
def test_captured_calls_have_workspaces_of_their_own(kind):
    """Two graphs over one cache, the second replayed first, on two streams at
    once and next to calls outside; then the cache's workspace grows, and the
    graphs replay again."""
    c = Call(kind, 12, 900, 32)
    want = c.want()
    big = Call(kind, 12, 900, 64)
    big.kv, big.bt = c.kv, c.bt
    grown = big.want()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs, graphs = [c.outputs(), c.outputs()], []
    for s, o in zip(streams, outs):
        with torch.cuda.stream(s):
            c(*c.outputs())  # (loads the kernels)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c(*o)
        graphs.append(g)
    dirty(c.bytes, torch.cuda.current_stream(), *streams)
    eager, large = c.outputs(), big.outputs()
    for again in range(3):
        for (out, scores), _ in zip(outs, graphs):
            out.fill_(7.0), scores.copy_(c.scores)
        eager[1].copy_(c.scores)
        torch.cuda.synchronize()
        for s, g in reversed(list(zip(streams, graphs))):
            with torch.cuda.stream(s):
                g.replay()
        c(*eager)
        torch.cuda.synchronize()
        assert same(outs[0], want) and same(outs[1], want) and same(eager, want), again
        if again == 1:
            for s in streams:
                big(*large, stream=s)
                s.synchronize()
                assert torch.equal(large[0], grown[0])
            dirty(c.bytes, torch.cuda.current_stream(), *streams)
    check_status_clean()
