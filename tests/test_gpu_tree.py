"""GPU parity of tree attention (pa_tree_attention) and of the accepted path's
commit (pa_tree_commit) against the fp64 oracle.

Tolerances, from the arithmetic.  A rounding to a type is off by at most half
a step, u = eps / 2 of it (bf16 2^-8, fp32 2^-24), relative to the value.
With A = sum_t p_t |V_t| of the exact probabilities:
* the logits are sums of D products in fp32, off by at most (D + 2) 2^-24
  sum |q k| scale, which the cases keep below 64, so a probability and the
  denominator are each off by at most dp = (D + 2) 2^-18 relative (130 of
  them: 5e-4 for D = 128), plus the exponential's own 2^-12;
* a bf16 cache goes through the tensor cores with probabilities rounded to
  bf16: another u(bf16) of each term;
* the weighted sum in fp32 over at most 2^12 terms adds 2^-12 of A;
* the output is rounded once: u |out|.
So |got - out| <= A (2 dp + 2^-11 + 2^-12 + u_p) + u |out| with u_p = 2^-8 for
bf16, 0 for fp32.
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_351_b200 as pa
from gpu_harness import check_status_clean
from oracle.tree import ancestors, pack_mask, tree_attention, tree_commit

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def bound(out, mag, dtype, D):
    dp = (D + 2) * 2.0 ** -18
    u_p, u = (2.0 ** -8, 2.0 ** -8) if dtype == "bf16" else (0.0, 2.0 ** -24)
    return mag * (2 * dp + 2.0 ** -11 + 2.0 ** -12 + u_p) + u * np.abs(out) + 1e-30


def random_parents(rng, n, reach=6):
    return [-1 if j == 0 else max(-1, j - 1 - int(rng.integers(0, reach))) for j in range(n)]


class Case:
    """Sequences of (committed, drafted) tokens over permuted blocks; every
    slot that no sequence holds is NaN."""

    def __init__(self, seed, pairs, H, hk, D, dtype, sees=None, extra_rows=0, max_q=None, std=1.0):
        rng = np.random.default_rng(seed)
        self.pairs, self.H, self.hk, self.D, self.dtype = pairs, H, hk, D, dtype
        self.n = [b for _, b in pairs]
        self.ctx = np.array([a + b for a, b in pairs], np.int32)
        self.qs = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.rows = int(self.qs[-1])
        self.T = self.rows + extra_rows
        nbs = [-(-int(c) // 16) for c in self.ctx]
        self.NB = sum(nbs) + 5
        perm = rng.permutation(self.NB)
        self.max_nb = max(1, max(nbs)) + 1
        self.tables = np.full((len(pairs), self.max_nb), -1, np.int32)
        off = 0
        for i, k in enumerate(nbs):
            self.tables[i, :k] = perm[off:off + k]
            off += k
        g = torch.Generator().manual_seed(seed)
        t = DT[dtype]
        self.kc = torch.full((self.NB, hk, 16, D), float("nan"), dtype=t)
        self.vc = torch.full((self.NB, hk, 16, D), float("nan"), dtype=t)
        for i, c in enumerate(self.ctx):
            for j in range(nbs[i]):
                m = min(16, int(c) - 16 * j)
                b = int(self.tables[i, j])
                self.kc[b, :, :m] = (torch.randn(hk, m, D, generator=g) * std).to(t)
                self.vc[b, :, :m] = torch.randn(hk, m, D, generator=g).to(t)
        self.q = torch.randn(self.T, H, D, generator=g).to(t)
        self.sees = [ancestors(random_parents(rng, m)) for m in self.n] if sees is None else sees
        self.max_q = max(1, max(self.n)) if max_q is None else max_q
        self.words = (self.max_q + 31) // 32
        self.mask = torch.from_numpy(pack_mask(self.sees, self.T, self.words))
        self.scale = 1.0 / math.sqrt(D)

    def device(self):
        self.dev = dict(kc=self.kc.to(DEV), vc=self.vc.to(DEV), q=self.q.to(DEV), mask=self.mask.to(DEV),
                        bt=torch.from_numpy(self.tables).to(DEV), cl=torch.from_numpy(self.ctx).to(DEV),
                        qs=torch.from_numpy(self.qs).to(DEV))
        return self.dev

    def workspace(self):
        n = pa.pa_tree_attention_workspace_bytes(self.H, self.hk, self.D, self.max_q)
        return torch.zeros(n, dtype=torch.uint8, device=DEV)

    def run(self, ws=None, out=None, part=0, **kw):
        d = self.device()
        d.update(kw)
        if out is None:
            out = torch.full((self.T, self.H, self.D), 7.0, dtype=DT[self.dtype], device=DEV)
        pa.pa_tree_attention(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], d["mask"], self.max_q,
                             self.scale, self.hk, workspace=ws, partition_tokens=part)
        torch.cuda.synchronize()
        return out

    def ref(self):
        return tree_attention(self.q[:self.rows].double().numpy(), self.kc.double().numpy(), self.vc.double().numpy(),
                              self.tables, self.ctx, self.sees, self.scale)

    def check(self, out, ref=None):
        want, mag = self.ref() if ref is None else ref
        got = out[:self.rows].double().cpu().numpy()
        err = np.abs(got - want)
        lim = bound(want, mag, self.dtype, self.D)
        assert not np.isnan(got).any()
        assert (err <= lim).all(), (err / lim).max()
        assert bool((out[self.rows:] == 7.0).all())  # rows of no sequence stay as they were


KINDS = [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)]
EDGE = [(0, 1), (1, 1), (15, 1), (16, 2), (17, 0), (0, 33), (31, 3), (63, 1), (64, 5), (65, 64), (130, 17), (0, 0),
        (257, 40), (100, 31), (100, 32), (5, 65)]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("H,hk", [(3, 3), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("split", [True, False])
def test_edges(dtype, D, H, hk, split):
    c = Case(H * 10 + hk, EDGE, H, hk, D, dtype, extra_rows=3)
    out = c.run(ws=c.workspace() if split else None)
    check_status_clean()
    c.check(out)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_one_sequence_cut_between_many_workers(dtype, D):
    """A long context over few heads: every unit is cut and merged."""
    c = Case(5, [(3000, 9)], 4, 2, D, dtype)
    ws = c.workspace()
    ref = c.ref()
    for _ in range(2):  # the counters are zero again after a call
        out = c.run(ws=ws)
        c.check(out, ref)
    check_status_clean()
    assert int(ws[: pa.PA_DECODE_WS_HEADER_BYTES].count_nonzero()) == 0


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("n", [129, 300])
def test_wide_trees(dtype, D, n):
    """More query rows than one tile of the kernel holds, and masks of many words."""
    rng = np.random.default_rng(n)
    sees = [ancestors(random_parents(rng, n, reach=40)), ancestors([-1])]
    c = Case(n, [(50, n), (200, 1)], 4, 2, D, dtype, sees=sees)
    out = c.run(ws=c.workspace())
    check_status_clean()
    c.check(out)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_rows_that_see_nothing(dtype, D):
    """No context and no bit: zero.  No context and only others' bits: those."""
    a, b = np.zeros((6, 6), bool), np.zeros((70, 70), bool)
    a[2, 5] = a[3, 0] = a[3, 4] = True  # a mask need not be a tree
    b[69, 0] = b[1, 69] = True
    c = Case(11, [(0, 6), (0, 70), (20, 6)], 4, 2, D, dtype, sees=[a, b, a])
    out = c.run(ws=c.workspace())
    check_status_clean()
    c.check(out)
    assert bool((out[0] == 0).all()) and bool((out[5] == 0).all())


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("split", [True, False])
def test_masked_tokens_may_hold_anything(dtype, D, bad, split):
    """Drafted tokens with NaN or infinite K and V change only the rows that see them."""
    n = 40
    sees = [ancestors(random_parents(np.random.default_rng(3), n))] * 2
    for s in sees:
        s[:, 7] = False
        s[9, 7] = True
    c = Case(13, [(300, n), (0, n)], 4, 2, D, dtype, sees=sees)
    for i in range(2):
        pos = int(c.ctx[i]) - n + 7
        blk, off = int(c.tables[i, pos // 16]), pos % 16
        c.kc[blk, :, off] = bad
        c.vc[blk, :, off, ::3] = bad
    out = c.run(ws=c.workspace() if split else None)
    check_status_clean()
    clean = [r for r in range(2 * n) if r % n != 9]
    # the oracle walks seen tokens only, so it is finite in these rows
    keep = [np.delete(s, 9, 0) for s in sees]
    want, mag = [], []
    for i in range(2):
        rows = [i * n + j for j in range(n) if j != 9]
        for r, s in zip(rows, keep[i]):
            one = np.zeros((n, n), bool)
            one[0] = s
            qq = np.zeros((n, c.H, D))
            qq[0] = c.q[r].double().numpy()
            o, m = tree_attention(qq, c.kc.double().numpy(), c.vc.double().numpy(), c.tables[i:i + 1],
                                  c.ctx[i:i + 1], [one], c.scale)
            want.append(o[0])
            mag.append(m[0])
    got = out[clean].double().cpu().numpy()
    err, lim = np.abs(got - np.stack(want)), bound(np.stack(want), np.stack(mag), dtype, D)
    assert (err <= lim).all(), np.nanmax(err / lim)
    assert not bool(torch.isfinite(out[9].float()).all())  # the row that sees it is not finite


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_seen_infinite_value_reaches_its_dims_only(dtype, D):
    """An infinite V of a seen drafted token: that dim is infinite, the others are right."""
    n = 12
    c = Case(17, [(90, n)], 4, 2, D, dtype, sees=[ancestors(list(range(-1, n - 1)))])
    pos = 90 + 4
    blk, off = int(c.tables[0, pos // 16]), pos % 16
    keep = c.vc[blk, :, off, 5].clone()
    ref = c.ref()
    c.vc[blk, :, off, 5] = float("inf")
    out = c.run(ws=c.workspace()).double().cpu().numpy()
    c.vc[blk, :, off, 5] = keep
    check_status_clean()
    assert np.isposinf(out[4:, :, 5]).all() and np.isfinite(out[:4]).all()
    rest = [d for d in range(D) if d != 5]
    lim = bound(ref[0], ref[1], dtype, D)
    assert (np.abs(out - ref[0])[..., rest] <= lim[..., rest]).all()
    assert (np.abs(out - ref[0])[:4] <= lim[:4]).all()


@pytest.mark.parametrize("dtype,D", KINDS)
def test_strided_inputs_and_wide_tables(dtype, D):
    """Rows of a wider buffer, a mask and a table with longer rows."""
    c = Case(19, [(70, 5), (3, 9), (0, 2)], 4, 2, D, dtype)
    T, H = c.T, c.H
    big_q = torch.zeros(T, H + 2, D + 64, dtype=DT[dtype], device=DEV)
    big_q[:, 1:H + 1, :D] = c.q.to(DEV)
    big_o = torch.full((T, H + 1, D + 32), 7.0, dtype=DT[dtype], device=DEV)
    big_m = torch.full((T, c.words + 3), -1, dtype=torch.int32, device=DEV)
    big_m[:, :c.words] = c.mask.to(DEV)
    big_t = torch.full((3, c.max_nb + 7), -5, dtype=torch.int32, device=DEV)
    big_t[:, :c.max_nb] = torch.from_numpy(c.tables).to(DEV)
    out = c.run(ws=c.workspace(), out=big_o[:, :H, :D], q=big_q[:, 1:H + 1, :D], mask=big_m, bt=big_t[:, :c.max_nb])
    check_status_clean()
    c.check(out)
    assert bool((big_o[:, H:] == 7).all()) and bool((big_o[:, :, D:] == 7).all())


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_graph_replay_on_a_side_stream(dtype, D):
    """A captured call replays on new inputs of the same buffers."""
    c = Case(23, [(500, 7), (40, 12)], 8, 2, D, dtype)
    d = c.device()
    ws, out = c.workspace(), torch.full((c.T, 8, D), 7.0, dtype=DT[dtype], device=DEV)
    s = torch.cuda.Stream()
    call = lambda: pa.pa_tree_attention(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"],  # noqa: E731
                                        d["mask"], c.max_q, c.scale, c.hk, workspace=ws)
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    c.q = torch.randn(c.T, 8, D).to(DT[dtype])
    d["q"].copy_(c.q)
    for _ in range(3):
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.check(out)
    check_status_clean()


def test_prepared_call_and_chain_equals_prefill():
    """A chain (every token's parent is the one before) is causal attention:
    pa_prefill on the same inputs agrees within both bounds."""
    pairs = [(100, 20), (0, 9), (15, 1), (700, 130)]
    c = Case(29, pairs, 8, 2, 128, "bf16", sees=[ancestors(list(range(-1, m - 1))) for _, m in pairs])
    d = c.device()
    out = torch.full((c.T, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    call = pa.prepare_tree_attention(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], d["mask"], c.max_q,
                                     c.scale, c.hk, workspace=c.workspace())
    call()
    ref = c.ref()
    c.check(out, ref)
    pre = torch.empty_like(out)
    pa.pa_prefill(pre, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], c.max_q, c.scale, c.hk)
    torch.cuda.synchronize()
    check_status_clean()
    diff = (out.double() - pre.double()).abs().cpu().numpy()
    assert (diff <= 2 * bound(ref[0], ref[1], "bf16", 128)).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 128)])
def test_few_units_with_many_shares(dtype, D):
    """One sequence, one kv head, a long context: tens of shares of one unit
    (the second launch), on one workspace next to a batch of many units."""
    a = Case(39, [(6000, 21)], 2, 1, D, dtype)
    b = Case(40, [(60, 3)] * 40, 8, 8, D, dtype)
    ws = a.workspace()
    n = b.workspace().numel()
    ws = torch.zeros(max(n, ws.numel()), dtype=torch.uint8, device=DEV)
    ra, rb = a.ref(), b.ref()
    for _ in range(2):
        a.check(a.run(ws=ws), ra)
        b.check(b.run(ws=ws), rb)
    check_status_clean()
    assert int(ws[: pa.PA_DECODE_WS_HEADER_BYTES].count_nonzero()) == 0


def test_two_streams_and_a_small_workspace():
    """Calls on two streams, each with its own workspace; a workspace below the
    size asked for leaves the context unsplit."""
    cases = [Case(41 + k, [(900, 9), (30, 4)], 8, 2, 128, "bf16") for k in range(2)]
    refs = [c.ref() for c in cases]
    devs, wss = [c.device() for c in cases], [c.workspace() for c in cases]
    outs = [torch.full((c.T, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, d, ws, out, s in zip(cases, devs, wss, outs, streams):
            pa.pa_tree_attention(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], d["mask"], c.max_q,
                                 c.scale, c.hk, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, out, ref in zip(cases, outs, refs):
        c.check(out, ref)
    small = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    cases[0].check(cases[0].run(ws=small), refs[0])
    cases[0].check(cases[0].run(ws=wss[0], part=-1), refs[0])
    check_status_clean()


@pytest.mark.parametrize("dtype,D", KINDS)
def test_one_row_with_any_stride(dtype, D):
    """The stride of a dimension of size 1 is never taken."""
    c = Case(45, [(33, 1)], 1, 1, D, dtype)
    flat = c.q.reshape(D).to(DEV)
    q = flat.as_strided((1, 1, D), (0, 0, 1))
    assert q.stride()[:2] == (0, 0)
    out = c.run(ws=c.workspace(), q=q)
    check_status_clean()
    c.check(out)


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("split", [True, False])
def test_scale_next_to_zero(dtype, D, split):
    """The least scales weigh all seen tokens alike (8 / scale is no float)."""
    c = Case(17, [(700, 9), (3, 40)], 4, 2, D, dtype)
    c.scale = 1e-38
    c.check(c.run(ws=c.workspace() if split else None))
    check_status_clean()


def test_bad_ranges_and_blocks_are_reported():
    c = Case(31, [(10, 5), (0, 4), (30, 3)], 4, 2, 128, "bf16", sees=None)
    ref = c.ref()
    qs = c.qs.copy()
    qs[1] = 40  # more rows than sequence 0 has tokens; sequence 1's become negative
    out = c.run(ws=c.workspace(), qs=torch.from_numpy(qs).to(DEV))
    st, bits = pa.pa_get_device_status()
    assert bits & pa.PA_DEV_BAD_CONTEXT
    got = out.double().cpu().numpy()
    assert (got[:9] == 7.0).all()  # skipped
    assert (np.abs(got[9:] - ref[0][9:]) <= bound(ref[0], ref[1], "bf16", 128)[9:]).all()  # the third is served
    bt = torch.from_numpy(c.tables).to(DEV)
    bt[2, 1] = c.NB
    out = c.run(ws=c.workspace(), bt=bt)
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_BLOCK
    got = out.double().cpu().numpy()
    assert (np.abs(got[:9] - ref[0][:9]) <= bound(ref[0], ref[1], "bf16", 128)[:9]).all()
    check_status_clean()


def test_more_sequences_than_threads():
    """600 sequences, most of them without a draft."""
    rng = np.random.default_rng(7)
    pairs = [(int(rng.integers(0, 40)), int(rng.integers(1, 4)) if k % 3 == 0 else 0) for k in range(600)]
    c = Case(37, pairs, 2, 1, 64, "bf16")
    out = c.run(ws=c.workspace())
    check_status_clean()
    c.check(out)


# ---- commit -----------------------------------------------------------------

def as_bytes(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


@pytest.mark.parametrize("dtype,D", KINDS + [("fp8", 128)])
@pytest.mark.parametrize("hk", [1, 3, 8])
def test_commit_moves_the_path(dtype, D, hk):
    pairs = [(10, 6), (0, 30), (16, 1), (31, 17), (5, 0), (100, 40), (3, 12)]
    paths = [[0, 2, 5], list(range(1, 30, 2)), [0], [3], [], list(range(40)), []]
    c = Case(41, pairs, hk, hk, D, dtype)
    d = c.device()
    acc = torch.full((len(pairs), 43), -9, dtype=torch.int32)
    for i, p in enumerate(paths):
        acc[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    cnt = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
    pa.pa_tree_commit(d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], acc.to(DEV), cnt)
    check_status_clean()
    for got, src in ((d["kc"], c.kc), (d["vc"], c.vc)):
        want = tree_commit(as_bytes(src), c.tables, c.ctx, c.n, paths)
        assert np.array_equal(as_bytes(got), want)


@pytest.mark.parametrize("hk", [1, 5])
def test_commit_long_paths(hk):
    """Paths over several rounds of 32, and ones that move nothing or one row far on."""
    pairs = [(7, 200), (16, 100), (0, 65), (40, 64), (3, 97)]
    rng = np.random.default_rng(5)
    paths = [sorted(rng.choice(200, 131, replace=False).tolist()), list(range(33)) + [99], list(range(65)),
             list(range(1, 64)), list(range(32)) + [40, 96]]
    c = Case(47, pairs, hk, hk, 128, "bf16")
    d = c.device()
    acc = torch.zeros(len(pairs), 131, dtype=torch.int32)
    for i, p in enumerate(paths):
        acc[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    cnt = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
    pa.pa_tree_commit(d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], acc.to(DEV), cnt)
    check_status_clean()
    for got, src in ((d["kc"], c.kc), (d["vc"], c.vc)):
        assert np.array_equal(as_bytes(got), tree_commit(as_bytes(src), c.tables, c.ctx, c.n, paths))
    # a fault in the second round: nothing moves
    d = c.device()
    acc[0, 40] = acc[0, 39]
    pa.pa_tree_commit(d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], acc.to(DEV), cnt)
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_CONTEXT
    want = tree_commit(as_bytes(c.kc), c.tables, c.ctx, c.n, [[]] + paths[1:])
    assert np.array_equal(as_bytes(d["kc"]), want)


def test_commit_refuses_bad_paths():
    """A path that does not ascend, leaves the draft or is too long, and a bad
    block: reported, and nothing of the sequence moves; the others do."""
    pairs = [(10, 6)] * 6
    paths = [[2, 1], [0, 6], [-1, 2], [1, 1], [2, 4], [3, 5]]
    c = Case(43, pairs, 2, 2, 64, "bf16")
    d = c.device()
    acc = torch.tensor(paths, dtype=torch.int32, device=DEV)
    cnt = torch.tensor([2, 2, 2, 2, 2, 2], dtype=torch.int32, device=DEV)
    pa.pa_tree_commit(d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], acc, cnt)
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_CONTEXT
    want = tree_commit(as_bytes(c.kc), c.tables, c.ctx, c.n, [[], [], [], [], [2, 4], [3, 5]])
    assert np.array_equal(as_bytes(d["kc"]), want)
    # more accepted than the path's row holds, a negative count, a block outside the pool
    d = c.device()
    d["bt"][5, 0] = c.NB
    cnt = torch.tensor([3, -1, 0, 0, 2, 2], dtype=torch.int32, device=DEV)
    pa.pa_tree_commit(d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], acc, cnt)
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_CONTEXT | pa.PA_DEV_BAD_BLOCK
    want = tree_commit(as_bytes(c.vc), c.tables, c.ctx, c.n, [[], [], [], [], [2, 4], []])
    assert np.array_equal(as_bytes(d["vc"]), want)
    check_status_clean()
