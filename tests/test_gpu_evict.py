"""GPU parity of the scored decode (pa_decode_scored) and of eviction
(pa_evict) against the fp64 oracle.

Tolerances of the scored decode, from the arithmetic (u = half a step of a
type: bf16 2^-8, f16 2^-11, fp32 2^-24; A = sum_t p_t |V_t|):
* logits are sums of D fp32 products (an e4m3 cache: of a query carried in 22
  bits), off by at most (D + 2) 2^-24 sum |q k| scale, the sum below 64 in
  these cases: a weight and the denominator are each off by dp = (D + 2)
  2^-18 relative, plus the exponential's 2^-12;
* the weighted sum adds 2^-12 of A (at most 2^12 terms in fp32); an e4m3 cache
  with grouped heads takes the probabilities in f16: 2^-11 more;
* out is rounded once: u |out|;
* a score adds at most 8 weights to a score below 2^4: (8 + 1) 2^-24 of the
  result, beside the weights' own 2 dp + 2^-11.
Eviction moves bytes and compares numbers: equal to the last bit.
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_351_b200 as pa
from gpu_harness import check_status_clean
from oracle.evict import evict, scored_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
KINDS = [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64), ("fp8", 128)]


def as_bytes(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


class Case:
    """Sequences over permuted blocks; slots that no sequence holds are NaN."""

    def __init__(self, seed, ctx, H, hk, D, dtype, spare=0, S=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.H, self.hk, self.D, self.dtype = H, hk, D, dtype
        self.ctx = np.array(ctx, np.int32)
        nbs = [-(-c // 16) for c in ctx]
        self.NB = sum(nbs) + spare + 3
        perm = rng.permutation(self.NB)
        self.max_nb = max(1, max(nbs)) + 1
        self.tables = np.full((len(ctx), self.max_nb), -1, np.int32)
        off = 0
        for i, k in enumerate(nbs):
            self.tables[i, :k] = perm[off:off + k]
            off += k
        self.free = perm[off:].astype(np.int32)
        nan = torch.full((self.NB, hk, 16, D), float("nan"))
        self.kc, self.vc = nan.to(DT[dtype]), nan.to(DT[dtype])
        self.ks = self.vs = None
        mul = 1.0
        if dtype == "fp8":
            self.ks = torch.rand(hk, generator=g) * 0.01 + 0.01
            self.vs = torch.rand(hk, generator=g) * 0.01 + 0.01
            mul = 70.0
        for i, c in enumerate(ctx):
            for j in range(nbs[i]):
                m, b = min(16, c - 16 * j), int(self.tables[i, j])
                self.kc[b, :, :m] = (torch.randn(hk, m, D, generator=g) * mul).to(DT[dtype])
                self.vc[b, :, :m] = (torch.randn(hk, m, D, generator=g) * mul).to(DT[dtype])
        self.q = torch.randn(len(ctx), H, D, generator=g).to(torch.bfloat16 if dtype == "fp8" else DT[dtype])
        self.S = self.max_nb * 16 + 3 if S is None else S
        self.scores = torch.rand(len(ctx), hk, self.S, generator=g)
        self.scale = 1.0 / math.sqrt(D)

    def wide(self):
        k, v = self.kc.double(), self.vc.double()
        if self.ks is not None:
            k, v = k * self.ks.double()[None, :, None, None], v * self.vs.double()[None, :, None, None]
        return k.numpy(), v.numpy()

    def device(self):
        t = lambda x: None if x is None else torch.as_tensor(x).to(DEV)  # noqa: E731
        self.d = dict(kc=t(self.kc), vc=t(self.vc), q=t(self.q), bt=t(self.tables), cl=t(self.ctx), ks=t(self.ks),
                      vs=t(self.vs), scores=t(self.scores))
        return self.d

    def workspace(self, part=0):
        n = pa.pa_decode_scored_workspace_bytes(len(self.ctx), self.H, self.hk, self.D, self.max_nb, part)
        return torch.zeros(n, dtype=torch.uint8, device=DEV)

    def run(self, part=0, ws=None):
        d = self.device()
        out = torch.full((len(self.ctx), self.H, self.D), 7.0, dtype=self.q.dtype, device=DEV)
        pa.pa_decode_scored(out, d["scores"], d["q"], d["kc"], d["vc"], d["bt"], d["cl"], self.scale, self.hk,
                            self.workspace(part) if ws is None else ws, k_scale=d["ks"], v_scale=d["vs"],
                            partition_tokens=part)
        torch.cuda.synchronize()
        return out, d["scores"]

    def ref(self):
        k, v = self.wide()
        return scored_decode(self.q.double().numpy(), k, v, self.tables, self.ctx, self.scale, self.scores.numpy())

    def check(self, out, scores, ref=None):
        want, mag, acc, add = self.ref() if ref is None else ref
        dp = (self.D + 2) * 2.0 ** -18
        u = 2.0 ** -24 if self.dtype == "f32" else 2.0 ** -8
        u_p = 2.0 ** -11 if self.dtype == "fp8" else 0.0
        got = out.double().cpu().numpy()
        lim = mag * (2 * dp + 2.0 ** -11 + 2.0 ** -12 + u_p) + u * np.abs(want) + 1e-30
        assert (np.abs(got - want) <= lim).all(), (np.abs(got - want) / lim).max()
        s = scores.double().cpu().numpy()
        lim = add * (2 * dp + 2.0 ** -11) + 9 * 2.0 ** -24 * np.abs(acc) + 1e-30
        assert (np.abs(s - acc) <= lim).all(), (np.abs(s - acc) / lim).max()


CTX = [1, 0, 15, 16, 17, 33, 100, 257, 0, 48, 1000]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("H,hk", [(3, 3), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("part", [0, -1])
def test_scored_decode(dtype, D, H, hk, part):
    c = Case(H * 10 + hk, CTX, H, hk, D, dtype)
    out, scores = c.run(part)
    check_status_clean()
    c.check(out, scores)
    past = torch.as_tensor(c.scores)
    for i, n in enumerate(CTX):  # entries past the context stay as they were
        assert torch.equal(scores[i, :, n:].cpu(), past[i, :, n:])


@pytest.mark.parametrize("dtype,D", KINDS)
def test_scored_decode_repeats_bitwise_and_matches_decode(dtype, D):
    """Two calls on one workspace: same bits, counters left at zero, and the
    output is pa_decode's."""
    c = Case(3, [3000, 700], 8, 2, D, dtype)
    ws = c.workspace()
    a, sa = c.run(ws=ws)
    b, sb = c.run(ws=ws)
    assert torch.equal(a, b) and torch.equal(sa, sb)
    assert int(ws[: pa.PA_DECODE_WS_HEADER_BYTES].count_nonzero()) == 0
    c.check(a, sa)
    d = c.d
    n = pa.pa_decode_workspace_bytes(2, 8, 2, D, c.max_nb)
    dws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    ref = torch.empty_like(a)
    if dtype == "fp8":
        pa.pa_decode_fp8(ref, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], c.scale, 2, d["ks"], d["vs"], workspace=dws)
    else:
        pa.pa_decode(ref, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], c.scale, 2, workspace=dws)
    torch.cuda.synchronize()
    check_status_clean()
    assert torch.equal(a, ref)


def test_scores_add_up_over_steps():
    """Ten steps: every step adds G weights of sum one to each kv head's row."""
    c = Case(5, [40, 7], 8, 2, 128, "bf16")
    c.scores.zero_()
    d = c.device()
    ws, out = c.workspace(), torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    call = pa.prepare_decode_scored(out, d["scores"], d["q"], d["kc"], d["vc"], d["bt"], d["cl"], c.scale, 2, ws)
    for _ in range(10):
        call()
    torch.cuda.synchronize()
    check_status_clean()
    total = d["scores"].double().sum(dim=2).cpu()
    assert bool((total - 40).abs().max() <= 40 * (2 * 130 * 2.0 ** -18 + 2.0 ** -11))
    c.scores = c.scores * 0
    _, _, _, add = c.ref()
    assert np.abs(d["scores"].double().cpu().numpy() - 10 * add).max() <= 10 * 4 * 2e-3


def test_scores_row_views_and_short_rows():
    """Rows of a wider, strided accumulator; a context longer than the row is
    reported and scored as far as the row goes."""
    c = Case(7, [50, 20], 4, 2, 64, "f32", S=32)
    d = c.device()
    big = torch.full((6, 5, 40), 2.0, device=DEV)
    view = big[1:5:2, ::3, :32]
    view.copy_(c.scores)
    out = torch.empty(2, 4, 64, device=DEV)
    pa.pa_decode_scored(out, view, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], c.scale, 2, c.workspace())
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_CONTEXT
    want, mag, acc, add = c.ref()
    assert np.abs(view.double().cpu().numpy() - acc).max() <= 1e-3
    rest = big.clone()
    rest[1:5:2, ::3, :32] = 2.0
    assert bool((rest == 2.0).all())
    check_status_clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_scored_decode_in_a_graph(dtype):
    c = Case(9, [300, 64, 5], 8, 2, 128, dtype)
    d, ws = c.device(), c.workspace()
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    call = lambda: pa.pa_decode_scored(out, d["scores"], d["q"], d["kc"], d["vc"], d["bt"], d["cl"],  # noqa: E731
                                       c.scale, 2, ws, k_scale=d["ks"], v_scale=d["vs"])
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    ref = c.ref()
    for _ in range(2):
        d["scores"].copy_(c.scores)
        g.replay()
        torch.cuda.synchronize()
        c.check(out, d["scores"], ref)
    check_status_clean()


# ---- eviction ----------------------------------------------------------------

def evict_case(seed, ctx, keep, hk, D, dtype, sink, recent, scores=None, pad=(0, 0)):
    """Runs pa_evict and checks every output against the oracle."""
    c = Case(seed, ctx, hk, hk, D, dtype, spare=sum(-(-min(k, n) // 16) for k, n in zip(keep, ctx)))
    if scores is not None:
        c.scores = scores(c)
    K = [min(k, n) for k, n in zip(keep, ctx)]
    dnb = [-(-k // 16) for k in K]
    dst = np.full((len(ctx), max(max(dnb), 1)), -1, np.int32)
    off = 0
    for i, k in enumerate(dnb):
        dst[i, :k] = c.free[off:off + k]
        off += k
    so = torch.full((len(ctx), hk, max(K) + pad[0]), 5.0)
    ko = torch.full((len(ctx), hk, max(K) + pad[1]), 99, dtype=torch.int32)
    d = c.device()
    so_d, ko_d = so.to(DEV), ko.to(DEV)
    pa.pa_evict(d["kc"], d["vc"], d["bt"], d["cl"], d["scores"], torch.from_numpy(dst).to(DEV),
                torch.tensor(keep, dtype=torch.int32, device=DEV), sink, recent, so_d, ko_d)
    torch.cuda.synchronize()
    check_status_clean()
    k2, v2, s2, p2 = evict(as_bytes(c.kc), as_bytes(c.vc), c.tables, c.ctx, c.scores.numpy(), dst, keep, sink, recent,
                           so.numpy(), ko.numpy())
    assert np.array_equal(ko_d.cpu().numpy(), p2)
    assert np.array_equal(so_d.cpu().numpy(), s2, equal_nan=True)
    assert np.array_equal(as_bytes(d["kc"]), k2) and np.array_equal(as_bytes(d["vc"]), v2)


LENS = [1, 0, 15, 16, 17, 100, 257, 700, 40, 64]
KEEP = [1, 5, 3, 16, 1, 64, 0, 300, 40, 63]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("hk", [1, 3])
@pytest.mark.parametrize("sink,recent", [(0, 0), (4, 16), (2, 1000), (1000, 1)])
def test_evict(dtype, D, hk, sink, recent):
    evict_case(11 + hk, LENS, KEEP, hk, D, dtype, sink, recent, pad=(9, 5))


@pytest.mark.parametrize("kind", ["zeros", "few values", "special", "one value above"])
@pytest.mark.parametrize("longest", [700, 1500, 5000])  # a warp a row (32, 64 keys a lane), a cluster a row
def test_evict_ties_and_special_scores(kind, longest):
    def make(c):
        g = torch.Generator().manual_seed(1)
        s = torch.zeros_like(c.scores)
        if kind == "few values":
            s = torch.randint(0, 3, s.shape, generator=g).float()
        elif kind == "special":
            pick = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1.0, -1.0, 1e-45, 3e38])
            s = pick[torch.randint(0, len(pick), s.shape, generator=g)]
        elif kind == "one value above":
            s[:, :, 37] = 1.0
        return s

    for sink, recent in ((0, 0), (4, 10)):
        evict_case(21, [longest, 64, 33, 100], [longest // 2, 20, 32, 7], 2, 64, "bf16", sink, recent, scores=make)


@pytest.mark.parametrize("n,keep", [(1024, 1000), (1025, 3), (2048, 1024), (2049, 2048), (20000, 2500), (5000, 4999),
                                    (70000, 37), (40000, 0), (40000, 36)])
def test_evict_long_rows(n, keep):
    evict_case(31, [n, 300], [keep, 200], 2, 64, "bf16", 4, 32)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_evict_many_rows(dtype, D):
    """Over four rows per SM: the kernel that chooses also moves."""
    rng = np.random.default_rng(35)
    ctx = [int(x) for x in rng.integers(0, 60, 150)]
    keep = [int(x) for x in rng.integers(0, 60, 150)]
    ctx[7], keep[7] = 1500, 700
    evict_case(35, ctx, keep, 5, D, dtype, 2, 5, pad=(3, 2))


@pytest.mark.parametrize("n,keep", [(450_000, 3000), (900, 300)])
def test_evict_rows_longer_than_shared_memory(n, keep):
    """A table and score rows of over 440,000 tokens: the scores are read from memory in every pass."""
    ctx, hk, D = [n, 50], 1, 64
    c = Case(33, ctx, hk, hk, D, "bf16", spare=-(-keep // 16) + 4, S=480_000)
    table = np.full((2, 30_000), -1, np.int32)
    table[:, :c.max_nb] = c.tables[:, :30_000]
    dst = np.full((2, -(-keep // 16)), -1, np.int32)
    dst[0] = c.free[:dst.shape[1]]
    dst[1, 0] = c.free[dst.shape[1]]
    d = c.device()
    so, ko = torch.zeros(2, hk, keep, device=DEV), torch.zeros(2, hk, keep, dtype=torch.int32, device=DEV)
    pa.pa_evict(d["kc"], d["vc"], torch.from_numpy(table).to(DEV), d["cl"], d["scores"],
                torch.from_numpy(dst).to(DEV), torch.tensor([keep, 16], dtype=torch.int32, device=DEV), 1, 5, so, ko)
    torch.cuda.synchronize()
    check_status_clean()
    k2, v2, s2, p2 = evict(as_bytes(c.kc), as_bytes(c.vc), c.tables, c.ctx, c.scores.numpy(), dst, [keep, 16], 1, 5,
                           so.cpu().numpy(), ko.cpu().numpy())
    assert np.array_equal(ko.cpu().numpy(), p2) and np.array_equal(so.cpu().numpy(), s2)
    assert np.array_equal(as_bytes(d["kc"]), k2) and np.array_equal(as_bytes(d["vc"]), v2)


def test_evict_keeps_scores_that_differ_in_one_bit():
    """Neighbouring floats: the choice goes by the last bit."""
    def make(c):
        base = np.float32(1.0).view(np.int32)
        v = (base + np.random.default_rng(2).permutation(c.S * c.hk * len(c.ctx)).astype(np.int32)).view(np.float32)
        return torch.from_numpy(v.reshape(len(c.ctx), c.hk, c.S).copy())

    evict_case(41, [3000, 513], [1000, 100], 2, 64, "f32", 0, 0, scores=make)


def test_evict_reports_what_does_not_fit():
    """Negative lengths, more tokens than the table or the row, more kept than
    an output holds: skipped and reported; the others are served."""
    c = Case(51, [40, 40, 40, 40], 2, 2, 64, "bf16", spare=8)
    d = c.device()
    dst = torch.from_numpy(c.free[:8].reshape(4, 2).copy()).to(DEV)
    cl = torch.tensor([40, -1, 100000, 40], dtype=torch.int32, device=DEV)
    keep = torch.tensor([33, 20, 20, 20], dtype=torch.int32, device=DEV)  # the first: more than the destination table
    so = torch.full((4, 2, 40), 5.0, device=DEV)
    ko = torch.full((4, 2, 40), 99, dtype=torch.int32, device=DEV)
    before = as_bytes(d["kc"])
    pa.pa_evict(d["kc"], d["vc"], d["bt"], cl, d["scores"], dst, keep, 0, 0, so, ko)
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_CONTEXT
    assert bool((so[:3] == 5).all()) and bool((ko[:3] == 99).all())
    assert bool((ko[3, :, 19] >= 0).all()) and bool((ko[3, :, 20:] == -1).all())
    after = as_bytes(d["kc"])
    changed = set(np.nonzero((after != before).any(axis=(1, 2, 3)))[0].tolist())
    assert changed <= set(c.free[6:8].tolist())
    # a destination block outside the pool: reported, its rows are not moved
    dst[3, 0] = c.NB
    pa.pa_evict(d["kc"], d["vc"], d["bt"], d["cl"], d["scores"], dst, keep - 14, 0, 0, so, ko)
    st, bits = pa.pa_get_device_status()
    assert bits == pa.PA_DEV_BAD_BLOCK
    check_status_clean()


def test_evict_in_a_graph_on_new_scores():
    c = Case(61, [200, 90], 2, 2, 128, "bf16", spare=8)
    d = c.device()
    dst = torch.from_numpy(c.free[:8].reshape(2, 4).copy()).to(DEV)
    keep = torch.tensor([60, 50], dtype=torch.int32, device=DEV)
    so = torch.empty(2, 2, 64, device=DEV)
    ko = torch.empty(2, 2, 60, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    call = pa.prepare_evict(d["kc"], d["vc"], d["bt"], d["cl"], d["scores"], dst, keep, 2, 8, so, ko)
    with torch.cuda.stream(s):
        call(stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(stream=s)
    for seed in (1, 2):
        c.scores = torch.rand(2, 2, c.S, generator=torch.Generator().manual_seed(seed))
        d["scores"].copy_(c.scores)
        g.replay()
        torch.cuda.synchronize()
        k2, v2, s2, p2 = evict(as_bytes(c.kc), as_bytes(c.vc), c.tables, c.ctx, c.scores.numpy(), dst.cpu().numpy(),
                               [60, 50], 2, 8, so.cpu().numpy(), ko.cpu().numpy())
        assert np.array_equal(ko.cpu().numpy(), p2) and np.array_equal(so.cpu().numpy(), s2)
        rows = np.unique(dst.cpu().numpy())
        assert np.array_equal(as_bytes(d["vc"])[rows][:, :, :, 0] != 0, v2[rows][:, :, :, 0] != 0)
    check_status_clean()
