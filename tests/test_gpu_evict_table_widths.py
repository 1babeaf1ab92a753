"""GPU parity of eviction (pa_evict) at every width of table that chooses
another kernel: the tokens that the table and the score rows have room for
(the smaller of the two) and the number of rows decide, not the lengths.

    up to 2,048          one CTA of 256 threads a row, 8 keys a lane
    up to 32,768         1 to 8 CTAs of 512 threads, 8 keys a lane, while the
                         rows are few (fewer CTAs than two per SM)
    up to 131,072        1 to 8 CTAs of 512 threads, 32 keys a lane
    above                8 CTAs of 512 threads that read the scores in every pass

Every output lies in a wider buffer whose other entries must stay as they
were.  Eviction moves bytes and compares numbers: equal to the last bit."""

import numpy as np
import pytest
import torch

import paged_kv_cache_351_b200 as pa
from gpu_harness import check_status_clean
from oracle.evict import evict
from test_gpu_evict import DEV, KINDS, Case, as_bytes

pytestmark = pytest.mark.gpu
LEFT, RIGHT = 5, 70  # entries of the output buffers before and behind each row


def check(seed, cap, ctx, keep, hk, sink, recent, scores=None, D=64, dtype="bf16"):
    K = [min(k, n) for k, n in zip(keep, ctx)]
    dnb = [-(-k // 16) for k in K]
    c = Case(seed, ctx, hk, hk, D, dtype, spare=sum(dnb), S=cap)
    if dtype == "f32":
        c.vc = c.vc * 0.75 - 0.25  # (the case's fp32 K and V are one tensor)
    if scores is not None:
        c.scores = scores(c.scores)
    table = np.full((len(ctx), -(-cap // 16)), -1, np.int32)
    w = min(table.shape[1], c.max_nb)
    table[:, :w] = c.tables[:, :w]
    dst = np.full((len(ctx), max(max(dnb), 1)), -1, np.int32)
    off = 0
    for i, k in enumerate(dnb):
        dst[i, :k] = c.free[off:off + k]
        off += k
    P = max(K) + 2
    so = torch.full((len(ctx), hk, LEFT + P + RIGHT), 5.0)
    ko = torch.full((len(ctx), hk, LEFT + P + RIGHT), 99, dtype=torch.int32)
    d = c.device()
    so_d, ko_d = so.to(DEV), ko.to(DEV)
    mid = slice(LEFT, LEFT + P)
    pa.pa_evict(d["kc"], d["vc"], torch.from_numpy(table).to(DEV), d["cl"], d["scores"], torch.from_numpy(dst).to(DEV),
                torch.tensor(keep, dtype=torch.int32, device=DEV), sink, recent, so_d[:, :, mid], ko_d[:, :, mid])
    torch.cuda.synchronize()
    check_status_clean()
    k2, v2, s2, p2 = evict(as_bytes(c.kc), as_bytes(c.vc), table, c.ctx, c.scores.numpy(), dst, keep, sink, recent,
                           so[:, :, mid].numpy(), ko[:, :, mid].numpy())
    so[:, :, mid], ko[:, :, mid] = torch.from_numpy(s2), torch.from_numpy(p2)
    assert torch.equal(ko_d.cpu(), ko)
    assert np.array_equal(so_d.cpu().numpy(), so.numpy(), equal_nan=True)
    assert np.array_equal(as_bytes(d["kc"]), k2) and np.array_equal(as_bytes(d["vc"]), v2)


# Above 131,072 tokens a warp owns a run of about cap / 128 of them.  Runs of
# 1,025, 1,094, 1,250 and 3,750 tokens are no multiple of the 32 that a warp
# takes at a time.
ABOVE = [131_073, 131_088, 140_000, 160_000, 480_000]


@pytest.mark.parametrize("cap", ABOVE)
@pytest.mark.parametrize("sink,recent", [(0, 0), (4, 32)])
def test_sequences_within_their_budget_keep_every_token_once(cap, sink, recent):
    """Nothing is chosen: the rows are copied, over several runs."""
    check(1, cap, [5000, 300, 0, 4100, 31], [5000, 400, 3, 9000, 31], 2, sink, recent)


@pytest.mark.parametrize("cap", ABOVE)
@pytest.mark.parametrize("sink,recent", [(4, 1500), (1300, 2), (0, 4990), (4000, 900), (0, 0)])
def test_protected_tokens_over_the_end_of_a_run_stay_once(cap, sink, recent):
    check(2, cap, [5000, 4200, 2051], [4995, 2600, 2050], 2, sink, recent)


@pytest.mark.parametrize("cap", [131_088, 160_000])
@pytest.mark.parametrize("kind", ["zeros", "few values", "nan and -inf"])
def test_ties_over_the_end_of_a_run(cap, kind):
    """Equal scores on both sides of a run's end: the lower positions stay."""
    def make(s):
        g = torch.Generator().manual_seed(4)
        if kind == "zeros":
            return torch.zeros_like(s)
        pick = torch.tensor([0.0, 1.0, 2.0] if kind == "few values" else [float("nan"), float("-inf"), -0.0, 0.0])
        return pick[torch.randint(0, len(pick), s.shape, generator=g)]

    check(3, cap, [5000, 2600, 1260], [1100, 2599, 600], 2, 4, 32, scores=make)


def test_a_row_as_long_as_the_table():
    check(5, 131_088, [131_088, 1100], [3000, 1099], 1, 4, 700)


WIDTHS = [2048, 2064, 4096, 4112, 8192, 8208, 16_384, 16_400, 32_768, 32_784, 65_536, 65_552, 131_072, 131_088]


@pytest.mark.parametrize("cap", WIDTHS)
@pytest.mark.parametrize("sink,recent", [(0, 0), (3, 40)])
def test_few_rows_on_either_side_of_every_width(cap, sink, recent):
    """Six rows; one of them fills the table (or 20,000 tokens of it)."""
    n = min(cap, 20_000)
    check(6, cap, [n, 700, 0], [n // 3, 700, 5], 2, sink, recent)


@pytest.mark.parametrize("cap", WIDTHS)
def test_many_rows_on_either_side_of_every_width(cap):
    """300 rows: a table over 2,048 tokens wide takes 32 keys a lane."""
    rng = np.random.default_rng(cap)
    ctx = [int(x) for x in rng.integers(0, 50, 150)]
    keep = [int(x) for x in rng.integers(0, 50, 150)]
    ctx[3], keep[3] = min(cap, 20_000), 1000
    ctx[149], keep[149] = 1900, 1899
    check(7, cap, ctx, keep, 2, 2, 5)


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("cap", [1000, 3000, 140_000])
def test_every_cache_type(dtype, D, cap):
    """K to K and V to V, for rows of every length in bytes."""
    check(8, cap, [1000, 333, 17], [500, 333, 16], 3, 2, 20, D=D, dtype=dtype)
