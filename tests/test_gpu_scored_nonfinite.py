"""Scored decode over a cache with NaN or infinite keys, whether a row is cut
between CTAs or not: a NaN makes the output and the weights of its rows NaN, a
logit of -infinity weighs nothing, and a row of nothing else is 0 / 0; other
rows and kv heads are right.  Tolerances: see test_gpu_evict."""

import numpy as np
import pytest
import torch

from gpu_harness import check_status_clean
from test_gpu_evict import KINDS, Case

pytestmark = pytest.mark.gpu


def own_values(c):
    """The case's fp32 K and V are one tensor."""
    if c.dtype == "f32":
        c.vc = c.vc * 0.75 - 0.25


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("H,hk", [(2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("part", [0, -1])
@pytest.mark.parametrize("ctx,at", [([4000, 700, 5], 2345), ([40, 300, 17], 39)])
def test_one_nan_key(dtype, D, H, hk, part, ctx, at):
    c = Case(H, ctx, H, hk, D, dtype)
    own_values(c)
    want, mag, acc, add = c.ref()
    b = int(c.tables[0, at // 16])
    c.kc[b, 1, at % 16, 3] = float("nan")
    out, scores = c.run(part)
    check_status_clean()
    got, s = out.double().cpu().numpy(), scores.double().cpu().numpy()
    g = H // hk
    assert np.isnan(got[0, g:]).all()
    assert np.isnan(s[0, 1, :ctx[0]]).all()
    assert np.array_equal(s[0, 1, ctx[0]:], c.scores[0, 1, ctx[0]:].double().numpy())
    # everything else as without the key
    got[0, g:], s[0, 1, :ctx[0]] = want[0, g:], acc[0, 1, :ctx[0]]
    c.check(torch.from_numpy(got), torch.from_numpy(s), (want, mag, acc, add))


@pytest.mark.parametrize("dtype,D", KINDS[:4])  # (e4m3 has no infinity)
@pytest.mark.parametrize("H,hk", [(2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("part", [0, -1])
def test_keys_of_no_weight(dtype, D, H, hk, part):
    """The first pages of a row (and with them whole shares), a single last
    token, every other page; then a row of such keys only."""
    ctx = [4000, 700, 33, 2500, 40]
    c = Case(H + 1, ctx, H, hk, D, dtype)
    own_values(c)
    c.q[..., 0] = c.q[..., 0].abs() + 0.25  # a key of -infinity in this dimension has that logit
    hit = [range(3000), range(16), [32], [t for t in range(2500) if t // 16 % 2], []]
    for i, ts in enumerate(hit):
        for t in ts:
            c.kc[int(c.tables[i, t // 16]), :, t % 16, 0] = float("-inf")
    out, scores = c.run(part)
    check_status_clean()
    ref = c.ref()
    c.check(out, scores, ref)
    for i in (0, 4):  # nothing else: one cut row, one whole
        for t in range(ctx[i]):
            c.kc[int(c.tables[i, t // 16]), 1, t % 16, 0] = float("-inf")
    out, scores = c.run(part)
    check_status_clean()
    got, s = out.double().cpu().numpy(), scores.double().cpu().numpy()
    g = H // hk
    for i in (0, 4):
        assert np.isnan(got[i, g:]).all() and np.isnan(s[i, 1, :ctx[i]]).all()
        got[i, g:], s[i, 1, :ctx[i]] = ref[0][i, g:], ref[2][i, 1, :ctx[i]]
    c.check(torch.from_numpy(got), torch.from_numpy(s), ref)
