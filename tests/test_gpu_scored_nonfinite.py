"""Scored decode over a cache with NaN or infinite keys: the weights of the
rows that see them are NaN, as the formula says, whether a row is cut between
CTAs or not; other rows and kv heads are right.  Tolerances: see
test_gpu_evict."""

import numpy as np
import pytest
import torch

from gpu_harness import check_status_clean
from test_gpu_evict import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("H,hk", [(2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("part", [0, -1])
@pytest.mark.parametrize("ctx,at", [([4000, 700, 5], 2345), ([40, 300, 17], 39)])
def test_one_nan_key(dtype, D, H, hk, part, ctx, at):
    c = Case(H, ctx, H, hk, D, dtype)
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
