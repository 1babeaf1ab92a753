"""Tree attention over caches with infinities and NaN in keys that rows do
see: what the formula gives in fp64 (a logit of -infinity weighs nothing, a
row of nothing else, a logit of +infinity or a NaN give NaN), in every kernel,
wherever the keys lie in a tile.  Tolerances: see test_gpu_tree."""

import numpy as np
import pytest
import torch

from gpu_harness import check_status_clean
from test_gpu_tree import KINDS, Case, bound

pytestmark = pytest.mark.gpu

# tokens of the drafts: at G = 2 up to 16, 32, 64, 128 and over 128 rows a kv head
DRAFTS = [5, 16, 30, 60, 100]


def positive_first_dim(c):
    """Queries whose first dimension is positive: a key of -infinity there has that logit."""
    c.q[..., 0] = c.q[..., 0].abs() + 0.25


def set_keys(c, i, tokens, value):
    for t in tokens:
        c.kc[int(c.tables[i, t // 16]), :, t % 16, 0] = value


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("n", DRAFTS)
@pytest.mark.parametrize("split", [True, False])
def test_leading_keys_of_no_weight(dtype, D, n, split):
    """The first tiles of a row (of a share, of a whole context) hold only
    logits of -infinity; finite ones follow."""
    c = Case(n, [(400, n), (129, 3), (0, n)], 4, 2, D, dtype)
    positive_first_dim(c)
    set_keys(c, 0, range(300), float("-inf"))
    set_keys(c, 1, range(129), float("-inf"))  # the whole context: the draft's own keys remain
    out = c.run(ws=c.workspace() if split else None)
    check_status_clean()
    c.check(out)


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("n", DRAFTS)
@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_key_that_makes_its_rows_nan(dtype, D, n, split, value):
    """One committed key of NaN, or of a logit of +infinity, in every position
    of a tile: the rows of its sequence are NaN, the others are right."""
    pairs = [(256, n), (90, 4)] + [(256, 1)] * 8
    c = Case(n + 1, pairs, 4, 2, D, dtype)
    positive_first_dim(c)
    ref = c.ref()
    clean = c.kc.clone()
    for i, (want, at) in enumerate([(0, 0), (0, 25), (0, 31), (0, 63), (0, 88), (0, 127), (0, 155), (0, 255)]):
        c.kc = clean.clone()
        set_keys(c, want, [at], value)
        set_keys(c, 2 + i, range(17 * i + 3, 17 * i + 4), value)
        out = c.run(ws=c.workspace() if split else None)[:c.rows].double().cpu().numpy()
        check_status_clean()
        hit = np.zeros(c.rows, bool)
        for s in (want, 2 + i):
            hit[c.qs[s]:c.qs[s + 1]] = True
        assert np.isnan(out[hit]).all(), at
        lim = bound(ref[0], ref[1], dtype, D)
        assert (np.abs(out - ref[0]) <= lim)[~hit].all(), at


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("n", DRAFTS)
@pytest.mark.parametrize("split", [True, False])
def test_rows_of_no_logit_above_minus_infinity(dtype, D, n, split):
    """0 / 0 where every key that a row sees has that logit; a row that sees
    nothing is still zero."""
    sees = [np.eye(n, dtype=bool), np.eye(n, dtype=bool), np.zeros((n, n), bool)]
    c = Case(n + 2, [(270, n), (0, n), (0, n)], 4, 2, D, dtype, sees=sees)
    positive_first_dim(c)
    set_keys(c, 0, list(range(270)) + [270 + n - 1], float("-inf"))
    set_keys(c, 1, [0, n - 1], float("-inf"))
    out = c.run(ws=c.workspace() if split else None).double().cpu().numpy()
    check_status_clean()
    assert np.isnan(out[n - 1]).all() and np.isnan(out[n]).all() and np.isnan(out[2 * n - 1]).all()
    assert (out[2 * n:] == 0).all()
    # the others see one key each: its value
    for i, rows in ((0, range(n - 1)), (1, range(1, n - 1))):
        for j in rows:
            t = int(c.ctx[i]) - n + j
            v = c.vc[int(c.tables[i, t // 16]), :, t % 16].double().numpy()
            want = np.repeat(v, 2, axis=0)
            assert (np.abs(out[c.qs[i] + j] - want) <= bound(want, np.abs(want), dtype, D)).all()
