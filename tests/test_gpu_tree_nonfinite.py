"""Tree attention over caches with infinities and NaN in keys that rows do
see: what the formula gives in fp64 (a logit of -infinity weighs nothing, a
row of nothing else, a logit of +infinity or a NaN give NaN), in every kernel,
wherever the keys lie in a tile.  Tolerances: see test_gpu_tree."""

import numpy as np
import pytest
import torch

from gpu_harness import check_status_clean
from test_gpu_tree import KINDS, Case

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
