"""Tree attention in every variant of its kernels: rows a unit, merge on the
spot or by a second launch, one or several units a sequence, on either side
of each border.  What decides is the largest draft times the query heads of a
kv head, the width of the tables and the number of units, not the lengths.

fp32: 16 rows a unit up to 16 (or where the tables hold little), 32 up to 32,
64 above; bf16: 128 up to 128, two halves of 128 above.  A unit for four CTAs
or more is merged by the second launch.

Each call runs three times on one workspace: the same bits, and counters of
zero behind it.  Tolerances: see test_gpu_tree."""

import numpy as np
import pytest
import torch

import paged_kv_cache_351_b200 as pa
from gpu_harness import check_status_clean
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

# (drafted tokens, query heads a kv head): 9 to 264 rows a kv head
ROWS = {"f32": [(9, 1), (16, 1), (17, 1), (8, 4), (33, 1), (16, 4), (65, 1), (10, 8), (33, 4)],
        "bf16": [(9, 1), (127, 1), (16, 8), (129, 1), (33, 4), (128, 2), (257, 1), (33, 8)]}


@pytest.mark.parametrize("dtype,n,G", [(dtype, n, G) for dtype, rows in ROWS.items() for n, G in rows])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("units", ["few", "many", "few in small tables"])
def test_rows_and_merges(dtype, D, n, G, units):
    if units == "many":
        pairs, hk = [(300 + 20 * i, n if i % 3 == 0 else max(1, n // 3)) for i in range(4 if n > 33 else 10)], 8
        pairs += [(20, 1)] * (20 - len(pairs))
    else:
        pairs, hk = [(2500 if units == "few" else 250, n), (70, max(1, n // 2))], 2
    c = Case(100 * n + G, pairs, hk * G, hk, D, dtype)
    # (the case's fp32 K and V are one tensor)
    v = torch.randn(c.vc.shape, generator=torch.Generator().manual_seed(n)).to(c.vc.dtype)
    c.vc = torch.where(c.vc.isnan(), c.vc, v)
    if units != "few in small tables":
        c.tables = np.pad(c.tables, ((0, 0), (0, 1300)), constant_values=-1)
    ws = c.workspace()
    out = c.run(ws=ws)
    check_status_clean()
    c.check(out)
    for _ in range(2):
        assert torch.equal(c.run(ws=ws), out)
    assert int(ws[: pa.PA_DECODE_WS_HEADER_BYTES].count_nonzero()) == 0
