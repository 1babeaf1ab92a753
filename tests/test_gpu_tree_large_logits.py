"""Tree attention where logits are so large that their rounding to fp32 is not
small beside 1: the key of the largest one has all the weight.

Tolerance: a logit is a sum of D fp32 products, off by at most e = (D + 2)
2^-24 sum |q k| scale.  Where the two largest logits of a row are more than 2 e
+ 64 apart, the largest keeps a share of 1 - n 2^-92 (n keys), far closer to 1
than the output's rounding, so the output is that key's value, rounded once
(the bounds of test_gpu_tree with |V| as the sum's size).  Rows whose largest
logits are nearer than that are left out; they must be few."""

import numpy as np
import pytest
import torch

from gpu_harness import check_status_clean
from test_gpu_tree import KINDS, Case, bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("n", [9, 30, 100])
@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("power", [20, 32, 60, 110])
def test_one_key_has_all_the_weight(dtype, D, n, split, power):
    c = Case(n + power, [(500, n), (40, 3), (0, n)], 4, 2, D, dtype)
    c.kc = (c.kc.double() * 2.0 ** power).to(c.kc.dtype)  # (exact)
    out = c.run(ws=c.workspace() if split else None)[:c.rows].double().cpu().numpy()
    check_status_clean()
    q, kc, vc = c.q.double().numpy(), c.kc.double().numpy(), c.vc.double().numpy()
    rows = apart = 0
    for i, sees in enumerate(c.sees):
        c0 = int(c.ctx[i]) - len(sees)
        for j in range(len(sees)):
            pos = list(range(c0)) + [c0 + u for u in range(len(sees)) if sees[j, u]]
            k, v = (np.stack([x[int(c.tables[i, t // 16]), :, t % 16] for t in pos]) for x in (kc, vc))
            for h in range(4):
                qr = q[int(c.qs[i]) + j, h]
                z, e = c.scale * (k[:, h // 2] @ qr), c.scale * (np.abs(k[:, h // 2]) @ np.abs(qr))
                top = np.sort(z)[-2:]
                got = out[int(c.qs[i]) + j, h]
                assert np.isfinite(got).all()
                rows += 1
                if len(top) == 2 and top[1] - top[0] <= 2 * (D + 2) * 2.0 ** -24 * e.max() + 64:
                    continue
                apart += 1
                want = v[z.argmax(), h // 2]
                assert (np.abs(got - want) <= bound(want, np.abs(want), dtype, D)).all()
    assert apart > 0.9 * rows
