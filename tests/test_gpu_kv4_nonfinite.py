"""Queries that hold a NaN or an infinity: their rows' outputs and log sums say so, and no
other row notices."""
import numpy as np
import pytest

from gpu_cases import say, to_dev
from kv4_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,ctx,hq,hkv,d", [
    ([1, 1], [40, 300], 4, 2, 128),        # finished in a block
    ([1], [9000], 8, 2, 64),               # joined from many
    ([7, 1], [5, 2000], 4, 1, 128),        # leading rows that see nothing
    ([500], [500], 32, 4, 64),             # many rows, whole row tiles
    ([300], [3000], 16, 2, 128),           # many rows, shares of them
])
def test_a_bad_query(gpu_lib, new, ctx, hq, hkv, d):
    import torch
    say(f"[kv4 nonfinite] new={new} ctx={ctx} d={d}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 64, seed=5).fill()
    out, lse = b.attention()
    T = sum(new)
    bad = [(0, 0), (T - 1, hq - 1), (T // 2, 1)]
    q = b.q.copy()
    for n, (row, head) in enumerate(bad):
        q[row, head, 3 * n] = (np.nan, np.inf, np.nan)[n]
    # a NaN or an infinity times codes of both signs and 0: the sums are NaN where a token is seen
    got, got_lse = b.attention(q=to_dev(q, torch))
    sees = torch.isfinite(lse)
    for row, head in bad:
        if sees[row, head]:
            assert bool(torch.isnan(got_lse[row, head])), (row, head)
            assert bool(torch.isnan(got[row, head]).all()), (row, head)
        else:
            assert float(got_lse[row, head]) == -np.inf and float(got[row, head].abs().max()) == 0
        got[row, head], got_lse[row, head] = out[row, head], lse[row, head]
    assert torch.equal(got, out) and torch.equal(got_lse, lse)
