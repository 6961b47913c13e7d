"""Neighbouring tokens whose value scales lie as far apart as fp16 lets them: whichever
outweighs the other, the output keeps the bits of the bound in kv4_cases."""
import numpy as np
import pytest

from gpu_cases import say
from kv4_cases import Batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ahead", [0, 10, 20, 26, 32])
@pytest.mark.parametrize("new,ctx,hq,hkv,d", [
    ([1, 1], [64, 700], 2, 2, 128),
    ([1], [6000], 4, 1, 64),
    ([20], [300], 4, 2, 128),
    ([500], [500], 32, 4, 64),
    ([600], [900], 16, 2, 128),
])
def test_neighbours_of_unlike_scales(gpu_lib, new, ctx, hq, hkv, d, ahead):
    """Every other token has values of some 2^-11, its neighbours 2^15; the scores of the
    first kind are ahead by `ahead` powers of two, so that either kind takes the sum (0, 10)
    or both have a part in it (26)."""
    import torch
    rng = np.random.default_rng(ahead)
    L, T = sum(ctx), sum(new)
    u = rng.standard_normal(d)
    u /= np.linalg.norm(u)
    # scores: q . k / sqrt(d), q = 4 u (and a little else), k = a u + a little else
    small = np.arange(L) % 2 == 0
    a = np.where(small, ahead * np.log(2), 0.0) * np.sqrt(d) / 4
    k = a[:, None, None] * u + 0.05 * rng.standard_normal((L, hkv, d))
    v = rng.uniform(-1, 1, (L, hkv, d)) * np.where(small, 2.0 ** -11, 6e4)[:, None, None]
    q = 4 * u + 0.05 * rng.standard_normal((T, hq, d))
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 32, seed=ahead, k=k.astype(np.float16), v=v.astype(np.float16),
              q=q.astype(np.float16)).fill()
    say(f"[kv4 neighbours] new={new} ctx={ctx} d={d} ahead={ahead}")
    check(*b.attention(), b.reference(), f"ahead {ahead}")
