"""Scores so large that neighbouring float32 values lie far apart: as long as queries and
keys are finite, so are the outputs."""
import numpy as np
import pytest

import oracle
from gpu_cases import say
from kv4_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [30.0, 300.0, 3000.0, 30000.0])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("new,ctx,hq,hkv,d", [
    ([1, 1], [64, 700], 2, 2, 128),
    ([1], [6000], 4, 1, 64),
    ([20], [300], 4, 2, 128),
    ([500], [500], 32, 4, 64),
    ([600], [900], 16, 2, 128),
])
def test_large_scores(gpu_lib, new, ctx, hq, hkv, d, size, sign):
    """Queries and keys of some `size` in each channel, along one direction, so that scores
    reach size^2 d / sqrt(d) (1e10), all positive or all negative. Products of an fp16 query and
    a code less its zero-point are exact in float32 and their sum of d is off by less than d
    2^-24 of the sum of magnitudes, once more by the scale and the exponent's factor; so
    whatever weights come of scores within that of the exact ones are right. In the tokens
    that can have the row's largest score the held values bound the output."""
    import torch
    rng = np.random.default_rng(int(size))
    L, T = sum(ctx), sum(new)
    u = rng.choice([-1.0, 1.0], d)
    k = size * u * rng.uniform(0.8, 1.2, (L, hkv, d))
    k[L // 2:] *= 1.3  # the largest are not the first
    q = sign * size * u * rng.uniform(0.9, 1.1, (T, hq, d))
    v = rng.standard_normal((L, hkv, d))
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 32, seed=9, k=k.astype(np.float16), v=v.astype(np.float16),
              q=q.astype(np.float16)).fill()
    out, lse = b.attention()
    got, got_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    say(f"[kv4 large scores] new={new} ctx={ctx} size={size} sign={sign}")
    assert np.isfinite(got).all() and np.isfinite(got_lse).all()
    row = 0
    for s, (n, c) in enumerate(zip(new, ctx)):
        kk, vv = (oracle.kv4_values(x[b.begin[s]:b.begin[s] + c]) for x in (b.k, b.v))
        for i in range(0, n, max(1, n // 7)):
            for h in range(hq):
                seen = c - n + i + 1
                qi, kh, vh = b.q[row + i, h].astype(np.float64), kk[:seen, h * hkv // hq], vv[:seen, h * hkv // hq]
                x = kh @ qi / np.sqrt(d)
                off = (d + 8) * 2.0 ** -24 * (np.abs(kh) @ np.abs(qi)).max() / np.sqrt(d)
                assert abs(got_lse[row + i, h] - (x.max() + np.log(np.exp(x - x.max()).sum()))) <= 2 * off + 1e-4
                # tokens that rounding cannot put ahead have at most e^-20 each of the weight
                near = x >= x.max() - 2 * off - 20
                lo, hi = vh[near].min(0), vh[near].max(0)
                eps = 2.0 ** -10 * np.abs(vh).max() + np.exp(-20) * seen * np.abs(vh).max()
                assert np.all(got[row + i, h] >= lo - eps) and np.all(got[row + i, h] <= hi + eps), (i, h)
        row += n


@pytest.mark.parametrize("scale", [1e-30, 1e16])
@pytest.mark.parametrize("new,ctx,hq", [([1], [70], 4), ([300], [300], 8)])
def test_scale_limits(gpu_lib, new, ctx, hq, scale):
    """The largest scale makes every row its best token's values (scores some 1e15 apart, all
    negative), a vanishing one their mean."""
    import torch
    rng = np.random.default_rng(1)
    d, c = 128, ctx[0]
    k = -np.abs(rng.standard_normal((c, 1, d))).astype(np.float16)
    q = np.abs(rng.standard_normal((new[0], hq, d))).astype(np.float16)
    b = Batch(gpu_lib, torch, new, ctx, hq, 1, d, 32, seed=2, k=k, q=q).fill()
    out, lse = b.attention(scale=scale)
    got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
    kk, vv = oracle.kv4_values(b.k)[:, 0], oracle.kv4_values(b.v)[:, 0]
    for i in range(0, new[0], 13):
        seen = c - new[0] + i + 1
        x = kk[:seen] @ b.q[i, 0].astype(np.float64)
        want = vv[x.argmax()] if scale > 1 else vv[:seen].mean(0)
        size = np.abs(want) if scale > 1 else np.abs(vv[:seen]).mean(0)
        assert np.all(np.abs(got[i, 0] - want) <= 2.0 ** -10 * size + 2.0 ** -24)
        if scale > 1:
            assert abs(got_lse[i, 0] / (scale * x.max()) - 1) < 1e-5
        else:
            assert abs(got_lse[i, 0] - np.log(seen)) < 1e-5
