"""Rows that hold a NaN or an infinity, and rows of zeros with eps = 0: what the norm's
definition makes of them reaches the output, in 8 bits through the row's scale."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import layer_to_dev, say, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [128, 4096, 28672, 40000])
@pytest.mark.parametrize("n_out", [0, 8])
def test_a_bad_row_stays_bad(gpu_lib, K, n_out):
    """Row 1 holds a NaN, row 3 an infinity, row 4 overflows the sum to one (the block
    before wrote an infinity), row 6 is zero with eps = 0; the others are as without them."""
    import torch
    say(f"[norm nonfinite] K={K} outliers={n_out}")
    rng = np.random.default_rng(K)
    x = rng.standard_normal((8, K)).astype(np.float16)
    res = rng.standard_normal((8, K)).astype(np.float16)
    w = (1 + 0.1 * rng.standard_normal(K)).astype(np.float16)
    out = np.sort(rng.choice(K, n_out, replace=False)).astype(np.int32)
    inner = np.setdiff1d(np.arange(K), out)  # channels that are not outliers
    good = x.copy()
    x[1, inner[5]] = np.nan
    x[3, inner[-1]] = -np.inf
    res[4, inner[7]] = np.inf
    x[6], res[6] = 0, 0
    bad = [1, 3, 4, 6]
    fine = [0, 2, 5, 7]
    xd, rd, wd, od = (to_dev(a, torch) for a in (x, res, w, out))
    xq, sx, xo, h = gpu_lib.add_rmsnorm_int8(xd, wd, rd, eps=0.0, outliers=od)
    values = gpu_lib.dequantize_act_int8(xq, sx, xo, od)
    y, _ = gpu_lib.add_rmsnorm(xd, wd, rd, eps=0.0)
    torch.cuda.synchronize()
    # all of a row with a NaN, or of zeros, is NaN; one with an infinity is NaN there
    nan = torch.isnan(y.float().cpu())
    assert bool(nan[1].all()) and bool(nan[6].all()) and bool(nan[3, inner[-1]]) and bool(nan[4, inner[7]])
    assert bool(torch.isnan(sx[bad]).all()) and bool(torch.isfinite(sx[fine]).all())
    assert bool(torch.isnan(values[bad][:, to_dev(inner, torch)]).all())
    assert bool(torch.isfinite(values[fine]).all())
    ref = gpu_lib.add_rmsnorm_int8(to_dev(good[fine], torch), wd, to_dev(res[fine], torch), eps=0.0, outliers=od)
    for got, want in zip((xq[fine], sx[fine], xo[fine], h[fine]), ref):
        assert torch.equal(got, want)


def test_a_bad_outlier(gpu_lib):
    """An infinity in an outlier channel: the other channels are 0 (divided by it), the
    outlier itself is NaN; a NaN there takes the whole row. A weight that is NaN, in every
    row's range."""
    import torch
    rng = np.random.default_rng(2)
    K, out = 512, np.array([3, 100], np.int32)
    x = rng.standard_normal((3, K)).astype(np.float16)
    x[0, 100] = np.inf
    x[2, 3] = np.nan
    w = np.ones(K, np.float16)
    od = to_dev(out, torch)
    xq, sx, xo, _ = gpu_lib.add_rmsnorm_int8(to_dev(x, torch), to_dev(w, torch), outliers=od)
    v = gpu_lib.dequantize_act_int8(xq, sx, xo, od).float().cpu()
    assert bool(torch.isnan(v[0, 100])) and float(v[0].nan_to_num().abs().max()) == 0.0
    assert bool(torch.isfinite(v[1]).all()) and bool(torch.isnan(v[2]).all())
    w[40] = np.nan
    _, sx, _, _ = gpu_lib.add_rmsnorm_int8(to_dev(x[1:2], torch), to_dev(w, torch), outliers=od)
    assert bool(torch.isnan(sx).all())


def test_the_product_shows_it(gpu_lib):
    """A bad row's products are NaN, its neighbours' those without it."""
    import torch
    M, N, K = 5, 300, 1024
    rng = np.random.default_rng(3)
    x = rng.standard_normal((M, K)).astype(np.float16)
    x[2, 700] = np.inf
    w = np.ones(K, np.float16)
    L = oracle.quantize_layer(workloads.random_weights(6, N, K), 0)
    D = layer_to_dev(L, torch)
    od = to_dev(np.array([8, 9], np.int32), torch)

    def product(rows):
        xq, sx, xo, _ = gpu_lib.add_rmsnorm_int8(to_dev(rows, torch), to_dev(w, torch), outliers=od)
        return gpu_lib.linear_w4a8_quantized(xq, sx, xo, od, D["packed"], D["scales"], D["zeros"])

    y = product(x)
    assert bool(torch.isnan(y[2]).all())
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], product(x[keep]))
