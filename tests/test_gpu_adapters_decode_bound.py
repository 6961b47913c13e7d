"""The decode kernel of three rows and more with adapters, against a bound without the GEMM's rounding of each weight: it
holds q - z exactly and applies the scale to a group's float32 sum. (That of one or two rows takes 1024 + z off a group's
sum of (1024 + q) x: sums of larger terms, whose bound is no closer than the one with rounded weights.)"""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import say
from rows_cases import factors, layer, run_adapters, worst

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["any", "one", "none"])
@pytest.mark.parametrize("M,N,K,r,n,per_mille", [
    (3, 17, 384, 16, 4, 0), (5, 300, 1536, 96, 5, 4), (7, 64, 4096, 32, 7, 0), (12, 48, 14336, 16, 12, 0),
    (16, 260, 2048, 24, 16, 4), (16, 1, 128, 8, 7, 0), (4, 64, 128, 256, 1, 4),
    (17, 130, 1024, 16, 3, 0), (33, 4097, 512, 64, 40, 0), (70, 300, 1024, 56, 6, 4),
    (300, 40, 8192, 24, 9, 0)])
def test_decode_kernels(gpu_lib, M, N, K, r, n, per_mille, kind):
    import torch
    say(f"[adapters decode bound] M={M} N={N} K={K} r={r} n={n} sparse={per_mille} rows={kind}")
    L = layer(M + N + K, N, K, per_mille)
    rng = np.random.default_rng(M + K)
    x = workloads.random_x(M + 5 * r, M, K)
    L1, L2 = factors(M + r, n, r, N, K)
    ids = {"any": rng.integers(-1, n, M), "one": np.full(M, n - 1), "none": np.full(M, -1)}[kind]
    scale = rng.uniform(0.25, 2.0, n).astype(np.float32)
    ref, bound = oracle.rows.linear_adapters(x, L["held"], L1, L2, ids, scale)
    y = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel="gemv", out_dtype=torch.float32)
    err = worst(y, ref, bound, f16=False)
    say(f"    {err:.3f} of the bound")
    assert err <= 1.0
