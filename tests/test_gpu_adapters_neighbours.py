"""A row of linear_adapters has the same bits whatever the batch's other rows hold, which adapters they name and where it
stands among them, in float32 as in fp16: by the decode kernels, by each GEMM with and without slices of K, and by both
down-projections."""
import numpy as np
import pytest

import workloads
from gpu_cases import say, to_dev
from rows_cases import factors, layer, run_adapters

pytestmark = pytest.mark.gpu


def check(wq, M, N, K, r, n, per_mille, kernel, seeds=8):
    import torch
    L = layer(M + N, N, K, per_mille)
    L1, L2 = factors(M + K, n, r, N, K)
    L2 *= np.float16(8)  # (the branch as large as the layer's own output: its terms' order shows)
    scale = np.random.default_rng(r).uniform(0.5, 2.0, n)
    for seed in range(seeds):
        rng = np.random.default_rng(seed)
        x, ids, p = workloads.random_x(seed, M, K), rng.integers(-1, n, M), rng.permutation(M)
        kept = rng.random(M) < 0.3
        others = np.where(kept, ids, rng.integers(-1, n, M))
        x2 = np.where(kept[:, None], x, workloads.random_x(100 + seed, M, K))
        for dtype in (torch.float32, torch.float16):
            y = run_adapters(wq, torch, L, x, L1, L2, ids, scale, kernel=kernel, out_dtype=dtype)
            moved = run_adapters(wq, torch, L, x[p], L1, L2, ids[p], scale, kernel=kernel, out_dtype=dtype)
            differ = (moved != y[to_dev(p, torch)]).sum().item()
            assert differ == 0, f"seed {seed}: {differ} outputs of a permuted batch differ ({dtype})"
            beside = run_adapters(wq, torch, L, x2, L1, L2, others, scale, kernel=kernel, out_dtype=dtype)
            rows = to_dev(kept, torch)
            differ = (beside[rows] != y[rows]).sum().item()
            assert differ == 0, f"seed {seed}: {differ} outputs beside other rows differ ({dtype})"


@pytest.mark.parametrize("M,N,K,r,n,per_mille", [
    (2, 300, 1024, 16, 3, 0), (5, 96, 384, 40, 4, 4), (16, 300, 1024, 16, 9, 0), (16, 130, 4096, 64, 40, 4),
    (48, 300, 1024, 16, 9, 0), (70, 2100, 1024, 8, 70, 0), (33, 4097, 512, 72, 5, 4)])
def test_decode_kernels(gpu_lib, M, N, K, r, n, per_mille):
    say(f"[neighbours decode] M={M} N={N} K={K} r={r} n={n}")
    check(gpu_lib, M, N, K, r, n, per_mille, "gemv")


@pytest.mark.parametrize("M,N,K,r,n,per_mille", [
    (40, 300, 1024, 16, 9, 0),      # slices of K, no two rows alike
    (64, 520, 4096, 64, 64, 0), (64, 520, 4096, 24, 5, 4), (33, 96, 8192, 8, 33, 0),
    (100, 300, 1152, 16, 30, 4), (100, 300, 4224, 16, 30, 0),  # tile GEMM, its slices
    (200, 256, 4096, 32, 12, 4), (300, 300, 2048, 8, 300, 0)])
def test_gemms(gpu_lib, M, N, K, r, n, per_mille):
    say(f"[neighbours gemm] M={M} N={N} K={K} r={r} n={n}")
    check(gpu_lib, M, N, K, r, n, per_mille, "gemm", seeds=4)


@pytest.mark.parametrize("M,N,K,r,n,kernel", [
    (300, 40, 8192, 24, 9, "gemv"), (131, 33, 16512, 40, 131, "gemv"), (400, 48, 1280, 80, 3, "gemm"),
    (2100, 16, 2048, 16, 30, "gemv"), (1100, 64, 256, 128, 20, "gemm"), (700, 270, 1152, 56, 5, "gemm")])
def test_down_projection_of_many_rows(gpu_lib, M, N, K, r, n, kernel):
    """(Its waves are dealt to the adapters of 16 rows: one to sixteen waves share K for a row.)"""
    say(f"[neighbours down] M={M} N={N} K={K} r={r} n={n}")
    check(gpu_lib, M, N, K, r, n, 0, kernel, seeds=4)
