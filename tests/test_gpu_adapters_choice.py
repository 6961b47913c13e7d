"""Which kernel AUTO takes beside adapters, told by its bits: the decode kernels for rows in the hundreds, the GEMM for
prompts on layers of any size."""
import numpy as np
import pytest

import workloads
from gpu_cases import say, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,n,kernel", [
    (1024, 256, 512, 2, "gemv"), (2048, 256, 512, 9, "gemv"), (100, 2048, 2048, 2, "gemv"), (200, 2048, 2048, 9, "gemv"),
    (64, 4096, 4096, 2, "gemv"), (128, 4096, 4096, 9, "gemv"),
    (512, 4096, 512, 2, "gemm"), (1024, 4096, 512, 9, "gemm"), (4096, 512, 512, 2, "gemm"), (4096, 1024, 1024, 9, "gemm"),
    (64, 8192, 4096, 300, "gemv"), (64, 8192, 8192, 2, "gemm"), (300, 4096, 4096, 2, "gemm"), (600, 4096, 4096, 9, "gemm"),
    (9000, 512, 128, 2, "gemm")])
def test_choice(gpu_lib, M, N, K, n, kernel):
    import torch
    say(f"[adapters choice] M={M} N={N} K={K} n={n}: {kernel}")
    g = torch.Generator(device="cuda").manual_seed(M + n)
    packed = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), dtype=torch.int32, device="cuda", generator=g)
    s = (torch.rand(N, K // 128, device="cuda", generator=g) * 0.01 + 0.005).half()
    z = torch.randint(0, 16, (N, K // 128), device="cuda", generator=g).half()
    x = to_dev(workloads.random_x(M, M, K), torch)
    L1 = (torch.randn(n, 8, K, device="cuda", generator=g) / K ** 0.5).half()
    L2 = torch.randn(n, N, 8, device="cuda", generator=g).half()
    ids = to_dev(np.random.default_rng(M).integers(-1, n, M).astype(np.int32), torch)
    y = {k: gpu_lib.linear_adapters(x, packed, s, z, L1, L2, ids, kernel=k, out_dtype=torch.float32)
         for k in ("auto", "gemv", "gemm")}
    assert not torch.equal(y["gemv"], y["gemm"])
    assert torch.equal(y["auto"], y[kernel])
