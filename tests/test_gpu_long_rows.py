"""Rows of any length that the entry points take: so long that the decode kernels' scales and zero-points, staged in LDS,
fill it with two tiles, or with one; and lengths just below 64 KB of it. The reference is a float64 product on the GPU of the
codes that the layer holds."""
import pytest

from gpu_cases import say

pytestmark = pytest.mark.gpu


def layer(torch, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), dtype=torch.int32, device="cuda", generator=g)
    s = (torch.rand(N, K // 128, device="cuda", generator=g) * 0.01 + 0.005).half()
    z = torch.randint(0, 16, (N, K // 128), device="cuda", generator=g).half()
    return packed, s, z


def held(torch, packed, s, z):
    q = torch.stack([(packed >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2).double()
    return (q - z.double().repeat_interleave(128, -1)) * s.double().repeat_interleave(128, -1)


def bound(x, w, s):
    """Float32 sums of K terms, and a rounding of each weight to fp16 in the GEMM. The decode kernels of one or two rows take
    (1024 + z) sum x off a group's sum of (1024 + q) x: two sums of 128 terms of at most 1040 |x|, times s."""
    M, K = x.shape
    mag = x.abs() @ w.abs().t()
    most = ((K + 8) * 2.0 ** -24 + 2.0 ** -11) * mag
    if M <= 2:
        most = most + 2 * 136 * 2.0 ** -24 * 1040 * (x.abs() @ s.double().repeat_interleave(128, -1).t())
    return most


SIZES = [(1, 48, 24576), (2, 48, 13312), (16, 8192, 47104), (16, 64, 94208),  # just below 64 KB
         (16, 8192, 138240), (5, 8200, 139520), (16, 40, 284160), (3, 40, 300032), (1, 64, 2 ** 19), (4, 64, 2 ** 19),
         (40, 64, 2 ** 19), (70, 8, 2 ** 19)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(gpu_lib, M, N, K):
    import torch
    say(f"[long rows] M={M} N={N} K={K} {gpu_lib.auto_kernel(M, N, K)}")
    packed, s, z = layer(torch, N, K, K)
    x = torch.randn(M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(M)).half()
    y = gpu_lib.linear(x, packed, s, z, out_dtype=torch.float32)
    rows = torch.arange(0, N, max(1, N // 40), device="cuda")
    w = held(torch, packed[rows], s[rows], z[rows])
    xd = x.double()
    assert ((y[:, rows].double() - xd @ w.t()).abs() <= bound(xd, w, s[rows])).all()


@pytest.mark.parametrize("M,N,K", SIZES)
def test_adapters(gpu_lib, M, N, K):
    import torch
    say(f"[long rows, adapters] M={M} N={N} K={K}")
    r, n = 8, 3
    g = torch.Generator(device="cuda").manual_seed(K + M)
    packed, s, z = layer(torch, N, K, K)
    x = torch.randn(M, K, device="cuda", generator=g).half()
    L1 = (torch.randn(n, r, K, device="cuda", generator=g) / K ** 0.5).half()
    L2 = torch.randn(n, N, r, device="cuda", generator=g).half()
    ids = (torch.arange(M, device="cuda") % (n + 1) - 1).int()
    y = gpu_lib.linear_adapters(x, packed, s, z, L1, L2, ids, out_dtype=torch.float32)
    rows = torch.arange(0, N, max(1, N // 40), device="cuda")
    w = held(torch, packed[rows], s[rows], z[rows])
    xd = x.double()
    ref, most = xd @ w.t(), bound(xd, w, s[rows])
    for m in range(M):
        a = int(ids[m])
        if a >= 0:
            one, two = L1[a].double(), L2[a][rows].double()
            t, up = one @ xd[m], (K + 8) * 2.0 ** -24 * (one.abs() @ xd[m].abs())
            ref[m] += two @ t
            # t's sum and its rounding to fp16, and r terms more in float32
            most[m] += two.abs() @ (up + 2.0 ** -11 * (t.abs() + up) + 2.0 ** -25 + (2 * r + 8) * 2.0 ** -24 * t.abs())
    assert ((y[:, rows].double() - ref).abs() <= most).all()


def test_a_kernel_that_does_not_fit(gpu_lib):
    """Asked for by name it is an error, which leaves nothing behind in HIP's state or on the stream."""
    import torch
    say("[long rows, refused]")
    N, K = 64, 2 ** 19
    packed, s, z = layer(torch, N, K, 1)
    x = torch.ones(4, K, dtype=torch.float16, device="cuda")
    want = gpu_lib.linear(x, packed, s, z)
    for _ in range(2):
        with pytest.raises(gpu_lib.WQError):
            gpu_lib.linear(x, packed, s, z, kernel="gemv")
        assert (torch.zeros(8, device="cuda") == 0).all()
        torch.cuda.synchronize()
        assert torch.equal(gpu_lib.linear(x, packed, s, z), want)
