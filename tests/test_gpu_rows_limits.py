"""Adapters, routing and experts at the far ends of what they take: batches of more rows than one launch, or a grid's second
dimension, holds; experts as wide as they may be. References in float64 on the GPU."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import say, to_dev
from rows_cases import worst
from test_gpu_long_rows import bound, held, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", ["gemv", "gemm"])
def test_adapters_of_more_rows_than_a_launch(gpu_lib, kernel):
    import torch
    M, N, K, n, r = 1_100_003, 9, 128, 3, 24
    say(f"[rows limits] adapters M={M} {kernel}")
    g = torch.Generator(device="cuda").manual_seed(1)
    packed, s, z = layer(torch, N, K, 2)
    x = torch.randn(M, K, device="cuda", generator=g).half()
    L1 = (torch.randn(n, r, K, device="cuda", generator=g) / K ** 0.5).half()
    L2 = torch.randn(n, N, r, device="cuda", generator=g).half()
    ids = torch.randint(-1, n + 1, (M,), device="cuda", generator=g, dtype=torch.int32)
    y = gpu_lib.linear_adapters(x, packed, s, z, L1, L2, ids, kernel=kernel, out_dtype=torch.float32).double()
    w = held(torch, packed, s, z)
    for at in range(0, M, 1 << 18):
        rows = slice(at, at + (1 << 18))
        xd = x[rows].double()
        ref, most = xd @ w.t(), bound(xd, w, s)
        for a in range(n):
            mine = ids[rows] == a
            one, two = L1[a].double(), L2[a].double()
            t, off = xd[mine] @ one.t(), (K + 8) * 2.0 ** -24 * (xd[mine].abs() @ one.abs().t())
            ref[mine] += t @ two.t()
            # t's sum and its rounding to fp16, and r terms more in float32
            off = off + 2.0 ** -11 * (t.abs() + off) + 2.0 ** -25 + (2 * r + 8) * 2.0 ** -24 * t.abs()
            most[mine] += off @ two.abs().t()
        assert ((y[rows] - ref).abs() <= most).all(), at


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_route_of_many_rows(gpu_lib, dtype):
    import torch
    M, E, k = 600_011, 33, 4
    say(f"[rows limits] route M={M} {dtype}")
    logits = torch.randn(M, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    logits = logits.to(getattr(torch, dtype))
    e, w = gpu_lib.moe_route(logits, k)
    top, order = torch.sort(logits.double(), dim=-1, descending=True, stable=True)
    assert torch.equal(e, order[:, :k].int())
    p = torch.exp(top[:, :k] - top[:, :1])
    p /= p.sum(-1, keepdim=True)
    # an exponential (its argument's rounding, of at most 16, and two of its own), a sum and a quotient
    assert ((w.double() - p).abs() <= p * 2.0 ** -24 * (2 * 16 + k + 8)).all()


def codes(rng, E, N, K):
    q = rng.integers(0, 16, (E, N, K), dtype=np.uint8)
    s = (rng.uniform(0.5, 1.5, (E, N, K // 128)) * 0.25 * K ** -0.5).astype(np.float16)
    z = rng.integers(0, 16, (E, N, K // 128)).astype(np.float16)
    packed = oracle.pack(q.reshape(-1, K)).reshape(E, N, -1)
    return (packed, s, z), [oracle.dequant(q[i], s[i], z[i]) for i in range(E)]


@pytest.mark.parametrize("H,I", [(65536, 128), (128, 65536), (16384, 1024)])
def test_experts_of_all_widths(gpu_lib, H, I):
    import torch
    E, k = 2, 2
    rng = np.random.default_rng(H)
    up, held_up = codes(rng, E, 2 * I, H)
    down, held_down = codes(rng, E, H, I)
    args = [to_dev(v, torch) for v in (*up, *down)]
    for M in (1, 4, 6, 40):
        say(f"[rows limits] experts M={M} {H} x {I}")
        x = workloads.random_x(M, M, H)
        e, w = rng.integers(-1, E, (M, k)), rng.uniform(0.1, 1.0, (M, k))
        ref, most = oracle.rows.moe_experts(x, e, w.astype(np.float32), held_up, held_down)
        y = gpu_lib.moe_experts(to_dev(x, torch), to_dev(e.astype(np.int32), torch),
                                to_dev(w.astype(np.float32), torch), *args, out_dtype=torch.float32)
        assert worst(y, ref, most, f16=False) <= 1.0


def test_experts_of_many_rows(gpu_lib):
    """70001 rows, more than 65535: many blocks of lists, and as many of the join."""
    import torch
    M, H, I, E, k = 70_001, 128, 128, 7, 3
    say(f"[rows limits] experts M={M}")
    rng = np.random.default_rng(5)
    up, held_up = codes(rng, E, 2 * I, H)
    down, held_down = codes(rng, E, H, I)
    x = workloads.random_x(7, M, H)
    e = rng.integers(-1, E, (M, k))
    w = rng.uniform(0.1, 1.0, (M, k)).astype(np.float32)
    ref, most = oracle.rows.moe_experts(x, e, w, held_up, held_down)
    y = gpu_lib.moe_experts(to_dev(x, torch), to_dev(e.astype(np.int32), torch), to_dev(w, torch),
                            *(to_dev(v, torch) for v in (*up, *down)), out_dtype=torch.float32)
    assert worst(y, ref, most, f16=False) <= 1.0
