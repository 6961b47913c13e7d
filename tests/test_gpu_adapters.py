"""Low-rank adapters that each row names, beside the 4-bit layer, against the float64 oracle, with bounds that count the
kernels' roundings (oracle/rows.py)."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import layer_to_dev, say, to_dev
from rows_cases import factors, layer, run_adapters, worst

pytestmark = pytest.mark.gpu

# (M, N, K, r, n, nnz per mille, kernel): each kernel and split of the product, ranks that fill a step and do not
SHAPES = [
    (1, 300, 1024, 8, 3, 0, "auto"), (1, 64, 128, 256, 1, 4, "auto"), (2, 130, 2048, 40, 5, 4, "auto"),
    (1, 33, 12288, 16, 2, 0, "auto"),     # a single row of a long layer
    (3, 17, 384, 16, 4, 0, "auto"), (5, 300, 1536, 96, 5, 4, "auto"), (16, 260, 2048, 24, 16, 4, "auto"),
    (16, 1, 128, 8, 7, 0, "auto"), (33, 4097, 512, 64, 40, 0, "gemv"),
    (16, 300, 1024, 32, 9, 4, "gemm"), (40, 300, 1024, 64, 11, 4, "auto"), (64, 520, 2048, 200, 64, 0, "auto"),
    (65, 520, 2048, 16, 9, 0, "auto"),
    (100, 300, 1152, 16, 30, 4, "gemm"),  # tile GEMM
    (130, 513, 384, 48, 3, 0, "gemm"), (200, 256, 4096, 128, 12, 4, "gemm"), (300, 300, 1152, 8, 300, 0, "gemm"),
    (70, 300, 1024, 56, 6, 4, "gemv"), (700, 270, 1024, 16, 5, 0, "gemm"), (530, 1000, 8320, 24, 3, 0, "gemm"),
    (64, 520, 2048, 72, 64, 0, "gemm"), (40, 300, 1024, 64, 11, 4, "gemm"), (80, 64, 2176, 24, 80, 0, "auto"),
    (300, 40, 8192, 24, 9, 0, "auto"), (131, 33, 16512, 40, 131, 0, "auto"),  # several chunks of K
    (2100, 16, 2048, 8, 30, 0, "auto"), (400, 48, 1280, 80, 3, 4, "auto"),
]


def _rows(rng, M, n, kind):
    """Adapters of M rows: any order, in runs as prompts are, or one for all."""
    if kind == "one":
        return np.full(M, rng.integers(n))
    ids = rng.integers(-1, n, M)
    return np.sort(ids) if kind == "runs" else ids


@pytest.mark.parametrize("kind", ["any", "runs", "one"])
@pytest.mark.parametrize("M,N,K,r,n,per_mille,kernel", SHAPES)
def test_parity(gpu_lib, M, N, K, r, n, per_mille, kernel, kind):
    import torch
    say(f"[adapters] M={M} N={N} K={K} r={r} n={n} sparse={per_mille} kernel={kernel} rows={kind}")
    L = layer(M + N + K, N, K, per_mille)
    rng = np.random.default_rng(M + r)
    x = workloads.random_x(M + 3 * r, M, K)
    L1, L2 = factors(M + r, n, r, N, K)
    ids, scale = _rows(rng, M, n, kind), rng.uniform(0.25, 2.0, n).astype(np.float32)
    y = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel=kernel)
    ref, bound = oracle.rows.linear_adapters(x, L["held"], L1, L2, ids, scale, rounded_weights=True)
    err = worst(y, ref, bound)
    say(f"    {err:.3f} of the bound")
    assert err <= 1.0
    y32 = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel=kernel, out_dtype=torch.float32)
    assert worst(y32, ref, bound, f16=False) <= 1.0
    assert torch.equal(y32.half(), y)


@pytest.mark.parametrize("M,N,K,r,n,kernel", [(1, 96, 512, 8, 2, "auto"), (7, 80, 1024, 24, 5, "auto"),
                                              (16, 64, 2048, 16, 20, "auto"), (60, 288, 1024, 32, 7, "gemm"),
                                              (150, 256, 1024, 40, 9, "gemm"), (90, 96, 384, 8, 90, "gemm"),
                                              (90, 96, 2048, 8, 90, "auto")])
def test_integers_are_exact(gpu_lib, M, N, K, r, n, kernel):
    """Integer operands whose every sum float32 holds: fp32 outputs are the oracle's, bit for bit."""
    import torch
    say(f"[adapters exact] M={M} N={N} K={K} r={r} n={n}")
    rng = np.random.default_rng(M * K + r)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    z = rng.integers(0, 16, (N, K // 128)).astype(np.float16)
    s = np.exp2(rng.integers(-1, 2, (N, K // 128))).astype(np.float16)
    L = dict(q=q, s=s, z=z, packed=oracle.pack(q), row_ptr=np.zeros(N + 1, np.int32), col=np.zeros(1, np.int32),
             val=np.zeros(1, np.float16), nnz=0)
    x = rng.integers(-2, 3, (M, K)).astype(np.float16)
    L1 = np.where(rng.random((n, r, K)) < 0.1, rng.integers(-2, 3, (n, r, K)), 0).astype(np.float16)
    L2 = rng.integers(-4, 5, (n, N, r)).astype(np.float16)
    ids, scale = rng.integers(-1, n, M), np.exp2(rng.integers(-1, 2, n)).astype(np.float32)
    ref, _ = oracle.rows.linear_adapters(x, oracle.dequant(q, s, z), L1, L2, ids, scale)
    y = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel=kernel, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), ref)


@pytest.mark.parametrize("M,kernel", [(1, "gemv_mfma"), (2, "gemv_mfma"), (16, "gemv_mfma"), (90, "gemv_mfma"),
                                      (48, "gemm"), (64, "gemm"), (90, "gemm"), (300, "gemm")])
def test_no_adapter_is_the_plain_product(gpu_lib, M, kernel):
    """Rows outside [0, n), of any value: the plain product's bits."""
    import torch
    N, K, n, r = 300, 1024, 3, 16
    L = layer(5, N, K, 4)
    x = workloads.random_x(M, M, K)
    L1, L2 = factors(1, n, r, N, K)
    D = layer_to_dev(L, torch)
    plain = gpu_lib.linear_sparse(to_dev(x, torch), D["packed"], D["scales"], D["zeros"], D["row_ptr"], D["col"],
                                  D["val"], kernel=kernel)
    out = np.resize(np.array([-1, n, -2 ** 31, 2 ** 31 - 1, 1 << 20], np.int64), M)
    assert torch.equal(run_adapters(gpu_lib, torch, L, x, L1, L2, out, kernel=kernel), plain)


@pytest.mark.parametrize("M,kernel", [(2, "auto"), (16, "auto"), (40, "gemm"), (64, "gemm"), (100, "auto"),
                                      (300, "gemm")])
def test_an_adapters_infinities_stay_its_own(gpu_lib, M, kernel):
    """Infinities and NaN in one adapter's factors, in its scale, or in one row: every other row is as it was."""
    import torch
    N, K, n, r = 300, 1024, 4, 24
    L = layer(6, N, K)
    x = workloads.random_x(M, M, K)
    L1, L2 = factors(2, n, r, N, K)
    ids = np.arange(M) % n
    scale = np.ones(n, np.float32)
    want = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel=kernel)
    bad = ids == 1
    for which in ("L1", "L2", "scale", "x"):
        a1, a2, sc, xx, rows = L1.copy(), L2.copy(), scale.copy(), x.copy(), bad
        if which == "L1":
            a1[1, 3, 5] = np.inf
            a1[1, 4, 6] = np.nan
        elif which == "L2":
            a2[1, :, 2] = np.inf
            a2[1, 7, 3] = np.nan
        elif which == "scale":
            sc[1] = np.nan
        else:
            rows = np.arange(M) == 1
            xx[1, 9] = np.inf
        y = run_adapters(gpu_lib, torch, L, xx, a1, a2, ids, sc, kernel=kernel)
        keep = to_dev(~rows, torch)
        assert torch.equal(y[keep], want[keep]), which
        assert not torch.isfinite(y[~keep].float()).all(), which


@pytest.mark.parametrize("seed", range(16))
def test_drawn_sizes(gpu_lib, seed):
    import torch
    rng = np.random.default_rng(200 + seed)
    M, N = int(np.exp(rng.uniform(0, np.log(600)))), int(np.exp(rng.uniform(0, np.log(1500))))
    K, r, n = 128 * int(rng.integers(1, 34)), 8 * int(rng.integers(1, 33)), int(np.exp(rng.uniform(0, np.log(60))))
    kind, kernel = rng.choice(["any", "runs", "one"]), rng.choice(["auto", "auto", "gemv", "gemm"])
    per_mille = int(rng.choice([0, 0, 4]))
    say(f"[adapters drawn] M={M} N={N} K={K} r={r} n={n} sparse={per_mille} kernel={kernel} rows={kind}")
    L = layer(300 + seed, N, K, per_mille)
    x = workloads.random_x(seed, M, K)
    L1, L2 = factors(seed, n, r, N, K)
    ids, scale = _rows(rng, M, n, kind), rng.uniform(-2.0, 2.0, n).astype(np.float32)
    y = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel=str(kernel))
    ref, bound = oracle.rows.linear_adapters(x, L["held"], L1, L2, ids, scale, rounded_weights=True)
    assert worst(y, ref, bound) <= 1.0
    assert torch.equal(run_adapters(gpu_lib, torch, L, x, L1, L2, ids, scale, kernel=str(kernel)), y)


@pytest.mark.parametrize("M,K", [(3, 512), (40, 1024), (300, 8192), (700, 2048)])
def test_subnormal_inputs_and_factors(gpu_lib, M, K):
    """fp16 values below 2^-14 count as all others do, in x and in L1 (t itself is brought back by the scale)."""
    import torch
    say(f"[adapters subnormal] M={M} K={K}")
    N, n, r = 64, 4, 24
    L = layer(11, N, K)
    rng = np.random.default_rng(M)
    L1, L2 = factors(5, n, r, N, K)
    ids = rng.integers(0, n, M)
    small = np.ldexp(rng.integers(-1023, 1024, (M, K)), -24).astype(np.float16)
    scale = np.full(n, 2.0 ** 14, np.float32)
    for x, a1 in ((small, L1), (workloads.random_x(M, M, K), np.ldexp(rng.integers(-1023, 1024, L1.shape), -24).astype(np.float16))):
        y = run_adapters(gpu_lib, torch, L, x, a1, L2, ids, scale, out_dtype=torch.float32)
        ref, bound = oracle.rows.linear_adapters(x, L["held"], a1, L2, ids, scale, rounded_weights=True)
        assert worst(y, ref, bound, f16=False) <= 1.0


@pytest.mark.parametrize("M,K,kernel", [(1, 512, "auto"), (9, 512, "auto"), (60, 1024, "gemm"), (60, 1024, "gemv"),
                                        (500, 8192, "auto")])
def test_workspaces_of_any_contents(gpu_lib, M, K, kernel):
    """A workspace of NaN gives the same bits, also where rows, or all of them, name no adapter."""
    import torch
    say(f"[adapters workspace] M={M} K={K}")
    N, n, r = 80, 5, 40
    L = layer(13, N, K)
    L1, L2 = factors(8, n, r, N, K)
    x = workloads.random_x(M, M, K)
    for ids in (np.arange(M) % n, np.arange(M) % (n + 2) - 1, np.full(M, -1)):
        want = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, kernel=kernel)
        assert torch.isfinite(want.float()).all()
        ws = torch.full((gpu_lib.linear_adapters_workspace_bytes(M, N, K, r),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(run_adapters(gpu_lib, torch, L, x, L1, L2, ids, kernel=kernel, workspace=ws), want)


def test_outputs_of_any_place(gpu_lib):
    """An output that begins four bytes into its memory, the bytes around it as they were."""
    import torch
    L1, L2 = factors(6, 3, 16, 48, 512)
    L = layer(12, 48, 512)
    for M in (1, 5, 16, 70):
        say(f"[adapters place] M={M}")
        x, ids = workloads.random_x(M, M, 512), np.arange(M) % 4 - 1
        for dtype, lead in ((torch.float32, 1), (torch.float16, 2)):
            want = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, out_dtype=dtype)
            room = torch.full((M * 48 + 2 * lead,), 7.0, dtype=dtype, device="cuda")
            out = room[lead:-lead].view(M, 48)
            run_adapters(gpu_lib, torch, L, x, L1, L2, ids, out_dtype=dtype, out=out)
            assert torch.equal(out, want) and (room[:lead] == 7).all() and (room[-lead:] == 7).all()


@pytest.mark.parametrize("M", [2, 64, 200])
def test_factors_beyond_32_bits(gpu_lib, M):
    """The last adapters of arrays of more than 2^32 bytes (and 2^31 elements)."""
    import torch
    N, K, n, r = 20480, 20480, 1700, 64
    say(f"[adapters far] M={M}")
    x = workloads.random_x(M, M, K)
    far = [0, n // 2, n - 2, n - 1]
    small1, small2 = factors(7, len(far), r, N, K)
    L1 = torch.empty(n, r, K, dtype=torch.float16, device="cuda")
    L2 = torch.empty(n, N, r, dtype=torch.float16, device="cuda")
    assert L1.numel() > 2 ** 31 and L2.numel() > 2 ** 31
    small1, small2 = to_dev(small1, torch), to_dev(small2, torch)
    for i, a in enumerate(far):
        L1[a], L2[a] = small1[i], small2[i]
    which = torch.arange(M, device="cuda") % len(far)
    packed = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")  # codes 0 of zero-point 0: no weights
    s = torch.ones(N, K // 128, dtype=torch.float16, device="cuda")
    xd = to_dev(x, torch)
    args = xd, packed, s, torch.zeros_like(s)
    y = gpu_lib.linear_adapters(*args, L1, L2, torch.tensor(far, device="cuda")[which].int())
    assert torch.equal(y, gpu_lib.linear_adapters(*args, small1, small2, which.int()))
    assert torch.isfinite(y.float()).all() and y.any(1).all()


def test_rows_do_not_depend_on_their_neighbours_or_order(gpu_lib):
    """A permuted batch gives the permuted rows, whichever adapters then share a tile."""
    import torch
    M, N, K, n, r = 48, 300, 1024, 9, 16
    L = layer(7, N, K)
    x = workloads.random_x(3, M, K)
    L1, L2 = factors(3, n, r, N, K)
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, n, M)
    p = rng.permutation(M)
    y = run_adapters(gpu_lib, torch, L, x, L1, L2, ids, kernel="gemv")
    assert torch.equal(run_adapters(gpu_lib, torch, L, x[p], L1, L2, ids[p], kernel="gemv"), y[to_dev(p, torch)])


def test_graph_streams_and_given_tensors(gpu_lib):
    """Captured once and replayed with other rows, adapters and inputs in place, eager work between; two streams at
    once with workspaces of their own; an output given; an empty batch."""
    import torch
    M, N, K, n, r = 16, 520, 2048, 6, 16
    L = layer(8, N, K)
    D = layer_to_dev(L, torch)
    L1, L2 = (to_dev(v, torch) for v in factors(4, n, r, N, K))
    x = torch.empty(M, K, dtype=torch.float16, device="cuda")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, dtype=torch.float16, device="cuda")
    nbytes = gpu_lib.linear_adapters_workspace_bytes(M, N, K, r)
    ws = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def call(out, w):
        return gpu_lib.linear_adapters(x, D["packed"], D["scales"], D["zeros"], L1, L2, ids, out=out, workspace=w)

    x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, ws[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert call(out, ws[0]) is out
    rng = np.random.default_rng(1)
    for i in range(4):
        x.copy_(to_dev(workloads.random_x(i, M, K), torch))
        ids.copy_(to_dev(rng.integers(-1, n, M).astype(np.int32), torch))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, call(None, None)), i
    other = torch.empty_like(out)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(other, ws[1])
    call(out, ws[0])
    torch.cuda.synchronize()
    assert torch.equal(out, got) and torch.equal(other, got)
    empty = gpu_lib.linear_adapters(x[:0], D["packed"], D["scales"], D["zeros"], L1, L2, ids[:0])
    assert tuple(empty.shape) == (0, N)


def test_refusals(gpu_lib):
    import torch
    M, N, K, n, r = 2, 64, 256, 3, 16
    L = layer(9, N, K)
    D = layer_to_dev(L, torch)
    L1, L2 = (to_dev(v, torch) for v in factors(4, n, r, N, K))
    x, ids = to_dev(workloads.random_x(0, M, K), torch), torch.zeros(M, dtype=torch.int32, device="cuda")

    def call(x=x, L1=L1, L2=L2, ids=ids, **kw):
        return gpu_lib.linear_adapters(x, D["packed"], D["scales"], D["zeros"], L1, L2, ids, **kw)

    for bad in (dict(ids=ids.long()), dict(L1=L1.float()), dict(ids=ids.cpu()), dict(out_dtype=torch.bfloat16),
                dict(adapter_scale=torch.ones(n, dtype=torch.float64, device="cuda")),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(ids=ids[:1]), dict(L1=L1[:2].contiguous()), dict(L2=L2[:, :, :8].contiguous()), dict(L1=L1[0]),
                dict(adapter_scale=torch.ones(n + 1, device="cuda")), dict(x=x[:, ::2]),
                dict(out=torch.empty(M, N + 1, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(gpu_lib.WQError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gpu_lib.WQError):  # rank 12
        call(L1=L1[:, :12].contiguous(), L2=L2[:, :, :12].contiguous())
