"""Expert routing and the mixture-of-experts layer against the float64 oracle, with bounds that count the kernels'
roundings (oracle/rows.py)."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import layer_to_dev, say, to_dev
from rows_cases import Moe, factors, layer, worst

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ route
def _route(wq, torch, logits, k, renormalize):
    e, w = wq.moe_route(to_dev(logits, torch), k, renormalize=renormalize)
    torch.cuda.synchronize()
    return e.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def _check_route(got, logits, k, renormalize):
    """Experts exactly; a weight is an exponential (its argument's rounding, 2^-24 of it, and two of its own), a sum of E
    such and a quotient."""
    experts, weights = oracle.rows.moe_route(logits, k, renormalize)
    assert np.array_equal(got[0], experts)
    x = np.asarray(logits, np.float64)
    spread = np.where(np.isfinite(x), x, 0.0)
    spread = spread.max(1, keepdims=True) - spread.min(1, keepdims=True)
    bound = weights * 2.0 ** -24 * (2 * spread + x.shape[1] + 8) + 2.0 ** -126
    same = np.isnan(weights)
    assert np.array_equal(same, np.isnan(got[1]))
    assert np.all(np.abs(got[1] - weights)[~same] <= bound[~same])


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (5, 63, 8), (64, 64, 6), (7, 65, 16), (33, 128, 8),
                                   (9, 160, 6), (4, 256, 8), (5, 257, 4), (3, 512, 16), (2, 1000, 16), (1, 1024, 1)])
def test_route(gpu_lib, M, E, k, renormalize, dtype):
    import torch
    say(f"[route] M={M} E={E} k={k} renormalize={renormalize} {dtype.__name__}")
    rng = np.random.default_rng(M * E + k)
    logits = (2 * rng.standard_normal((M, E))).astype(dtype)
    _check_route(_route(gpu_lib, torch, logits, k, renormalize), logits, k, renormalize)


@pytest.mark.parametrize("E", [5, 64, 100, 300])
def test_route_ties_masks_and_extremes(gpu_lib, E):
    import torch
    rng = np.random.default_rng(E)
    k = min(E, 8)
    top = np.finfo(np.float32).max
    rows = [np.zeros(E), np.full(E, -np.inf), rng.integers(-1, 2, E), np.where(rng.random(E) < 0.5, -0.0, 0.0),
            np.where(np.arange(E) == E - 1, 3.0, -np.inf), np.where(rng.random(E) < 0.9, -np.inf, 1.0),
            np.full(E, -top), np.where(np.arange(E) == 2, -top, -np.inf), np.full(E, top),
            np.where(np.arange(E) % 2, -1e4, 1e4), 1e30 * rng.standard_normal(E)]
    logits = np.array(rows, np.float32)
    for renormalize in (True, False):
        say(f"[route extremes] E={E} renormalize={renormalize}")
        _check_route(_route(gpu_lib, torch, logits, k, renormalize), logits, k, renormalize)
    # NaN is the largest and makes its row's weights NaN; infinities as the formula has them
    odd = rng.standard_normal((3, E)).astype(np.float32)
    odd[0, 3] = np.nan
    odd[1, [1, 4]] = np.inf
    odd[2, 0] = np.inf
    e, w = _route(gpu_lib, torch, odd, k, True)
    assert e[0, 0] == 3 and np.isnan(w[0]).all()
    assert e[1, :2].tolist() == [1, 4] and np.isnan(w[1]).all()
    assert e[2, 0] == 0 and np.isnan(w[2]).all()


# ------------------------------------------------------------------ experts
def _pick(rng, M, E, k, none=0.1, spread=True):
    """Distinct experts of each row, some slots empty; spread = False: the same few for all rows."""
    e = np.array([rng.permutation(E if spread else min(E, k + 1))[:k] for _ in range(M)]).reshape(M, k)
    e[rng.random((M, k)) < none] = -1
    return e.astype(np.int32), rng.uniform(0.05, 1.0, (M, k)).astype(np.float32)


@pytest.mark.parametrize("spread", [True, False])
@pytest.mark.parametrize("M,H,I,E,k", [
    (1, 128, 128, 1, 1), (1, 256, 384, 8, 2), (2, 512, 128, 3, 3), (5, 384, 640, 10, 4), (16, 256, 256, 4, 2),
    (17, 128, 256, 2, 2), (40, 384, 128, 6, 3), (64, 256, 256, 16, 6), (65, 256, 128, 5, 2), (130, 128, 384, 30, 8),
    (3, 2176, 128, 4, 2), (4, 128, 2176, 5, 2), (33, 1024, 1024, 7, 2),
])
def test_experts(gpu_lib, M, H, I, E, k, spread):
    import torch
    say(f"[experts] M={M} H={H} I={I} E={E} k={k} spread={spread}")
    rng = np.random.default_rng(M * H + I)
    moe = Moe(torch, H + I, H, I, E)
    x = workloads.random_x(M, M, H)
    e, w = _pick(rng, M, E, k, spread=spread)
    ref, bound = moe.reference(x, e, w)
    y = moe.run(gpu_lib, torch, x, e, w)
    err = worst(y, ref, bound)
    say(f"    {err:.3f} of the bound")
    assert err <= 1.0
    y32 = moe.run(gpu_lib, torch, x, e, w, out_dtype=torch.float32)
    assert worst(y32, ref, bound, f16=False) <= 1.0
    assert torch.equal(y32.half(), y)


def test_rows_stand_alone(gpu_lib):
    """The same bits run after run; a row alone, in a larger batch or in another order is right, and has the same bits
    whatever its neighbours hold; rows and slots of no expert give zeros."""
    import torch
    say("[experts rows]")
    M, H, I, E, k = 70, 256, 384, 6, 3
    rng = np.random.default_rng(5)
    moe = Moe(torch, 9, H, I, E)
    x = workloads.random_x(4, M, H)
    e, w = _pick(rng, M, E, k)
    e[11] = -1
    e[12] = [E, 2 ** 31 - 1, -2 ** 31]
    ref, bound = moe.reference(x, e, w)
    y = moe.run(gpu_lib, torch, x, e, w)
    assert not y[11].any() and not y[12].any()
    for _ in range(5):
        assert torch.equal(moe.run(gpu_lib, torch, x, e, w), y)
    p = rng.permutation(M)
    assert worst(moe.run(gpu_lib, torch, x[p], e[p], w[p]), ref[p], bound[p]) <= 1.0
    for m in (0, 63, 64, 69):
        one = slice(m, m + 1)
        assert worst(moe.run(gpu_lib, torch, x[one], e[one], w[one]), ref[one], bound[one]) <= 1.0
    x[7, 3], w[8, 1], e[8, 1] = np.inf, np.nan, 2
    y = moe.run(gpu_lib, torch, workloads.random_x(4, M, H), e, np.where(np.isnan(w), 1, w))
    got = moe.run(gpu_lib, torch, x, e, w)
    rest = [m for m in range(M) if m not in (7, 8)]
    assert torch.equal(got[rest], y[rest])
    assert not torch.isfinite(got[8].float()).any()


def test_an_expert_named_twice(gpu_lib):
    """Its weights add up."""
    import torch
    say("[experts twice]")
    H, I, E = 256, 128, 3
    moe = Moe(torch, 3, H, I, E)
    x = workloads.random_x(1, 4, H)
    e = np.array([[1, 1, 1], [0, 2, 0], [2, -1, 2], [1, 0, 2]])
    w = np.array([[0.5, 0.25, 0.125], [0.5, 0.25, 1.0], [1.0, 9.0, 0.5], [0.1, 0.2, 0.3]])
    ref, bound = moe.reference(x, e, w)
    assert worst(moe.run(gpu_lib, torch, x, e, w), ref, bound) <= 1.0


def test_gates_of_all_sizes(gpu_lib):
    """Gates far below and above zero: silu ends in 0 and in the gate itself."""
    import torch
    say("[experts gates]")
    H, I, E, M = 128, 256, 2, 6
    moe = Moe(torch, 4, H, I, E)
    rng = np.random.default_rng(0)
    x = workloads.random_x(2, M, H) * np.array([1e-4, 0.1, 1, 10, 30, 60], np.float16)[:, None]
    e, w = _pick(rng, M, E, 2, none=0.0)
    ref, bound = moe.reference(x, e, w)
    assert worst(moe.run(gpu_lib, torch, x, e, w, out_dtype=torch.float32), ref, bound, f16=False) <= 1.0


def test_large_batches_of_small_layers(gpu_lib):
    """Many blocks of 64 rows, all slots of the lists in use, many experts."""
    import torch
    say("[experts many]")
    H, I, E, k, M = 128, 128, 40, 16, 200
    moe = Moe(torch, 5, H, I, E)
    rng = np.random.default_rng(1)
    x = workloads.random_x(2, M, H)
    e, w = _pick(rng, M, E, k, none=0.0)
    ref, bound = moe.reference(x, e, w)
    assert worst(moe.run(gpu_lib, torch, x, e, w), ref, bound) <= 1.0


@pytest.mark.parametrize("M", [2, 9, 60, 200])
def test_weights_beyond_32_bits(gpu_lib, M):
    """The last experts of arrays of more than 2^32 bytes, in turn with the first: the bits of a layer of just those."""
    import torch
    say(f"[experts far] M={M}")
    H, I, E, k = 4096, 2048, 1024, 2
    moe = Moe(torch, 8, 256, 128, 4)  # (of this size: its words fill the large arrays' rows again and again)
    far = torch.tensor([0, E // 2, E - 2, E - 1], device="cuda")
    big, small = [], []
    for i, shape in enumerate([(E, 2 * I, H // 8), (E, 2 * I, H // 128), (E, 2 * I, H // 128),
                               (E, H, I // 8), (E, H, I // 128), (E, H, I // 128)]):
        src = moe.args[i].flatten()
        t = torch.empty(shape, dtype=src.dtype, device="cuda")
        n = t[0].numel()
        own = torch.stack([src.roll(j).repeat(-(-n // src.numel()))[:n].view(shape[1:]) for j in range(4)])
        for j in range(4):
            t[far[j].item()] = own[j]
        big.append(t)
        small.append(own)
    assert big[0].numel() * 4 > 2 ** 32 and big[3].numel() * 4 >= 2 ** 32
    rng = np.random.default_rng(M)
    x = to_dev((workloads.random_x(M, M, H).astype(np.float32) / 64).astype(np.float16), torch)
    e, w = _pick(rng, M, 4, k, none=0.0)
    w = to_dev(w, torch)
    want = gpu_lib.moe_experts(x, to_dev(e, torch), w, *small)
    got = gpu_lib.moe_experts(x, to_dev(far.cpu().numpy().astype(np.int32)[e], torch), w, *big)
    assert torch.isfinite(want.float()).all() and want.any(1).all()
    assert torch.equal(got, want)


def test_subnormal_inputs(gpu_lib):
    """fp16 values below 2^-14 in x count as all others do, and the inner activations of such sizes keep theirs."""
    import torch
    H, I, E, k = 256, 128, 3, 2
    moe = Moe(torch, 10, H, I, E)
    rng = np.random.default_rng(2)
    for M in (2, 12, 60):
        say(f"[experts subnormal] M={M}")
        x = np.ldexp(rng.integers(-1023, 1024, (M, H)), -24).astype(np.float16)
        x[M // 2:] = np.ldexp(rng.integers(-1023, 1024, (M - M // 2, H)), -18).astype(np.float16)
        e, w = _pick(rng, M, E, k, none=0.0)
        ref, bound = moe.reference(x, e, w)
        assert worst(moe.run(gpu_lib, torch, x, e, w, out_dtype=torch.float32), ref, bound, f16=False) <= 1.0


def test_outputs_of_any_place(gpu_lib):
    """An output that begins four bytes into its memory, the bytes around it as they were."""
    import torch
    H, I, E, k = 384, 128, 5, 2
    moe = Moe(torch, 11, H, I, E)
    rng = np.random.default_rng(3)
    for M in (1, 4, 5, 33):
        say(f"[experts place] M={M}")
        x = workloads.random_x(M, M, H)
        e, w = _pick(rng, M, E, k)
        for dtype, lead in ((torch.float32, 1), (torch.float16, 2)):
            want = moe.run(gpu_lib, torch, x, e, w, out_dtype=dtype)
            room = torch.full((M * H + 2 * lead,), 7.0, dtype=dtype, device="cuda")
            out = room[lead:-lead].view(M, H)
            moe.run(gpu_lib, torch, x, e, w, out_dtype=dtype, out=out)
            assert torch.equal(out, want) and (room[:lead] == 7).all() and (room[-lead:] == 7).all()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_sizes(gpu_lib, seed):
    """Rows up to three blocks of the lists, experts that many rows name and that none does."""
    import torch
    rng = np.random.default_rng(100 + seed)
    H, I = (128 * int(rng.integers(1, 6)) for _ in range(2))
    E, k = int(rng.integers(1, 25)), int(rng.integers(1, 9))
    k = min(k, E)
    M = int(np.exp(rng.uniform(0, np.log(500))))
    say(f"[experts drawn] M={M} H={H} I={I} E={E} k={k}")
    moe = Moe(torch, 30 + seed, H, I, E)
    x = workloads.random_x(seed, M, H)
    p = rng.dirichlet(np.full(E, 0.5)) + 1e-3
    e = np.array([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(M)]).reshape(M, k)
    e[rng.random((M, k)) < 0.05] = -1
    w = rng.uniform(-1, 1, (M, k)).astype(np.float32)
    ref, bound = moe.reference(x, e, w)
    y = moe.run(gpu_lib, torch, x, e, w)
    assert worst(y, ref, bound) <= 1.0
    assert torch.equal(moe.run(gpu_lib, torch, x, e, w), y)


@pytest.mark.parametrize("M", [1, 4, 7, 70, 250])
def test_workspaces_of_any_contents(gpu_lib, M):
    """A workspace of NaN gives the same bits, also where rows, or all of them, name no expert."""
    import torch
    say(f"[experts workspace] M={M}")
    H, I, E, k = 256, 128, 7, 3
    moe = Moe(torch, 14, H, I, E)
    rng = np.random.default_rng(M)
    x = workloads.random_x(M, M, H)
    for none in (0.0, 0.7, 1.0):
        e, w = _pick(rng, M, E, k, none=none)
        want = moe.run(gpu_lib, torch, x, e, w)
        ref, bound = moe.reference(x, e, w)
        assert worst(want, ref, bound) <= 1.0
        ws = torch.full((gpu_lib.moe_experts_workspace_bytes(M, H, I, k),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(moe.run(gpu_lib, torch, x, e, w, workspace=ws), want)
        assert none < 1.0 or not want.any()


def test_layer_from_logits_in_a_graph(gpu_lib):
    """Route and experts captured together and replayed on other inputs, eager work between; two streams at once with
    workspaces of their own."""
    import torch
    say("[experts graph]")
    M, H, I, E, k = 20, 256, 384, 8, 2
    moe = Moe(torch, 6, H, I, E)
    x = torch.zeros(M, H, dtype=torch.float16, device="cuda")
    logits = torch.zeros(M, E, device="cuda")
    out = torch.empty(M, H, dtype=torch.float16, device="cuda")
    ws = [torch.empty(gpu_lib.moe_experts_workspace_bytes(M, H, I, k), dtype=torch.uint8, device="cuda")
          for _ in range(2)]

    def step(out, w):
        experts, weights = gpu_lib.moe_route(logits, k)
        return gpu_lib.moe_experts(x, experts, weights, *moe.args, out=out, workspace=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out, ws[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, ws[0])
    rng = np.random.default_rng(3)
    for i in range(4):
        xs, ls = workloads.random_x(i, M, H), rng.standard_normal((M, E)).astype(np.float32)
        x.copy_(to_dev(xs, torch))
        logits.copy_(to_dev(ls, torch))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step(None, None)), i
        e, w = oracle.rows.moe_route(ls, k)
        ref, bound = moe.reference(xs, e, w)
        # (the weights' own error: 2^-24 (2 x 8 + 8 + 8) of each, see _check_route)
        assert worst(got, ref, bound + 2.0 ** -19 * np.abs(ref)) <= 1.0
    other = torch.empty_like(out)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(other, ws[1])
    step(out, ws[0])
    torch.cuda.synchronize()
    assert torch.equal(out, got) and torch.equal(other, got)


@pytest.mark.parametrize("M", [1, 4, 14, 90])
def test_a_layer_with_adapters_and_experts(gpu_lib, M):
    """A decoder block's second half as it is served: a 4-bit projection with each request's adapter, a router's logits
    by another 4-bit layer, the choice, the experts; each step against the oracle on the step before's outputs, and the
    whole in a graph, replayed on other inputs with eager work between."""
    import torch
    say(f"[block] M={M}")
    K, H, I, E, k, n, r = 512, 256, 384, 16, 4, 5, 16
    proj, router = layer(20, H, K, 4), layer(21, E, H, 0, 0.2)
    P, R = layer_to_dev(proj, torch), layer_to_dev(router, torch)
    moe = Moe(torch, 12, H, I, E)
    L1, L2 = factors(13, n, r, H, K)
    d1, d2 = to_dev(L1, torch), to_dev(L2, torch)
    x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")

    def step():
        h = gpu_lib.linear_adapters(x, P["packed"], P["scales"], P["zeros"], d1, d2, ids, None, P["row_ptr"], P["col"],
                                    P["val"])
        logits = gpu_lib.linear(h, R["packed"], R["scales"], R["zeros"], out_dtype=torch.float32)
        experts, weights = gpu_lib.moe_route(logits, k)
        return h, logits, experts, weights, gpu_lib.moe_experts(h, experts, weights, *moe.args)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    rng = np.random.default_rng(M)
    for i in range(3):
        xs, a = workloads.random_x(i, M, K), rng.integers(-1, n, M)
        x.copy_(to_dev(xs, torch))
        ids.copy_(to_dev(a.astype(np.int32), torch))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(g, t) for g, t in zip(got, step())), i
        h, logits, e, w, y = (t.cpu().numpy() for t in got)
        ref, bound = oracle.rows.linear_adapters(xs, proj["held"], L1, L2, a, rounded_weights=True)
        assert worst(got[0], ref, bound) <= 1.0
        _check_route((e, w.astype(np.float64)), logits, k, True)
        ref, bound = moe.reference(h, e, w)
        assert worst(got[4], ref, bound) <= 1.0


def test_empty_batches_and_refusals(gpu_lib):
    import torch
    H, I, E, k, M = 256, 128, 3, 2, 4
    moe = Moe(torch, 7, H, I, E)
    x = to_dev(workloads.random_x(1, M, H), torch)
    e = torch.zeros(M, k, dtype=torch.int32, device="cuda")
    w = torch.ones(M, k, device="cuda")
    assert tuple(gpu_lib.moe_experts(x[:0], e[:0], w[:0], *moe.args).shape) == (0, H)
    assert tuple(gpu_lib.moe_route(torch.zeros(0, 8, device="cuda"), 2)[0].shape) == (0, 2)

    def call(x=x, e=e, w=w, args=moe.args, **kw):
        return gpu_lib.moe_experts(x, e, w, *args, **kw)

    for bad in (dict(e=e.long()), dict(w=w.half()), dict(x=x.float()), dict(e=e.cpu()),
                dict(args=[moe.args[0].float()] + moe.args[1:]), dict(out_dtype=torch.float64),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(TypeError):
            call(**bad)
    swapped = moe.args[3:] + moe.args[:3]
    for bad in (dict(e=e[:2]), dict(w=w[:, :1].contiguous()), dict(args=swapped), dict(x=x[:, :128].contiguous()),
                dict(args=moe.args[:1] + [moe.args[1][:, :, :1].contiguous()] + moe.args[2:]),
                dict(out=torch.empty(M, I, dtype=torch.float16, device="cuda")), dict(w=w.t().contiguous().t())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(gpu_lib.WQError):
        call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gpu_lib.WQError):
        call(e=e.repeat(1, 9).contiguous(), w=w.repeat(1, 9).contiguous())
    with pytest.raises(TypeError):
        gpu_lib.moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError):
        gpu_lib.moe_route(torch.zeros(2, 8, device="cuda", dtype=torch.float64), 2)
    for E, k in ((8, 0), (8, 9), (1025, 2), (40, 17)):
        with pytest.raises(gpu_lib.WQError):
            gpu_lib.moe_route(torch.zeros(2, E, device="cuda"), k)
