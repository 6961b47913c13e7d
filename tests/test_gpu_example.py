"""The example's attention block: the operators together, prompts first, then single
tokens, eager and in a graph."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
from gpu_cases import say
from kv4_cases import check

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(__file__), os.pardir, "examples", "w4a8kv4_attention.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("w4a8kv4_attention", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _batch(torch, wq, lengths, room, hkv, d, page=32):
    pages = -(-(max(lengths) + room) // page)
    B = len(lengths)
    cache = wq.kv4_cache(B * pages, page, hkv, d)
    cache.fill_(0xFF)  # NaN scales and zero-points wherever no token was written
    table = torch.randperm(B * pages, device="cuda").int().view(B, pages)
    starts = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda")
    return cache, table, starts, torch.tensor(lengths, dtype=torch.int32, device="cuda"), pages * page


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (4, 4, 128)])
def test_block(gpu_lib, example, hq, hkv, d):
    """Each operator's part of the block against the oracle, on the block's own inputs."""
    import torch
    lengths, hidden = [150, 1, 33, 64], 512
    say(f"[block] hq={hq} hkv={hkv} d={d}")
    torch.manual_seed(d)
    block = example.AttentionBlock(hidden, hq, hkv, d)
    cache, table, starts, ctx, room = _batch(torch, gpu_lib, lengths, 0, hkv, d)
    x, res = (torch.randn(sum(lengths), hidden, device="cuda").half() for _ in range(2))
    out, h = block(x, res, cache, table, starts, ctx, max(lengths), max(lengths))
    q, k, v, h2 = block.project(x, res)
    assert torch.equal(h, h2)
    # (the sum is rounded to fp16 once)
    exact = x.double() + res.double()
    assert bool(((h.double() - exact).abs() <= 2.0 ** -11 * exact.abs()).all())
    rk, rv = gpu_lib.kv4_read(cache, table, starts, ctx, tokens=sum(lengths), head_dim=d, max_new=max(lengths))
    kn, vn, qn = k.cpu().numpy(), v.cpu().numpy(), q.cpu().numpy()
    hk, hv = oracle.kv4_values(kn), oracle.kv4_values(vn)
    assert np.array_equal(rk.cpu().numpy(), hk.astype(np.float16))
    assert np.array_equal(rv.cpu().numpy(), hv.astype(np.float16))
    o, lse = gpu_lib.kv4_attention(q, cache, table, starts, ctx, max_q=max(lengths), max_ctx=max(lengths),
                                   return_lse=True)
    at = np.cumsum([0] + lengths)
    refs = [oracle.kv4_attention(qn[a:b], hk[a:b], hv[a:b]) for a, b in zip(at[:-1], at[1:])]
    check(o, lse, tuple(np.concatenate(r) for r in zip(*refs)))
    assert torch.equal(out, gpu_lib.linear(o.view(sum(lengths), -1), *block.o))


def test_decode_graph(gpu_lib, example):
    """Steps replayed from a graph, with eager work between them, equal eager steps bit for
    bit: outputs, and the cache that they leave."""
    import torch
    lengths, hidden, hq, hkv, d = [40, 1, 64, 95], 512, 8, 2, 64
    say("[block graph]")
    torch.manual_seed(1)
    block = example.AttentionBlock(hidden, hq, hkv, d)
    cache, table, starts, ctx, room = _batch(torch, gpu_lib, lengths, 8, hkv, d)
    x, res = (torch.randn(sum(lengths), hidden, device="cuda").half() for _ in range(2))
    out, h = block(x, res, cache, table, starts, ctx, max(lengths), room)
    last = starts[1:].long() - 1
    x, res = out[last].contiguous(), h[last].contiguous()
    one = torch.arange(len(lengths) + 1, dtype=torch.int32, device="cuda")
    first = [t.clone() for t in (x, res, cache, ctx)]

    def step():
        ctx.add_(1)
        out, h = block(x, res, cache, table, one, ctx, 1, room)
        x.copy_(out)
        res.copy_(h)

    eager = []
    for _ in range(5):
        step()
        eager.append((x.clone(), res.clone()))
    left = cache.clone()
    graph, _ = example.captured(step)
    for t, was in zip((x, res, cache, ctx), first):
        t.copy_(was)
    for i in range(5):
        noise = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(noise)
        assert torch.isfinite(x).all()
        assert torch.equal(x, eager[i][0]) and torch.equal(res, eager[i][1]), i
    assert torch.equal(cache, left)


def test_command(gpu_lib, example, capsys, monkeypatch):
    say("[example]")
    monkeypatch.setattr("sys.argv", ["w4a8kv4_attention.py", "--steps", "3"])
    example.main()
    assert "finite: True" in capsys.readouterr().out
