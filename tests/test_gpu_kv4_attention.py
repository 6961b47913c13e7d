"""Attention over the 4-bit cache against the float64 oracle on the values the cache
holds, with bounds derived in kv4_cases."""
import numpy as np
import pytest

import oracle
from gpu_cases import say, to_dev
from kv4_cases import Batch, check, out_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (8, 2), (7, 1), (16, 1), (12, 4), (40, 1)])
def test_single_tokens(gpu_lib, hq, hkv, d):
    """One new token a sequence, every length around a tile's and a page's end."""
    import torch
    ctx = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]
    say(f"[kv4 decode] hq={hq} hkv={hkv} d={d}")
    b = Batch(gpu_lib, torch, [1] * len(ctx), ctx, hq, hkv, d, 64, seed=hq + d).fill()
    check(*b.attention(), b.reference())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,ctx,hq,hkv,page", [
    ([2, 3, 5], [2, 40, 333], 8, 2, 32),           # a few rows: one column tile of 16 or 20
    ([4, 1, 7], [4, 70, 90], 16, 2, 64),           # up to 56 rows: both kernels
    ([33], [33], 4, 1, 32),                        # 132 rows: two row tiles of the last kernel
    ([64, 64], [64, 200], 4, 4, 96),
    ([130, 1, 0, 17], [300, 400, 0, 17], 8, 2, 64),
    ([257], [1000], 6, 2, 128),
    ([1, 1, 200, 1], [1, 900, 200, 33], 28, 4, 64),
])
def test_several_tokens(gpu_lib, new, ctx, hq, hkv, page, d):
    import torch
    say(f"[kv4 chunks] new={new} ctx={ctx} hq={hq} hkv={hkv} page={page} d={d}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, page, seed=sum(ctx) + d).fill()
    check(*b.attention(), b.reference())


@pytest.mark.parametrize("new,ctx,hq,hkv,d,window,page", [
    ([500], [500], 32, 4, 64, 0, 64),                        # whole row tiles
    ([500, 333], [500, 1000], 16, 2, 128, 0, 32),
    ([300], [3000], 16, 2, 128, 0, 64),                      # shares of them, joined
    ([200] * 12, [2400] * 6 + [200, 1111, 2399, 201, 999, 31], 10, 2, 64, 0, 96),
    ([65], [20000], 16, 1, 128, 0, 64),                      # many shares of one
    ([130], [72000], 16, 1, 64, 0, 128),
    ([500, 1, 40, 1, 0], [3000, 2500, 100, 1, 70], 16, 2, 128, 0, 64),   # single tokens beside them
    ([600], [1500], 16, 2, 128, 500, 32),                    # windows
    ([700, 600], [300, 2000], 16, 2, 128, 0, 64),            # leading rows that see nothing
    ([700, 600], [300, 2000], 16, 2, 128, 70, 64),
    ([160] * 80, list(range(160, 240)), 7, 1, 64, 0, 32),    # more than 64 sequences
])
def test_many_rows(gpu_lib, new, ctx, hq, hkv, d, window, page):
    import torch
    say(f"[kv4 many rows] new={new} ctx={ctx} hq={hq} hkv={hkv} d={d} window={window} page={page}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, page, seed=sum(ctx) + d).fill()
    check(*b.attention(window=window), b.reference(window=window))


@pytest.mark.parametrize("hint", [20, 600])
@pytest.mark.parametrize("B,hkv", [(3, 4), (100, 1), (150, 2)])
def test_less_work_than_blocks(gpu_lib, B, hkv, hint):
    """Batches small enough for one item a block, also of more than 64 sequences, some of
    them idle or empty, with the lengths within the bounds given and beyond them."""
    import torch
    rng = np.random.default_rng(B)
    new = rng.integers(0, 6, B).tolist()
    ctx = [int(n + rng.integers(0, 600 - n)) if n else int(rng.integers(0, 300)) for n in new]
    new[1], ctx[1], new[2], ctx[2] = 3, 2, 5, 599
    say(f"[kv4 small batch] B={B} hkv={hkv} max_ctx={hint}")
    b = Batch(gpu_lib, torch, new, ctx, 7 * hkv, hkv, 64, 32, seed=B).fill()
    check(*b.attention(max_ctx=hint), b.reference())


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 10000])
@pytest.mark.parametrize("new,ctx,hq,hkv", [([1, 1, 1], [1, 95, 400], 4, 2), ([5, 3], [77, 300], 6, 2),
                                            ([90, 1], [250, 120], 4, 1)])
def test_window(gpu_lib, window, new, ctx, hq, hkv):
    """A sliding window, with the page of what it has passed given to somebody else: its
    entries name pages of NaN, and whatever stands there may not be noticed."""
    import torch
    say(f"[kv4 window] {window} new={new} ctx={ctx}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, 128, 32, seed=window).fill()
    ref = b.reference(window=window)
    free = (set(range(b.num_pages)) - set(b.table.cpu().numpy().ravel().tolist())).pop()
    table = b.table.cpu().numpy().copy()
    for i, (n, c) in enumerate(zip(new, ctx)):
        passed = max(0, c - n - window + 1) // 32
        table[i, :passed] = free
    b.table = to_dev(table, torch)
    check(*b.attention(window=window), ref)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(gpu_lib, d):
    """Padded slots (a row, no token), sequences of no rows, more rows than tokens: rows of
    0 with -infinity, in every kernel and split."""
    import torch
    for new, ctx in (([1, 1, 1], [0, 5, 0]), ([1], [0]), ([0, 0, 1], [0, 9, 3]), ([40, 3], [7, 1]),
                     ([100, 1, 100], [0, 0, 60])):
        say(f"[kv4 empty rows] new={new} ctx={ctx} d={d}")
        b = Batch(gpu_lib, torch, new, ctx, 4, 2, d, 32, seed=1).fill()
        check(*b.attention(), b.reference())
        check(*b.attention(max_ctx=5000), b.reference())


@pytest.mark.parametrize("hint_q,hint_ctx", [(0, 0), (1, 1), (1, 100000), (1000, 40), (None, None), (60, 2500)])
@pytest.mark.parametrize("new,ctx,hq,hkv", [([1, 1, 1], [2300, 1, 77], 8, 2), ([60, 1, 9], [2500, 900, 9], 8, 2),
                                            ([300, 1, 9], [1500, 900, 9], 16, 2)])
def test_hints_only_shape_the_launch(gpu_lib, hint_q, hint_ctx, new, ctx, hq, hkv):
    """max_q and max_ctx far too small and far too large: other splits, the same rows."""
    import torch
    say(f"[kv4 hints] max_q={hint_q} max_ctx={hint_ctx} new={new}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, 128, 64, seed=3).fill()
    check(*b.attention(max_q=hint_q, max_ctx=hint_ctx), b.reference())


@pytest.mark.parametrize("new,ctx,hq,hkv,d", [([1], [20000], 8, 2, 128), ([1, 1], [9000, 40], 32, 1, 64),
                                              ([20], [6000], 16, 2, 128), ([300], [5000], 4, 1, 64)])
def test_long_sequences_are_split(gpu_lib, new, ctx, hq, hkv, d):
    import torch
    say(f"[kv4 long] new={new} ctx={ctx} hq={hq} d={d}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 128, seed=8).fill()
    assert gpu_lib.kv4_attention_workspace_bytes(sum(new), len(new), hq, hkv, d, max(new), max(ctx)) > 0
    check(*b.attention(), b.reference())


@pytest.mark.parametrize("new,ctx", [([1, 1], [700, 2100]), ([50], [1200]), ([1900], [1900])])
def test_values_and_scores_of_all_sizes(gpu_lib, new, ctx):
    """Value scales that grow along the sequence from 2^-13 to 2^11, and from large to small;
    scores that rise and fall by hundreds: the running reference moves, and moves back
    nothing."""
    import torch
    hq, hkv, d = 4, 2, 128
    L = sum(ctx)
    rng = np.random.default_rng(11)
    ramp = 2.0 ** np.linspace(-11, 13, L)[:, None, None]
    base = rng.standard_normal((L, hkv, d))
    rise = np.linspace(0.1, 30, L)[:, None, None]
    for name, k, v in (("growing values", base, base * ramp), ("falling values", base, base * ramp[::-1]),
                       ("rising scores", base * rise, base), ("falling scores", base * rise[::-1], base),
                       ("both", base * rise, base * ramp[::-1]), ("tiny values", base, base * 1e-4),
                       ("huge values", base, np.clip(base * 2e4, -65504, 65504))):
        b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 64, seed=12, k=k.astype(np.float16),
                  v=v.astype(np.float16)).fill()
        say(f"[kv4 ranges] {name} new={new}")
        check(*b.attention(), b.reference(), name)


def test_one_token_takes_all(gpu_lib):
    """A key far ahead of the others: its held value comes back, to the rounding of its
    weight times its value scale (2^-11) and of the output (2^-11)."""
    import torch
    d, ctx = 128, 200
    rng = np.random.default_rng(4)
    k = (0.01 * rng.standard_normal((ctx, 1, d))).astype(np.float16)
    q = rng.standard_normal((1, 1, d)).astype(np.float16)
    k[77] = 20 * q[0]
    b = Batch(gpu_lib, torch, [1], [ctx], 1, 1, d, 32, k=k, q=q, seed=4).fill()
    out, lse = b.attention()
    held = oracle.kv4_values(b.v[77:78])[0]
    assert np.all(np.abs(out.cpu().numpy()[0] - held) <= 2.0 ** -10 * np.abs(held))


def test_equal_scores_average(gpu_lib):
    """A zero query weighs all tokens alike: the mean of the held values, and log(ctx)."""
    import torch
    for new, ctx in ((1, 1000), (70, 300)):
        b = Batch(gpu_lib, torch, [new], [ctx], 2, 1, 64, 64, seed=6, q=np.zeros((new, 2, 64), np.float16)).fill()
        out, lse = b.attention()
        check(out, lse, b.reference())
        assert abs(float(lse[-1, 0]) - np.log(ctx)) < 1e-5


def test_scale_slices_and_out(gpu_lib):
    """Another scale, queries as a slice of a wider projection, an output given."""
    import torch
    d, hq, hkv = 64, 6, 3
    b = Batch(gpu_lib, torch, [5, 1, 50], [50, 300, 60], hq, hkv, d, 32, seed=7).fill()
    wide = torch.randn(56, (hq + 2 * hkv) * d, device="cuda").half()
    wide[:, :hq * d] = to_dev(b.q.reshape(56, -1), torch)
    q = wide[:, :hq * d].unflatten(1, (hq, d))
    assert not q.is_contiguous()
    for scale in (0.02, 1.0):
        out = torch.empty(56, hq, d, device="cuda", dtype=torch.float16)
        got, lse = b.attention(q=q, scale=scale, out=out)
        assert got is out
        check(got, lse, b.reference(scale=scale), f"scale {scale}")


def test_chunks_join_by_lse(gpu_lib):
    """Two halves of a sequence's tokens, attended to apart by queries that see all of each,
    joined by their log sums: the whole."""
    import torch
    d, hq, hkv = 128, 4, 2
    b = Batch(gpu_lib, torch, [1], [600], hq, hkv, d, 64, seed=13).fill()
    out, lse = b.attention()
    first = Batch(gpu_lib, torch, [1], [256], hq, hkv, d, 64, seed=1, k=b.k[:256], v=b.v[:256], q=b.q).fill()
    second = Batch(gpu_lib, torch, [1], [344], hq, hkv, d, 64, seed=2, k=b.k[256:], v=b.v[256:], q=b.q).fill()
    (o1, l1), (o2, l2) = first.attention(), second.attention()
    w = torch.softmax(torch.stack((l1, l2)).double(), 0)[..., None]
    whole = w[0] * o1.double() + w[1] * o2.double()
    assert float((whole - out.double()).abs().max()) < 2e-3
    assert float((torch.logaddexp(l1, l2) - lse).abs().max()) < 1e-4


def test_deterministic_and_other_streams(gpu_lib):
    import torch
    b = Batch(gpu_lib, torch, [1, 60, 3], [3000, 700, 90], 8, 2, 128, 64, seed=14).fill()
    say("[kv4 streams]")
    out, lse = b.attention()
    q = to_dev(b.q, torch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, lse2 = b.wq.kv4_attention(q, b.cache, b.table, b.seq_start, b.ctx_len, max_q=60, max_ctx=3000,
                                         return_lse=True)
    side.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_graph_of_a_decode_step(gpu_lib):
    """Append and attention captured once and replayed as the sequences grow (lengths and
    inputs in place): every replay equals the eager call and the oracle."""
    import torch
    hq, hkv, d, steps = 8, 2, 128, 5
    start = [30, 63, 200]
    ctx = [c + steps for c in start]
    b = Batch(gpu_lib, torch, [1] * 3, ctx, hq, hkv, d, 32, seed=15).fill(start)
    k, v = torch.empty(3, hkv, d, device="cuda", dtype=torch.float16), None
    v = torch.empty_like(k)
    q = torch.empty(3, hq, d, device="cuda", dtype=torch.float16)
    out = torch.empty_like(q)
    ws = torch.empty(max(gpu_lib.kv4_attention_workspace_bytes(3, 3, hq, hkv, d, 1, 600), 1), dtype=torch.uint8,
                     device="cuda")
    lens = to_dev(np.array(start, np.int32), torch)

    def step():
        lens.add_(1)
        gpu_lib.kv4_append(k, v, b.cache, b.table, b.seq_start, lens, max_new=1)
        gpu_lib.kv4_attention(q, b.cache, b.table, b.seq_start, lens, max_q=1, max_ctx=600, out=out, workspace=ws)

    qs = np.random.default_rng(16).standard_normal((steps, 3, hq, d)).astype(np.float16)
    say("[kv4 graph]")
    graph = torch.cuda.CUDAGraph()
    k.zero_(), v.zero_(), q.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warm-up outside the graph; its token is overwritten by the first replay
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    lens.copy_(to_dev(np.array(start, np.int32), torch))
    for i in range(steps):
        rows = [b.begin[s] + start[s] + i for s in range(3)]
        k.copy_(to_dev(b.k[rows], torch))
        v.copy_(to_dev(b.v[rows], torch))
        q.copy_(to_dev(qs[i], torch))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = gpu_lib.kv4_attention(q, b.cache, b.table, b.seq_start, lens, max_q=1, max_ctx=600)
        torch.cuda.synchronize()
        assert torch.equal(got, eager), i
        for s in range(3):
            n = start[s] + i + 1
            kk, vv = (oracle.kv4_values(x[b.begin[s]:b.begin[s] + n]) for x in (b.k, b.v))
            o, _, spread = oracle.kv4_attention(qs[i, s:s + 1], kk, vv)
            assert out_error(got[s:s + 1], o, spread) <= 1.0
