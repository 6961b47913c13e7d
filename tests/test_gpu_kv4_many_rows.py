"""The attention's kernel for many rows where masks, empty rows, strides, scales and streams
are those that the few rows' kernel is tested with. Each test says which kernels its batch
must take, so that a change of the choice between them shows here; bounds as in kv4_cases."""
import numpy as np
import pytest

from gpu_cases import say, to_dev
from kv4_cases import Batch, check

pytestmark = pytest.mark.gpu


def plan(wq, new, ctx, hq, hkv, d, window=0, max_q=None, max_ctx=None):
    return wq.kv4_attention_plan(sum(new), len(new), hq, hkv, d, max(new) if max_q is None else max_q,
                                 max(ctx) if max_ctx is None else max_ctx, window)


def takes_many_rows(wq, shares, new, ctx, hq, hkv, d, **kw):
    p = plan(wq, new, ctx, hq, hkv, d, **kw)
    assert p["many_rows"] and p["shares"] == shares, p


@pytest.mark.parametrize("new,ctx,hq,hkv,d,window,shares", [
    *[([500], [500], 32, 4, 64, w, False) for w in (1, 2, 31, 32, 33, 100, 10000)],
    *[([260, 260], [700, 300], 32, 4, 128, w, False) for w in (1, 33, 100, 257)],
    ([640], [4000], 32, 2, 128, 1, False),
    ([640], [4000], 32, 2, 128, 33, False),
    ([640], [4000], 32, 2, 128, 700, True),
    ([640], [4000], 32, 2, 128, 1500, True),
    ([300, 310], [2600, 2700], 32, 2, 128, 1500, True),   # with single rows' kernel beside it
])
def test_window(gpu_lib, new, ctx, hq, hkv, d, window, shares):
    """A sliding window, with the pages of what it has passed given to somebody else: their
    entries name a page of NaN, and whatever stands there may not be noticed."""
    import torch
    say(f"[kv4 many rows, window] {window} new={new} ctx={ctx} d={d}")
    takes_many_rows(gpu_lib, shares, new, ctx, hq, hkv, d, window=window)
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 32, seed=window).fill()
    ref = b.reference(window=window)
    table = b.table.cpu().numpy().copy()
    used = {int(p) for i, c in enumerate(ctx) for p in table[i, :-(-c // 32)]}
    free = (set(range(b.num_pages)) - used).pop()
    for i, (n, c) in enumerate(zip(new, ctx)):
        table[i, :max(0, c - n - window + 1) // 32] = free
    b.table = to_dev(table, torch)
    check(*b.attention(window=window), ref)


@pytest.mark.parametrize("new,ctx,hq,hkv,d,max_ctx,shares", [
    ([400, 400], [0, 900], 32, 2, 128, None, False),        # no tokens at all beside many
    ([400, 390], [300, 380], 32, 4, 64, None, False),       # the first rows see nothing
    ([1200, 1200], [3, 1150], 16, 4, 64, None, False),
    ([560, 520, 500], [5000, 2300, 0], 32, 2, 128, None, True),
    ([900], [700], 32, 2, 128, 9000, True),                 # shares made for more than there is
    ([600], [0], 32, 2, 128, 9000, True),
])
@pytest.mark.parametrize("window", [0, 70])
def test_rows_that_see_nothing(gpu_lib, new, ctx, hq, hkv, d, max_ctx, shares, window):
    import torch
    say(f"[kv4 many rows, empty] new={new} ctx={ctx} d={d} max_ctx={max_ctx} window={window}")
    takes_many_rows(gpu_lib, shares and window == 0, new, ctx, hq, hkv, d, max_ctx=max_ctx, window=window)
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 32, seed=1).fill()
    kw = {} if max_ctx is None else {"max_ctx": max_ctx}
    check(*b.attention(window=window, **kw), b.reference(window=window))


@pytest.mark.parametrize("new,ctx,hq,hkv,d,page,shares", [([500], [500], 30, 3, 64, 32, False),
                                                         ([260, 260], [700, 300], 28, 4, 128, 96, False),
                                                         ([640], [3000], 28, 2, 128, 64, True),
                                                         ([700], [2600], 52, 4, 64, 128, True)])
def test_scale_slices_and_out(gpu_lib, new, ctx, hq, hkv, d, page, shares):
    """Other scales, queries as a slice of a wider projection, an output given."""
    import torch
    say(f"[kv4 many rows, slices] new={new} ctx={ctx} hq={hq} d={d}")
    takes_many_rows(gpu_lib, shares, new, ctx, hq, hkv, d)
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, page, seed=7).fill()
    T = sum(new)
    wide = torch.randn(T, (hq + 2 * hkv) * d, device="cuda").half()
    wide[:, hkv * d:(hkv + hq) * d] = to_dev(b.q.reshape(T, -1), torch)
    q = wide[:, hkv * d:(hkv + hq) * d].unflatten(1, (hq, d))
    assert not q.is_contiguous()
    for scale in (0.02, 1.0):
        out = torch.full((T, hq, d), float("nan"), device="cuda", dtype=torch.float16)
        got, lse = b.attention(q=q, scale=scale, out=out)
        assert got is out
        check(got, lse, b.reference(scale=scale), f"scale {scale}")


@pytest.mark.parametrize("new,ctx,hq,hkv,d,few,shares", [([500], [500], 32, 4, 64, False, False),
                                                        ([640], [4000], 32, 2, 128, False, True),
                                                        ([640, 2, 1], [4000, 50, 3000], 32, 2, 128, True, True)])
def test_deterministic_and_other_streams(gpu_lib, new, ctx, hq, hkv, d, few, shares):
    import torch
    say(f"[kv4 many rows, streams] new={new} ctx={ctx}")
    p = plan(gpu_lib, new, ctx, hq, hkv, d)
    assert p["many_rows"] and p["few_rows"] == few and p["shares"] == shares, p
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 64, seed=14).fill()
    out, lse = b.attention()
    check(out, lse, b.reference())
    q = to_dev(b.q, torch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, lse2 = b.wq.kv4_attention(q, b.cache, b.table, b.seq_start, b.ctx_len, max_q=max(new),
                                         max_ctx=max(ctx), return_lse=True)
    side.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # a workspace full of something else
    ws = torch.full((gpu_lib.kv4_attention_workspace_bytes(sum(new), len(new), hq, hkv, d, max(new), max(ctx)) + 1,),
                    0xFF, device="cuda", dtype=torch.uint8)
    third, lse3 = b.attention(workspace=ws)
    assert torch.equal(out, third) and torch.equal(lse, lse3)


@pytest.mark.parametrize("new,ctx,hq,hkv,d,shares", [([500], [500], 32, 4, 64, False), ([640], [3000], 32, 2, 128, True)])
def test_values_and_scores_of_all_sizes(gpu_lib, new, ctx, hq, hkv, d, shares):
    """Value scales along the sequence from 2^-13 to 2^11 and back, scores that rise and fall by
    hundreds, equal scores."""
    import torch
    takes_many_rows(gpu_lib, shares, new, ctx, hq, hkv, d)
    L = sum(ctx)
    rng = np.random.default_rng(11)
    ramp = 2.0 ** np.linspace(-11, 13, L)[:, None, None]
    base = rng.standard_normal((L, hkv, d))
    rise = np.linspace(0.1, 30, L)[:, None, None]
    for name, k, v in (("growing values", base, base * ramp), ("falling values", base, base * ramp[::-1]),
                       ("rising scores", base * rise, base), ("falling scores", base * rise[::-1], base),
                       ("both", base * rise, base * ramp[::-1]), ("equal scores", base * 0, base),
                       ("huge values", base, np.clip(base * 2e4, -65504, 65504))):
        b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 64, seed=12, k=k.astype(np.float16),
                  v=v.astype(np.float16)).fill()
        say(f"[kv4 many rows, ranges] {name} new={new}")
        check(*b.attention(), b.reference(), name)
