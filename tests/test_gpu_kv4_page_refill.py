"""Blocks that walk many pages of one sequence: the decode kernel holds the numbers of 64 pages
at a time and loads the next ones between tiles that are on their way."""
import pytest

from gpu_cases import say
from kv4_cases import Batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,ctx,hq,hkv,page", [
    ([1], [9000], 4, 1, 32),           # 282 pages of one tile
    ([1, 3], [8190, 6400], 2, 1, 32),
    ([20], [7000], 4, 2, 32),          # more rows than one column of queries
    ([1], [20000], 1, 1, 96),          # pages of three tiles
])
@pytest.mark.parametrize("window", [0, 5000])
def test_many_pages_in_one_block(gpu_lib, new, ctx, hq, hkv, page, d, window):
    """With a bound on the lengths of one token a sequence has one share, so one block takes
    all its pages, in a shuffled order."""
    import torch
    say(f"[kv4 pages] new={new} ctx={ctx} page={page} d={d} window={window}")
    plan = gpu_lib.kv4_attention_plan(sum(new), len(new), hq, hkv, d, max(new), 1, window)
    assert plan["few_rows"] and not plan["many_rows"]
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, page, seed=sum(ctx)).fill()
    check(*b.attention(max_ctx=1, window=window), b.reference(window=window))
