"""What the cache attention launches, from the host's plan (CPU only): the choice itself and
the shape of the joins."""
import pytest

import quantized_gemm_rtn_amd as wq
from test_kv4_abi import lib  # noqa: F401


def plan(new, ctx, hq, hkv, d, window=0):
    return wq.kv4_attention_plan(sum(new), len(new), hq, hkv, d, max(new), max(ctx), window)


def test_sizes(lib):  # noqa: F811
    f = lib.wq_kv4_attention_plan
    for bad in ((0, 1, 8, 8, 128, 1, 10, 0), (1, 0, 8, 8, 128, 1, 10, 0), (1, 1, 9, 8, 128, 1, 10, 0),
                (1, 1, 8, 8, 96, 1, 10, 0), (1, 1, 8, 8, 128, -1, 10, 0), (1, 1, 8, 8, 128, 1, -1, 0),
                (1, 1, 8, 8, 128, 1, 10, -1), (1, 1, 8, 8, 128, 1, 10, 1 << 31)):
        assert f(*bad) == 0
    with pytest.raises(ValueError):
        plan([1], [10], 9, 8, 128)


def test_single_tokens(lib):  # noqa: F811
    """One token each: the kernel for few rows; joined where the sequences are split, by more
    waves where a row has more partials."""
    assert plan([1], [32], 32, 8, 128) == dict(few_rows=True, many_rows=False, shares=False, join_waves=0)
    assert plan([1] * 64, [8192] * 64, 64, 8, 128)["join_waves"] == 1
    assert plan([1], [131071], 32, 8, 128)["join_waves"] == 16


@pytest.mark.parametrize("T,B,hq,hkv,max_q,max_ctx,waves", [
    (33, 1, 4, 1, 33, 4937, 4),      # 5 items in 512 shares
    (76, 1, 7, 1, 76, 1914, 4),      # 17 in 512
    (178, 1, 4, 1, 178, 780, 1),     # 23 in as many shares as items have eights of tiles
    (2, 2, 8, 1, 1, 17868, 16),      # 2 in 512
])
def test_partials_of_a_row(lib, T, B, hq, hkv, max_q, max_ctx, waves):  # noqa: F811
    """A row's partials are those of its own item of 32 rows, of which a sequence has several:
    not all shares of the sequence."""
    p = wq.kv4_attention_plan(T, B, hq, hkv, 128, max_q, max_ctx)
    assert p["few_rows"] and not p["many_rows"] and p["join_waves"] == waves


@pytest.mark.parametrize("T,B,hq,hkv,d,max_q,max_ctx,window,many", [
    (33, 1, 4, 1, 128, 33, 4937, 0, False),        # 14 us, 42 with the other kernel
    (52, 1, 64, 8, 128, 52, 6838, 0, False),       # 43, 58
    (344, 43, 16, 1, 64, 8, 4008, 0, False),       # 34, 43
    (1309, 11, 8, 8, 128, 119, 2419, 2300, False),  # 54, 61
    (272, 16, 64, 8, 128, 17, 1217, 0, True),      # 48, 60
    (476, 4, 32, 4, 64, 163, 453, 0, True),        # 22, 31
    (2048, 1, 32, 8, 128, 2048, 2048, 0, True),
    (16384, 64, 64, 8, 128, 256, 4096, 0, True),
])
def test_the_faster_kernel_is_taken(lib, T, B, hq, hkv, d, max_q, max_ctx, window, many):  # noqa: F811
    """Batches of more than 96 rows a sequence whose times with either kernel differ by more
    than a tenth."""
    p = wq.kv4_attention_plan(T, B, hq, hkv, d, max_q, max_ctx, window)
    assert p["many_rows"] == many


def test_no_workspace_where_nothing_is_split(lib):  # noqa: F811
    f = lib.wq_kv4_attention_workspace_bytes
    # more key/value heads than half the blocks that run at once: one share a head
    for hkv in (257, 512, 600):
        for T, q in ((1, 1), (200, 200), (2000, 2000)):
            assert f(T, 1, hkv, hkv, 128, q, 4096) == 0
    assert f(2000, 1, 256, 256, 128, 2000, 4096) > 0
