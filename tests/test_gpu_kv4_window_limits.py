"""Windows up to the largest that is taken (2^31 - 1, a common way to say "none") with
sequences whose leading rows stand before the first token."""
import pytest

from gpu_cases import say
from kv4_cases import Batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 40, 2 ** 30, 400])
@pytest.mark.parametrize("new,ctx,hq,hkv,d", [
    ([8], [3], 4, 2, 128),                 # few rows, all in one item
    ([5, 1], [1, 3], 2, 1, 64),
    ([40, 3, 1], [7, 100, 0], 4, 2, 128),  # more row tiles than one
    ([700, 600], [300, 400], 16, 2, 128),  # many rows
])
def test_windows_beyond_the_context(gpu_lib, window, new, ctx, hq, hkv, d):
    """A window of at least the tokens that a sequence has hides none of them: the bits of
    the call without one, and the oracle's."""
    import torch
    say(f"[kv4 large window] {window} new={new} ctx={ctx} d={d}")
    b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 32, seed=sum(new)).fill()
    out, lse = b.attention(window=window)
    check(out, lse, b.reference(), f"window {window}")
    if window > 10 ** 6:
        plain, plain_lse = b.attention()
        assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
