"""Scales that would carry scores past the kernels' mark of a row that has seen nothing are
refused before any HIP call (the fake device addresses are never dereferenced)."""
import pytest

from test_kv4_abi import attention, lib  # noqa: F401


@pytest.mark.parametrize("scale", [1.1e16, 1e20, 1e29, 3e38])
def test_scales_past_the_mark(lib, scale):  # noqa: F811
    assert attention(lib, scale=scale) == -4


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e16])
def test_scales_up_to_it(lib, scale):  # noqa: F811
    assert attention(lib, scale=scale, T=0) == 0
    assert attention(lib, scale=scale, ws=None, max_ctx=100000) == -6  # the next check
