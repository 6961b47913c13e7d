"""Workspaces: the binding refuses one that is not a whole piece of the inputs' device (CPU
only)."""
import types

import pytest

import quantized_gemm_rtn_amd as wq

HERE = types.SimpleNamespace(get_device=lambda: -1)   # an input in host memory
THERE = types.SimpleNamespace(get_device=lambda: 0)   # and one on a GPU


def test_a_workspace_is_a_whole_piece_of_the_device():
    import torch
    w = torch.zeros(64, 8, dtype=torch.float32)
    assert wq._workspace_bytes(None, THERE) == 0
    assert wq._workspace_bytes(w, HERE) == 2048
    assert wq._workspace_bytes(w[3:], HERE) == 61 * 32
    with pytest.raises(TypeError):
        wq._workspace_bytes(w, THERE)        # host memory, which the GPU must not write
    with pytest.raises(TypeError):
        wq._workspace_bytes(b"0" * 64, THERE)
    for view in (w[:, :4], w.t(), w[::2]):   # numel * element_size is not what lies behind them
        with pytest.raises(ValueError):
            wq._workspace_bytes(view, HERE)
