"""Every entry point that takes a workspace refuses host memory and strided views, before it
launches anything."""
import pytest

import oracle
import workloads
from gpu_cases import layer_to_dev, to_dev

pytestmark = pytest.mark.gpu


def test_refusals(gpu_lib):
    import torch
    import numpy as np
    N, K, M, r = 64, 1024, 4, 32
    W = workloads.random_weights(3, N, K)
    L = oracle.quantize_layer(W, 0)
    D = layer_to_dev(L, torch)
    x = to_dev(workloads.random_x(1, M, K), torch)
    layer = (D["packed"], D["scales"], D["zeros"])
    od = to_dev(np.array([1, 2], np.int32), torch)
    perm = torch.arange(K, dtype=torch.int32, device="cuda")
    xq, sx, xo = gpu_lib.quantize_act_int8(x, od)
    low = [torch.zeros(*s, dtype=torch.float16, device="cuda") for s in ((r, K), (N, r))]
    cache = gpu_lib.kv4_cache(4, 32, 2, 64)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    start, ctx = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1], [100]))
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    calls = {
        "quantize_rtn": lambda ws: gpu_lib.quantize_rtn(to_dev(W, torch), 10, workspace=ws),
        "quantize_rtn_act_order": lambda ws: gpu_lib.quantize_rtn_act_order(to_dev(W, torch), perm, 10, workspace=ws),
        "linear": lambda ws: gpu_lib.linear(x, *layer, workspace=ws),
        "linear_lowrank": lambda ws: gpu_lib.linear_lowrank(x, *layer, *low, workspace=ws),
        "linear_act_order": lambda ws: gpu_lib.linear_act_order(x, perm, *layer, workspace=ws),
        "linear_w4a8": lambda ws: gpu_lib.linear_w4a8(x, od, *layer, workspace=ws),
        "linear_w4a8_quantized": lambda ws: gpu_lib.linear_w4a8_quantized(xq, sx, xo, od, *layer, workspace=ws),
        "kv4_attention": lambda ws: gpu_lib.kv4_attention(q, cache, table, start, ctx, workspace=ws),
    }
    size = 1 << 24
    for name, call in calls.items():
        with pytest.raises(TypeError, match="workspace"):
            call(torch.zeros(size, dtype=torch.uint8))
        with pytest.raises(ValueError, match="workspace"):
            call(torch.zeros(2, size, dtype=torch.uint8, device="cuda").t())
        call(torch.zeros(size, dtype=torch.uint8, device="cuda"))
        call(torch.zeros(size // 4, dtype=torch.float32, device="cuda"))
    torch.cuda.synchronize()
