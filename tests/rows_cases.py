"""Shared helpers of the tests of products whose weights a row chooses (imported by test_gpu_adapters.py, test_gpu_moe.py
and others): layers on the CPU and their copies on the GPU."""
import numpy as np

import oracle
import workloads
from gpu_cases import layer_to_dev, to_dev


def layer(seed, N, K, per_mille=0, sigma=0.02):
    """A quantized layer and its held weights (float64, sparse entries added)."""
    L = oracle.quantize_layer(workloads.random_weights(seed, N, K, sigma), N * K * per_mille // 1000)
    w = oracle.dequant(L["q"], L["s"], L["z"])
    for n in range(N):
        a, b = L["row_ptr"][n], L["row_ptr"][n + 1]
        w[n, L["col"][a:b]] += L["val"][a:b].astype(np.float64)
    L["held"], L["nnz"] = w, int(L["row_ptr"][-1])
    return L


def factors(seed, n, r, N, K):
    rng = np.random.default_rng(seed)
    return ((rng.standard_normal((n, r, K)) / K ** 0.5).astype(np.float16),
            (0.1 * rng.standard_normal((n, N, r))).astype(np.float16))


def run_adapters(wq, torch, L, x, L1, L2, adapter, scale=None, **kw):
    D = layer_to_dev(L, torch)
    csr = (D["row_ptr"], D["col"], D["val"]) if L["nnz"] else (None, None, None)
    y = wq.linear_adapters(to_dev(x, torch), D["packed"], D["scales"], D["zeros"], to_dev(L1, torch), to_dev(L2, torch),
                           to_dev(np.asarray(adapter, np.int32), torch),
                           None if scale is None else to_dev(np.asarray(scale, np.float32), torch), *csr, **kw)
    torch.cuda.synchronize()
    return y


def stacked(seed, E, N, K, sigma):
    """E layers [N, K]: their tensors stacked, and held weights."""
    layers = [layer(seed + e, N, K, 0, sigma) for e in range(E)]
    return {k: np.stack([L[k] for L in layers]) for k in ("packed", "s", "z")}, [L["held"] for L in layers]


class Moe:
    """A mixture-of-experts layer on the CPU and the GPU."""

    def __init__(self, torch, seed, H, I, E):
        self.H, self.I, self.E = H, I, E
        self.up, self.held_up = stacked(seed, E, 2 * I, H, H ** -0.5)
        self.down, self.held_down = stacked(seed + 1000, E, H, I, I ** -0.5)
        self.args = [to_dev(p[k], torch) for p in (self.up, self.down) for k in ("packed", "s", "z")]

    def run(self, wq, torch, x, experts, weights, **kw):
        y = wq.moe_experts(to_dev(x, torch), to_dev(np.asarray(experts, np.int32), torch),
                           to_dev(np.asarray(weights, np.float32), torch), *self.args, **kw)
        torch.cuda.synchronize()
        return y

    def reference(self, x, experts, weights):
        return oracle.rows.moe_experts(x, experts, weights, self.held_up, self.held_down)


def worst(y, ref, bound, f16=True):
    """The largest |y - ref| as a multiple of its bound."""
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    most = np.maximum(oracle.rows.rounded(ref, bound, f16), 1e-300)  # (a row of no terms: 0, and no error)
    return float(np.max(np.abs(got - ref) / most)) if got.size else 0.0
