"""The norm with the residual's addition against float64, in fp16 and in 8 bits."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import layer_to_dev, say, to_dev

pytestmark = pytest.mark.gpu

# y is h times two float32 factors and a sum's root, each within a few float32 roundings
# (K additions of squares, all positive, in chains of at most 64 and a tree), then one
# rounding to fp16: half an ulp, 2^-11 of the value (2^-25 below the smallest normal).
F32 = 2.0 ** -19


def _case(M, K, seed, n_out=0, scale=1.0):
    rng = np.random.default_rng(seed)
    x = (scale * rng.standard_normal((M, K))).astype(np.float16)
    res = (2 * scale * rng.standard_normal((M, K))).astype(np.float16)
    w = (1 + 0.1 * rng.standard_normal(K)).astype(np.float16)
    out = np.sort(rng.choice(K, n_out, replace=False)).astype(np.int32)
    res[:, out] = res[:, out] * np.float16(20)
    return x, res, w, out


def _close16(got, ref):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(g - ref) <= (2.0 ** -11 + F32) * np.abs(ref) + 2.0 ** -25), np.abs(g - ref).max()


SIZES = [(1, 16), (1, 128), (3, 48), (2, 4096), (7, 1040), (33, 8192), (5, 16400), (2, 28672), (2, 32768), (2, 40000),
         (300, 256), (70000, 32)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("with_residual", [True, False])
def test_fp16(gpu_lib, M, K, with_residual):
    import torch
    x, res, w, _ = _case(M, K, M + K)
    res = res if with_residual else None
    say(f"[norm fp16] M={M} K={K} residual={with_residual}")
    xd = to_dev(x, torch)
    y, h = gpu_lib.add_rmsnorm(xd, to_dev(w, torch), None if res is None else to_dev(res, torch))
    torch.cuda.synchronize()
    ry, rh = oracle.add_rmsnorm(x, w, res)
    _close16(y, ry)
    if res is None:
        assert h is xd
    else:
        _close16(h, rh)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("n_out", [0, 1, 8, 16])
def test_int8(gpu_lib, M, K, n_out):
    """The integers are those of the exact quotient, except where that lies within a few
    float32 roundings of a half; scales and outliers are within theirs."""
    import torch
    x, res, w, out = _case(M, K, M + K + n_out, n_out)
    say(f"[norm int8] M={M} K={K} outliers={n_out}")
    od = to_dev(out, torch)
    xq, sx, xo, h = gpu_lib.add_rmsnorm_int8(to_dev(x, torch), to_dev(w, torch), to_dev(res, torch), outliers=od)
    torch.cuda.synchronize()
    ry, rh = oracle.add_rmsnorm(x, w, res)
    quot, s = oracle.norm_int8(ry, out)
    _close16(h, rh)
    got_s = sx.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got_s - s) <= F32 * s)
    q = xq.cpu().numpy().reshape(M, K // 16, 16)
    order = [0, 2, 4, 6, 1, 3, 5, 7, 8, 10, 12, 14, 9, 11, 13, 15]
    nat = np.empty_like(q)
    nat[:, :, order] = q
    nat = nat.reshape(M, K).astype(np.float64)
    assert np.all(np.abs(nat - quot) <= 0.5 + 128 * F32)
    assert np.all(np.abs(nat) <= 127) and np.all(nat[:, out] == 0)
    xo = xo.cpu()
    _close16(xo[:, :n_out], ry[:, out])
    assert bool((xo[:, n_out:] == 0).all())
    # and the values they stand for
    v = gpu_lib.dequantize_act_int8(xq, sx, xo.cuda(), od)
    want = nat * got_s[:, None]
    want[:, out] = xo[:, :n_out].numpy()
    _close16(v, want)


def test_zero_rows_and_in_place(gpu_lib):
    import torch
    x, res, w, _ = _case(4, 512, 3)
    x[1] = 0
    res[1] = 0
    xd, rd, wd = (to_dev(a, torch) for a in (x, res, w))
    ry, rh = oracle.add_rmsnorm(x, w, res)
    xq, sx, xo, h = gpu_lib.add_rmsnorm_int8(xd, wd, rd, h=rd)
    torch.cuda.synchronize()
    assert h is rd and float(sx[1]) == 1.0 and bool((xq[1] == 0).all())
    _close16(rd, rh)
    y, h = gpu_lib.add_rmsnorm(xd, wd, to_dev(res, torch), h=xd, out=torch.empty_like(xd))
    torch.cuda.synchronize()
    assert h is xd and bool((y[1] == 0).all())
    _close16(y, ry)
    _close16(xd, rh)
    e, _ = gpu_lib.add_rmsnorm(xd[:0], wd)
    assert tuple(e.shape) == (0, 512)


@pytest.mark.parametrize("K", [512, 28672, 40000])
def test_long_rows_in_place(gpu_lib, K):
    """Rows longer than the registers hold are read again: the sum in place of the
    residual must not be what is read."""
    import torch
    x, res, w, out = _case(3, K, K, 4)
    rd = to_dev(res, torch)
    xq, sx, xo, h = gpu_lib.add_rmsnorm_int8(to_dev(x, torch), to_dev(w, torch), rd, outliers=to_dev(out, torch), h=rd)
    a = gpu_lib.add_rmsnorm_int8(to_dev(x, torch), to_dev(w, torch), to_dev(res, torch), outliers=to_dev(out, torch))
    for p, q in zip((xq, sx, xo, h), a):
        assert torch.equal(p, q)
    y1, _ = gpu_lib.add_rmsnorm(to_dev(x, torch), to_dev(w, torch), to_dev(res, torch))
    rd = to_dev(res, torch)
    y2, _ = gpu_lib.add_rmsnorm(to_dev(x, torch), to_dev(w, torch), rd, h=rd)
    assert torch.equal(y1, y2) and torch.equal(rd, h)


def test_feeds_the_product(gpu_lib):
    """Norm, then the INT8 product, against float64 on the integers the norm gave; and the
    product equals linear_w4a8's on the same activations."""
    import torch
    M, N, K = 19, 300, 1024
    x, res, w, out = _case(M, K, 5, 8)
    W = workloads.random_weights(6, N, K)
    L = oracle.quantize_layer(W, 0)
    D = layer_to_dev(L, torch)
    od = to_dev(out, torch)
    xq, sx, xo, _ = gpu_lib.add_rmsnorm_int8(to_dev(x, torch), to_dev(w, torch), to_dev(res, torch), outliers=od)
    y = gpu_lib.linear_w4a8_quantized(xq, sx, xo, od, D["packed"], D["scales"], D["zeros"], out_dtype=torch.float32)
    vals = gpu_lib.dequantize_act_int8(xq, sx, xo, od).float().cpu().numpy().astype(np.float64)
    ref = vals @ oracle.dequant(L["q"], L["s"], L["z"]).T
    err = oracle.rel_err_inf(y.cpu().numpy(), ref)
    say(f"[norm product] rel err {err:.2e}")
    assert err <= oracle.TOL
    z = to_dev(x, torch)
    a = gpu_lib.quantize_act_int8(z, od)
    one = gpu_lib.linear_w4a8_quantized(*a, od, D["packed"], D["scales"], D["zeros"])
    two = gpu_lib.linear_w4a8(z, od, D["packed"], D["scales"], D["zeros"])
    assert torch.equal(one, two)
