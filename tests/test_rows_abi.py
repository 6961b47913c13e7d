"""Refusals of the adapter, routing and mixture-of-experts entry points: bad arguments come back as a status, before any
HIP call (the fake device addresses are never dereferenced); and the oracle's pins."""
import ctypes

import numpy as np
import pytest

import oracle
import quantized_gemm_rtn_amd as wq
from test_kv4_abi import lib  # noqa: F401

A = ctypes.c_void_p(0x7F0000000000)      # aligned fake device addresses
A2 = ctypes.c_void_p(0x7F0000100000)
MIS = ctypes.c_void_p(0x7F0000000008)    # 8-byte aligned only
ODD = ctypes.c_void_p(0x7F0000000002)
BYTE = ctypes.c_void_p(0x7F0000000001)


def adapters(lib, x=A, M=4, K=256, packed=A, scales=A, zeros=A, N=64, group=128, row_ptr=None, col=None, val=None,
             nnz=0, L1=A, L2=A, scale=A, n=3, r=16, adapter=A, y=A2, y_dtype=0, kernel=0, ws=A, nbytes=1 << 30):
    return lib.wq_linear_adapters(x, M, K, packed, scales, zeros, N, group, row_ptr, col, val, nnz, L1, L2, scale, n,
                                  r, adapter, y, y_dtype, kernel, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(packed=None), -1), (dict(scales=None), -1), (dict(zeros=None), -1), (dict(y=None), -1),
    (dict(L1=None), -1), (dict(L2=None), -1), (dict(adapter=None), -1), (dict(nnz=3), -1),
    (dict(row_ptr=A, nnz=3), -1), (dict(group=64), -4), (dict(y_dtype=2), -4), (dict(kernel=7), -4), (dict(r=12), -4),
    (dict(r=264), -4), (dict(r=0), -2), (dict(r=-8), -2), (dict(n=0), -2), (dict(n=(1 << 20) + 1), -2),
    (dict(M=-1), -2), (dict(N=0), -2), (dict(K=200), -2), (dict(K=0), -2), (dict(M=1 << 24), -2),
    (dict(x=MIS), -3), (dict(packed=MIS), -3), (dict(L1=MIS), -3), (dict(L2=MIS), -3), (dict(scale=ODD), -3),
    (dict(adapter=ODD), -3), (dict(y=ODD), -3), (dict(ws=MIS), -3), (dict(ws=None), -6), (dict(nbytes=255), -6),
    (dict(M=0, x=None, y=None, adapter=None, ws=None, nbytes=0), 0),
])
def test_adapters_validation(lib, kw, status):  # noqa: F811
    assert adapters(lib, **kw) == status


def test_adapters_workspace(lib):  # noqa: F811
    f = lib.wq_linear_adapters_workspace_bytes
    assert f(4, 64, 256, 16) == 256 + lib.wq_linear_workspace_bytes(4, 64, 256)   # t: 4 rows of 32 fp16
    assert f(5, 64, 256, 40) == 768 + lib.wq_linear_workspace_bytes(5, 64, 256)   # 5 rows of 64
    for bad in ((0, 64, 256, 16), (4, 0, 256, 16), (4, 64, 200, 16), (4, 64, 256, 12), (4, 64, 256, 0),
                (4, 64, 256, 264), (1 << 24, 64, 256, 16)):
        assert f(*bad) == 0


def route(lib, logits=A, dtype=1, M=4, E=8, k=2, renorm=1, experts=A, weights=A):
    return lib.wq_moe_route(logits, dtype, M, E, k, renorm, experts, weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), -1), (dict(experts=None), -1), (dict(weights=None), -1), (dict(dtype=2), -4),
    (dict(E=1025), -4), (dict(k=17, E=20), -4), (dict(E=0), -2), (dict(k=0), -2), (dict(k=9), -2), (dict(M=-1), -2),
    (dict(M=1 << 28), -2), (dict(M=(1 << 25) + 1, E=1, k=1), -2), (dict(logits=ODD), -3), (dict(logits=BYTE, dtype=0), -3), (dict(experts=ODD), -3),
    (dict(weights=ODD), -3), (dict(M=0, logits=None, experts=None, weights=None), 0),
])
def test_route_validation(lib, kw, status):  # noqa: F811
    assert route(lib, **kw) == status


def experts(lib, x=A, M=4, H=256, ids=A, weights=A, k=2, E=8, up=A, up_s=A, up_z=A, I=384, down=A, down_s=A, down_z=A,
            group=128, y=A2, y_dtype=0, ws=A, nbytes=1 << 30):
    return lib.wq_moe_experts(x, M, H, ids, weights, k, E, up, up_s, up_z, I, down, down_s, down_z, group, y, y_dtype,
                              ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(up=None), -1), (dict(up_s=None), -1),
    (dict(up_z=None), -1), (dict(down=None), -1), (dict(down_s=None), -1), (dict(down_z=None), -1), (dict(y=None), -1),
    (dict(group=64), -4), (dict(y_dtype=3), -4), (dict(E=1025), -4), (dict(k=17), -4), (dict(E=0), -2), (dict(k=0), -2),
    (dict(M=-1), -2), (dict(M=65535 * 64 + 1, H=128, I=128), -2), (dict(H=200), -2), (dict(I=64), -2), (dict(I=0), -2),
    (dict(H=1 << 16, I=1 << 14), -2), (dict(M=1 << 22, H=512), -2), (dict(x=MIS), -3), (dict(up=MIS), -3),
    (dict(down=MIS), -3), (dict(up_s=BYTE), -3), (dict(up_z=BYTE), -3), (dict(down_s=BYTE), -3), (dict(down_z=BYTE), -3),
    (dict(ids=ODD), -3), (dict(weights=ODD), -3), (dict(y=ODD), -3), (dict(ws=MIS), -3), (dict(ws=None), -6),
    (dict(nbytes=1024), -6), (dict(M=0, x=None, ids=None, weights=None, y=None, ws=None, nbytes=0), 0),
])
def test_experts_validation(lib, kw, status):  # noqa: F811
    assert experts(lib, **kw) == status


def test_experts_workspace(lib):  # noqa: F811
    f = lib.wq_moe_experts_workspace_bytes
    last = 0
    for M in range(1, 1000):
        n = f(M, 256, 384, 2)
        assert n >= M * 2 * 384 * 2 and n >= last
        last = n
    for bad in ((0, 256, 384, 2), (4, 200, 384, 2), (4, 256, 100, 2), (4, 256, 384, 0), (4, 256, 384, 17),
                (4, 1 << 16, 1 << 14, 2)):
        assert f(*bad) == 0


def test_binding_refuses_host_tensors(lib):  # noqa: F811
    import torch
    x = torch.zeros(2, 256, dtype=torch.float16)
    with pytest.raises(TypeError):
        wq.linear_adapters(x, x, x, x, x, x, x)
    with pytest.raises(TypeError):
        wq.moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError):
        wq.moe_route([[1.0]], 1)
    with pytest.raises(TypeError):
        wq.moe_experts(x, x, x, x, x, x, x, x, x)


# ---------------------------------------------------------------- the oracle's pins
def test_oracle_adapters_pins():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((4, 6)).astype(np.float16), rng.standard_normal((5, 6))
    L1, L2 = rng.standard_normal((2, 3, 6)).astype(np.float16), rng.standard_normal((2, 5, 3)).astype(np.float16)
    y, bound = oracle.rows.linear_adapters(x, w, L1, L2, [1, -1, 0, 2], [2.0, 0.5])
    for m, (a, s) in enumerate([(1, 0.5), (None, 0), (0, 2.0), (None, 0)]):
        for n in range(5):
            v = sum(float(x[m, k]) * w[n, k] for k in range(6))
            if a is not None:
                v += s * sum(sum(float(x[m, k]) * float(L1[a, c, k]) for k in range(6)) * float(L2[a, n, c])
                             for c in range(3))
            assert np.isclose(y[m, n], v)
    assert np.all(bound > 0) and np.all(bound < 1e-2)


def test_oracle_route_pins():
    e, w = oracle.rows.moe_route([[0.0, np.log(2.0), np.log(2.0), -np.inf]], 2)
    assert e.tolist() == [[1, 2]] and np.allclose(w, [[0.5, 0.5]])
    e, w = oracle.rows.moe_route([[0.0, np.log(2.0), np.log(2.0), -np.inf]], 4, renormalize=False)
    assert e.tolist() == [[1, 2, 0, -1]] and np.allclose(w, [[0.4, 0.4, 0.2, 0.0]])
    e, w = oracle.rows.moe_route([[-np.inf] * 3, [0.0, np.nan, 9.0]], 2)
    assert e.tolist() == [[-1, -1], [1, 2]] and np.all(w[0] == 0) and np.all(np.isnan(w[1]))


def test_oracle_experts_pins():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 4)).astype(np.float16)
    up, down = rng.standard_normal((2, 6, 4)), rng.standard_normal((2, 4, 3))
    ids, wt = np.array([[0, 1], [1, 1], [-1, 0]]), np.array([[0.25, 0.75], [0.5, 0.25], [9.0, 2.0]])
    y, bound = oracle.rows.moe_experts(x, ids, wt, up, down)
    for m in range(3):
        v = np.zeros(4)
        for j in range(2):
            if ids[m, j] >= 0:
                gu = up[ids[m, j]] @ x[m].astype(np.float64)
                h = np.array([gu[i] / (1 + np.exp(-gu[i])) * gu[3 + i] for i in range(3)])
                v += wt[m, j] * (down[ids[m, j]] @ h)
        assert np.allclose(y[m], v)
    assert np.all(bound > 0) and np.all(bound < 1e-1)
