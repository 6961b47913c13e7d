"""Refusals of the norm and cache entry points: bad arguments come back as a status, before
any HIP call (the fake device addresses are never dereferenced); the binding's own checks;
and the oracle's pins."""
import ctypes

import numpy as np
import pytest

import oracle
import quantized_gemm_rtn_amd as wq

A = ctypes.c_void_p(0x7F0000000000)      # aligned fake device addresses
A2 = ctypes.c_void_p(0x7F0000100000)
A3 = ctypes.c_void_p(0x7F0000200000)
MIS = ctypes.c_void_p(0x7F0000000008)    # 8-byte aligned only
ODD = ctypes.c_void_p(0x7F0000000002)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(wq.LIB_PATH):
        import quantized_gemm_rtn_amd.build as b
        b.build()
    return wq.load()


# ---------------------------------------------------------------- norm
def norm(lib, x=A, residual=A2, weight=A3, M=4, K=256, eps=1e-5, h=A, y=A2):
    return lib.wq_add_rmsnorm(x, residual, weight, M, K, eps, h, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(weight=None), -1), (dict(y=None), -1),
    (dict(eps=-1e-9), -4), (dict(eps=float("nan")), -4), (dict(eps=float("inf")), -4),
    (dict(M=-1), -2), (dict(K=0), -2), (dict(K=24), -2), (dict(M=1 << 20, K=4096), -2), (dict(K=1 << 31), -2),
    (dict(x=MIS), -3), (dict(residual=MIS), -3), (dict(weight=MIS), -3), (dict(h=MIS), -3), (dict(y=MIS), -3),
    (dict(M=0, x=None, y=None, residual=None, h=None), 0),
])
def test_norm_validation(lib, kw, status):
    assert norm(lib, **kw) == status


def norm8(lib, x=A, K=256, M=4, outliers=A2, n_out=8, xq=A, sx=A2, xo=A3, eps=1e-5):
    return lib.wq_add_rmsnorm_int8(x, None, A3, M, K, eps, outliers, n_out, None, xq, sx, xo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(outliers=None), -1), (dict(xq=None), -1), (dict(sx=None), -1), (dict(xo=None), -1),
    (dict(n_out=17), -4), (dict(n_out=-1), -4), (dict(eps=-1.0), -4), (dict(K=100), -2), (dict(xq=MIS), -3),
    (dict(xo=MIS), -3), (dict(sx=ODD), -3), (dict(outliers=ODD), -3),
    (dict(M=0, x=None, xq=None, sx=None, xo=None), 0),
])
def test_norm_int8_validation(lib, kw, status):
    assert norm8(lib, **kw) == status


def test_dequantize_validation(lib):
    f = lib.wq_dequantize_act_int8
    assert f(None, A, A, None, 0, 4, 256, A2, None) == -1
    assert f(A, A, None, A2, 2, 4, 256, A2, None) == -1
    assert f(A, A, A, None, 2, 4, 256, A2, None) == -1
    assert f(A, A, A, A2, 17, 4, 256, A2, None) == -4
    assert f(A, A, A, A2, 2, 4, 20, A2, None) == -2
    assert f(A, A, A, A2, 2, -1, 256, A2, None) == -2
    assert f(MIS, A, A, A2, 2, 4, 256, A2, None) == -3
    assert f(None, None, None, None, 0, 0, 256, None, None) == 0


def w4a8q(lib, xq=A, sx=A2, xo=A3, M=4, K=256, outliers=A, n_out=8, N=64, group=128, y=A2, y_dtype=0, ws=A,
          ws_bytes=1 << 20):
    return lib.wq_linear_w4a8_quantized(xq, sx, xo, M, K, outliers, n_out, A2, A3, A, N, group, y, y_dtype, ws,
                                        ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xq=None), -1), (dict(sx=None), -1), (dict(xo=None), -1), (dict(outliers=None), -1), (dict(y=None), -1),
    (dict(n_out=17), -4), (dict(group=64), -4), (dict(y_dtype=2), -4), (dict(K=200), -2), (dict(N=0), -2),
    (dict(xq=MIS), -3), (dict(xo=MIS), -3), (dict(ws=None), -6), (dict(ws_bytes=64 * 32 - 1), -6), (dict(ws=MIS), -3),
    (dict(M=0, xq=None, sx=None, xo=None, y=None, ws=None, ws_bytes=0), 0),
])
def test_w4a8_quantized_validation(lib, kw, status):
    assert w4a8q(lib, **kw) == status
    assert lib.wq_linear_w4a8_quantized_workspace_bytes(64) == 64 * 32
    assert lib.wq_linear_w4a8_quantized_workspace_bytes(0) == 0


# ---------------------------------------------------------------- cache
def test_page_bytes(lib):
    assert lib.wq_kv4_page_bytes(32, 128) == 32 * 136
    assert lib.wq_kv4_page_bytes(96, 64) == 96 * 72
    for bad in ((0, 128), (-32, 128), (16, 128), (33, 128), (64, 96), (64, 256), (64, 0), (1 << 40, 128)):
        assert lib.wq_kv4_page_bytes(*bad) == 0


def append(lib, k=A, ks=1024, v=A2, vs=1024, T=4, hkv=8, d=128, start=A, ctx=A2, B=2, max_new=4, table=A3,
           max_pages=4, cache=A, num_pages=10, page=64):
    return lib.wq_kv4_append(k, ks, v, vs, T, hkv, d, start, ctx, B, max_new, table, max_pages, cache, num_pages, page,
                             None)


SHARED = [
    (dict(start=None), -1), (dict(ctx=None), -1), (dict(table=None), -1), (dict(cache=None), -1),
    (dict(d=96), -4), (dict(d=0), -4), (dict(page=16), -4), (dict(page=0), -4), (dict(page=-64), -4),
    (dict(T=-1), -2), (dict(B=-1), -2), (dict(B=(1 << 20) + 1), -2), (dict(hkv=0), -2), (dict(num_pages=0), -2),
    (dict(num_pages=1 << 31), -2), (dict(max_pages=0), -2), (dict(max_pages=(1 << 24) + 1), -2),
    (dict(T=1 << 31), -2), (dict(start=ODD), -3), (dict(ctx=ODD), -3), (dict(table=ODD), -3), (dict(cache=MIS), -3),
    (dict(T=0), 0), (dict(B=0), 0),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(ks=1016), -2), (dict(vs=0), -2), (dict(max_new=-1), -2),
    (dict(hkv=65536, ks=1 << 30, vs=1 << 30), -2), (dict(ks=1028), -3), (dict(vs=1026), -3), (dict(k=MIS), -3),
    (dict(v=MIS), -3), (dict(T=0, k=None, v=None, start=None, ctx=None, table=None, cache=None), 0),
])
def test_append_validation(lib, kw, status):
    assert append(lib, **kw) == status


def read(lib, cache=A, num_pages=10, page=64, T=4, hkv=8, d=128, start=A, ctx=A2, B=2, max_new=4, table=A3,
         max_pages=4, k=A, v=A2):
    return lib.wq_kv4_read(cache, num_pages, page, T, hkv, d, start, ctx, B, max_new, table, max_pages, k, v, None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(max_new=-1), -2), (dict(k=MIS), -3), (dict(v=MIS), -3),
])
def test_read_validation(lib, kw, status):
    assert read(lib, **kw) == status


def attention(lib, q=A, qs=4096, T=4, hq=32, hkv=8, d=128, start=A, ctx=A2, B=4, max_q=1, max_ctx=100, table=A3,
              max_pages=4, cache=A, num_pages=10, page=64, scale=0.1, window=0, out=A, lse=None, ws=A, nbytes=1 << 40):
    return lib.wq_kv4_attention(q, qs, T, hq, hkv, d, start, ctx, B, max_q, max_ctx, table, max_pages, cache,
                                num_pages, page, scale, window, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(q=None), -1), (dict(out=None), -1), (dict(scale=0.0), -4), (dict(scale=-1.0), -4),
    (dict(scale=float("nan")), -4), (dict(scale=float("inf")), -4), (dict(hq=12), -2), (dict(hq=4), -2),
    (dict(qs=4088), -2), (dict(max_q=-1), -2), (dict(max_ctx=-1), -2), (dict(max_ctx=(1 << 30) + 1), -2),
    (dict(window=-1), -2), (dict(window=1 << 31), -2), (dict(q=MIS), -3), (dict(qs=4097), -3), (dict(out=ODD), -3),
    (dict(lse=ODD), -3), (dict(max_ctx=100000, ws=None), -6), (dict(max_ctx=100000, nbytes=16), -6),
    (dict(max_ctx=100000, ws=MIS), -3),
])
def test_attention_validation(lib, kw, status):
    assert attention(lib, **kw) == status


def test_grid_and_work_limits(lib):
    """Batch times heads stays below 2^24 (a grid has 2^32 threads), and the tokens that
    all rows may see within 64-bit sums."""
    assert append(lib, B=1 << 19, hkv=32, ks=4096, vs=4096) == -2
    assert read(lib, B=1 << 19, hkv=32) == -2
    assert attention(lib, B=1 << 19) == -2
    assert lib.wq_kv4_attention_workspace_bytes(4, 1 << 19, 32, 8, 128, 1, 100) == 0
    assert lib.wq_kv4_attention_workspace_bytes(4, (1 << 19) - 1, 32, 8, 128, 1, 100) > 0
    assert attention(lib, T=1 << 24, hq=64, qs=8192, hkv=1, max_pages=1 << 24) == -2


def test_attention_workspace(lib):
    f = lib.wq_kv4_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128, 1, 32) == 0                 # one tile: nothing to split
    a = f(1, 1, 32, 8, 128, 1, 100000)
    assert 0 < a < 1 << 26
    # a longer bound never needs less, so one workspace serves every shorter batch
    for T, B, hq, hkv, d, q in ((1, 1, 32, 8, 128, 1), (16, 16, 32, 32, 128, 1), (40, 8, 28, 4, 64, 5),
                                (700, 3, 32, 8, 128, 600), (2048, 1, 64, 8, 128, 2048)):
        last = 0
        for ctx in range(0, 20000, 97):
            n = f(T, B, hq, hkv, d, q, ctx)
            assert n >= last
            last = n
    for bad in ((0, 1, 8, 8, 128, 1, 10), (1, 0, 8, 8, 128, 1, 10), (1, 1, 9, 8, 128, 1, 10), (1, 1, 8, 8, 96, 1, 10),
                (1, 1, 8, 8, 128, -1, 10), (1, 1, 8, 8, 128, 1, -1), (1, 1, 4, 8, 128, 1, 10)):
        assert f(*bad) == 0


def test_binding_refuses_host_tensors_and_shapes(lib):
    import torch
    x = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        wq.add_rmsnorm(x, x[0])
    with pytest.raises(TypeError):
        wq.kv4_append(x.view(2, 1, 64), x.view(2, 1, 64), x, x, x, x)
    with pytest.raises(ValueError):
        wq.kv4_cache(4, 48, 2, 128)
    with pytest.raises(ValueError):
        wq.kv4_cache(4, 64, 2, 80)
    assert wq.kv4_page_bytes(64, 80) == 0


# ---------------------------------------------------------------- the oracle's pins
def test_oracle_quantizer_pins():
    # values on the grid -7.. 8 in steps of 0.5 come back exactly; range 7.5, s = 0.5, z = 7
    x = (np.arange(16) - 7).astype(np.float16) * np.float16(0.5)
    q, s, z = oracle.kv4_quantize(x[None])
    assert s[0] == np.float16(0.5) and z[0] == 7 and np.array_equal(q[0], np.arange(16))
    assert np.array_equal(oracle.kv4_values(x[None])[0], x.astype(np.float64))
    # all positive: the range is widened to 0, z = 0
    q, s, z = oracle.kv4_quantize(np.full((1, 64), 3.0, np.float16))
    assert z[0] == 0 and np.all(q == 15) and abs(float(s[0]) - 0.2) < 1e-4
    # zeros hold 0, at the smallest scale
    q, s, z = oracle.kv4_quantize(np.zeros((1, 64), np.float16))
    assert s[0] == np.float16(2.0 ** -14) and np.all(oracle.kv4_values(np.zeros((1, 64), np.float16)) == 0)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)).astype(np.float16)
    _, s, _ = oracle.kv4_quantize(x)
    assert np.all(np.abs(oracle.kv4_values(x) - x) <= 0.51 * s.astype(np.float64)[:, None] + 16 * 2.0 ** -11 * s.astype(np.float64)[:, None])


def test_oracle_attention_pins():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((3, 4, 64))
    k, v = rng.standard_normal((2, 7, 2, 64))
    out, lse, _ = oracle.kv4_attention(q, k, v)
    for i in range(3):
        for h in range(4):
            w = np.array([np.exp(q[i, h] @ k[t, h // 2] / 8) for t in range(5 + i)])
            assert np.allclose(out[i, h], (w[:, None] * v[:5 + i, h // 2]).sum(0) / w.sum())
            assert np.isclose(lse[i, h], np.log(w.sum()))
    # a window of one: each row its own value; fewer tokens than rows: empty rows first
    out, lse, _ = oracle.kv4_attention(q, k, v, window=1)
    assert np.allclose(out[:, 0], v[4:, 0])
    out, lse, _ = oracle.kv4_attention(q, k[:1], v[:1])
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.allclose(out[2, 0], v[0, 0])


def test_oracle_norm_pins():
    x = np.array([[3.0, 4.0]])
    y, h = oracle.add_rmsnorm(x, np.array([1.0, 2.0]), eps=0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]) and np.array_equal(h, x)
    q, s = oracle.norm_int8(np.array([[1.0, -254.0, 1000.0], [0.0, 0.0, 5.0]]), [2])
    assert np.allclose(s, [2.0, 1.0]) and np.allclose(q, [[0.5, -127.0, 0.0], [0, 0, 0]])
