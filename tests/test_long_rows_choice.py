"""Which kernel AUTO takes where a row is so long that the decode kernels' scales and zero-points do not fit their LDS."""
from test_kv4_abi import lib  # noqa: F401

GEMV, GEMM = 1, 2


def test_long_rows(lib):  # noqa: F811
    # 16 rows of (s, z) pairs of K / 128 groups, four bytes each, beside four waves' slots
    for M in (1, 2, 5, 16):
        assert lib.wq_auto_kernel(M, 64, 28672) == GEMV
        assert lib.wq_auto_kernel(M, 64, 262144) == GEMV
        assert lib.wq_auto_kernel(M, 64, 1 << 19) == GEMM
    for M in (17, 64, 65):
        assert lib.wq_auto_kernel(M, 64, 1 << 19) == GEMM
