"""Python binding of libwq.so, the gfx950 W4A16 group-quantized linear.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind include/wq.h.  PyTorch provides device memory and the current
stream.  There is no fallback: if the library is missing, every call raises.

Entry points (the same names as the C ABI, without the ``wq_`` prefix):

* ``quantize_rtn(W, sparse_k)``  split + RTN INT4 group quantization
* ``pack(codes)``                eight codes per 32-bit word
* ``linear(x, packed, scales, zeros)``
* ``linear_sparse(x, packed, scales, zeros, row_ptr, col, val)``
* ``linear_lowrank(x, packed, scales, zeros, L1, L2, row_ptr, col, val)``
  the same plus a rank-r fp16 branch (x . L1^T) . L2^T
* ``quantize_rtn_act_order(W, perm)``, ``linear_act_order(x, perm, ...)``
  act-order layers, kept in the permuted channel order
* ``quantize_act_int8(x, outliers)``, ``linear_w4a8(x, outliers, ...)``
  INT8 activations with fp16 outlier channels on the same INT4 layer
* ``add_rmsnorm(x, weight, residual)``, ``add_rmsnorm_int8(...)``
  root-mean-square norm of x + residual, in fp16 or as the INT8 activations of
  ``linear_w4a8_quantized``; ``dequantize_act_int8`` gives their values
* ``kv4_cache(...)``, ``kv4_append(k, v, cache, ...)``, ``kv4_read(cache, ...)``,
  ``kv4_attention(q, cache, ...)``
  a paged key/value cache in 4 bits and causal attention over it
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libwq.so")
GROUP = 128

WQ_OK = 0
STATUS = {0: "WQ_OK", -1: "WQ_ERR_NULL", -2: "WQ_ERR_SHAPE", -3: "WQ_ERR_ALIGN",
          -4: "WQ_ERR_UNSUPPORTED", -5: "WQ_ERR_HIP", -6: "WQ_ERR_WORKSPACE", -7: "WQ_ERR_SCRATCH"}
KERNELS = {"auto": 0, "gemv": 1, "gemm": 2, "gemv_mfma": 3}

# name -> (restype, argtypes) for every symbol declared in include/wq.h
_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
SIGNATURES = {
    "wq_quantize_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "wq_quantize_rtn": (ctypes.c_int, [_vp, _i64, _i64, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "wq_quantize_rtn_bits": (ctypes.c_int, [_vp, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                            _sz, _vp]),
    "wq_pack": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp]),
    "wq_pack_bits": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "wq_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "wq_linear": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i32, _vp, _i32, _vp, _sz, _vp]),
    "wq_linear_sparse": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64,
                                        _vp, _i32, _vp, _sz, _vp]),
    "wq_linear_sparse_bits": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64,
                                             _vp, _i32, _i32, _vp, _sz, _vp]),
    "wq_linear_sparse_kernel": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64,
                                               _vp, _i32, _i32, _vp, _sz, _vp]),
    "wq_linear_lowrank_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "wq_linear_lowrank": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64,
                                         _vp, _vp, _i64, _vp, _i32, _i32, _vp, _sz, _vp]),
    "wq_quantize_act_order_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "wq_quantize_rtn_act_order": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                                 _vp, _sz, _vp]),
    "wq_linear_act_order_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "wq_linear_act_order": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64,
                                           _vp, _i32, _i32, _vp, _sz, _vp]),
    "wq_quantize_act_int8": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "wq_linear_w4a8_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "wq_linear_w4a8": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _vp, _i32, _vp, _sz,
                                      _vp]),
    "wq_linear_w4a8_quantized_workspace_bytes": (_sz, [_i64]),
    "wq_linear_w4a8_quantized": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _vp,
                                                _i32, _vp, _sz, _vp]),
    "wq_add_rmsnorm": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, ctypes.c_float, _vp, _vp, _vp]),
    "wq_add_rmsnorm_int8": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, ctypes.c_float, _vp, _i64, _vp, _vp, _vp, _vp,
                                           _vp]),
    "wq_dequantize_act_int8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]),
    "wq_kv4_page_bytes": (_sz, [_i64, _i64]),
    "wq_kv4_append": (ctypes.c_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp,
                                     _i64, _i64, _vp]),
    "wq_kv4_read": (ctypes.c_int, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp,
                                   _vp]),
    "wq_kv4_attention_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i64, _i64, _i64]),
    "wq_kv4_attention_plan": (ctypes.c_int, [_i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64]),
    "wq_kv4_attention": (ctypes.c_int, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp,
                                        _i64, _i64, ctypes.c_float, _i64, _vp, _vp, _vp, _sz, _vp]),
    "wq_linear_sparse_noalloc": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64,
                                                _vp, _i32, _vp]),
    "wq_auto_kernel": (ctypes.c_int, [_i64, _i64, _i64]),
    "wq_last_hip_error": (ctypes.c_int, []),
    "wq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}

_lib = None


class WQError(RuntimeError):
    def __init__(self, fn, status, lib):
        msg = lib.wq_status_string(status).decode() if lib is not None else ""
        super().__init__(f"{fn} returned {STATUS.get(status, status)}: {msg}")
        self.status = status


def load():
    """Load libwq.so (built by ``python -m quantized_gemm_rtn_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m quantized_gemm_rtn_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _check(fn, rc):
    if rc != WQ_OK:
        raise WQError(fn, rc, _lib)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    import torch
    # the current stream's handle; a Stream object around it would cost 2 us a call
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _need(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace_bytes(workspace, like):
    """Bytes of a workspace that the GPU will write: a whole piece of the inputs' device."""
    if workspace is None:
        return 0
    try:
        here = workspace.get_device() == like.get_device()
    except AttributeError:
        here = False
    if not here:
        raise TypeError("workspace must be a tensor on the inputs' device")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.nbytes


def quantize_workspace_bytes(N, K, sparse_k):
    return int(load().wq_quantize_workspace_bytes(N, K, sparse_k))


def quantize_rtn(W, sparse_k: int = 0, group: int = GROUP, workspace=None, bits: int = 4):
    """Dense-and-sparse split and RTN INT4 quantization of ``W`` (float32 [N, K]).

    ``group``: 128, a larger multiple of 128 dividing K, or -1 (one group per
    row); ``bits``: 2 to 4 (codes of fewer bits in the same 4-bit packing). Returns a dict with ``codes`` uint8 [N, K], ``scales``/``zeros``
    float16 [N, K/128] (a coarser group's values repeated in each of its
    128-channel slots), and the sparse part ``row_ptr`` int32 [N+1], ``col``
    int32 [sparse_k], ``val`` float16 [sparse_k]."""
    import torch
    lib = load()
    _need(W, torch.float32, "W")
    N, K = W.shape
    dev = W.device
    # metadata slots per row: one per 64 channels for group 64, else one per 128
    G = K // 64 if group == 64 else K // GROUP
    codes = torch.empty((N, K), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, max(G, 1)), dtype=torch.float16, device=dev)
    zeros = torch.empty((N, max(G, 1)), dtype=torch.float16, device=dev)
    row_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(sparse_k, 1), dtype=torch.int32, device=dev)
    val = torch.empty(max(sparse_k, 1), dtype=torch.float16, device=dev)
    nbytes = int(lib.wq_quantize_workspace_bytes(N, K, sparse_k))
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    rc = lib.wq_quantize_rtn_bits(_p(W), N, K, group, bits, sparse_k, _p(codes), _p(scales), _p(zeros),
                                  _p(row_ptr), _p(col), _p(val), _p(workspace), _workspace_bytes(workspace, W),
                                  _stream(W))
    _check("wq_quantize_rtn_bits", rc)
    return dict(codes=codes, scales=scales[:, :G], zeros=zeros[:, :G], row_ptr=row_ptr,
                col=col[:sparse_k], val=val[:sparse_k])


def pack(codes, bits: int = 4):
    """Eight INT4 codes per 32-bit word, or (bits = 3) 32 3-bit codes per three
    words (returned as int32 bit patterns, [N, K/8] or [N, 3K/32])."""
    import torch
    lib = load()
    _need(codes, torch.uint8, "codes")
    N, K = codes.shape
    width = K // 8 if bits == 4 else 3 * K // 32
    packed = torch.empty((N, width), dtype=torch.int32, device=codes.device)
    _check("wq_pack_bits", lib.wq_pack_bits(_p(codes), N, K, bits, _p(packed), _stream(codes)))
    return packed


def _layer_format(packed, scales, K, N):
    """(bits, group) of a layer from its tensors' shapes: [N, K/8] words are 4-bit
    codes and [N, 3K/32] 3-bit ones; [N, K/128] metadata is group 128, [N, K/64]
    group 64."""
    if packed.shape[0] != N:
        raise ValueError("inconsistent shapes")
    if packed.shape[1] * 8 == K:
        bits = 4
    elif K % 32 == 0 and packed.shape[1] == 3 * K // 32:
        bits = 3
    else:
        raise ValueError("packed must be [N, K/8] (4-bit) or [N, 3K/32] (3-bit)")
    if tuple(scales.shape) == (N, K // GROUP):
        group = GROUP
    elif tuple(scales.shape) == (N, K // 64):
        group = 64
    else:
        raise ValueError("scales must be [N, K/128] or [N, K/64]")
    return bits, group


def linear_workspace_bytes(M, N, K):
    return int(load().wq_linear_workspace_bytes(M, N, K))


def linear_sparse(x, packed, scales, zeros, row_ptr=None, col=None, val=None, out_dtype=None,
                  kernel: str = "auto", out=None, workspace=None):
    """y = x . dequant(packed, scales, zeros)^T (+ W_sparse x when CSR is given).

    The layer's format follows from the shapes: 4-bit ([N, K/8] words) or 3-bit
    ([N, 3K/32]) codes, one (s, z) per 128 ([N, K/128]) or 64 ([N, K/64]) input
    channels. ``workspace`` (uint8 device tensor of ``linear_workspace_bytes``
    bytes) lets the GEMM split K; when omitted, one is allocated per call."""
    import torch
    lib = load()
    out_dtype = torch.float16 if out_dtype is None else out_dtype
    _need(x, torch.float16, "x")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    _need(zeros, torch.float16, "zeros")
    M, K = x.shape
    N = packed.shape[0]
    bits, group = _layer_format(packed, scales, K, N)
    if zeros.shape != scales.shape:
        raise ValueError("inconsistent shapes")
    nnz = 0
    if row_ptr is not None:
        _need(row_ptr, torch.int32, "row_ptr")
        if row_ptr.numel() != N + 1:
            raise ValueError("row_ptr must have N+1 entries")
        nnz = int(col.numel()) if col is not None else 0
        if nnz:
            _need(col, torch.int32, "col")
            _need(val, torch.float16, "val")
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _need(out, out_dtype, "out")
    y_dtype = 1 if out_dtype == torch.float32 else 0
    if workspace is None:
        nbytes = int(lib.wq_linear_workspace_bytes(M, N, K))
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    wbytes = _workspace_bytes(workspace, x)
    rc = lib.wq_linear_sparse_bits(_p(x), M, K, _p(packed), bits, _p(scales), _p(zeros), N, group,
                                   _p(row_ptr), _p(col) if nnz else None, _p(val) if nnz else None, nnz,
                                   _p(out), y_dtype, KERNELS[kernel], _p(workspace), wbytes, _stream(x))
    _check("wq_linear_sparse_bits", rc)
    return out


def linear_sparse_noalloc(x, packed, scales, zeros, out, row_ptr=None, col=None, val=None, group: int = GROUP):
    """``linear_sparse`` through ``wq_linear_sparse_noalloc``: no workspace, the
    library's per-GPU scratch instead; ``out`` (float16 or float32 [M, N]) must be
    given, so the call allocates nothing."""
    import torch
    lib = load()
    _need(x, torch.float16, "x")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    _need(zeros, torch.float16, "zeros")
    M, K = x.shape
    N = packed.shape[0]
    if packed.shape[1] * 8 != K or scales.shape != (N, K // group) or zeros.shape != scales.shape:
        raise ValueError("inconsistent shapes")
    if out.dtype not in (torch.float16, torch.float32):
        raise TypeError("out must be float16 or float32")
    _need(out, out.dtype, "out")
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    nnz = 0
    if row_ptr is not None:
        _need(row_ptr, torch.int32, "row_ptr")
        if row_ptr.numel() != N + 1:
            raise ValueError("row_ptr must have N+1 entries")
        nnz = int(col.numel()) if col is not None else 0
        if nnz:
            _need(col, torch.int32, "col")
            _need(val, torch.float16, "val")
    rc = lib.wq_linear_sparse_noalloc(_p(x), M, K, _p(packed), _p(scales), _p(zeros), N, group, _p(row_ptr),
                                      _p(col) if nnz else None, _p(val) if nnz else None, nnz, _p(out),
                                      1 if out.dtype == torch.float32 else 0, _stream(x))
    _check("wq_linear_sparse_noalloc", rc)
    return out


def last_hip_error() -> int:
    """hipError_t of this thread's last launch that failed inside the library (0 if none)."""
    return int(load().wq_last_hip_error())


def linear(x, packed, scales, zeros, out_dtype=None, kernel: str = "auto", out=None, workspace=None):
    return linear_sparse(x, packed, scales, zeros, None, None, None, out_dtype, kernel, out, workspace)


def linear_lowrank_workspace_bytes(M, N, K, r):
    return int(load().wq_linear_lowrank_workspace_bytes(M, N, K, r))


def linear_lowrank(x, packed, scales, zeros, L1, L2, row_ptr=None, col=None, val=None, out_dtype=None,
                   kernel: str = "auto", out=None, group: int = GROUP, workspace=None):
    """y = x . dequant(packed, scales, zeros)^T (+ W_sparse x when CSR is given)
    + (x . L1^T) . L2^T, with L1 [r, K] and L2 [N, r] fp16 (r a multiple of 32).

    ``workspace`` (uint8 device tensor of ``linear_lowrank_workspace_bytes``
    bytes) is allocated per call when omitted."""
    import torch
    lib = load()
    out_dtype = torch.float16 if out_dtype is None else out_dtype
    _need(x, torch.float16, "x")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    _need(zeros, torch.float16, "zeros")
    _need(L1, torch.float16, "L1")
    _need(L2, torch.float16, "L2")
    M, K = x.shape
    N = packed.shape[0]
    r = L1.shape[0]
    if packed.shape[1] * 8 != K or scales.shape != (N, K // group) or zeros.shape != scales.shape:
        raise ValueError("inconsistent shapes")
    if L1.shape != (r, K) or L2.shape != (N, r):
        raise ValueError("L1 must be [r, K] and L2 [N, r]")
    nnz = 0
    if row_ptr is not None:
        _need(row_ptr, torch.int32, "row_ptr")
        if row_ptr.numel() != N + 1:
            raise ValueError("row_ptr must have N+1 entries")
        nnz = int(col.numel()) if col is not None else 0
        if nnz:
            _need(col, torch.int32, "col")
            _need(val, torch.float16, "val")
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _need(out, out_dtype, "out")
    y_dtype = 1 if out_dtype == torch.float32 else 0
    if workspace is None:
        nbytes = int(lib.wq_linear_lowrank_workspace_bytes(max(M, 1), N, K, r))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    wbytes = _workspace_bytes(workspace, x)
    rc = lib.wq_linear_lowrank(_p(x), M, K, _p(packed), _p(scales), _p(zeros), N, group,
                               _p(row_ptr) if nnz else None, _p(col) if nnz else None, _p(val) if nnz else None,
                               nnz, _p(L1), _p(L2), r, _p(out), y_dtype, KERNELS[kernel], _p(workspace), wbytes,
                               _stream(x))
    _check("wq_linear_lowrank", rc)
    return out


def quantize_rtn_act_order(W, perm, sparse_k: int = 0, group: int = GROUP, workspace=None):
    """``quantize_rtn`` of ``W[:, perm]`` (``perm`` int32 [K], a permutation): the
    layer of an act-order quantization, kept in the permuted channel order (its
    CSR columns are positions in that order). Same return value as
    ``quantize_rtn``."""
    import torch
    lib = load()
    _need(W, torch.float32, "W")
    _need(perm, torch.int32, "perm")
    N, K = W.shape
    if perm.numel() != K:
        raise ValueError("perm must have K entries")
    dev = W.device
    G = K // GROUP
    codes = torch.empty((N, K), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, max(G, 1)), dtype=torch.float16, device=dev)
    zeros = torch.empty((N, max(G, 1)), dtype=torch.float16, device=dev)
    row_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(sparse_k, 1), dtype=torch.int32, device=dev)
    val = torch.empty(max(sparse_k, 1), dtype=torch.float16, device=dev)
    nbytes = int(lib.wq_quantize_act_order_workspace_bytes(N, K, sparse_k))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    wbytes = _workspace_bytes(workspace, W)
    rc = lib.wq_quantize_rtn_act_order(_p(W), N, K, group, _p(perm), sparse_k, _p(codes), _p(scales), _p(zeros),
                                       _p(row_ptr), _p(col), _p(val), _p(workspace), wbytes, _stream(W))
    _check("wq_quantize_rtn_act_order", rc)
    return dict(codes=codes, scales=scales[:, :G], zeros=zeros[:, :G], row_ptr=row_ptr,
                col=col[:sparse_k], val=val[:sparse_k])


def linear_act_order_workspace_bytes(M, N, K):
    return int(load().wq_linear_act_order_workspace_bytes(M, N, K))


def linear_act_order(x, perm, packed, scales, zeros, row_ptr=None, col=None, val=None, out_dtype=None,
                     kernel: str = "auto", out=None, group: int = GROUP, workspace=None):
    """y = x . W^T for a layer kept in permuted channel order (``perm`` int32
    [K]; from ``quantize_rtn_act_order``): x, in the original order, has its
    columns gathered through ``perm`` and then meets the layer as in
    ``linear_sparse``."""
    import torch
    lib = load()
    out_dtype = torch.float16 if out_dtype is None else out_dtype
    _need(x, torch.float16, "x")
    _need(perm, torch.int32, "perm")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    _need(zeros, torch.float16, "zeros")
    M, K = x.shape
    N = packed.shape[0]
    if perm.numel() != K or packed.shape[1] * 8 != K or scales.shape != (N, K // group) or \
            zeros.shape != scales.shape:
        raise ValueError("inconsistent shapes")
    nnz = 0
    if row_ptr is not None:
        _need(row_ptr, torch.int32, "row_ptr")
        if row_ptr.numel() != N + 1:
            raise ValueError("row_ptr must have N+1 entries")
        nnz = int(col.numel()) if col is not None else 0
        if nnz:
            _need(col, torch.int32, "col")
            _need(val, torch.float16, "val")
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _need(out, out_dtype, "out")
    y_dtype = 1 if out_dtype == torch.float32 else 0
    if workspace is None:
        nbytes = int(lib.wq_linear_act_order_workspace_bytes(max(M, 1), N, K))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    wbytes = _workspace_bytes(workspace, x)
    rc = lib.wq_linear_act_order(_p(x), M, K, _p(perm), _p(packed), _p(scales), _p(zeros), N, group,
                                 _p(row_ptr) if row_ptr is not None else None, _p(col) if nnz else None,
                                 _p(val) if nnz else None, nnz, _p(out), y_dtype, KERNELS[kernel], _p(workspace),
                                 wbytes, _stream(x))
    _check("wq_linear_act_order", rc)
    return out


def quantize_act_int8(x, outliers):
    """Per-row INT8 activations with fp16 outlier channels (``outliers`` int32
    [n_out], n_out <= 16): returns ``xq`` int8 [M, K] in the products' byte order,
    ``sx`` float32 [M] and ``xo`` float16 [M, 16]."""
    import torch
    lib = load()
    _need(x, torch.float16, "x")
    _need(outliers, torch.int32, "outliers")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    sx = torch.empty(max(M, 1), dtype=torch.float32, device=x.device)
    xo = torch.empty((max(M, 1), 16), dtype=torch.float16, device=x.device)
    n_out = outliers.numel()
    _check("wq_quantize_act_int8", lib.wq_quantize_act_int8(_p(x), M, K, _p(outliers) if n_out else None, n_out,
                                                            _p(xq), _p(sx), _p(xo), _stream(x)))
    return xq, sx[:M], xo[:M]


def linear_w4a8_workspace_bytes(M, N, K):
    return int(load().wq_linear_w4a8_workspace_bytes(M, N, K))


def linear_w4a8(x, outliers, packed, scales, zeros, out_dtype=None, out=None, group: int = GROUP, workspace=None):
    """y = W4A8 product with fp16 outlier channels (``outliers`` int32 [n_out],
    n_out <= 16): the INT8 activations are made per call."""
    import torch
    lib = load()
    out_dtype = torch.float16 if out_dtype is None else out_dtype
    _need(x, torch.float16, "x")
    _need(outliers, torch.int32, "outliers")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    _need(zeros, torch.float16, "zeros")
    M, K = x.shape
    N = packed.shape[0]
    if packed.shape[1] * 8 != K or scales.shape != (N, K // group) or zeros.shape != scales.shape:
        raise ValueError("inconsistent shapes")
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _need(out, out_dtype, "out")
    if workspace is None:
        nbytes = int(lib.wq_linear_w4a8_workspace_bytes(max(M, 1), N, K))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    wbytes = _workspace_bytes(workspace, x)
    n_out = outliers.numel()
    rc = lib.wq_linear_w4a8(_p(x), M, K, _p(outliers) if n_out else None, n_out, _p(packed), _p(scales), _p(zeros),
                            N, group, _p(out), 1 if out_dtype == torch.float32 else 0, _p(workspace), wbytes,
                            _stream(x))
    _check("wq_linear_w4a8", rc)
    return out


def linear_w4a8_quantized(xq, sx, xo, outliers, packed, scales, zeros, out_dtype=None, out=None, group: int = GROUP,
                          workspace=None):
    """``linear_w4a8`` of activations that are already INT8: ``xq``, ``sx``, ``xo`` from
    ``quantize_act_int8`` or ``add_rmsnorm_int8`` with the same ``outliers``."""
    import torch
    lib = load()
    out_dtype = torch.float16 if out_dtype is None else out_dtype
    _need(xq, torch.int8, "xq")
    _need(sx, torch.float32, "sx")
    _need(xo, torch.float16, "xo")
    _need(outliers, torch.int32, "outliers")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    _need(zeros, torch.float16, "zeros")
    M, K = xq.shape
    N = packed.shape[0]
    if packed.shape[1] * 8 != K or scales.shape != (N, K // group) or zeros.shape != scales.shape:
        raise ValueError("inconsistent shapes")
    if sx.numel() != M or tuple(xo.shape) != (M, 16):
        raise ValueError("sx must be [M] and xo [M, 16]")
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    else:
        _need(out, out_dtype, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    if workspace is None:
        workspace = torch.empty(int(lib.wq_linear_w4a8_quantized_workspace_bytes(N)), dtype=torch.uint8,
                                device=xq.device)
    wbytes = _workspace_bytes(workspace, xq)
    n_out = outliers.numel()
    rc = lib.wq_linear_w4a8_quantized(_p(xq), _p(sx), _p(xo), M, K, _p(outliers) if n_out else None, n_out,
                                      _p(packed), _p(scales), _p(zeros), N, group, _p(out),
                                      1 if out_dtype == torch.float32 else 0, _p(workspace), wbytes, _stream(xq))
    _check("wq_linear_w4a8_quantized", rc)
    return out


def _norm_args(x, weight, residual, h):
    import torch
    _need(x, torch.float16, "x")
    _need(weight, torch.float16, "weight")
    M, K = x.shape
    if weight.numel() != K:
        raise ValueError("weight must have K entries")
    for t, name in ((residual, "residual"), (h, "h")):
        if t is not None:
            _need(t, torch.float16, name)
            if t.shape != x.shape:
                raise ValueError(f"{name} must have the shape of x")
    # the sum is only written where there is something to add, or a place for it is given
    return M, K, torch.empty_like(x) if h is None and residual is not None else h


def add_rmsnorm(x, weight, residual=None, eps: float = 1e-5, out=None, h=None):
    """Root-mean-square norm of ``x + residual`` (float16 [M, K]): returns ``(y, h)``,
    y = h / sqrt(mean(h^2) + eps) * weight and h the sum, the next block's residual
    (``x`` itself when ``residual`` is None). ``h`` may be ``x`` or ``residual``, to
    update it in place."""
    import torch
    lib = load()
    M, K, h = _norm_args(x, weight, residual, h)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, torch.float16, "out")
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    _check("wq_add_rmsnorm", lib.wq_add_rmsnorm(_p(x), _p(residual), _p(weight), M, K, eps, _p(h), _p(out),
                                                _stream(x)))
    return out, x if h is None else h


def add_rmsnorm_int8(x, weight, residual=None, eps: float = 1e-5, outliers=None, h=None):
    """``add_rmsnorm`` with its output in 8 bits, as ``linear_w4a8_quantized`` reads it:
    returns ``(xq, sx, xo, h)``, int8 [M, K] in the products' byte order, one float32
    scale per row, and the float16 values [M, 16] of the ``outliers`` channels (int32,
    at most 16)."""
    import torch
    lib = load()
    M, K, h = _norm_args(x, weight, residual, h)
    n_out = 0
    if outliers is not None:
        _need(outliers, torch.int32, "outliers")
        n_out = outliers.numel()
    xq = torch.empty_like(x, dtype=torch.int8)
    sx = x.new_empty(M, dtype=torch.float32)
    xo = x.new_empty((M, 16))
    rc = lib.wq_add_rmsnorm_int8(_p(x), _p(residual), _p(weight), M, K, eps, _p(outliers) if n_out else None, n_out,
                                 _p(h), _p(xq), _p(sx), _p(xo), _stream(x))
    _check("wq_add_rmsnorm_int8", rc)
    return xq, sx, xo, x if h is None else h


def dequantize_act_int8(xq, sx, xo=None, outliers=None):
    """The float16 values [M, K] that INT8 activations stand for, in channel order."""
    import torch
    lib = load()
    _need(xq, torch.int8, "xq")
    _need(sx, torch.float32, "sx")
    M, K = xq.shape
    n_out = 0 if outliers is None else outliers.numel()
    if n_out:
        _need(outliers, torch.int32, "outliers")
        _need(xo, torch.float16, "xo")
    if sx.numel() != M or (n_out and tuple(xo.shape) != (M, 16)):
        raise ValueError("sx must be [M] and xo [M, 16]")
    out = torch.empty_like(xq, dtype=torch.float16)
    rc = lib.wq_dequantize_act_int8(_p(xq), _p(sx), _p(xo) if n_out else None, _p(outliers) if n_out else None, n_out,
                                    M, K, _p(out), _stream(xq))
    _check("wq_dequantize_act_int8", rc)
    return out


def kv4_page_bytes(page_tokens, head_dim):
    return int(load().wq_kv4_page_bytes(page_tokens, head_dim))


def kv4_cache(num_pages: int, page_tokens: int, kv_heads: int, head_dim: int, device="cuda"):
    """An empty 4-bit key/value cache: uint8 [num_pages, kv_heads, page bytes], for pages
    of ``page_tokens`` tokens (a multiple of 32) and ``head_dim`` 64 or 128."""
    import torch
    nbytes = kv4_page_bytes(page_tokens, head_dim)
    if nbytes == 0:
        raise ValueError("page_tokens must be a multiple of 32 and head_dim 64 or 128")
    return torch.empty((num_pages, kv_heads, nbytes), dtype=torch.uint8, device=device)


def _rows(t, name, heads, head_dim):
    """Elements between the tokens of ``t`` [T, heads, head_dim], whose heads must be
    contiguous (a slice of a wider projection's output is)."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be {torch.float16}, got {t.dtype}")
    tokens, h, d = t.shape if t.dim() == 3 else (0, 0, 0)
    if h != heads or d != head_dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {head_dim}]")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != head_dim and heads > 1):
        raise ValueError(f"{name}: each token's heads must be contiguous")
    return s0 if tokens > 1 else heads * head_dim


def _kv4_view(cache, page_table, seq_start, ctx_len, head_dim):
    """(B, max_pages, num_pages, page_tokens, kv_heads) of a batch and its cache."""
    import torch
    _need(cache, torch.uint8, "cache")
    _need(page_table, torch.int32, "page_table")
    _need(seq_start, torch.int32, "seq_start")
    _need(ctx_len, torch.int32, "ctx_len")
    if cache.dim() != 3:
        raise ValueError("cache must be [num_pages, kv_heads, page bytes], as kv4_cache makes it")
    num_pages, kv_heads, nbytes = cache.shape
    B = ctx_len.numel()
    tile = kv4_page_bytes(32, head_dim)
    if tile == 0 or nbytes == 0 or nbytes % tile:
        raise ValueError(f"the cache's pages of {nbytes} bytes do not hold whole tiles of head_dim {head_dim}")
    if seq_start.numel() != B + 1:
        raise ValueError("seq_start must have one entry more than ctx_len")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, pages]")
    return B, page_table.shape[1], num_pages, nbytes // tile * 32, kv_heads


def kv4_append(k, v, cache, page_table, seq_start, ctx_len, max_new=None):
    """Quantizes new tokens' keys and values (float16 [T, kv_heads, head_dim]; slices of a
    wider projection's output are fine) into ``cache``.

    Sequence b's tokens are the rows ``seq_start[b]`` to ``seq_start[b + 1]`` (int32
    [B + 1]), the last of its ``ctx_len[b]`` (int32 [B]) tokens; token t is in page
    ``page_table[b, t // page_tokens]`` (int32 [B, pages]). ``max_new``: the most new
    tokens of a sequence, if known (it shapes the launch only)."""
    lib = load()
    T, head_dim = k.shape[0], k.shape[-1]
    B, max_pages, num_pages, page_tokens, kv_heads = _kv4_view(cache, page_table, seq_start, ctx_len, head_dim)
    ks, vs = _rows(k, "k", kv_heads, head_dim), _rows(v, "v", kv_heads, head_dim)
    if v.shape[0] != T:
        raise ValueError("k and v must have the same tokens")
    rc = lib.wq_kv4_append(_p(k), ks, _p(v), vs, T, kv_heads, head_dim, _p(seq_start), _p(ctx_len), B,
                           T if max_new is None else max_new, _p(page_table), max_pages, _p(cache), num_pages,
                           page_tokens, _stream(k))
    _check("wq_kv4_append", rc)


def kv4_read(cache, page_table, seq_start, ctx_len, tokens: int, head_dim: int, max_new=None):
    """The keys and values of each sequence's last tokens as ``cache`` holds them: float16
    [tokens, kv_heads, head_dim] each, rows as in ``kv4_append`` (those of no sequence are
    not written)."""
    import torch
    lib = load()
    B, max_pages, num_pages, page_tokens, kv_heads = _kv4_view(cache, page_table, seq_start, ctx_len, head_dim)
    k = cache.new_empty((tokens, kv_heads, head_dim), dtype=torch.float16)
    v = torch.empty_like(k)
    rc = lib.wq_kv4_read(_p(cache), num_pages, page_tokens, tokens, kv_heads, head_dim, _p(seq_start), _p(ctx_len), B,
                         tokens if max_new is None else max_new, _p(page_table), max_pages, _p(k), _p(v),
                         _stream(cache))
    _check("wq_kv4_read", rc)
    return k, v


def kv4_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim, max_q, max_ctx):
    return int(load().wq_kv4_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim, max_q, max_ctx))


def kv4_attention_plan(T, B, q_heads, kv_heads, head_dim, max_q, max_ctx, window: int = 0) -> dict:
    """What ``kv4_attention`` launches for these sizes: ``few_rows`` and ``many_rows``, its two
    kernels, ``shares`` (many rows dealt out in equal shares), and ``join_waves``, the waves
    that join a row of split sequences (0 for none)."""
    p = load().wq_kv4_attention_plan(T, B, q_heads, kv_heads, head_dim, max_q, max_ctx, window)
    if p == 0:
        raise ValueError("invalid sizes")
    return {"few_rows": bool(p & 1), "many_rows": bool(p & 2), "shares": bool(p & 4), "join_waves": p >> 8}


def kv4_attention(q, cache, page_table, seq_start, ctx_len, max_q=None, max_ctx=None, scale=None, window: int = 0,
                  out=None, return_lse: bool = False, workspace=None):
    """Causal attention of new tokens' queries (float16 [T, q_heads, head_dim]; a slice of
    a wider projection's output is fine) over ``cache``, to which their keys and values
    are already appended; sequences and pages as in ``kv4_append``.

    A row sees the tokens up to its own, with ``window`` > 0 only the last ``window`` of
    them; a row that sees none gives 0, one of no sequence is not written. ``scale`` (at most
    1e16) is 1 / sqrt(head_dim) when omitted.
    ``max_q`` and ``max_ctx``, the most new tokens and the most tokens of a sequence,
    shape the launch only (the largest possible when omitted). Returns the float16
    output [T, q_heads, head_dim], with ``return_lse`` also float32 [T, q_heads], the log
    of each row's sum of exponentials. ``workspace`` (uint8 device tensor of
    ``kv4_attention_workspace_bytes`` bytes) is allocated per call when omitted."""
    import torch
    lib = load()
    T, q_heads, head_dim = q.shape
    B, max_pages, num_pages, page_tokens, kv_heads = _kv4_view(cache, page_table, seq_start, ctx_len, head_dim)
    qs = _rows(q, "q", q_heads, head_dim)
    max_q = T if max_q is None else max_q
    max_ctx = max_pages * page_tokens if max_ctx is None else max_ctx
    if out is None:
        out = q.new_empty((T, q_heads, head_dim))
    else:
        _need(out, torch.float16, "out")
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    lse = q.new_empty((T, q_heads), dtype=torch.float32) if return_lse else None
    if workspace is None:
        nbytes = int(lib.wq_kv4_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim, max_q, max_ctx))
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    wbytes = _workspace_bytes(workspace, q)
    rc = lib.wq_kv4_attention(_p(q), qs, T, q_heads, kv_heads, head_dim, _p(seq_start), _p(ctx_len), B, max_q, max_ctx,
                              _p(page_table), max_pages, _p(cache), num_pages, page_tokens,
                              head_dim ** -0.5 if scale is None else scale, window, _p(out), _p(lse), _p(workspace),
                              wbytes, _stream(q))
    _check("wq_kv4_attention", rc)
    return (out, lse) if return_lse else out


def auto_kernel(M, N, K) -> str:
    k = int(load().wq_auto_kernel(M, N, K))
    return {1: "gemv", 2: "gemm"}[k]
