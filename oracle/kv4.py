"""CPU oracle of the norm and of the 4-bit key/value cache with its attention.

TEST INFRASTRUCTURE ONLY, like the rest of this package: plain numpy, nothing shared with
the HIP library. The quantizer runs in IEEE float32 (its results are integers and fp16 bit
patterns), everything else in float64.
"""
from __future__ import annotations

import numpy as np

from .ref import FP16_MIN_NORMAL, QMAX


def add_rmsnorm(x, weight, residual=None, eps=1e-5):
    """``(y, h)`` in float64: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + float(np.float32(eps))) * np.asarray(weight, np.float64)
    return y, h


def norm_int8(y, outliers=()):
    """``(q, s)`` of float64 rows y: s = amax / 127 over the channels that are not outliers
    (1 when that is 0), and the exact quotients y / s (not yet rounded), 0 on outliers."""
    y = np.array(y, np.float64)
    y[:, list(outliers)] = 0.0
    amax = np.max(np.abs(y), axis=1) if y.shape[1] else np.zeros(y.shape[0])
    s = np.where(amax > 0, amax / 127.0, 1.0)
    return y / s[:, None], s


def kv4_quantize(x):
    """Codes, fp16 scale and zero-point of each group x[..., :] (fp16): asymmetric 4-bit
    with the range widened to hold 0, in float32 steps rounded half to even."""
    x = np.asarray(x, np.float32)
    hi = np.maximum(x.max(-1), np.float32(0))
    lo = np.minimum(x.min(-1), np.float32(0))
    s = np.maximum(((hi - lo) / np.float32(QMAX)).astype(np.float32), FP16_MIN_NORMAL).astype(np.float16)
    sf = s.astype(np.float32)
    z = np.clip(np.rint((-lo / sf).astype(np.float32)), 0, QMAX)
    q = np.clip(np.rint((x / sf[..., None]).astype(np.float32)) + z[..., None], 0, QMAX)
    return q.astype(np.uint8), s, z.astype(np.float16)


def kv4_values(x):
    """The float64 values the cache holds for groups x[..., :]."""
    q, s, z = kv4_quantize(x)
    return (q.astype(np.float64) - z.astype(np.float64)[..., None]) * s.astype(np.float64)[..., None]


def kv4_attention(q, k, v, scale=None, window=0):
    """One sequence: q [n, q heads, d], held keys and values [ctx, kv heads, d] (float64
    values), the rows being the last n of ctx positions (or fewer: leading rows see
    nothing). Returns ``(out, lse, spread)`` in float64, spread = the weighted mean of
    |v|, which bounds how far rounded weights can move an output."""
    q = np.asarray(q, np.float64)
    n, hq, d = q.shape
    ctx, hkv = k.shape[0], k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, spread = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    pos = ctx - n + np.arange(n)[:, None]
    t = np.arange(ctx)[None]
    see = t <= pos
    if window:
        see &= t > pos - window
    some = see.any(1)
    for h in range(hq):
        if not some.any():
            break
        x = scale * (q[:, h] @ k[:, h // (hq // hkv)].T)
        x = np.where(see, x, -np.inf)[some]
        top = x.max(1, keepdims=True)
        w = np.exp(x - top)
        total = w.sum(1, keepdims=True)
        vh = v[:, h // (hq // hkv)]
        out[some, h] = (w @ vh) / total
        spread[some, h] = (w @ np.abs(vh)) / total
        lse[some, h] = (np.log(total) + top)[:, 0]
    return out, lse, spread
