"""CPU oracle of the products whose weights a row chooses: low-rank adapters beside a shared layer, expert routing, and
a mixture-of-experts layer.

TEST INFRASTRUCTURE ONLY, like the rest of this package: plain numpy in float64, nothing shared with the HIP library.
Each product also returns a bound on what a correct kernel may be off by, from its roundings:

* a sum of n float32 terms, in any order, is off by at most n 2^-24 times the sum of the terms' magnitudes;
* a value rounded to fp16 by at most 2^-11 of it, or 2^-25 where it is subnormal.
"""
from __future__ import annotations

import numpy as np

U32, U16, TINY = 2.0 ** -24, 2.0 ** -11, 2.0 ** -25


def _product(x, w, dx=0.0, extra=8):
    """x . w^T in float64 and its bound, x [m, k] off by dx, w [n, k] exact operands."""
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    return y, (x.shape[1] + extra) * U32 * mag + (dx @ np.abs(w).T if np.ndim(dx) else 0.0)


def linear_adapters(x, w, L1, L2, adapter, scale=None, rounded_weights=False):
    """``(y, bound)``, both [M, N]: y[m] = x[m] w^T + scale[a] (x[m] L1[a]^T) L2[a]^T, a = adapter[m], no adapter outside
    [0, n). ``w`` [N, K] float64: the layer's held weights, its sparse entries added. ``rounded_weights``: the kernel
    rounds each weight to fp16 (the GEMM does, the decode kernels do not)."""
    x = np.asarray(x, np.float64)
    y, bound = _product(x, w)
    if rounded_weights:
        bound = bound + U16 * (np.abs(x) @ np.abs(w).T)
    L1, L2 = np.asarray(L1, np.float64), np.asarray(L2, np.float64)
    for m, a in enumerate(np.asarray(adapter)):
        if not 0 <= a < L1.shape[0]:
            continue
        s = 1.0 if scale is None else float(np.float32(scale[a]))
        t, dt = _product(x[m:m + 1] * s, L1[a])
        dt = dt + U16 * (np.abs(t) + dt) + TINY
        v, dv = _product(t, L2[a], dt)
        y[m] += v[0]
        # the branch's terms join the same float32 sum
        bound[m] += dv[0] + (L1.shape[2] + L1.shape[1]) * U32 * (np.abs(t) @ np.abs(L2[a]).T)[0]
    return y, bound


def moe_route(logits, top_k, renormalize=True):
    """``(experts, weights)`` in float64: each row's top_k largest (equal ones by index, NaN the largest, -infinity
    never) and their softmax."""
    logits = np.asarray(logits, np.float64)
    M, E = logits.shape
    experts, weights = np.full((M, top_k), -1, np.int32), np.zeros((M, top_k))
    for m in range(M):
        row = logits[m]
        order = sorted(range(E), key=lambda e: (0 if np.isnan(row[e]) else 1, 0.0 if np.isnan(row[e]) else -row[e], e))
        chosen = [e for e in order if row[e] != -np.inf][:top_k]
        if not chosen:
            continue
        with np.errstate(invalid="ignore"):
            p = np.exp(row - row[chosen[0]])
        total = p[chosen].sum() if renormalize else p.sum()
        experts[m, :len(chosen)] = chosen
        weights[m, :len(chosen)] = p[chosen] / total
    return experts, weights


def moe_experts(x, experts, weights, gate_up, down):
    """``(y, bound)``, both [M, H]: the layer of held weights gate_up [E][2 I, H] and down [E][H, I], float64."""
    x = np.asarray(x, np.float64)
    M, H = x.shape
    y, bound = np.zeros((M, H)), np.zeros((M, H))
    mag = np.zeros((M, H))
    terms = 0
    for e in range(len(gate_up)):
        w = np.where(np.asarray(experts) == e, np.asarray(weights, np.float64), 0.0).sum(1)
        rows = np.nonzero((np.asarray(experts) == e).any(1))[0]
        if len(rows) == 0:
            continue
        gu, dgu = _product(x[rows], gate_up[e])
        I = gu.shape[1] // 2
        g, u, dg, du = gu[:, :I], gu[:, I:], dgu[:, :I], dgu[:, I:]
        sig = 1.0 / (1.0 + np.exp(-g))
        # |silu'| <= 1.1; the exponential's argument and value, the sum, the quotient: a few roundings each
        silu, dsilu = g * sig, 1.1 * dg + (8 + np.abs(g)) * U32 * np.abs(g * sig)
        h = silu * u
        dh = np.abs(u) * dsilu + (np.abs(silu) + dsilu) * du + 2 * U32 * np.abs(h)
        dh = dh + U16 * (np.abs(h) + dh) + TINY
        v, dv = _product(h, down[e], dh)
        y[rows] += w[rows, None] * v
        bound[rows] += np.abs(w[rows, None]) * dv
        mag[rows] += np.abs(w[rows, None]) * (np.abs(h) @ np.abs(down[e]).T)
        terms += 1
    return y, bound + (terms + 32) * U32 * mag


def rounded(y, bound, f16=True):
    """The bound of y after its one rounding to the output's type."""
    return bound + (U16 if f16 else U32) * (np.abs(y) + bound) + (TINY if f16 else 0.0)
