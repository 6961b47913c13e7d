"""Shared helpers of the cache tests: a batch of sequences with its page table, on the
GPU, and the oracle's outputs for it (imported by test_gpu_kv4_*.py)."""
import numpy as np

import oracle
from gpu_cases import to_dev


class Batch:
    """Sequences of `ctx` tokens, the last `new` of them new, in pages of `page` tokens.

    The cache is filled with 0xFF first (NaN scales and zero-points, codes of 15), and the
    page table's unused entries point outside the cache: neither may be noticed."""

    def __init__(self, wq, torch, new, ctx, hq, hkv, d, page=64, seed=0, k=None, v=None, q=None, extra_pages=3):
        self.wq, self.torch = wq, torch
        self.new, self.ctx, self.hq, self.hkv, self.d, self.page = list(new), list(ctx), hq, hkv, d, page
        B = len(new)
        rng = np.random.default_rng(seed)
        L, T = sum(ctx), sum(new)
        self.k = (rng.standard_normal((L, hkv, d)) + rng.standard_normal((1, hkv, d))).astype(np.float16) \
            if k is None else k
        self.v = (0.6 * rng.standard_normal((L, hkv, d))).astype(np.float16) if v is None else v
        self.q = rng.standard_normal((T, hq, d)).astype(np.float16) if q is None else q
        per = [-(-c // page) for c in ctx]
        self.num_pages = sum(per) + extra_pages
        order = rng.permutation(self.num_pages)
        width = max(max(per), 1) + 1
        table = np.full((B, width), 1 << 30, np.int32)
        table[:, 1::2] = -7
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = to_dev(table, torch)
        self.seq_start = to_dev(np.cumsum([0] + self.new).astype(np.int32), torch)
        self.ctx_len = to_dev(np.array(ctx, np.int32), torch)
        self.begin = np.cumsum([0] + self.ctx)
        self.cache = wq.kv4_cache(max(self.num_pages, 1), page, hkv, d)
        self.cache.fill_(0xFF)

    def fill(self, upto=None):
        """Appends every token (of sequence b the first upto[b]) in one call."""
        upto = self.ctx if upto is None else upto
        rows = np.concatenate([np.arange(self.begin[b], self.begin[b] + n) for b, n in enumerate(upto)]) \
            if sum(upto) else np.zeros(0, np.int64)
        start = to_dev(np.cumsum([0] + list(upto)).astype(np.int32), self.torch)
        if len(rows):
            self.wq.kv4_append(to_dev(self.k[rows], self.torch), to_dev(self.v[rows], self.torch), self.cache,
                               self.table, start, to_dev(np.array(upto, np.int32), self.torch),
                               max_new=max(upto))
        return self

    def attention(self, **kw):
        kw.setdefault("max_q", max(self.new))
        kw.setdefault("max_ctx", max(self.ctx))
        q = kw.pop("q", None)
        out, lse = self.wq.kv4_attention(to_dev(self.q, self.torch) if q is None else q, self.cache, self.table,
                                         self.seq_start, self.ctx_len, return_lse=True, **kw)
        self.torch.cuda.synchronize()
        return out, lse

    def reference(self, scale=None, window=0):
        outs, lses, spreads, row = [], [], [], 0
        for b, (n, c) in enumerate(zip(self.new, self.ctx)):
            k = oracle.kv4_values(self.k[self.begin[b]:self.begin[b] + c]) if c else np.zeros((0, self.hkv, self.d))
            v = oracle.kv4_values(self.v[self.begin[b]:self.begin[b] + c]) if c else np.zeros((0, self.hkv, self.d))
            o, ls, sp = oracle.kv4_attention(self.q[row:row + n], k, v, scale, window)
            row += n
            outs.append(o)
            lses.append(ls)
            spreads.append(sp)
        return np.concatenate(outs), np.concatenate(lses), np.concatenate(spreads)


# A weight times its value scale is rounded to fp16 (half an ulp: 2^-11 of it, so at most
# 2^-11 spread in the sum), the output once more (2^-11 of it); fp32 scores of a few tens
# are off by some 1e-6 each, which the weights inherit, and weights far below their row's
# largest are held to 2^-25 of 2^9: 2^-13 spread covers both.
def out_error(out, ref, spread):
    """The largest |out - ref| as a multiple of its bound."""
    o = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all()
    bound = 2.0 ** -11 * (spread + np.abs(ref)) + 2.0 ** -13 * spread + 2.0 ** -24
    return float(np.max(np.abs(o - ref) / bound)) if o.size else 0.0


def check(out, lse, ref, tag=""):
    o, ls, spread = ref
    err = out_error(out, o, spread)
    got = lse.cpu().numpy().astype(np.float64)
    none = np.isneginf(ls)
    assert np.array_equal(none, np.isneginf(got)), tag
    assert (out.float().cpu().numpy()[none] == 0).all(), tag
    off = float(np.max(np.abs(got[~none] - ls[~none]) / (1e-4 + 2e-6 * np.abs(ls[~none])))) if (~none).any() else 0.0
    print(f"    {tag} out {err:.3f}, lse {off:.3f} of their bounds", flush=True)
    assert err <= 1.0, (tag, err)
    assert off <= 1.0, (tag, off)
