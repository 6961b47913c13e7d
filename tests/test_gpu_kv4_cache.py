"""The 4-bit cache's writer and reader against the oracle's quantizer: every value the
cache holds equals the oracle's, rounded to fp16, bit for bit."""
import numpy as np
import pytest

import oracle
from gpu_cases import f16_bits_host, say, to_dev
from kv4_cases import Batch

pytestmark = pytest.mark.gpu


def _expect(b, new):
    """fp16 bits of the last new[i] tokens of each sequence of b, zeros where there is none."""
    ks, vs = [], []
    for i, n in enumerate(new):
        have = min(n, b.ctx[i])
        end = b.begin[i] + b.ctx[i]
        for src, dst in ((b.k, ks), (b.v, vs)):
            held = oracle.kv4_values(src[end - have:end]).astype(np.float16) if have else \
                np.zeros((0, b.hkv, b.d), np.float16)
            dst.append(np.concatenate([np.zeros((n - have, b.hkv, b.d), np.float16), held]))
    return np.concatenate(ks), np.concatenate(vs)


def _same(t, ref):
    # -0 and +0 are the same value (a code at its zero-point)
    got = t.cpu().numpy()
    return got.shape == ref.shape and np.array_equal(got, ref)


def _read(wq, torch, b, new, **kw):
    start = to_dev(np.cumsum([0] + list(new)).astype(np.int32), torch)
    k, v = wq.kv4_read(b.cache, b.table, start, b.ctx_len, tokens=sum(new), head_dim=b.d, **kw)
    torch.cuda.synchronize()
    return k, v


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx,hkv,page", [
    ([1], 1, 32), ([31, 32, 33], 2, 32), ([64, 1, 200, 5], 3, 96), ([0, 7, 0, 130], 2, 64), ([777], 5, 256),
])
def test_append_and_read(gpu_lib, ctx, hkv, page, d):
    import torch
    say(f"[kv4 append] ctx={ctx} hkv={hkv} page={page} d={d}")
    b = Batch(gpu_lib, torch, ctx, ctx, hkv, hkv, d, page, seed=sum(ctx) + d).fill()
    k, v = _read(gpu_lib, torch, b, ctx)
    ek, ev = _expect(b, ctx)
    assert _same(k, ek) and _same(v, ev)


@pytest.mark.parametrize("d", [64, 128])
def test_token_by_token_and_in_chunks(gpu_lib, d):
    """A tile filled token by token, in chunks that end inside it and at once holds the
    same bytes; tokens of other sequences and pages stay as they were."""
    import torch
    ctx = [70, 45]
    a = Batch(gpu_lib, torch, ctx, ctx, 2, 2, d, 32, seed=5).fill()
    b = Batch(gpu_lib, torch, ctx, ctx, 2, 2, d, 32, seed=5).fill([33, 0])
    say(f"[kv4 append in steps] d={d}")
    at = [33, 0]
    steps = [[1, 1], [1, 20], [10, 1], [1, 1], [24, 22]]
    for new in steps:
        at = [x + n for x, n in zip(at, new)]
        rows = np.concatenate([np.arange(b.begin[i] + at[i] - new[i], b.begin[i] + at[i]) for i in range(2)])
        gpu_lib.kv4_append(to_dev(b.k[rows], torch), to_dev(b.v[rows], torch), b.cache, b.table,
                           to_dev(np.cumsum([0] + new).astype(np.int32), torch),
                           to_dev(np.array(at, np.int32), torch), max_new=1)
    torch.cuda.synchronize()
    assert at == ctx
    for x, y in zip(_read(gpu_lib, torch, a, ctx), _read(gpu_lib, torch, b, ctx)):
        assert torch.equal(x, y)
    # pages of no sequence still hold what they held
    used = set(a.table.cpu().numpy().ravel().tolist())
    for p in range(a.num_pages):
        if p not in used:
            assert bool((b.cache[p] == 0xFF).all())


@pytest.mark.parametrize("d", [64, 128])
def test_groups_at_the_edges(gpu_lib, d):
    """All equal, all positive, all negative, zero, one spike, the widest range, values
    below the smallest scale."""
    import torch
    rng = np.random.default_rng(3)
    g = [np.zeros(d), np.full(d, 3.0), np.full(d, -0.25), np.abs(rng.standard_normal(d)) + 5,
         -np.abs(rng.standard_normal(d)) - 5, np.eye(1, d, 7)[0] * 100, np.where(np.arange(d) % 2, 65504.0, -65504.0),
         rng.standard_normal(d) * 1e-5, rng.standard_normal(d) * 2.0 ** -14, np.linspace(0, 15, d).round(),
         np.linspace(-7, 8, d).round() * 0.5]
    x = np.stack(g).astype(np.float16)[:, None, :]
    say(f"[kv4 edge groups] d={d}")
    n = len(g)
    b = Batch(gpu_lib, torch, [n], [n], 1, 1, d, 32, k=x, v=x[::-1].copy()).fill()
    k, v = _read(gpu_lib, torch, b, [n])
    ek, ev = _expect(b, [n])
    assert _same(k, ek) and _same(v, ev)
    # codes that a group's own grid holds exactly come back exactly
    assert np.array_equal(k.cpu().numpy()[-2:], x[-2:])


def test_slices_padded_slots_and_hints(gpu_lib):
    """k and v as slices of one wider projection, a slot with a row but no token, hints
    that are too small and too large."""
    import torch
    d, hkv, hq = 128, 2, 4
    new, ctx = [3, 1, 40, 1], [10, 0, 41, 33]
    for hint in (0, 1, 40, 100000, None):
        b = Batch(gpu_lib, torch, new, ctx, hq, hkv, d, 64, seed=9)
        b.fill([max(c - n, 0) for c, n in zip(ctx, new)])
        rows = np.concatenate([np.arange(b.begin[i] + c - n, b.begin[i] + c) if c else np.array([0])
                               for i, (n, c) in enumerate(zip(new, ctx))])
        wide = torch.randn(sum(new), (hq + 2 * hkv) * d, device="cuda").half()
        wide[:, hq * d:(hq + hkv) * d] = to_dev(b.k[rows].reshape(len(rows), -1), torch)
        wide[:, (hq + hkv) * d:] = to_dev(b.v[rows].reshape(len(rows), -1), torch)
        k, v = wide[:, hq * d:].unflatten(1, (2 * hkv, d)).split(hkv, 1)
        say(f"[kv4 slices] max_new={hint}")
        gpu_lib.kv4_append(k, v, b.cache, b.table, b.seq_start, b.ctx_len, max_new=hint)
        got = _read(gpu_lib, torch, b, new, max_new=hint)
        for x, e in zip(got, _expect(b, new)):
            assert _same(x, e)
        whole = _read(gpu_lib, torch, b, ctx)
        for x, e in zip(whole, _expect(b, ctx)):
            assert _same(x, e)


def test_cache_beyond_4_gib(gpu_lib):
    """Pages whose offset passes 32 bits (bytes and, at d = 128, half that many words)."""
    import torch
    d, hkv, page = 128, 8, 256
    size = gpu_lib.kv4_page_bytes(page, d) * hkv
    pages = (9 << 30) // size
    ctx = [300, 40]
    b = Batch(gpu_lib, torch, [1, 1], ctx, hkv, hkv, d, page, seed=2)
    b.cache = gpu_lib.kv4_cache(pages, page, hkv, d)
    say(f"[kv4 large cache] {b.cache.numel() / 2**30:.1f} GiB")
    b.table = to_dev(np.array([[pages - 1, pages // 2 + 3, 0], [pages - 2, 0, 0]], np.int32), torch)
    b.fill()
    for x, e in zip(_read(gpu_lib, torch, b, ctx), _expect(b, ctx)):
        assert _same(x, e)


def test_lengths_outside_the_arrays_are_clamped(gpu_lib):
    """Starts, lengths and page numbers that do not fit give wrong values at most: the
    call ends, and nothing outside the named pages changes."""
    import torch
    d = 64
    b = Batch(gpu_lib, torch, [4, 4], [40, 20], 1, 1, d, 32, seed=4).fill()
    say("[kv4 clamped]")
    guard = b.cache.clone()
    k = torch.zeros(8, 1, d, device="cuda", dtype=torch.float16)
    table = torch.full_like(b.table, -5)
    for start, ctx in (([0, 4, 1 << 20], [40, 20]), ([-3, 6, 2], [1 << 30, -9]), ([0, 8, 8], [5, 1 << 30])):
        s, c = to_dev(np.array(start, np.int32), torch), to_dev(np.array(ctx, np.int32), torch)
        gpu_lib.kv4_append(k, k, b.cache, table, s, c)
        gpu_lib.kv4_read(b.cache, table, s, c, tokens=8, head_dim=d)
        gpu_lib.kv4_attention(k, b.cache, table, s, c)
        torch.cuda.synchronize()
    # every page number was below the cache: only page 0 was written
    assert torch.equal(guard[1:], b.cache[1:])
