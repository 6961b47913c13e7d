"""Mixture-of-experts layers of more active experts than one scan of 64 holds, up to all 1024 that a layer may have and a
block's lists can name, evenly used and not; and a layer made by the library's own quantizer."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_cases import say, to_dev
from rows_cases import worst

pytestmark = pytest.mark.gpu
H = I = 128


class Codes:
    """A layer of random codes; held weights are made for the experts that are asked for."""

    def __init__(self, seed, E):
        rng = np.random.default_rng(seed)
        self.E, self.parts = E, []
        for N, K in ((2 * I, H), (H, I)):
            q = rng.integers(0, 16, (E, N, K), dtype=np.uint8)
            s = (rng.uniform(0.5, 1.5, (E, N, K // 128)) * 0.25 * K ** -0.5).astype(np.float16)
            z = rng.integers(0, 16, (E, N, K // 128)).astype(np.float16)
            self.parts.append((q, s, z))

    def args(self, torch):
        out = []
        for q, s, z in self.parts:
            packed = oracle.pack(q.reshape(-1, q.shape[2])).reshape(q.shape[0], q.shape[1], -1)
            out += [to_dev(v, torch) for v in (packed, s, z)]
        return out

    def reference(self, x, experts, weights):
        """The oracle's result, of a layer of just the experts that rows name."""
        named = np.unique(experts[(experts >= 0) & (experts < self.E)])
        place = np.full(self.E, -1)
        place[named] = np.arange(len(named))
        few = np.where((experts >= 0) & (experts < self.E), place[np.clip(experts, 0, self.E - 1)], -1)
        held = [[oracle.dequant(q[e], s[e], z[e]) for e in named] for q, s, z in self.parts]
        return len(named), *oracle.rows.moe_experts(x, few, weights, *held)


def check(wq, layer, x, e, w, least):
    import torch
    active, ref, bound = layer.reference(x, e, w)
    assert active >= least
    args = layer.args(torch)
    call = [to_dev(x, torch), to_dev(e.astype(np.int32), torch), to_dev(w.astype(np.float32), torch), *args]
    y = wq.moe_experts(*call, out_dtype=torch.float32)
    err = worst(y, ref, bound, f16=False)
    say(f"    {active} active, {err:.3f} of the bound")
    assert err <= 1.0
    assert torch.equal(wq.moe_experts(*call), y.half())


@pytest.mark.parametrize("M", [64, 200])
@pytest.mark.parametrize("E,least", [(65, 65), (128, 128), (129, 129), (1024, 600)])
def test_evenly_used(gpu_lib, E, least, M):
    k = 16
    say(f"[many experts] E={E} M={M}")
    rng = np.random.default_rng(E + M)
    x = workloads.random_x(M, M, H)
    e = np.array([rng.permutation(E)[:k] for _ in range(M)])
    check(gpu_lib, Codes(E, E), x, e, rng.uniform(0.05, 1.0, (M, k)), least)


def test_every_pair_an_expert_of_its_own(gpu_lib):
    """64 rows of sixteen slots, 1024 experts: lists as full as they get, each expert with one pair."""
    say("[many experts] a pair each")
    rng = np.random.default_rng(1)
    e = rng.permutation(1024).reshape(64, 16)
    check(gpu_lib, Codes(2, 1024), workloads.random_x(3, 64, H), e, rng.uniform(0.05, 1.0, e.shape), 1024)


@pytest.mark.parametrize("M,k", [(64, 16), (130, 7)])
def test_a_few_crowded_among_hundreds_of_single_ones(gpu_lib, M, k):
    """Two experts that every row names (more than 32 pairs), one that a third of the rows do, and hundreds that one row
    does; an expert that the layer's last number has; slots of none."""
    say(f"[many experts] crowded, M={M} k={k}")
    E = 700
    rng = np.random.default_rng(M)
    single = rng.permutation(np.arange(10, E - 1))
    e = np.empty((M, k), np.int64)
    at = 0
    for m in range(M):
        row = [3, 500] + ([77] if m % 3 == 0 else []) + ([E - 1] if m % 20 == 0 else [])
        while len(row) < k:
            row.append(single[at % len(single)] if rng.random() < 0.9 else -1)
            at += 1
        e[m] = rng.permutation(row)
    check(gpu_lib, Codes(5, E), workloads.random_x(7, M, H), e, rng.uniform(-1.0, 1.0, e.shape), 400)


def test_a_layer_from_the_quantizer(gpu_lib):
    """Each expert's matrices by quantize_rtn and pack, stacked, as a user makes them."""
    import torch
    say("[experts from the quantizer]")
    E, M, k = 6, 9, 2
    rng = np.random.default_rng(9)
    shapes = (2 * I, H), (H, I)
    W = [[(rng.standard_normal(s) * s[1] ** -0.5).astype(np.float32) for s in shapes] for _ in range(E)]
    args, held = [], []
    for i in range(2):
        made = [gpu_lib.quantize_rtn(to_dev(W[e][i], torch)) for e in range(E)]
        args += [torch.stack([gpu_lib.pack(q["codes"]) for q in made]), torch.stack([q["scales"] for q in made]),
                 torch.stack([q["zeros"] for q in made])]
        held.append([oracle.dequant(*(q[n].cpu().numpy() for n in ("codes", "scales", "zeros"))) for q in made])
    x = workloads.random_x(1, M, H)
    e = np.array([rng.permutation(E)[:k] for _ in range(M)])
    w = rng.uniform(0.1, 1.0, (M, k)).astype(np.float32)
    ref, bound = oracle.rows.moe_experts(x, e, w, *held)
    y = gpu_lib.moe_experts(to_dev(x, torch), to_dev(e.astype(np.int32), torch), to_dev(w, torch), *args)
    assert worst(y, ref, bound) <= 1.0


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("M,E,k", [(192, 9, 5), (205, 20, 5), (257, 20, 4), (341, 12, 3), (342, 12, 3), (512, 30, 2),
                                   (513, 30, 2), (512, 5, 1), (1100, 40, 1)])
def test_rows_around_a_block_of_lists(gpu_lib, M, E, k, same):
    """As many rows as one block's lists hold (512, and 1024 pairs), one more, and several blocks of them; all on the same
    experts, whose pairs then fill up to sixteen tiles, or spread."""
    say(f"[experts lists] M={M} E={E} k={k} same={same}")
    rng = np.random.default_rng(M + k)
    x = workloads.random_x(M, M, H)
    e = np.array([np.arange(k) if same else rng.permutation(E)[:k] for _ in range(M)])
    check(gpu_lib, Codes(E + M, E), x, e, rng.uniform(0.05, 1.0, (M, k)), k)
