"""Cases of the operators whose rows choose their weights: inputs, plain forms, and the framework's calls.

Three operators of a serving step whose rows belong to many requests:

* ``adapters``  y = x W^T + W_sparse x + s_a (x L1_a^T) L2_a^T: one 4-bit layer shared by all rows, and a low-rank
                adapter that each row names (or none);
* ``route``     softmax over the logits of all experts, the largest few of each row and their weights;
* ``experts``   a mixture-of-experts layer for a few tokens: y = sum over a row's experts e of
                w (silu(x G_e^T) * (x U_e^T)) D_e^T, all matrices in 4 bits.

``own`` is set from outside: false runs the plain forms below (elementary torch operations in float32, rounded once at
the end), true the framework's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 128
QMAX = 15
MIN_SCALE = 2.0 ** -14


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one request, its adapter beside the up-projection: latency
        dict(name="adapters_one_row", op="adapters", M=1, N=11008, K=4096, r=16, n=8, seg=1, none=0.0, sparse=0.0),
        # a decode batch with outliers beside the 4-bit weights, some requests without an adapter
        dict(name="adapters_batch_sparse", op="adapters", M=16, N=4096, K=4096, r=32, n=12, seg=1, none=0.2,
             sparse=0.0045),
        # a large decode batch, every request with an adapter of its own, on a long row-parallel shard
        dict(name="adapters_batch_many", op="adapters", M=64, N=8192, K=3584, r=64, n=64, seg=1, none=0.0, sparse=0.0),
        # odd sizes: drafted tokens of a few requests, a rank that fills no step, a ragged layer
        dict(name="adapters_odd", op="adapters", M=77, N=1001, K=1408, r=24, n=5, seg=5, none=0.1, sparse=0.0005),
        # prompts of several requests in one batch
        dict(name="adapters_prompts", op="adapters", M=2048, N=14336, K=4096, r=16, n=9, seg=300, none=0.1,
             sparse=0.0),
        # one token's choice of two among eight: latency
        dict(name="route_one", op="route", M=1, E=8, k=2, dtype="fp32", renorm=True, masked=0.0),
        # prompts, many experts, fp16 logits (so with ties), some experts masked
        dict(name="route_prompts", op="route", M=8191, E=160, k=8, dtype="fp16", renorm=False, masked=0.05),
        # one token, two of eight large experts
        dict(name="experts_one_token", op="experts", M=1, H=4096, I=14336, E=8, k=2, skew=0.5, none=0.0),
        # one token, eight of many small experts: latency
        dict(name="experts_one_small", op="experts", M=1, H=2048, I=1024, E=64, k=8, skew=0.5, none=0.0),
        # a decode batch that meets all of the large experts
        dict(name="experts_batch", op="experts", M=16, H=4096, I=14336, E=8, k=2, skew=0.5, none=0.0),
        # a decode batch on many small experts, uneven, with sizes that fill no tile evenly
        dict(name="experts_batch_small", op="experts", M=33, H=2176, I=1408, E=60, k=6, skew=1.0, none=0.03),
        # drafted tokens of a large batch: more rows than one pass of the layer holds
        dict(name="experts_drafts", op="experts", M=150, H=4096, I=1536, E=32, k=4, skew=0.7, none=0.0),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters", "route", "experts", "experts", "experts"])
    if op == "adapters":
        K = GROUP * _log(rng, 1, 112)
        N = _log(rng, 1, min(14336, 14336 * 4096 // K))
        M = _log(rng, 1, 2048)
        return dict(op=op, M=M, N=N, K=K, r=8 * _log(rng, 1, 16), n=_log(rng, 1, 64),
                    seg=rng.choice([1, 1, _log(rng, 2, 500)]), none=rng.choice([0.0, 0.0, 0.2, 0.9]),
                    sparse=rng.choice([0.0, 0.0, 0.0005, 0.0045]))
    if op == "route":
        E = _log(rng, 1, 512)
        return dict(op=op, M=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 16)), dtype=rng.choice(["fp32", "fp16"]),
                    renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.1, 0.95]))
    H = GROUP * _log(rng, 1, 32)
    I = GROUP * _log(rng, 1, 112)
    E = _log(rng, 1, max(1, min(128, 8 * 4096 * 14336 // (H * I))))
    k = rng.randint(1, min(E, 10))
    return dict(op=op, M=_log(rng, 1, 150), H=H, I=I, E=E, k=k, skew=rng.choice([0.0, 0.5, 1.0]),
                none=rng.choice([0.0, 0.0, 0.1]))


def _adapter_of_rows(case):
    """The adapter of each row (-1: none), requests of about `seg` rows one after the other."""
    r = random.Random(case["M"] * 1000003 + case["n"] * 31 + case["r"])
    out = []
    while len(out) < case["M"]:
        a = -1 if r.random() < case["none"] else r.randrange(case["n"])
        out += [a] * (1 if case["seg"] == 1 else r.randint(max(1, case["seg"] // 2), case["seg"] + case["seg"] // 2))
    return out[:case["M"]]


def _experts_of_rows(case):
    """The experts of each row, distinct (-1: none): uneven popularity, as a router's."""
    r = random.Random(case["M"] * 1000003 + case["E"] * 31 + case["k"])
    order = r.sample(range(case["E"]), case["E"])
    out = []
    for _ in range(case["M"]):
        keys = sorted((r.gammavariate(1, 1) * (1 + i) ** case["skew"], e) for i, e in enumerate(order))
        out.append([-1 if r.random() < case["none"] else e for _, e in keys[:case["k"]]])
    return out


def _nnz(case):
    return int(case["sparse"] * case["N"] * case["K"])


def work(case):
    if case["op"] == "adapters":
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        rows = [a for a in _adapter_of_rows(case) if a >= 0]
        nnz = _nnz(case)
        nbytes = N * K // 2 + 4 * N * K // GROUP + 2 * M * (K + N) + 2 * len(set(rows)) * r * (K + N) + 4 * M
        if nnz:
            nbytes += 6 * nnz + 4 * (N + 1)
        return dict(bytes=nbytes, flops=2 * M * N * K + 2 * M * nnz + 2 * len(rows) * r * (K + N))
    if case["op"] == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=case["M"] * (case["E"] * size + 8 * case["k"]), flops=4 * case["M"] * case["E"])
    used = [e for row in _experts_of_rows(case) for e in row if e >= 0]
    M, H, I = case["M"], case["H"], case["I"]
    return dict(bytes=len(set(used)) * 3 * H * I * (GROUP // 2 + 4) // GROUP + 4 * M * H + 8 * M * case["k"],
                flops=6 * len(used) * H * I)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _quantize(w):
    """w [N, K] float32 -> packed codes int32 [N, K / 8], fp16 scales and zero-points [N, K / 128]: asymmetric 4-bit
    codes, code 8 t + i in bits 4 i .. 4 i + 3 of word t."""
    N, K = w.shape
    g = w.view(N, K // GROUP, GROUP)
    high, low = g.amax(-1), g.amin(-1)
    s = ((high - low) / QMAX).clamp_min(MIN_SCALE).half()
    sf = s.float()
    z = torch.round(-low / sf).clamp(0, QMAX)
    q = (torch.round(g / sf[..., None]) + z[..., None]).clamp(0, QMAX).to(torch.int32).view(N, K // 8, 8)
    word = q[..., 0].clone()
    for i in range(1, 8):
        word |= q[..., i] << (4 * i)
    return word, s, z.half()


def _layer(N, K, g, sigma):
    return _quantize(torch.randn(N, K, device=DEV, generator=g) * sigma)


def _inputs_adapters(case, seed):
    g, M, N, K, r, n = _gen(seed), case["M"], case["N"], case["K"], case["r"], case["n"]
    packed, scales, zeros = _layer(N, K, g, 0.02)
    out = dict(packed=packed, scales=scales, zeros=zeros)
    out["x"] = torch.randn(M, K, device=DEV, generator=g).half()
    # an adapter's branch is a fraction of the layer's output, as after fine-tuning
    out["L1"] = (torch.randn(n, r, K, device=DEV, generator=g) / K ** 0.5).half()
    out["L2"] = (torch.randn(n, N, r, device=DEV, generator=g) * 0.1).half()
    out["scale"] = torch.rand(n, device=DEV, generator=g) * 2 + 0.25
    out["rows"] = _adapter_of_rows(case)
    out["adapter"] = torch.tensor(out["rows"], dtype=torch.int32, device=DEV)
    nnz = _nnz(case)
    if nnz:
        # distinct places, in order: CSR with ascending columns
        at = torch.randint(0, N * K, (nnz + nnz // 8 + 64,), device=DEV, generator=g)
        at = torch.unique(at)
        at = at[torch.randperm(at.numel(), device=DEV, generator=g)[:nnz]].sort().values
        row = torch.div(at, K, rounding_mode="floor")
        out["col"] = (at - row * K).int()
        out["val"] = (torch.randn(at.numel(), device=DEV, generator=g) * 0.1).half()
        out["row"] = row
        counts = torch.bincount(row, minlength=N)
        out["row_ptr"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0))).int()
    return out


def _inputs_route(case, seed):
    g, M, E = _gen(seed), case["M"], case["E"]
    logits = torch.randn(M, E, device=DEV, generator=g) * 1.5 + torch.randn(E, device=DEV, generator=g) * 0.5
    if case["masked"]:
        hide = torch.rand(M, E, device=DEV, generator=g) < case["masked"]
        logits.masked_fill_(hide, -math.inf)
    return dict(logits=logits if case["dtype"] == "fp32" else logits.half())


def _inputs_experts(case, seed):
    g, M, H, I, E, k = _gen(seed), case["M"], case["H"], case["I"], case["E"], case["k"]

    def stack(N, K, sigma):
        parts = (torch.empty(E, N, K // 8, dtype=torch.int32, device=DEV),
                 torch.empty(E, N, K // GROUP, dtype=torch.float16, device=DEV),
                 torch.empty(E, N, K // GROUP, dtype=torch.float16, device=DEV))
        for e in range(E):
            for p, v in zip(parts, _layer(N, K, g, sigma)):
                p[e] = v
        return parts

    out = dict(gate_up=stack(2 * I, H, H ** -0.5), down=stack(H, I, I ** -0.5))
    out["x"] = torch.randn(M, H, device=DEV, generator=g).half()
    out["rows"] = _experts_of_rows(case)
    out["experts"] = torch.tensor(out["rows"], dtype=torch.int32, device=DEV)
    w = torch.rand(M, k, device=DEV, generator=g) + 0.05
    out["weights"] = w / w.sum(-1, keepdim=True)
    return out


def prepare(case, seed):
    st = {"adapters": _inputs_adapters, "route": _inputs_route, "experts": _inputs_experts}[case["op"]](case, seed)
    st["case"] = case
    if own and case["op"] != "route":
        # a serving program keeps its workspace
        import quantized_gemm_rtn_amd as wq
        if case["op"] == "adapters":
            n = wq.linear_adapters_workspace_bytes(case["M"], case["N"], case["K"], case["r"])
        else:
            n = wq.moe_experts_workspace_bytes(case["M"], case["H"], case["I"], case["k"])
        st["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms
def _values(packed, scales, zeros):
    """The float32 weights [N, K] that a 4-bit layer stands for."""
    N, words = packed.shape
    shift = torch.arange(0, 32, 4, dtype=torch.int32, device=packed.device)
    q = ((packed[..., None] >> shift) & 15).float().view(N, words * 8 // GROUP, GROUP)
    return ((q - zeros.float()[..., None]) * scales.float()[..., None]).view(N, words * 8)


def _where(rows):
    """{index: positions} of a list of indices, those of at least 0."""
    at = {}
    for i, a in enumerate(rows):
        if a >= 0:
            at.setdefault(a, []).append(i)
    return at


def _plain_adapters(st):
    x = st["x"].float()
    w = _values(st["packed"], st["scales"], st["zeros"])
    if "row" in st:
        w[st["row"], st["col"].long()] += st["val"].float()
    y = x @ w.t()
    for a, rows in _where(st["rows"]).items():
        rows = torch.tensor(rows, device=DEV)
        t = (x[rows] @ st["L1"][a].float().t()) * st["scale"][a]
        y[rows] += t @ st["L2"][a].float().t()
    return y.half()


def _plain_route(st):
    case = st["case"]
    logits = st["logits"].float()
    top, chosen = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, chosen = top[:, :case["k"]], chosen[:, :case["k"]]
    largest = top[:, :1].masked_fill(top[:, :1] == -math.inf, 0)
    total = torch.exp(logits - largest).sum(-1, keepdim=True)
    p = torch.exp(top - largest)
    if case["renorm"]:
        total = p.sum(-1, keepdim=True)
    weights = p / total.masked_fill(total == 0, 1)
    return dict(experts=torch.where(top == -math.inf, -1, chosen).int(), weights=weights)


def _plain_experts(st):
    case = st["case"]
    M, H, I, k = case["M"], case["H"], case["I"], case["k"]
    x = st["x"].float()
    slots = torch.zeros(M * k, H, device=DEV)
    flat = [e for row in st["rows"] for e in row]
    for e, at in _where(flat).items():
        at = torch.tensor(at, device=DEV)
        gu = x[torch.div(at, k, rounding_mode="floor")] @ _values(*(p[e] for p in st["gate_up"])).t()
        h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
        slots[at] = (h @ _values(*(p[e] for p in st["down"])).t()) * st["weights"].view(-1)[at, None]
    return slots.view(M, k, H).sum(1).half()


def run(st):
    case = st["case"]
    if not own:
        return {"adapters": _plain_adapters, "route": _plain_route, "experts": _plain_experts}[case["op"]](st)
    import quantized_gemm_rtn_amd as wq
    if case["op"] == "adapters":
        csr = (st["row_ptr"], st["col"], st["val"]) if "row" in st else (None, None, None)
        return wq.linear_adapters(st["x"], st["packed"], st["scales"], st["zeros"], st["L1"], st["L2"], st["adapter"],
                                  st["scale"], *csr, workspace=st["workspace"])
    if case["op"] == "route":
        experts, weights = wq.moe_route(st["logits"], case["k"], renormalize=case["renorm"])
        return dict(experts=experts, weights=weights)
    return wq.moe_experts(st["x"], st["experts"], st["weights"], *st["gate_up"], *st["down"],
                          workspace=st["workspace"])


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_weights(packed, scales, zeros):
    q = torch.stack([(packed >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2).double()
    s, z = (v.double().repeat_interleave(GROUP, -1) for v in (scales, zeros))
    return s * (q - z)


def exact(case, seed):
    if case["op"] == "adapters":
        i = _inputs_adapters(case, seed)
        x = i["x"].double()
        y = x @ _exact_weights(i["packed"], i["scales"], i["zeros"]).t()
        if "row" in i:
            sparse = torch.zeros(case["N"], case["K"], dtype=torch.float64, device=DEV)
            sparse[i["row"], i["col"].long()] = i["val"].double()
            y += x @ sparse.t()
        for a in range(case["n"]):
            mine = (i["adapter"] == a).nonzero()[:, 0]
            if mine.numel():
                y[mine] += x[mine] @ i["L1"][a].double().t() @ i["L2"][a].double().t() * i["scale"][a].double()
        return y
    if case["op"] == "route":
        logits = _inputs_route(case, seed)["logits"].double()
        M, E, k = case["M"], case["E"], case["k"]
        left = logits.clone()
        index = torch.arange(E, device=DEV)
        experts = torch.full((M, k), -1, dtype=torch.int32, device=DEV)
        weights = torch.zeros(M, k, dtype=torch.float64, device=DEV)
        log_total = torch.logsumexp(logits, -1)
        for j in range(k):
            best = left.max(-1).values
            at = torch.where(left == best[:, None], index, E).min(-1).values
            live = best > -math.inf
            experts[live, j] = at[live].int()
            weights[live, j] = torch.exp(best - log_total)[live]
            left[torch.arange(M, device=DEV), at] = -math.inf
        if case["renorm"]:
            weights /= weights.sum(-1, keepdim=True).clamp_min(1e-300)
        return dict(experts=experts, weights=weights)
    i = _inputs_experts(case, seed)
    x, I = i["x"].double(), case["I"]
    y = torch.zeros(case["M"], case["H"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        row, slot = (i["experts"] == e).nonzero(as_tuple=True)
        if row.numel() == 0:
            continue
        gu = x[row] @ _exact_weights(*(p[e] for p in i["gate_up"])).t()
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        # a row names an expert at most once: no two of these rows are the same
        y[row] += h @ _exact_weights(*(p[e] for p in i["down"])).t() * i["weights"][row, slot].double()[:, None]
    return y
