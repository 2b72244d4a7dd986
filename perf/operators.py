"""What the expert-layer and adapter operators are measured on.

Four operators: the router (``moe_route``), the mixture-of-experts layer for a
few tokens (``moe_layer``, timed from the router's logits as a decoding step
runs it), low-rank adapters of many requests beside a shared projection
(``lora_apply``) and their backward pass (``lora_backward``).

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the package.  ``exact`` computes them in 64
bits from the definitions, expert by expert and segment by segment.
"""

import math

import torch

own = False

_FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _route(name, T, E, k, dtype, renorm=True, masked=0.0):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype,
            "renorm": renorm, "masked": masked}


def _moe(name, T, E, k, D, F, dtype, fmt="e4m3", act="silu"):
    return {"name": name, "op": "moe", "T": T, "E": E, "k": k, "D": D, "F": F,
            "dtype": dtype, "fmt": fmt, "act": act}


def _lora(name, op, T, S, n, R, K, N, dtype, bare=0, split="even"):
    return {"name": name, "op": op, "T": T, "S": S, "n": n, "R": R, "K": K, "N": N,
            "dtype": dtype, "bare": bare, "split": split}


def listed():
    return [
        # one decoding token against many experts: pure latency
        _route("route 1 token 128 experts", 1, 128, 8, "bf16"),
        # the expert workload's 8192 tokens, top 2 of 8, sorted for the grouped GEMM
        _route("route 8192 tokens 8 experts", 8192, 8, 2, "f32"),
        # the smallest layer: a single token, all of it latency
        _moe("moe 1 token 8x1024", 1, 8, 2, 1024, 1024, "bf16"),
        # one decoding token through the expert workload's widths (4096, 14336)
        _moe("moe 1 token 8x14336", 1, 8, 2, 4096, 14336, "bf16"),
        # odd widths, E5M2 weights, a handful of tokens
        _moe("moe 7 tokens odd e5m2", 7, 10, 3, 1000, 1430, "bf16", "e5m2", "gelu_tanh"),
        # a decoding batch over many narrow experts, fp32 activations
        _moe("moe 24 tokens 64x1408", 24, 64, 8, 2048, 1408, "f32"),
        # the largest batch of the few-token form, every expert touched
        _moe("moe 128 tokens 8x14336", 128, 8, 2, 4096, 14336, "bf16"),
        # eight requests decoding one token each, every one with its own adapter
        _lora("lora 8 requests 1 token", "lora", 8, 8, 8, 16, 4096, 4096, "bf16", 0, "ones"),
        # ragged requests at odd widths, some without an adapter, fp32 activations
        _lora("lora ragged odd", "lora", 333, 17, 5, 24, 1000, 1001, "f32", 3, "ragged"),
        # prompts of four requests beside the qkv projection (8192 -> 10240)
        _lora("lora 4096 tokens qkv", "lora", 4096, 4, 3, 64, 8192, 10240, "bf16"),
        # a small training step of four adapters
        _lora("lora backward 256 tokens", "lora_backward", 256, 8, 4, 8, 1024, 1024, "bf16", 1,
              "ragged"),
        # a training step of three adapters beside the attention output projection
        _lora("lora backward 4096 tokens", "lora_backward", 4096, 4, 3, 32, 8192, 8192, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "lora", "lora_backward"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "route":
        E = _log(rng, 4, 256)
        T = _log(rng, 1, 8192 if E <= 64 else 2048)
        c = _route("", T, E, rng.randint(1, min(8, E)), dtype, rng.random() < 0.7,
                   rng.choice([0.0, 0.2]))
    elif op == "moe":
        E = _log(rng, 4, 64)
        D = _log(rng, 128, 4096)
        F = _log(rng, 128, min(14336, 400_000_000 // (E * D)))
        c = _moe("", _log(rng, 1, 128), E, rng.randint(1, min(8, E)), D, F, dtype,
                 rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["silu", "gelu_tanh"]))
    else:
        T = _log(rng, 1, 4096)
        S = _log(rng, 1, min(T, 64))
        n = rng.randint(1, min(8, S))
        R = rng.choice([4, 8, 13, 16, 24, 32, 48, 64])
        K, N = _log(rng, 64, 8192), _log(rng, 64, 8192)
        c = _lora("", op, T, S, n, R, K, N, dtype, rng.randint(0, S - n),
                  "ones" if S == T else rng.choice(["even", "ragged"]))
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs
def _codes(g, E, rows, cols, fmt):
    """Expert weights ~ N(0, 0.02), quantised with each expert's amax; the row
    stride is a multiple of 16 bytes."""
    t, top = _FP8[fmt]
    w = torch.zeros(E, rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, device="cuda")
    for e in range(E):
        v = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
        amax = v.abs().max()
        s[e] = amax / top
        w[e, :, :cols] = (v * (top / amax)).to(t).view(torch.uint8)
    return w[:, :, :cols], s


def _segments(case, g):
    """Row offsets and adapter of each request: `bare` requests have none, the
    others take the adapters in turn, in a shuffled order."""
    T, S = case["T"], case["S"]
    if case["split"] == "ones":
        offs = list(range(S + 1))
    elif case["split"] == "even":
        offs = [T * i // S for i in range(S + 1)]
    else:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")
        offs = [0] + sorted(cuts.tolist()) + [T]
    with_one = S - case["bare"]
    ids = torch.tensor([i % case["n"] for i in range(with_one)] + [-1] * case["bare"])
    ids = ids.cuda()[torch.randperm(S, generator=g, device="cuda")]
    return torch.tensor(offs, dtype=torch.int32).cuda(), ids.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)

    st = {"case": case}
    if case["op"] in ("route", "moe"):
        T, E = case["T"], case["E"]
        logits = normal(T, E, dtype=dt if case["op"] == "route" else torch.float32)
        if case.get("masked"):
            off = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
            logits = logits.masked_fill(off, -math.inf)
        st["logits"] = logits
    if case["op"] == "moe":
        D, F = case["D"], case["F"]
        st["x"] = normal(T, D)
        st["w13"], st["s13"] = _codes(g, E, 2 * F, D, case["fmt"])
        st["w2"], st["s2"] = _codes(g, E, D, F, case["fmt"])
    if case["op"] in ("lora", "lora_backward"):
        T, n, R, K, N = (case[c] for c in "TnRKN")
        bf = torch.bfloat16
        st["offs"], st["ids"] = _segments(case, g)
        st["x"] = normal(T, K)
        st["A"] = normal(n, R, K, sigma=K ** -0.5, dtype=bf)
        st["B"] = normal(n, R, N, sigma=0.05, dtype=bf)
        st["alpha"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        if case["op"] == "lora":
            st["base"] = normal(T, N, dtype=bf)
        else:
            st["dy"] = normal(T, N, sigma=0.01)
            st["dx_base"] = normal(T, K, sigma=0.01, dtype=bf)
            st["v"] = normal(T, R, dtype=torch.float32)
    return st


# -------------------------------------------------------------- plain forms
def _plain_route(logits, k, renorm):
    z = logits.float()
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    m = z.amax(1, keepdim=True)
    some = m > -math.inf
    m = torch.where(some, m, torch.zeros_like(m))
    p = torch.exp(top - m)
    s = p.sum(1, keepdim=True) if renorm else torch.exp(z - m).sum(1, keepdim=True)
    w = torch.where(some, p / s, torch.zeros_like(p))
    return torch.where(top > -math.inf, ids, -1).to(torch.int32), w


def _plain_sort(ids, E):
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.argsort(flat, stable=True).to(torch.int32)
    bounds = torch.arange(E + 1, device=flat.device)
    offs = (flat[None, :] < bounds[:, None]).sum(1).to(torch.int32)
    return offs, order


def _act(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_moe(st, ids, w):
    c = st["case"]
    t = _FP8[c["fmt"]][0]
    x = st["x"].float()
    gu = torch.matmul(x, st["w13"].view(t).float().transpose(1, 2)) * st["s13"][:, None, None]
    h = _act(gu[..., :c["F"]], c["act"]) * gu[..., c["F"]:]
    ye = torch.matmul(h, st["w2"].view(t).float().transpose(1, 2)) * st["s2"][:, None, None]
    share = torch.zeros(c["T"], c["E"] + 1, device=x.device)
    share.scatter_add_(1, torch.where(ids < 0, c["E"], ids).long(), w)
    return (ye * share[:, :c["E"]].t()[:, :, None]).sum(0).to(torch.bfloat16)


def _rows_of(st):
    """[T][n]: 1 where the row's request uses the adapter."""
    c = st["case"]
    row = torch.arange(c["T"], device="cuda")
    seg = (row[:, None] >= st["offs"][None, 1:]).sum(1)
    return (st["ids"][seg][:, None] == torch.arange(c["n"], device="cuda")).float()


def _plain_lora(st):
    c = st["case"]
    T, n, R = c["T"], c["n"], c["R"]
    on = _rows_of(st)[:, :, None]
    A = st["A"].float().reshape(n * R, -1)
    B = st["B"].float().reshape(n * R, -1)
    va = (st["x"].float() @ A.t()).view(T, n, R) * on
    delta = (va * st["alpha"][:, None]).reshape(T, n * R) @ B
    return (st["base"].float() + delta).to(torch.bfloat16), va.sum(1)


def _plain_lora_backward(st):
    c = st["case"]
    T, n, R = c["T"], c["n"], c["R"]
    on = _rows_of(st)[:, :, None] * st["alpha"][:, None]
    A = st["A"].float().reshape(n * R, -1)
    B = st["B"].float().reshape(n * R, -1)
    x, dy = st["x"].float(), st["dy"].float()
    dv = ((dy @ B.t()).view(T, n, R) * on).reshape(T, n * R)
    va = (st["v"][:, None, :] * on).reshape(T, n * R)
    dx = (st["dx_base"].float() + dv @ A).to(torch.bfloat16)
    return dx, (dv.t() @ x).view(n, R, -1), (va.t() @ dy).view(n, R, -1)


def run(state):
    c = state["case"]
    if own:
        import precision_linear_algebra_gb300 as fl
    if c["op"] == "route":
        if own:
            ids, w, offs, order = fl.moe_route(state["logits"], c["k"], renormalise=c["renorm"])
        else:
            ids, w = _plain_route(state["logits"], c["k"], c["renorm"])
            offs, order = _plain_sort(ids, c["E"])
        return {"ids": ids, "weights": w, "m_offsets": offs, "order": order}
    if c["op"] == "moe":
        if own:
            ids, w, _, _ = fl.moe_route(state["logits"], c["k"], sort=False)
            y = fl.moe_layer(state["x"], ids, w, state["w13"], state["s13"], state["w2"],
                             state["s2"], fmt=c["fmt"], activation=c["act"])
        else:
            ids, w = _plain_route(state["logits"], c["k"], True)
            y = _plain_moe(state, ids, w)
        return {"ids": ids, "weights": w, "y": y}
    if c["op"] == "lora":
        if own:
            out, v = fl.lora_apply(state["base"], state["x"], state["A"], state["B"],
                                   state["alpha"], state["offs"], state["ids"])
        else:
            out, v = _plain_lora(state)
        return {"out": out, "v": v}
    if own:
        dx, dA, dB = fl.lora_backward(state["dy"], state["x"], state["v"], state["A"],
                                      state["B"], state["alpha"], state["offs"], state["ids"],
                                      state["dx_base"])
    else:
        dx, dA, dB = _plain_lora_backward(state)
    return {"dx": dx, "dA": dA, "dB": dB}


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}[c["dtype"]]
    if c["op"] == "route":
        return {"bytes": c["T"] * c["E"] * size + c["T"] * c["k"] * 12 + 4 * c["E"] + 4,
                "flops": 3 * c["T"] * c["E"]}
    if c["op"] == "moe":
        # experts that T tokens with k different ones each touch, on average
        touched = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
        dim = c["D"] * c["F"]
        return {"bytes": touched * (3 * dim + 8) + c["T"] * (c["D"] * (size + 2) + 4 * c["E"]
                                                             + 8 * c["k"]),
                "flops": 6 * dim * c["T"] * c["k"]}
    T, n, R, K, N = (c[d] for d in "TnRKN")
    if c["op"] == "lora":
        return {"bytes": T * (K * size + 4 * N + 4 * R) + n * R * (K + N) * 2,
                "flops": 2 * T * R * (K + N)}
    return {"bytes": T * (K * size + N * size + 4 * K + 4 * R) + n * R * (K + N) * 6,
            "flops": 4 * T * R * (K + N)}


# ------------------------------------------------------------ in 64 bits
def _exact_route(z, k, renorm):
    z = z.double().cpu()
    T, E = z.shape
    key = torch.argsort(-z, dim=1, stable=True)[:, :k]
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    chosen = torch.gather(z, 1, key)
    live = chosen > -math.inf
    ids[live] = key[live].to(torch.int32)
    whole = torch.logsumexp(chosen if renorm else z, dim=1, keepdim=True)
    w[live] = torch.exp(chosen - whole)[live]
    return ids, w


def _exact_moe(st, ids, w):
    c = st["case"]
    t = _FP8[c["fmt"]][0]
    y = torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        tok, we = tok.cuda(), w[tok, slot].cuda()
        gu = st["x"][tok].double() @ st["w13"][e].view(t).double().t() * st["s13"][e].double()
        g, u = gu[:, :c["F"]], gu[:, c["F"]:]
        if c["act"] == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            h = g * u * (1 + torch.tanh((2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3))) / 2
        ye = h @ st["w2"][e].view(t).double().t() * st["s2"][e].double()
        y.index_add_(0, tok, ye * we[:, None])
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("route", "moe"):
        ids, w = _exact_route(st["logits"], case["k"], case.get("renorm", True))
        if case["op"] == "route":
            return {"ids": ids, "weights": w, "m_offsets": None, "order": None}
        return {"ids": ids, "weights": w, "y": _exact_moe(st, ids, w)}
    x, A, B = st["x"].double(), st["A"].double(), st["B"].double()
    alpha = st["alpha"].double()
    offs, ids = st["offs"].tolist(), st["ids"].tolist()
    segs = [(lo, hi, i) for lo, hi, i in zip(offs, offs[1:], ids) if i >= 0 and hi > lo]
    if case["op"] == "lora":
        out = st["base"].double()
        v = torch.zeros(case["T"], case["R"], dtype=torch.float64, device="cuda")
        for lo, hi, i in segs:
            v[lo:hi] = x[lo:hi] @ A[i].t()
            out[lo:hi] += alpha[i] * (v[lo:hi] @ B[i])
        return {"out": out, "v": v}
    dy, v, dx = st["dy"].double(), st["v"].double(), st["dx_base"].double()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for lo, hi, i in segs:
        dv = alpha[i] * (dy[lo:hi] @ B[i].t())
        dx[lo:hi] += dv @ A[i]
        dA[i] += dv.t() @ x[lo:hi]
        dB[i] += alpha[i] * (v[lo:hi].t() @ dy[lo:hi])
    return {"dx": dx, "dA": dA, "dB": dB}
