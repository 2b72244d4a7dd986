"""What the FP8 key/value cache and its attention are measured on.

Four operators on a paged cache of FP8 codes with one scale for each token and
head: writing it (``kv_append``), reading it back (``kv_read``), attention over it
for packed sequences of any number of rows, from a decoding token to a whole
prompt (``kv_attention``), and the same for a batch whose sequences share a prefix
(``kv_attention`` with ``prefix_table``).

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits, on sequences padded to the longest; with ``own`` true it calls the
package.  ``exact`` computes them in 64 bits from the definitions, sequence by
sequence and head by head.
"""

import math
import random

import torch

own = False

_FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, S, rows, ctx, H, G, D, page, dtype="bf16", fmt="e4m3", split="even",
          prefix=0):
    """S sequences of up to `rows` rows after up to `ctx` cached tokens; H heads of
    keys and values, G query heads on each."""
    return {"name": name, "op": op, "S": S, "rows": rows, "ctx": ctx, "H": H, "G": G, "D": D,
            "page": page, "dtype": dtype, "fmt": fmt, "split": split, "prefix": prefix}


def listed():
    return [
        # one decoding step of 64 requests: a token each, all of it latency
        _case("append 64 requests 1 token", "append", 64, 1, 2000, 8, 8, 128, 64),
        # a prompt batch of the transformer workload, 2 x 2048 tokens, fp32, odd pages
        _case("append 2 prompts of 2048 f32", "append", 2, 2048, 0, 8, 8, 128, 48, "f32"),
        # ragged requests at an odd head width, E5M2, read back in fp32
        _case("read ragged odd e5m2", "read", 7, 333, 0, 5, 1, 80, 16, "f32", "e5m2", "ragged"),
        # eight long contexts read back whole, to be moved or re-quantised
        _case("read 8 contexts of 8192", "read", 8, 8192, 0, 8, 1, 128, 64),
        # one request decoding alone: latency
        _case("decode 1 request 2048", "attention", 1, 1, 2047, 8, 8, 128, 64),
        # a decoding batch with ragged contexts: the cache's bytes
        _case("decode 64 requests ragged 8192", "attention", 64, 1, 8191, 8, 8, 128, 64,
              split="ragged"),
        # a few draft tokens a request, odd head width and pages, fp32 queries, E5M2
        _case("decode 9 requests 3 rows odd", "attention", 9, 3, 3001, 3, 5, 80, 24, "f32", "e5m2",
              "ragged"),
        # one very long context
        _case("decode 1 request 131072", "attention", 1, 1, 131071, 8, 8, 128, 256),
        # two prompts of the attention workload: 64 heads of 128, 2048 tokens each
        _case("prompt 2 x 2048", "attention", 2, 2048, 0, 8, 8, 128, 64),
        # packed prompts of different lengths after cached contexts, narrow heads
        _case("prompt 6 ragged odd", "attention", 6, 1001, 777, 4, 3, 64, 16, split="ragged"),
        # a decoding batch behind one system prompt
        _case("prefix 64 requests 8192", "attention", 64, 1, 511, 8, 8, 128, 64, split="ragged",
              prefix=8192),
        # a few requests behind a short prefix that ends inside a page, fp32 queries
        _case("prefix 5 requests odd", "attention", 5, 2, 100, 2, 7, 96, 32, "f32", "e4m3",
              "ragged", prefix=777),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "read", "decode", "decode", "prompt", "prompt", "prefix"])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    page = rng.choice([16, 24, 48, 64, 100, 128, 256])
    dtype, fmt = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["e4m3", "e4m3", "e5m2"])
    split = rng.choice(["even", "ragged"])
    H = rng.choice([1, 2, 3, 4, 8])
    if kind in ("append", "read"):
        S = _log(rng, 1, 64)
        c = _case("", kind, S, _log(rng, 1, 16384 // S), rng.choice([0, 1, 500]), H, 1, D, page,
                  dtype, fmt, split)
    elif kind == "decode":
        S = _log(rng, 1, 64)
        c = _case("", "attention", S, rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 131072 // S), H,
                  rng.choice([1, 2, 4, 5, 8, 16]), D, page, dtype, fmt, split)
    elif kind == "prompt":
        S = _log(rng, 1, 8)
        c = _case("", "attention", S, _log(rng, 16, 4096 // S), rng.choice([0, 0, 100, 1000]), H,
                  rng.choice([1, 2, 3, 4]), D, page, dtype, fmt, split)
        while work(c)["flops"] > 1.3e11:  # no more than the largest listed
            c["rows"] = c["rows"] * 3 // 4
    else:
        S = _log(rng, 2, 64)
        c = _case("", "attention", S, rng.choice([1, 1, 2, 4]), _log(rng, 1, 512), H,
                  rng.choice([1, 4, 7, 8]), D, page, dtype, fmt, split, _log(rng, 64, 8192))
    del c["name"]
    return c


def _lengths(case):
    """(rows, length with them) of each sequence; the first has the most."""
    rows, ctx = [case["rows"]], [case["ctx"]]
    rng = random.Random(case["S"] * 1000003 + case["rows"] * 1009 + case["ctx"])
    for _ in range(case["S"] - 1):
        if case["split"] == "even":
            rows.append(case["rows"])
            ctx.append(case["ctx"])
        else:
            rows.append(_log(rng, 1, case["rows"]))
            ctx.append(rng.randint(0, case["ctx"]))
    return rows, [n + c for n, c in zip(rows, ctx)]


# ------------------------------------------------------------------- inputs
def _cache_rows(g, shape, fmt):
    """Codes and scales of N(0, 1) rows whose size varies from token to token."""
    t, top = _FP8[fmt]
    x = torch.randn(*shape, generator=g, device="cuda")
    amax = x.abs().amax(-1, keepdim=True)
    codes = (x * (top / amax)).to(t).view(torch.uint8)
    size = torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device="cuda"))
    return codes, amax.squeeze(-1) / top * size


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    S, H, G, D, page = (case[k] for k in ("S", "H", "G", "D", "page"))
    rows, lens = _lengths(case)
    need = [-(-n // page) for n in lens]
    shared = -(-case["prefix"] // page)
    pages = sum(need) + shared + 3
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(S, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    offs = [0]
    for n in rows:
        offs.append(offs[-1] + n)
    T = offs[-1]
    st = {"case": case, "table": table, "most": max(rows), "longest": max(lens), "T": T,
          "offs": torch.tensor(offs, dtype=torch.int32).cuda(),
          "lens": torch.tensor(lens, dtype=torch.int32).cuda()}
    if case["prefix"]:
        st["prefix_table"] = ids[at:at + shared].clone()
        st["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32).cuda()
    st["kc"], st["ks"] = _cache_rows(g, (pages, H, page, D), case["fmt"])
    st["vc"], st["vs"] = _cache_rows(g, (pages, H, page, D), case["fmt"])
    if case["op"] == "append":
        # rows of a fused projection, query heads first
        qkv = torch.randn(T, (G + 2) * H, D, generator=g, device="cuda").to(dt)
        st["k"], st["v"] = qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
    elif case["op"] == "attention":
        st["q"] = (1.5 * torch.randn(T, G * H, D, generator=g, device="cuda")).to(dt)
    return st


# -------------------------------------------------------------- plain forms
def _places(st):
    """Page and place in it of each row's own position."""
    page = st["case"]["page"]
    row = torch.arange(st["T"], device="cuda")
    seg = (row[:, None] >= st["offs"][None, 1:]).sum(1)
    pos = st["lens"][seg] - st["offs"][seg + 1] + row
    return st["table"][seg, pos // page].long(), pos % page


def _plain_append(st):
    t, top = _FP8[st["case"]["fmt"]]
    at, place = _places(st)
    for x, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        x = x.float()
        amax = x.abs().amax(-1)
        fine = (amax > 0) & (top / amax < math.inf)
        up = torch.where(fine, top / amax, torch.ones_like(amax))
        q = (x * up[..., None]).clamp(-top, top).to(t)
        codes[at, :, place] = q.view(torch.uint8)
        scales[at, :, place] = torch.where(fine, amax / top, torch.ones_like(amax))


def _values(codes, scales, at, place, fmt):
    """Cached rows in 32 bits: [..., H, D]."""
    c = codes[at, :, place].view(_FP8[fmt][0]).float()
    return c * scales[at, :, place][..., None]


def _plain_read(st):
    c = st["case"]
    at, place = _places(st)
    dt = _TYPES[c["dtype"]]
    return (_values(st["kc"], st["ks"], at, place, c["fmt"]).to(dt),
            _values(st["vc"], st["vs"], at, place, c["fmt"]).to(dt))


def _plain_attention(st):
    c = st["case"]
    S, H, G, D, page, fmt = (c[k] for k in ("S", "H", "G", "D", "page", "fmt"))
    n, L, T = st["most"], st["longest"], st["T"]
    tok = torch.arange(L, device="cuda")
    at, place = st["table"][:, tok // page].long(), (tok % page).expand(S, L)
    # [S, H, L, D]; rows behind a sequence's end are garbage and masked below
    K = _values(st["kc"], st["ks"], at, place, fmt).transpose(1, 2)
    V = _values(st["vc"], st["vs"], at, place, fmt).transpose(1, 2)
    rows = st["offs"][1:] - st["offs"][:-1]
    i = torch.arange(n, device="cuda")
    r = (st["offs"][:-1, None] + i).clamp(max=T - 1)
    q = st["q"].float()[r].view(S, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * n, D)
    q = q * D ** -0.5
    pos = (st["lens"] - rows)[:, None] + i
    seen = (tok[None, None] <= pos[:, :, None]) & (tok[None, None] < st["lens"][:, None, None])
    s = (q @ K.transpose(2, 3)).view(S, H, G, n, L)
    s = s.masked_fill(~seen[:, None, None], -math.inf).view(S, H, G * n, L)
    if c["prefix"]:
        tok = torch.arange(c["prefix"], device="cuda")
        at, place = st["prefix_table"][tok // page].long(), tok % page
        Kp = _values(st["kc"], st["ks"], at, place, fmt).transpose(0, 1)
        Vp = _values(st["vc"], st["vs"], at, place, fmt).transpose(0, 1)
        qp = q.transpose(0, 1).reshape(H, S * G * n, D)
        sp = (qp @ Kp.transpose(1, 2)).view(H, S, G * n, c["prefix"]).transpose(0, 1)
        s = torch.cat([sp, s], -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    own_p = p[..., c["prefix"]:]
    o = own_p @ V
    if c["prefix"]:
        pp = p[..., :c["prefix"]].transpose(0, 1).reshape(H, S * G * n, c["prefix"])
        o = o + (pp @ Vp).view(H, S, G * n, D).transpose(0, 1)
    o = (o / total).view(S, H, G, n, D)
    lse = (m + torch.log(total)).view(S, H, G, n)
    row = torch.arange(T, device="cuda")
    seg = (row[:, None] >= st["offs"][None, 1:]).sum(1)
    j = row - st["offs"][seg]
    return (o.permute(0, 3, 1, 2, 4)[seg, j].reshape(T, H * G, D).to(torch.bfloat16),
            lse.permute(0, 3, 1, 2)[seg, j].reshape(T, H * G))


def run(state):
    st, c = state, state["case"]
    if own:
        import precision_linear_algebra_gb300 as fl
        cache = fl.KVCache(st["kc"], st["vc"], st["ks"], st["vs"], c["fmt"])
    if c["op"] == "append":
        if own:
            fl.kv_append(st["k"], st["v"], cache, st["offs"], st["lens"], st["table"])
        else:
            _plain_append(st)
        t = _FP8[c["fmt"]][0]
        return {"k": st["kc"].view(t), "v": st["vc"].view(t), "k_scale": st["ks"],
                "v_scale": st["vs"]}
    if c["op"] == "read":
        if own:
            k, v = fl.kv_read(cache, st["offs"], st["lens"], st["table"], st["T"],
                              dtype=_TYPES[c["dtype"]])
        else:
            k, v = _plain_read(st)
        return {"k": k, "v": v}
    if own:
        out, lse = fl.kv_attention(st["q"], cache, st["offs"], st["lens"], st["table"],
                                   max_rows=st["most"], prefix_table=st.get("prefix_table"),
                                   prefix_len=st.get("prefix_len"))
    else:
        out, lse = _plain_attention(st)
    return {"out": out, "lse": lse}


def work(case):
    c = case
    rows, lens = _lengths(c)
    T, size = sum(rows), {"f32": 4, "bf16": 2}[c["dtype"]]
    H, Hq, D = c["H"], c["H"] * c["G"], c["D"]
    if c["op"] in ("append", "read"):
        return {"bytes": T * H * (2 * D * size + 2 * D + 8), "flops": 4 * T * H * D}
    seen = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(rows, lens)) + T * c["prefix"]
    return {"bytes": (sum(lens) + c["prefix"]) * H * (2 * D + 8) + T * Hq * (D * (size + 2) + 4),
            "flops": 4 * D * Hq * seen}


# ------------------------------------------------------------ in 64 bits
def _sequence(codes, scales, pages, n, fmt):
    """The first n tokens of a list of pages: [H, n, D] in 64 bits."""
    x = codes[pages.long()].view(_FP8[fmt][0]).double() * scales[pages.long()].double()[..., None]
    x = x.transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :n]


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    H, G, D, page, fmt = (c[k] for k in ("H", "G", "D", "page", "fmt"))
    offs, lens, T = st["offs"].tolist(), st["lens"].tolist(), st["T"]
    if c["op"] == "append":
        t, top = _FP8[fmt]
        res = {}
        for name, x, codes, scales in (("k", st["k"], st["kc"], st["ks"]),
                                       ("v", st["v"], st["vc"], st["vs"])):
            codes, scales, x = codes.view(t).double(), scales.double(), x.double()
            for s, length in enumerate(lens):
                n = offs[s + 1] - offs[s]
                pos = torch.arange(length - n, length, device="cuda")
                at, place = st["table"][s][pos // page].long(), pos % page
                rows = x[offs[s]:offs[s + 1]]
                step = rows.abs().amax(-1) / top
                codes[at, :, place] = rows / step[..., None]
                scales[at, :, place] = step
            res[name], res[name + "_scale"] = codes, scales
        return res
    if c["op"] == "read":
        k = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
        for s, length in enumerate(lens):
            first = length - (offs[s + 1] - offs[s])
            for x, codes, scales in ((k, st["kc"], st["ks"]), (v, st["vc"], st["vs"])):
                whole = _sequence(codes, scales, st["table"][s][:-(-length // page)], length, fmt)
                x[offs[s]:offs[s + 1]] = whole[:, first:].transpose(0, 1)
        return {"k": k, "v": v}
    if work(c)["flops"] > 4e11:
        return None
    out = torch.empty(T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, H * G, dtype=torch.float64, device="cuda")
    for s, length in enumerate(lens):
        lo, hi = offs[s], offs[s + 1]
        pages = st["table"][s][:-(-length // page)]
        K = _sequence(st["kc"], st["ks"], pages, length, fmt)
        V = _sequence(st["vc"], st["vs"], pages, length, fmt)
        if c["prefix"]:
            K = torch.cat([_sequence(st["kc"], st["ks"], st["prefix_table"], c["prefix"], fmt), K], 1)
            V = torch.cat([_sequence(st["vc"], st["vs"], st["prefix_table"], c["prefix"], fmt), V], 1)
        whole = K.shape[1]
        ahead = torch.ones(hi - lo, whole, dtype=torch.bool, device="cuda").triu(whole - hi + lo + 1)
        for h in range(H * G):
            s2 = st["q"][lo:hi, h].double() @ K[h // G].t() / math.sqrt(D)
            s2[ahead] = -math.inf
            lse[lo:hi, h] = torch.logsumexp(s2, 1)
            out[lo:hi, h] = torch.softmax(s2, 1) @ V[h // G]
    return {"out": out, "lse": lse}
