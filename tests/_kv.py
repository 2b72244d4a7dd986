"""Inputs and 64-bit references of the key/value cache's tests.

Every place of the cache that no token uses holds NaN codes and NaN scales, and so
do the rows of page tables behind a sequence's end (page numbers outside the cache):
a kernel that lets any of it in returns NaN.

Bounds of the attention.  A score is off by at most

    d = X (2^-22 + (D / 16 + 8) 2^-23),   X = the largest sum of |scale q_i k_i|

2^-22 for an FP32 q as the sum of two halves (a BF16 one is exact), one cut of 2^-23
for each of the D / 16 steps on the tensor cores (FP32 products are exact there: 11
and 4 significant bits), 8 more for the products with the scales, the exponent and
the sum with log2 of V's scale, each of them 2^-24 of a value up to a few X.  exp of
that is off by e = 1.01 d + 2^-21 relatively (ex2.approx 2^-22), twice where numerator
and denominator err apart; weights are rounded by 2^-11; sums of n weights in
steps of 16 lose n / 16 2^-23 and in FP32 n 2^-24.  So, with A = sum p |v|,

    |out - ref| <= 2^-8 |out| + A (2^-11 + 2 e + (n / 16 + 64) 2^-23),
    |lse - ref| <= e + (n / 16 + 64) 2^-23 + 2^-22 (1 + |lse|)

where 2^-8 is BF16's rounding.  Weights 2^-21 below the largest are off by 2^-32 of
it each, which 2^-11 of the largest covers for n < 2^21."""

import math

import numpy as np

TOP = {"e4m3": 448.0, "e5m2": 57344.0}


def fp8(fmt):
    import torch
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2


def make(lens, rows, H, G, D, page, q="bfloat16", fmt="e4m3", prefix=0, inside=False, seed=0,
         pad_rows=0, sigma=1.0, spare=3):
    """A cache with sequences of `lens` tokens, the last `rows` of each being the
    call's.  inside: the heads lie inside a page's tokens."""
    import torch
    import precision_linear_algebra_gb300 as fl
    g = torch.Generator(device="cuda").manual_seed(seed + sum(lens) + H + G + D + page)
    S = len(lens)
    need = [-(-n // page) for n in lens]
    shared = -(-prefix // page)
    P = sum(need) + shared + spare
    shape = (P, page, H) if inside else (P, H, page)
    codes = [torch.full((*shape, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full(shape, math.nan, device="cuda") for _ in "kv"]
    if inside:
        codes, scales = [c.transpose(1, 2) for c in codes], [s.transpose(1, 2) for s in scales]
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, max(need + [1]) + 1), 2 ** 30, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    c = dict(H=H, G=G, D=D, page=page, fmt=fmt, lens=list(lens), rows=list(rows), prefix=prefix,
             table=table, prefix_table=ids[at:at + shared].clone(),
             kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             prefix_len=torch.tensor([prefix], dtype=torch.int32, device="cuda"))
    seqs = [(table[s], n) for s, n in enumerate(lens)] + [(c["prefix_table"], prefix)]
    for pages, n in seqs:
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        p, place = pages[j // page].long(), j % page
        for code, scale in zip(codes, scales):
            x = torch.randn(n, H, D, generator=g, device="cuda")
            amax = x.abs().amax(-1, keepdim=True)
            code[p, :, place] = (x * (TOP[fmt] / amax)).to(fp8(fmt)).view(torch.uint8)
            size = torch.exp(0.5 * torch.randn(n, H, generator=g, device="cuda")) * sigma
            scale[p, :, place] = amax[..., 0] / TOP[fmt] * size
    c["cache"] = fl.KVCache(codes[0], codes[1], scales[0], scales[1], fmt)
    offs = [0]
    for n in rows:
        offs.append(offs[-1] + n)
    c["offs"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    T = offs[-1] + pad_rows
    c["T"] = T
    c["q"] = (1.5 * torch.randn(T, H * G, D, generator=g, device="cuda")).to(getattr(torch, q))
    return c


def tokens(c, s, n=None):
    """K and V of sequence s (-1: the prefix), [H][n][D] in 64 bits."""
    import torch
    pages = c["prefix_table"] if s < 0 else c["table"][s]
    n = (c["prefix"] if s < 0 else c["lens"][s]) if n is None else n
    j = torch.arange(n, device="cuda")
    p, place = pages[j // c["page"]].long(), j % c["page"]
    cache = c["cache"]
    res = []
    for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = codes[p, :, place].view(fp8(c["fmt"])).double() * scales[p, :, place].double()[..., None]
        res.append(x.transpose(0, 1))
    return res


def reference(c, causal=True, scale=None, q=None):
    """(out, its bound, lse, its bound), and the rows' NaN where a token is."""
    import torch
    T, H, G, D = c["T"], c["H"], c["G"], c["D"]
    scale = D ** -0.5 if scale is None else scale
    q = (c["q"] if q is None else q).double() * scale
    out = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    ob = torch.zeros_like(out)
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    lb = torch.zeros_like(lse)
    row = 0
    Kp, Vp = tokens(c, -1)
    for s, (n, rows) in enumerate(zip(c["lens"], c["rows"])):
        K, V = tokens(c, s)
        K, V = torch.cat([Kp, K], 1), torch.cat([Vp, V], 1)
        total = K.shape[1]
        if total and rows:
            j = torch.arange(total, device="cuda") - c["prefix"]
            pos = torch.arange(n - rows, n, device="cuda")
            # every row sees the whole prefix
            seen = (j[None, :] < 0) | (j[None, :] <= (pos[:, None] if causal else n))
            for h in range(H * G):
                qh, k, v = q[row:row + rows, h], K[h // G], V[h // G]
                x = (qh @ k.t()).masked_fill(~seen, -math.inf)
                X = (qh.abs() @ k.abs().t()).masked_fill(~seen, 0.0).nan_to_num(0.0).amax(1)
                m = x.amax(1, keepdim=True)
                some = m > -math.inf
                p = torch.where(some, torch.exp(x - torch.where(some, m, 0.0)), 0.0)
                l = p.sum(1, keepdim=True)
                pn = torch.where(some, p / l, 0.0)
                # 0 weights do not let a NaN of a token that is not seen in
                o = torch.where(some, pn @ v.nan_to_num(0.0, 0.0, 0.0), 0.0)
                bad = (~v.isfinite()).double()
                if bad.any():
                    o[(seen.double() @ bad) > 0] = math.nan
                A = pn @ v.abs().nan_to_num(0.0, 0.0, 0.0)
                d = X * (2.0 ** -22 + (D / 16 + 8) * 2.0 ** -23)
                e = 1.01 * d + 2.0 ** -21
                chain = (total / 16 + 64) * 2.0 ** -23
                out[row:row + rows, h] = o
                ob[row:row + rows, h] = A * (2.0 ** -11 + 2 * e + chain)[:, None]
                z = torch.where(some, m + torch.log(l), -math.inf)[:, 0]
                lse[row:row + rows, h] = z
                lb[row:row + rows, h] = e + chain + 2.0 ** -22 * (1 + z.abs())
        row += rows
    ob += 2.0 ** -8 * (out.abs() + ob)
    return out, ob, lse, lb


def close(got, want, bound):
    """Whether got is within the bound, NaN and -inf where want is."""
    import torch
    got = got.double()
    odd = ~want.isfinite()
    inf = want == -math.inf
    ok = torch.where(inf, got == -math.inf, torch.where(odd, ~got.isfinite(), (got - want).abs() <= bound))
    return bool(ok.all())


def attend(fl, c, causal=True, **kw):
    import torch
    if c["prefix"]:
        kw.setdefault("prefix_table", c["prefix_table"])
        kw.setdefault("prefix_len", c["prefix_len"])
    q = kw.pop("q", c["q"])
    return fl.kv_attention(q, c["cache"], c["offs"], c["kv_lens"], c["table"], causal=causal, **kw)


def check(fl, c, causal=True, scale=None, **kw):
    import torch
    out, lse = attend(fl, c, causal, scale=scale, **kw)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rl, lb = reference(c, causal, scale)
    used = sum(c["rows"])
    assert close(lse[:used], rl[:used], lb[:used])
    assert close(out[:used], ro[:used], ob[:used])
    fine = ro[:used].isfinite()
    err = (out[:used].double() - ro[:used])[fine]
    assert err.norm() <= 2.0 ** -8 * ro[:used][fine].norm() + 1e-30
    return out, lse
