"""GPU: what the attention over the key/value cache makes of its limits: calls without
rows, sides without tokens, weights that underflow, V's scales and rows of any size.
Bounds are those of _kv.py."""

import math

import pytest

from _helpers import lib
from _kv import attend, check, close, fp8, make, reference, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("D", [64, 256])
def test_segments_without_rows(D, prefix):
    """max_rows 0 is the rows of the longest segment of a padded batch in an idle step."""
    import torch
    fl = lib()
    c = make((70, 0), (0, 0), 2, 4, D, 16, prefix=prefix, pad_rows=5)
    out = torch.full((5, 8, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 8), 9.0, device="cuda")
    attend(fl, c, out=out, lse=lse, max_rows=0)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.all(out == 9.0) and torch.all(lse == 9.0)
    c["offs"][1:] = 1       # a segment with a row, of more than max_rows
    attend(fl, c, out=out, lse=lse, max_rows=0)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert torch.all(out == 9.0) and torch.all(lse == 9.0)


@pytest.mark.parametrize("what", ["k", "k_scale", "v_scale"])
@pytest.mark.parametrize("rows,tokens", [(1, 100), (2, 20000), (70, 100), (70, 20000)])
def test_nan_beside_a_side_without_tokens(rows, tokens, what):
    """A row that a token made NaN stays so, its logarithm too, where the prefix or what
    follows it has no tokens; with many tokens its result is a joined one."""
    import torch
    fl = lib()
    c = make((tokens,), (rows,), 2, 2, 64, 16)
    want, wl = check(fl, c)
    bad = 0x7F if what == "k" else math.nan
    getattr(c["cache"], what)[int(c["table"][0, 1]), 1, 3] = bad
    out, lse = attend(fl, c, prefix_table=c["table"][0, :3].contiguous(),
                      prefix_len=torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out[:, :2], want[:, :2]) and torch.isnan(out[:, 2:]).all()
    assert (lse[:, :2] - wl[:, :2]).abs().max() < 1e-5 and torch.isnan(lse[:, 2:]).all()
    c = make((0, 0), (rows, rows), 2, 2, 64, 16, prefix=tokens)
    want, wl = check(fl, c)
    getattr(c["cache"], what)[int(c["prefix_table"][1]), 1, 3] = bad
    out, lse = attend(fl, c)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.equal(out[:, :2], want[:, :2]) and torch.isnan(out[:, 2:]).all()
    assert torch.equal(lse[:, :2], wl[:, :2]) and torch.isnan(lse[:, 2:]).all()


@pytest.mark.parametrize("rows,tokens,first", [(1, 40, 32), (1, 384, 256), (2, 20000, 15000),
                                               (100, 640, 384)])
def test_not_finite_value_of_a_negligible_token(rows, tokens, first):
    """Every token from `first` on has a weight that underflows, those of a whole warp or
    CTA among them; a V that is not finite still reaches its element of the rows."""
    import torch
    fl = lib()
    c = make((tokens,), (rows,), 1, 1, 64, 16)
    cache, j = c["cache"], torch.arange(first, tokens, device="cuda")
    page, place = c["table"][0][j // 16].long(), j % 16
    sign = torch.where(torch.randn(64, device="cuda") > 0, 1.0, -1.0)
    c["q"] = (sign * (1 + torch.rand(c["q"].shape, device="cuda"))).to(torch.bfloat16)
    cache.k[page, 0, place] = (-448 * sign).to(fp8("e4m3")).view(torch.uint8)
    cache.k_scale[page, 0, place] = 1.0
    cache.v[page[1], 0, place[1], 5] = 0x7F
    out, lse = check(fl, c)
    assert torch.isnan(out[:, 0, 5]).all() and int(torch.isnan(out).sum()) == rows
    assert torch.isfinite(lse).all()


def _endless(fl, S_long, rows, len_long, D, short_rows, prefix=None):
    """Sequences of the greatest length, all of their pages the same one, and a short one;
    out and lse to be left alone."""
    import torch
    page = 2 ** 20
    cache = fl.kv_cache(1, 1, page, D)
    table = torch.zeros(S_long + 1, 2 ** 11, dtype=torch.int32, device="cuda")
    lens = torch.tensor([len_long] * S_long + [200], dtype=torch.int32, device="cuda")
    offs = torch.tensor([rows * i for i in range(S_long + 1)] + [rows * S_long + short_rows],
                        dtype=torch.int32, device="cuda")
    T = rows * S_long + short_rows
    q = torch.ones(T, 1, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    lse = torch.full((T, 1), 5.0, device="cuda")
    fl.kv_attention(q, cache, offs, lens, table, max_rows=max(rows, short_rows), out=out, lse=lse)
    torch.cuda.synchronize()
    return fl.device_status(), out, lse


@pytest.mark.parametrize("S,rows,short", [(40, 64, 100), (140, 256, 3)])
def test_too_much_work_for_either_kernel_writes_nothing(S, rows, short):
    """2^31 tiles of short segments, or of long ones, beside one of the other kind."""
    import torch
    fl = lib()
    status, out, lse = _endless(fl, S, rows, 2 ** 31 - 4096, 16, short)
    assert status == fl.FP8LA_ERR_DEVICE_ARG
    assert torch.all(out == 5.0) and torch.all(lse == 5.0)


@pytest.mark.parametrize("D,rows,G,pages", [(256, 8192, 128, 64), (16, 32768, 64, 256)])
def test_too_much_work_for_the_prefix_writes_nothing(D, rows, G, pages):
    """2^31 tiles of the prefix, by either kernel, before sequences without tokens."""
    import torch
    fl = lib()
    cache = fl.kv_cache(1, 1, 2 ** 16 if D > 128 else 2 ** 20, D)
    table = torch.zeros(1, pages * (1 if D > 128 else 8), dtype=torch.int32, device="cuda")
    most = table.shape[1] * cache.shape[2]
    plen = torch.tensor([min(most, 2 ** 31 - 4096)], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.ones(rows, G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    lse = torch.full((rows, G), 5.0, device="cuda")
    fl.kv_attention(q, cache, offs, lens, table, out=out, lse=lse, prefix_table=table[0],
                    prefix_len=plen)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert torch.all(out == 5.0) and torch.all(lse == 5.0)


SPREADS = {
    "small first": lambda j, n, r: -148.0 if j == 0 else 2.0,
    "small last": lambda j, n, r: -140.0 if j == n - 1 else 2.0,
    "large first": lambda j, n, r: 100.0 if j == 0 else -40.0,
    "large last": lambda j, n, r: 100.0 if j == n - 1 else -40.0,
    "in turn": lambda j, n, r: 90.0 if j % 2 else -110.0,
    "rising": lambda j, n, r: -145.0 + 260.0 * j / n,
    "falling": lambda j, n, r: 115.0 - 260.0 * j / n,
    "any": lambda j, n, r: r.uniform(-145.0, 115.0),
    "all small": lambda j, n, r: r.uniform(-148.0, -130.0),
    "all large": lambda j, n, r: r.uniform(100.0, 115.0),
}


@pytest.mark.parametrize("spread", list(SPREADS))
@pytest.mark.parametrize("scale", [0.0, 0.125, 4.0, 60.0])
@pytest.mark.parametrize("rows,tokens,prefix", [(1, 70, 0), (3, 900, 0), (100, 300, 0),
                                                (2, 90, 150), (80, 100, 200)])
def test_scales_of_v_over_all_exponents(rows, tokens, prefix, scale, spread):
    """Whatever V's scales are, each token's mass and value count: with sharp scores a
    small one's alone, with scores of 0 all masses the same."""
    import random
    import torch
    fl = lib()
    r = random.Random(rows + tokens)
    c = make((tokens,), (rows,), 2, 2, 64, 16, prefix=prefix)
    for pages, n in ((c["table"][0], tokens), (c["prefix_table"], prefix)):
        j = torch.arange(n, device="cuda")
        size = torch.tensor([2.0 ** SPREADS[spread](i, n, r) for i in range(n)],
                            dtype=torch.float64, device="cuda").float()
        for h in range(2):
            c["cache"].v_scale[pages[j // 16].long(), h, j % 16] = size
    out, lse = attend(fl, c, scale=scale)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rl, lb = reference(c, scale=scale)
    # BF16's subnormals are 2^-133 apart, FP32's 2^-149
    assert close(out, ro, ob + 2.0 ** -134 + 2.0 ** -148)
    assert close(lse, rl, lb)


def _sink(c, s, j, x, value_scale=1.0):
    """Token j of sequence s (-1: the prefix) gets a score of about x in every row, and a
    row of V of zeros as kv_append writes it."""
    import torch
    cache, D, page = c["cache"], c["D"], c["page"]
    pages = c["prefix_table"] if s < 0 else c["table"][s]
    p, place = int(pages[j // page]), j % page
    u = c["u"]
    code = (u * (448.0 / float(u.abs().max()))).to(fp8("e4m3" if c["fmt"] == "e4m3" else "e5m2"))
    got = float((code.float() * u).sum()) * D ** -0.5
    for h in range(c["H"]):
        cache.k[p, h, place] = code.view(torch.uint8)
        cache.k_scale[p, h, place] = x / got
        cache.v[p, h, place] = torch.tensor([0, 0x80] * (D // 2), dtype=torch.uint8, device="cuda")
        cache.v_scale[p, h, place] = value_scale


def _with_direction(c):
    """Queries near one direction, so that a token can have the same score in all rows."""
    import torch
    D = c["D"]
    u = torch.randn(D, device="cuda").to(torch.bfloat16).float()
    c["u"] = u
    c["q"] = (u + 0.05 * torch.randn(c["q"].shape, device="cuda")).to(c["q"].dtype)
    return c


@pytest.mark.parametrize("fmt,sigma", [("e5m2", 1.0), ("e4m3", 0.05), ("e4m3", 1e-4), ("e4m3", 1e-6),
                                       ("e5m2", 1e-12)])
@pytest.mark.parametrize("x", [0.0, 5.0, 10.0, 20.0, 60.0])
@pytest.mark.parametrize("rows,tokens,D,prefix,q", [
    (1, 300, 64, 0, "bfloat16"), (2, 2000, 128, 0, "float32"), (3, 200, 256, 0, "bfloat16"),
    (130, 400, 128, 0, "bfloat16"), (70, 300, 64, 0, "float32"), (4, 100, 64, 300, "bfloat16"),
    (90, 100, 128, 500, "bfloat16")])
def test_rows_of_zeros_in_v(rows, tokens, D, prefix, q, x, fmt, sigma):
    """Tokens whose V is zero (a sink, a null key, padding), whose scale is 1 as kv_append
    writes it, far above the others'; they take mass and no precision."""
    import torch
    fl = lib()
    c = _with_direction(make((tokens,), (rows,), 2, 2, D, 16, q, fmt, prefix=prefix))
    c["cache"].v_scale.mul_(sigma)
    for j in (0, 1, 17, tokens - rows, tokens // 2):
        _sink(c, 0, j, x)
    if prefix:
        _sink(c, -1, 0, x)
        _sink(c, -1, prefix - 1, x / 2)
    check(fl, c)


@pytest.mark.parametrize("rows,D", [(1, 64), (2, 128), (90, 128), (1, 256)])
def test_nothing_but_zeros_in_v(rows, D):
    """All of V zero: out is 0, the logarithms are as ever."""
    import torch
    fl = lib()
    c = make((700, 40), (rows, min(rows, 40)), 2, 2, D, 16)
    c["cache"].v.fill_(0)
    c["cache"].v_scale.copy_(torch.where(c["cache"].v_scale.isnan(), math.nan, 1.0))
    out, _ = check(fl, c)
    assert torch.all(out == 0)


def test_rows_of_zeros_written_by_append():
    """The same through kv_append, in a program's order: append, attend."""
    import torch
    fl = lib()
    H, G, D, T = 2, 4, 128, 500
    g = torch.Generator(device="cuda").manual_seed(1)
    for fmt, rows in (("e5m2", 1), ("e4m3", 100)):
        cache = fl.kv_cache(-(-T // 16), H, 16, D, fmt)
        table = torch.arange(-(-T // 16), dtype=torch.int32, device="cuda").view(1, -1)
        offs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        u = torch.randn(D, generator=g, device="cuda")
        k = torch.randn(T, H, D, generator=g, device="cuda")
        v = 1e-3 * torch.randn(T, H, D, generator=g, device="cuda")
        k[:4], v[:4] = 1.5 * u, 0.0
        fl.kv_append(k, v, cache, offs, offs[1:], table)
        q = (u + 0.1 * torch.randn(rows, H * G, D, generator=g, device="cuda")).to(torch.bfloat16)
        c = dict(H=H, G=G, D=D, page=16, fmt=fmt, lens=[T], rows=[rows], prefix=0, table=table,
                 prefix_table=table[0, :0], cache=cache, q=q, T=rows, kv_lens=offs[1:],
                 offs=torch.tensor([0, rows], dtype=torch.int32, device="cuda"))
        assert float(cache.v_scale[0, 0, 0]) == 1.0
        check(fl, c)


def _lost(c, scale):
    """What an element may lose beside its bound, where the tokens that make it weigh next to
    nothing: a weight is a half, 2^-24 apart at the least where the row's largest one times
    V's scale is 2^7, so off by 2^-32 of that largest; and a part of a row weighs a product
    of two exponentials, of 2^-126 or more each, so 2^-252 or 0."""
    import torch
    T, H, G, D = c["T"], c["H"], c["G"], c["D"]
    res = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    cache, row = c["cache"], 0
    for s, (n, rows) in enumerate(zip(c["lens"], c["rows"])):
        at = []
        for pages, m in ((c["prefix_table"], c["prefix"]), (c["table"][s], n)):
            j = torch.arange(m, device="cuda")
            at.append((pages[j // c["page"]].long(), j % c["page"]))
        page, place = (torch.cat(x) for x in zip(*at))
        K, V = (torch.cat(x, 1) for x in zip(tokens(c, -1), tokens(c, s)))
        j = torch.arange(K.shape[1], device="cuda") - c["prefix"]
        seen = j[None] <= torch.arange(n - rows, n, device="cuda")[:, None]
        for h in range(H * G):
            x = c["q"][row:row + rows, h].double() * scale @ K[h // G].t()
            p = torch.softmax(x.masked_fill(~seen, -math.inf), 1)
            size = cache.v_scale[page, h // G, place].double()
            codes = V[h // G].abs() / size[:, None]
            some = (codes.amax(1) > 0).double()     # rows of zeros do not count
            top = (p * size * some).amax(1, keepdim=True)
            res[row:row + rows, h] = (2.0 ** -32 * top * (seen.double() @ codes) +
                                      torch.where(p < 2.0 ** -251, p, 0.0) @ V[h // G].abs())
        row += rows
    return res


@pytest.mark.parametrize("seed", range(60))
def test_drawn_values(seed):
    """Scales of V of any exponent, rows of zeros with any scale and scores of any
    sharpness together, on drawn shapes."""
    import random
    import torch
    fl = lib()
    r = random.Random(seed)
    S = r.choice([1, 2, 5])
    lens = [r.choice([r.randint(1, 40), r.randint(1, 900)]) for _ in range(S)]
    rows = [r.randint(1, n) if r.random() < 0.5 else min(n, r.randint(1, 3)) for n in lens]
    prefix = r.choice([0, 0, r.randint(1, 400)])
    c = make(lens, rows, r.choice([1, 2]), r.choice([1, 3, 8]), 16 * r.choice([1, 4, 5, 8, 8, 16]),
             r.choice([5, 16, 48]), r.choice(["bfloat16", "float32"]), r.choice(["e4m3", "e5m2"]),
             prefix=prefix, inside=r.random() < 0.3, seed=seed)
    cache, H, page = c["cache"], c["H"], c["page"]
    low, high = sorted((r.uniform(-145, 110), r.uniform(-145, 110)))
    some, zeros = r.choice([0.0, 0.02, 0.5, 1.0]), r.choice([0.0, 0.02, 0.5])
    g = torch.Generator(device="cuda").manual_seed(seed)
    for pages, n in [(c["table"][s], n) for s, n in enumerate(lens)] + [(c["prefix_table"], prefix)]:
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        p, place = pages[j // page].long(), j % page
        for h in range(H):
            v = cache.v_scale[p, h, place]
            pick = torch.rand(n, generator=g, device="cuda") < some
            e = low + (high - low) * torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
            v = torch.where(pick, torch.exp2(e).float(), v)
            z = torch.rand(n, generator=g, device="cuda") < zeros
            one = torch.rand(n, generator=g, device="cuda") < 0.7
            cache.v_scale[p, h, place] = torch.where(z & one, 1.0, v)
            codes = cache.v[p, h, place]
            codes[z] &= 0x80
            cache.v[p, h, place] = codes
    scale = r.choice([0.0, c["D"] ** -0.5, 2.0, 30.0])
    out, lse = attend(fl, c, scale=scale, max_rows=r.choice([None, max(rows)]))
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rl, lb = reference(c, scale=scale)
    assert close(out, ro, ob + 1.01 * _lost(c, scale) + 2.0 ** -134 + 2.0 ** -148)
    assert close(lse, rl, lb)
