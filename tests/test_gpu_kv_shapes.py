"""GPU: the key/value cache's calls on drawn shapes, and the forms of the many-row kernel
one by one: both formats and row types, heads inside a page's tokens, a prefix, sequences
whose sums are long.  Bounds are those of _kv.py."""

import math
import random

import numpy as np
import pytest

import oracle
from _helpers import lib
from _kv import attend, check, close, fp8, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inside", [False, True])
@pytest.mark.parametrize("q", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("D", [48, 64, 80, 128])
def test_many_rows_in_every_form(D, fmt, q, inside):
    fl = lib()
    c = make((300, 129, 700), (300, 70, 90), 2, 2, D, 24, q, fmt, inside=inside)
    check(fl, c)
    c = make((40, 0, 130), (40, 70, 130), 2, 2, D, 16, q, fmt, prefix=333, inside=inside)
    check(fl, c)
    check(fl, c, causal=False)


def _mean_error(c, few, heads, got, gl):
    """The mean relative error of some rows and heads, all of them within their bounds."""
    import torch
    G = len(heads) // c["H"]
    q = c["q"][few][:, heads]
    # without causal a row sees what the last one of its sequence sees
    each = [reference(dict(c, lens=c["lens"][:1], rows=[1], T=1, G=G, q=q[i:i + 1]), scale=0.01)
            for i in range(len(few))]
    ro, ob, rl, lb = (torch.cat(x) for x in zip(*each))
    got, gl = got[few][:, heads], gl[few][:, heads]
    assert close(got, ro, ob) and close(gl, rl, lb)
    return ((got.double() - ro) / ro).mean().abs().item()


def _mean_bound(H, D):
    """A cut of 2^-23 at most for each 16 tokens of a piece of 32768 (of a warp's), all the
    same way: 2^-12.  And BF16's roundings, each even over 2^-8 of a value at most, so with a
    variance of 2^-16 / 3: with nearly even weights all rows have the same results, so that
    only those of the H D columns are independent; four of their mean's deviations."""
    return 2.0 ** -12 + 4 * 2.0 ** -8 / math.sqrt(3 * H * D)


@pytest.mark.parametrize("q", ["bfloat16", "float32"])
@pytest.mark.parametrize("D,n", [(64, 32768), (128, 32768), (128, 131072)])
def test_long_sums(D, n, q):
    """Values of one sign, whose sums the tensor cores cut: errors do not grow with the
    length."""
    import torch
    fl = lib()
    H, G = 8, 64
    c = make((n,), (80,), H, G, D, 64, q, spare=0)
    c["cache"].v.bitwise_and_(0x7F)
    out, lse = attend(fl, c, causal=False, scale=0.01)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    mean = _mean_error(c, [0, 1, 41, 79], [h * G + i for h in range(H) for i in (0, 63)], out, lse)
    assert mean <= _mean_bound(H, D)


def test_long_sums_of_few_rows():
    """The same for the few-row kernel, 131072 tokens of a sequence a piece, a fourth of
    which a warp adds up: 512 sequences of the same pages."""
    import torch
    fl = lib()
    S, n, H, G, D = 512, 2 ** 20, 1, 8, 128
    c = make((n,), (1,), H, G, D, 64, spare=0)
    c["cache"].v.bitwise_and_(0x7F)
    q = (1.5 * torch.randn(S, H * G, D, device="cuda")).to(torch.bfloat16)
    out, lse = fl.kv_attention(q, c["cache"], torch.arange(S + 1, dtype=torch.int32, device="cuda"),
                               c["kv_lens"].expand(S).contiguous(),
                               c["table"].expand(S, -1).contiguous(),
                               max_rows=1, scale=0.01)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    mean = _mean_error(dict(c, q=q), [0, 31, 200, 511], list(range(8)), out, lse)
    assert mean <= _mean_bound(H, D)


@pytest.mark.parametrize("rows,H,G,lens", [
    (1, 8, 8, [140000 + 811 * i for i in range(60)]),         # few rows: two pieces each
    (40, 8, 4, [34000 + 4600 * i for i in range(20)]),        # many: two to four
    (100, 1, 3, [90000, 100, 70000]),                         # parts of several CTAs
])
@pytest.mark.parametrize("prefix", [0, 20000])
def test_pieces(rows, H, G, lens, prefix):
    """Parts that go through in several pieces, items that one CTA does whole and those
    that are shared, behind a prefix too; sequences share pages."""
    import torch
    fl = lib()
    n = max(lens)
    c = make((n,), (rows,), H, G, 64, 64, prefix=prefix)
    S = len(lens)
    c.update(lens=lens, rows=[rows] * S, T=S * rows, table=c["table"].expand(S, -1).contiguous(),
             kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             offs=torch.arange(S + 1, dtype=torch.int32, device="cuda") * rows)
    c["q"] = (1.5 * torch.randn(S * rows, H * G, 64, device="cuda")).to(torch.bfloat16)
    out, lse = attend(fl, c, max_rows=rows)
    again, lse2 = attend(fl, c, max_rows=rows)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    for s in sorted({0, 1, S // 2, S - 1}):
        for h in sorted({0, H - 1}):
            lo = s * rows
            one = dict(c, lens=[lens[s]], rows=[rows], T=rows, H=1, G=G, table=c["table"][s:s + 1],
                       q=c["q"][lo:lo + rows, h * G:(h + 1) * G])
            one["cache"] = fl.KVCache(*(t[:, h:h + 1] for t in (
                c["cache"].k, c["cache"].v, c["cache"].k_scale, c["cache"].v_scale)))
            ro, ob, rl, lb = reference(one)
            assert close(out[lo:lo + rows, h * G:(h + 1) * G], ro, ob)
            assert close(lse[lo:lo + rows, h * G:(h + 1) * G], rl, lb)


def _drawn(seed):
    r = random.Random(seed)
    S = r.choice([1, 1, 2, 3, 7, 20])
    many = r.random() < 0.4
    lens = [r.choice([0, 1, r.randint(1, 40), r.randint(1, 700)]) for _ in range(S)]
    rows = [r.randint(0, n + r.choice([0, 0, 3])) if many else min(n, r.randint(0, 4)) for n in lens]
    if sum(rows) == 0:
        rows[0] = 1
    return dict(lens=lens, rows=rows, H=r.choice([1, 2, 3, 4]), G=r.choice([1, 2, 3, 5, 8, 9]),
                D=16 * r.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 11, 16]), page=r.randint(1, 130),
                q=r.choice(["bfloat16", "float32"]), fmt=r.choice(["e4m3", "e5m2"]),
                prefix=r.choice([0, 0, 1, r.randint(2, 300)]), inside=r.random() < 0.5, seed=seed,
                pad_rows=r.choice([0, 2])), r.random() < 0.7, r.random() < 0.5


@pytest.mark.parametrize("seed", range(60))
def test_drawn_attention(seed):
    import torch
    fl = lib()
    shape, causal, tight = _drawn(seed)
    c = make(**shape)
    T, Hq, D = c["T"], c["H"] * c["G"], c["D"]
    out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 9.0, device="cuda")
    check(fl, c, causal, out=out, lse=lse, max_rows=max(c["rows"]) if tight else None)
    used = sum(c["rows"])
    assert torch.all(out[used:] == 9.0) and torch.all(lse[used:] == 9.0)


@pytest.mark.parametrize("seed", range(20))
def test_drawn_append_and_read(seed):
    import torch
    fl = lib()
    r = random.Random(1000 + seed)
    S = r.choice([1, 2, 5])
    lens = [r.randint(0, 40) for _ in range(S)]
    rows = [r.randint(0, n) for n in lens]
    H, D, page = r.choice([1, 2, 3, 5]), 16 * r.randint(1, 16), r.randint(1, 20)
    dt, fmt = r.choice([torch.bfloat16, torch.float32]), r.choice(["e4m3", "e5m2"])
    T = sum(rows)
    need = [-(-n // page) for n in lens]
    cache = fl.kv_cache(sum(need) + 1, H, page, D, fmt)
    ids = np.random.default_rng(seed).permutation(sum(need) + 1).astype(np.int32)
    table = np.full((S, max(need) + 1), -1, np.int32)
    at, places = 0, []
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
        places += [(table[s, j // page], j % page) for j in range(lens[s] - rows[s], lens[s])]
    offs = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    kvl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.from_numpy(table).cuda()
    g = torch.Generator().manual_seed(seed)
    x = [(torch.randn(T + 2, H, D, generator=g) * torch.exp(3 * torch.randn(T + 2, H, 1, generator=g)))
         .to(dt) for _ in "kv"]
    fl.kv_append(x[0].cuda(), x[1].cuda(), cache, offs, kvl, table)
    k, v = fl.kv_read(cache, offs, kvl, table, T, dtype=torch.float32)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for a, codes, scales, back in ((x[0], cache.k, cache.k_scale, k), (x[1], cache.v, cache.v_scale, v)):
        want_c, want_s = np.zeros(codes.shape, np.uint8), np.ones(scales.shape, np.float32)
        f = a.float().numpy()
        for t, (p, place) in enumerate(places):
            for h in range(H):
                q, _, sc = oracle.quantize_pertensor(f[t, h][None], fmt)
                want_c[p, h, place], want_s[p, h, place] = q[0], sc
        assert np.array_equal(codes.cpu().numpy(), want_c)
        assert np.array_equal(scales.cpu().numpy(), want_s)
        for t, (p, place) in enumerate(places):
            value = codes[p, :, place].view(fp8(fmt)).float() * scales[p, :, place][:, None]
            assert torch.equal(back[t], value)
