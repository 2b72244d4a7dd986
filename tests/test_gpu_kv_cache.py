"""GPU: rows quantised into the key/value cache, and read back.

Both are exact: codes and scales equal the per-tensor quantiser's oracle on each
(row, head) bit for bit, and a value read back is one FP32 product, rounded to BF16
where that is asked for."""

import math

import numpy as np
import pytest

import oracle
from _helpers import lib
from _kv import fp8

pytestmark = pytest.mark.gpu

def setup(lens, rows, H, D, page, fmt, inside=False, seed=0, width=None):
    """A cache of 0xA5 codes and scales of 7, and where each row goes."""
    import torch
    import precision_linear_algebra_gb300 as fl
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 2
    shape = (P, page, H) if inside else (P, H, page)
    codes = [torch.full((*shape, D), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full(shape, 7.0, device="cuda") for _ in "kv"]
    if inside:
        codes, scales = [c.transpose(1, 2) for c in codes], [s.transpose(1, 2) for s in scales]
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((len(lens), (width or max(need)) + 1), -7, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    offs = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    places = [(table[s, j // page], j % page) for s, (n, r) in enumerate(zip(lens, rows))
              for j in range(n - r, n)]
    dev = [torch.from_numpy(a).cuda() for a in (offs, np.array(lens, np.int32), table)]
    return fl.KVCache(*codes, *scales, fmt), dev, places


def values(rng, T, H, D, special=True):
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x *= np.exp(2 * rng.standard_normal((T, H, 1))).astype(np.float32)
    if special and T >= 4:
        x[0, 0] = 0.0
        x[1, 0, ::3] = -0.0
        x[2, -1, 1] = np.nan
        x[3, -1, 0] = np.inf
        x[1, -1] *= np.float32(1e-38)      # 448 / amax overflows: scale 1
    return x


CASES = [
    # lens, rows, H, D, page, dtype, fmt, heads inside
    ((5, 1, 9), (5, 1, 3), 3, 64, 4, "float32", "e4m3", False),
    ((33, 70), (0, 70), 1, 16, 16, "bfloat16", "e4m3", False),
    ((100,), (37,), 8, 128, 7, "bfloat16", "e5m2", True),
    ((20, 300, 1), (20, 1, 1), 5, 80, 1, "float32", "e5m2", False),
    ((64, 64), (64, 64), 2, 256, 64, "float32", "e4m3", True),
    ((17, 0, 4), (8, 0, 4), 4, 48, 5, "bfloat16", "e4m3", False),
    ((40,), (40,), 33, 96, 24, "float32", "e4m3", False),
]


@pytest.mark.parametrize("lens,rows,H,D,page,dtype,fmt,inside", CASES)
@pytest.mark.parametrize("layout", ["dense", "fused", "odd", "heads first"])
def test_append_and_read(lens, rows, H, D, page, dtype, fmt, inside, layout):
    import torch
    fl = lib()
    cache, (offs, kvl, table), places = setup(lens, rows, H, D, page, fmt, inside)
    T, pad = sum(rows), 2
    rng = np.random.default_rng(T + D)
    dt = getattr(torch, dtype)
    x = [torch.from_numpy(values(rng, T + pad, H, D)).to(dt) for _ in "kv"]
    if layout == "fused":
        whole = torch.zeros(T + pad, 3 * H, D, dtype=dt, device="cuda")
        dev = [whole[:, H:2 * H], whole[:, 2 * H:]]
    elif layout == "odd":
        dev = [torch.zeros((T + pad) * (H * D + 3) + 1, dtype=dt, device="cuda")[1:].view(
            T + pad, H * D + 3)[:, :H * D].unflatten(1, (H, D)) for _ in "kv"]
    elif layout == "heads first":
        dev = [torch.zeros(H, T + pad, D, dtype=dt, device="cuda").transpose(0, 1) for _ in "kv"]
    else:
        dev = [torch.zeros(T + pad, H, D, dtype=dt, device="cuda") for _ in "kv"]
    for d, a in zip(dev, x):
        d.copy_(a)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    fl.kv_append(dev[0], dev[1], cache, offs, kvl, table)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for a, codes, scales, c0, s0 in ((x[0], cache.k, cache.k_scale, before[0], before[2]),
                                     (x[1], cache.v, cache.v_scale, before[1], before[3])):
        want_c, want_s = c0.cpu().numpy().copy(), s0.cpu().numpy().copy()
        f = a.float().numpy()
        for t, (p, place) in enumerate(places):
            for h in range(H):
                q, _, sc = oracle.quantize_pertensor(f[t, h][None], fmt)
                want_c[p, h, place], want_s[p, h, place] = q[0], sc
        assert np.array_equal(codes.cpu().numpy(), want_c)
        assert np.array_equal(scales.cpu().numpy(), want_s)
    # back: the same rows, into the same layouts, rows behind the last left alone
    for d in dev:
        d.fill_(7.0)
    fl.kv_read(cache, offs, kvl, table, T + pad, k=dev[0], v=dev[1])
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for d, codes, scales in ((dev[0], cache.k, cache.k_scale), (dev[1], cache.v, cache.v_scale)):
        got = d.float().cpu()
        assert torch.all(got[T:] == 7.0)
        if T:
            p = torch.tensor([int(a) for a, _ in places])
            place = torch.tensor([int(b) for _, b in places])
            c = codes.cpu()[p, :, place].view(fp8(fmt)).float()
            want = (c * scales.cpu()[p, :, place][..., None]).to(dt).float()
            assert torch.equal(got[:T].nan_to_num(12345.0), want.nan_to_num(12345.0))
    if layout == "fused":
        assert torch.all(whole[:, :H] == 0)


def test_read_other_dtype_and_fresh_outputs():
    import torch
    fl = lib()
    cache, (offs, kvl, table), _ = setup((50, 3), (50, 2), 2, 64, 16, "e4m3")
    x = torch.randn(52, 2, 64, device="cuda")
    fl.kv_append(x, 2 * x, cache, offs, kvl, table)
    k32, v32 = fl.kv_read(cache, offs, kvl, table, 52, dtype=torch.float32)
    k16, v16 = fl.kv_read(cache, offs, kvl, table, 52)
    assert k16.dtype == torch.bfloat16 and torch.equal(k32.to(torch.bfloat16), k16)
    assert torch.equal(v32, 2 * k32) and torch.equal(v32.to(torch.bfloat16), v16)
    # half a step of E4M3: 2^-4 of the value, or of the smallest normal's step
    amax = x.abs().amax(-1, keepdim=True)
    assert ((k32 - x).abs() <= 2.0 ** -4 * x.abs() + amax / 448 * 2.0 ** -10 + 1e-6 * amax).all()


@pytest.mark.parametrize("what", ["offsets decrease", "offsets first", "offsets past", "length",
                                  "negative length", "shorter than its rows"])
def test_bad_segments(what):
    import torch
    fl = lib()
    cache, (offs, kvl, table), _ = setup((20, 20), (4, 4), 2, 64, 8, "e4m3")
    if what == "offsets decrease":
        offs = torch.tensor([0, 6, 4], dtype=torch.int32, device="cuda")
    elif what == "offsets first":
        offs = torch.tensor([1, 4, 8], dtype=torch.int32, device="cuda")
    elif what == "offsets past":
        offs = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    else:
        n = {"length": 1000, "negative length": -1}.get(what, 3)
        kvl = torch.tensor([20, n], dtype=torch.int32, device="cuda")
    x = torch.randn(8, 2, 64, device="cuda")
    fl.kv_append(x, x, cache, offs, kvl, table)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert torch.all(cache.k == 0xA5) and torch.all(cache.v_scale == 7.0)
    k = torch.full((8, 2, 64), 3.0, device="cuda")
    v = k.clone()
    fl.kv_read(cache, offs, kvl, table, 8, k=k, v=v)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert torch.all(k == 3.0) and torch.all(v == 3.0)


@pytest.mark.parametrize("page", [-1, 10 ** 6])
def test_bad_page(page):
    """Rows of a page outside the cache are left out, the others are written."""
    import torch
    fl = lib()
    cache, (offs, kvl, table), places = setup((20, 20), (4, 20), 2, 64, 8, "e4m3")
    good = cache.k.clone()
    x = torch.randn(24, 2, 64, device="cuda")
    fl.kv_append(x, x, cache, offs, kvl, table)
    want = cache.k.clone()
    cache.k.copy_(good)
    lost = int(table[1, 1])
    want[lost] = good[lost]
    table = table.clone()
    table[1, 1] = page
    fl.kv_append(x, x, cache, offs, kvl, table)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert torch.equal(cache.k, want)
    k = torch.full((24, 2, 64), 3.0, device="cuda")
    v = k.clone()
    fl.kv_read(cache, offs, kvl, table, 24, k=k, v=v)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    rows = torch.arange(24, device="cuda")
    out = (rows >= 4 + 8) & (rows < 4 + 16)
    assert torch.all(k[out] == 3.0) and torch.all(k[~out] != 3.0)


def test_many_segments_and_none():
    import torch
    fl = lib()
    S = 1024
    lens = [(i * 7) % 5 + 1 for i in range(S)]
    rows = [min(n, i % 3) for i, n in enumerate(lens)]
    cache, (offs, kvl, table), places = setup(lens, rows, 1, 16, 2, "e4m3")
    x = torch.randn(sum(rows), 1, 16, device="cuda")
    fl.kv_append(x, x, cache, offs, kvl, table)
    k, _ = fl.kv_read(cache, offs, kvl, table, sum(rows), dtype=torch.float32)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    amax = x.abs().amax(-1, keepdim=True)
    assert ((k - x).abs() <= 2.0 ** -4 * x.abs() + amax / 448 * 2.0 ** -10 + 1e-6 * amax).all()
    # no rows, no segments
    before = cache.k.clone()
    fl.kv_append(x[:0], x[:0], cache, offs * 0, kvl, table)
    fl.kv_append(x, x, cache, offs[:1], kvl[:0], table[:0])
    torch.cuda.synchronize()
    assert fl.device_status() == 0 and torch.equal(cache.k, before)
