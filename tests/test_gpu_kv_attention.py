"""GPU: attention over the FP8 key/value cache against its definition in 64 bits;
the bounds are derived in _kv.py."""

import math

import pytest

from _helpers import lib
from _kv import attend, check, close, fp8, make, reference

pytestmark = pytest.mark.gpu

FEW = [
    # lens, rows, H, G, D, page
    ((1,), (1,), 1, 1, 64, 1),
    ((17,), (1,), 1, 8, 128, 16),
    ((63, 64, 65), (1, 1, 1), 2, 4, 128, 64),
    ((130, 1, 500), (2, 1, 3), 3, 5, 80, 24),
    ((1000,), (4,), 8, 8, 128, 100),
    ((257, 33), (1, 7), 2, 3, 96, 7),
    ((300, 40, 2), (1, 4, 2), 1, 16, 256, 48),
    ((90, 1200), (1, 1), 4, 1, 16, 13),
    ((5000, 3, 777, 64), (1, 1, 1, 1), 2, 2, 192, 128),
]


@pytest.mark.parametrize("lens,rows,H,G,D,page", FEW)
@pytest.mark.parametrize("q", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_few_rows(lens, rows, H, G, D, page, q, fmt):
    fl = lib()
    c = make(lens, rows, H, G, D, page, q, fmt, inside=fmt == "e5m2")
    check(fl, c, max_rows=max(rows))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,rows,H,G,D,page,q", [
    ((50, 300), (50, 300), 2, 1, 64, 16, "bfloat16"),
    ((400,), (129,), 1, 4, 128, 64, "bfloat16"),
    ((1000, 7), (77, 7), 2, 3, 80, 24, "float32"),
    ((260, 130, 515), (260, 1, 300), 1, 8, 128, 48, "bfloat16"),
    ((200, 333), (200, 100), 1, 2, 256, 100, "bfloat16"),
    ((384,), (384,), 1, 2, 128, 32, "float32"),
])
def test_many_rows(lens, rows, H, G, D, page, q, causal):
    fl = lib()
    c = make(lens, rows, H, G, D, page, q)
    check(fl, c, causal)


@pytest.mark.parametrize("prefix", [1, 64, 777])
@pytest.mark.parametrize("lens,rows,H,G,D,page,q", [
    ((1, 20, 300), (1, 1, 1), 2, 8, 128, 64, "bfloat16"),
    ((0, 5, 90), (0, 2, 3), 3, 2, 80, 24, "float32"),
    ((130,), (130,), 1, 4, 64, 16, "bfloat16"),
])
def test_prefix(prefix, lens, rows, H, G, D, page, q):
    fl = lib()
    c = make(lens, rows, H, G, D, page, q, prefix=prefix)
    check(fl, c, max_rows=max(rows))
    check(fl, c, causal=False)


def test_prefix_of_no_tokens():
    import torch
    fl = lib()
    c = make((90, 4), (1, 2), 2, 4, 64, 16)
    want = attend(fl, c)
    got = attend(fl, c, prefix_table=c["table"][0, :3].contiguous(),
                 prefix_len=torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.equal(got[0], want[0])
    assert (got[1] - want[1]).abs().max() < 1e-6


def test_one_long_sequence():
    """Work of one sequence over all SMs, many partial results for each row."""
    fl = lib()
    c = make((40000,), (1,), 1, 8, 128, 256)
    check(fl, c, max_rows=1)
    c = make((20001, 60), (3, 1), 2, 2, 64, 100, "float32")
    check(fl, c, max_rows=3)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_see_nothing(D):
    """Sequences without tokens, and causal rows before a sequence's begin."""
    import torch
    fl = lib()
    c = make((0, 5, 3, 0), (1, 9, 3, 4), 2, 3, D, 4)
    out, lse = check(fl, c)
    assert torch.all(out[:5] == 0) and torch.all(lse[:5] == -math.inf)
    out, lse = check(fl, c, causal=False)
    assert torch.all(lse[13:] == -math.inf) and torch.all(lse[1:13] > -math.inf)


def test_rows_behind_the_last_segment_are_left():
    import torch
    fl = lib()
    c = make((70, 9), (2, 1), 2, 4, 64, 16, pad_rows=5)
    out = torch.full((8, 8, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 8), 9.0, device="cuda")
    check(fl, c, out=out, lse=lse)
    assert torch.all(out[3:] == 9.0) and torch.all(lse[3:] == 9.0)


@pytest.mark.parametrize("rows", [1, 40])
def test_strided_and_misaligned(rows):
    """q a slice of a fused projection, out with heads first or at odd addresses."""
    import torch
    fl = lib()
    c = make((rows + 90, rows + 2), (rows, rows), 2, 4, 64, 16)
    want, wl = check(fl, c)
    T = c["T"]
    fused = torch.randn(T, 12, 64, device="cuda").to(torch.bfloat16)
    fused[:, :8] = c["q"]
    odd = torch.zeros(T * 600 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, 600)
    odd[:, 3:515] = c["q"].flatten(1)
    first = torch.zeros(8, T, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    out = torch.zeros(T * 515 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, 515)
    wide = torch.zeros(T, 11, device="cuda")
    for q, o, l in ((fused[:, :8], first, None),
                    (odd[:, 3:515].unflatten(1, (8, 64)), out[:, :512].unflatten(1, (8, 64)),
                     wide[:, :8])):
        got, gl = attend(fl, c, q=q, out=o, lse=l)
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        assert torch.equal(got, want) and torch.equal(gl, wl)
    assert torch.all(out[:, 512:] == 0) and torch.all(wide[:, 8:] == 0)


@pytest.mark.parametrize("rows", [1, 3, 70])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_values_that_are_not_finite(rows, fmt):
    """A NaN reaches the rows that see it and no others: all of them in K, one
    element in V."""
    import torch
    fl = lib()
    c = make((rows + 100, rows), (rows, rows), 2, 2, 64, 16, fmt=fmt)
    cache = c["cache"]

    def put(t, s, j, h, d, value):
        t[(int(c["table"][s, j // 16]), h, j % 16) + ((d,) if d is not None else ())] = value

    put(cache.v, 0, 40, 0, 5, 0xFF)                      # seen by every row
    put(cache.v, 0, rows + 99, 1, 7, 0x7F)               # by the last row only
    put(cache.v, 1, rows - 1, 0, 63, 0x7C if fmt == "e5m2" else 0x7F)
    put(cache.k, 1, rows // 2, 1, 0, 0x7F)               # by the rows from there on
    out, lse = attend(fl, c)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rl, lb = reference(c)
    first = rows + rows // 2
    assert torch.isnan(out[first:, 2:]).all() and torch.isnan(lse[first:, 2:]).all()
    ro[first:, 2:] = math.nan
    rl[first:, 2:] = math.nan
    assert close(out, ro, ob) and close(lse, rl, lb)
    assert int((~out[:rows].isfinite()).sum()) == 2 * rows + 2


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("value", [math.nan, math.inf, 0.0, -1.0])
def test_scales_that_are_not_positive(which, value):
    import torch
    fl = lib()
    c = make((40, 30), (2, 1), 1, 2, 64, 16)
    getattr(c["cache"], which)[int(c["table"][0, 2]), 0, 39 - 32] = value
    out, lse = attend(fl, c)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rl, lb = reference(c)
    keep = [0, 2]       # the row before the token, and the other sequence
    assert close(out[keep], ro[keep], ob[keep])
    if which == "v_scale" or math.isnan(value):
        assert torch.isnan(out[1]).all()


@pytest.mark.parametrize("sigma", [1e-30, 1e-6, 1e6, 1e30])
def test_scales_of_any_size(sigma):
    """V's values far from 1 (K's then at 1 as scores go by them)."""
    import torch
    fl = lib()
    c = make((500, 70), (2, 1), 2, 4, 64, 16)
    c["cache"].v_scale.mul_(sigma)
    check(fl, c)
    c["cache"].k_scale.mul_(sigma)
    check(fl, c, scale=0.125 / sigma)


def test_scales_that_differ_from_token_to_token():
    """V's scales over 40 binades within a sequence."""
    import torch
    fl = lib()
    c = make((900, 70), (1, 1), 2, 4, 64, 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    size = torch.exp2(40 * torch.rand(c["cache"].v_scale.shape, generator=g, device="cuda") - 20)
    c["cache"].v_scale.mul_(torch.exp2(torch.floor(torch.log2(size))))
    check(fl, c)


@pytest.mark.parametrize("q", ["bfloat16", "float32"])
@pytest.mark.parametrize("size", [1e-36, 1e-3, 30.0, 1e30])
def test_queries_of_any_size(q, size):
    """Elements and rows of very different sizes, and scores that make softmax pick
    one token."""
    import torch
    fl = lib()
    c = make((300, 40), (3, 40), 2, 2, 128, 16, q)
    T = c["T"]
    f = torch.exp2(torch.randint(-12, 1, (T, 4, 128), device="cuda").float())
    c["q"] = (c["q"].float() * f * size).to(getattr(torch, q))
    check(fl, c, scale=0.1 / size if size != 30.0 else None)


def test_sharp_and_flat():
    """One token takes all, or all are the same."""
    import torch
    fl = lib()
    c = make((2000,), (1,), 1, 8, 128, 64)
    check(fl, c, scale=50.0)
    check(fl, c, scale=0.0)
    check(fl, c, scale=-0.3)


@pytest.mark.parametrize("what", ["offsets", "length", "page", "prefix length", "max_rows"])
def test_bad_arguments_on_the_device(what):
    import torch
    fl = lib()
    c = make((70, 90, 50), (1, 2, 1), 2, 4, 64, 16, prefix=40)
    good, gl = check(fl, c)
    kw = {}
    if what == "offsets":
        c["offs"] = torch.tensor([0, 2, 1, 4], dtype=torch.int32, device="cuda")
    elif what == "length":
        c["kv_lens"] = torch.tensor([70, 10 ** 6, 50], dtype=torch.int32, device="cuda")
    elif what == "prefix length":
        c["prefix_len"] = torch.tensor([16 * 3 + 1], dtype=torch.int32, device="cuda")
    elif what == "max_rows":
        kw["max_rows"] = 1
    else:
        c["table"][1, 2] = -5
    out = torch.full_like(good, 5.0)
    lse = torch.full_like(gl, 5.0)
    attend(fl, c, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    if what == "page":
        assert torch.isnan(out[1:3]).all()
        assert torch.equal(out[[0, 3]], good[[0, 3]]) and torch.equal(lse[[0, 3]], gl[[0, 3]])
    else:
        assert torch.all(out == 5.0) and torch.all(lse == 5.0)


def test_many_segments():
    fl = lib()
    lens = [(i * 37) % 150 for i in range(1024)]
    rows = [min(n, (i * 5) % 3) for i, n in enumerate(lens)]
    c = make(lens, rows, 1, 4, 64, 16)
    check(fl, c, max_rows=2)


@pytest.mark.parametrize("rows", [1, 60])
def test_repeats_bit_for_bit(rows):
    import torch
    fl = lib()
    c = make([rows + 500 + 71 * i for i in range(7)], [rows] * 7, 2, 4, 128, 64, prefix=300)
    first = attend(fl, c)
    for _ in range(3):
        again = attend(fl, c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_rows_do_not_depend_on_their_neighbours_values():
    """A row's result stays the same where other sequences' queries and tokens
    change, their lengths being the same."""
    import torch
    fl = lib()
    c = make((300, 200), (1, 1), 2, 4, 128, 64)
    want, wl = attend(fl, c)
    for j in range(4):
        c["cache"].k[int(c["table"][1, j])] = 0x7F
    c["q"][1] = math.inf
    got, gl = attend(fl, c)
    assert torch.equal(got[0], want[0]) and torch.equal(gl[0], wl[0])
