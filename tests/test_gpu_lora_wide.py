"""GPU: the adapters' tcgen05 kernels beyond plain contiguous forward calls: in
place, as the backward pass uses them, inside padded rows, with segments that
are refused, with values that are not finite.  From 2048 rows, 64 rows a segment
and 2^23 outputs on, at ranks 17 to 64, all three kernels of a call are theirs;
from 128 rows on, V's and the gradients' are.  Bounds as in test_gpu_lora.py."""

import pytest

from _helpers import lib
from test_gpu_lora import check_backward, check_forward, make, random_v, segments

pytestmark = pytest.mark.gpu

FORWARD = ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")
BACKWARD = ("A", "B", "alpha", "m_offsets", "adapter_ids", "dx_base")

# Ragged, with an empty segment, two without an adapter and rows after the last;
# tiles of 128 rows end inside each.
LENGTHS, IDS, ROWS = [700, 0, 129, 900, 63, 300, 201], [0, 1, -1, 1, -1, 2, 0], 2305


def apply(fl, c, **kw):
    return fl.lora_apply(*[c[k] for k in FORWARD], **kw)


def backward(fl, c, v, **kw):
    return fl.lora_backward(c["dy"], c["x"], v, *[c[k] for k in BACKWARD], **kw)


@pytest.mark.parametrize("R", [17, 32, 48, 64])
def test_backward(R):
    """expand with A as its factor and no alpha."""
    c = make(ROWS, LENGTHS, IDS, 3, R, 4104, 264)
    check_backward(lib(), c, random_v(c))


@pytest.mark.parametrize("R", [32, 64])
@pytest.mark.parametrize("lengths,ids", [(LENGTHS, IDS), ([2305], [0]), ([], []),
                                         ([1000, 1305], [-1, 0])])
def test_in_place(lengths, ids, R):
    """out is base and dx is dx_base: rows without an adapter are left alone."""
    import torch
    fl = lib()
    c = make(ROWS, lengths, ids, 3, R, 4104, 4104)
    out, v = check_forward(fl, c)
    d = dict(c, base=c["base"].clone())
    o2, v2 = apply(fl, d, out=d["base"])
    assert o2 is d["base"] and torch.equal(o2, out) and torch.equal(v2, v)
    dx, dA, dB = check_backward(fl, c, v)
    d = dict(c, dx_base=c["dx_base"].clone())
    got = backward(fl, d, v, dx=d["dx_base"])
    assert got[0] is d["dx_base"]
    for a, b in zip(got, (dx, dA, dB)):
        assert torch.equal(a, b)


def inside(t, left, row, fill=float("nan")):
    """t in the middle of rows of `row` elements."""
    import torch
    wide = torch.full((*t.shape[:-1], row), fill, dtype=t.dtype, device="cuda")
    part = wide[..., left:left + t.shape[-1]]
    part.copy_(t)
    return part


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,lengths,ids,R,K,N", [
    (ROWS, LENGTHS, IDS, 40, 4099, 4101),
    (ROWS, LENGTHS, IDS, 64, 67, 4129),
    (300, [170, 0, 129], [1, 0, 2], 8, 321, 130),
    (300, [170, 0, 129], [1, 0, 2], 100, 130, 321),
])
def test_padded_rows(T, lengths, ids, R, K, N, xt):
    """Widths that are no multiple of 8, in rows padded to one with NaN: what
    lies beyond a row's end is neither read into a sum nor written."""
    import torch
    fl = lib()
    c = make(T, lengths, ids, 3, R, K, N, xt=xt)
    v = random_v(c)
    up = lambda t, extra=16: (t.shape[-1] + 7) // 8 * 8 + extra
    wide = ("base", "x", "dy", "dx_base", "A", "B")
    d = dict(c, **{k: inside(c[k], 8, up(c[k])) for k in wide})
    out = inside(torch.zeros_like(c["base"]), 8, up(c["base"]), 7.0)
    vv = inside(torch.zeros_like(v), 4, up(v), 7.0)
    check_forward(fl, d, out=out, v=vv)
    dx = inside(torch.zeros_like(c["dx_base"]), 8, up(c["dx_base"]), 7.0)
    check_backward(fl, d, inside(v, 4, up(v)), dx=dx)
    for t, left in ((out, 8), (vv, 4), (dx, 8)):
        assert (t._base[:, :left] == 7).all()
        assert (t._base[:, left + t.shape[1]:] == 7).all()


@pytest.mark.parametrize("K", [72, 200, 1000, 1992])
@pytest.mark.parametrize("R", [8, 24, 64, 128])
def test_fp32_rows_that_end_inside_a_stage(K, R):
    """FP32 x and dy of long segments, whose last stage is not whole."""
    c = make(700, [300, 0, 399], [1, 0, 0], 2, R, K, K + 8, xt="float32")
    check_forward(lib(), c)
    check_backward(lib(), c, random_v(c))


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,K,R", [(ROWS, 4104, 32), (400, 264, 24)])
@pytest.mark.parametrize("offs,ids", [
    ([0, 300, 200], [0, 1]),        # decreasing
    ([1, 300, 400], [0, 1]),        # does not start at 0
    ([0, 300, 100000], [0, 1]),     # past the last row
    ([0, 300, 400], [0, 2]),        # no such adapter
    ([0, 300, 400], [-2, 1]),
])
def test_bad_segments_write_nothing(T, K, R, offs, ids, xt):
    import torch
    fl = lib()
    c = make(T, [300, 100], [0, 1], 2, R, K, K, xt=xt)
    v = random_v(c)
    c["m_offsets"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    c["adapter_ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    outs = [torch.full_like(t, 3.0) for t in (c["base"], v, c["dx_base"])]
    grads = [torch.full((2, R, K), 3.0, device="cuda") for _ in range(2)]
    apply(fl, c, out=outs[0], v=outs[1])
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    backward(fl, c, v, dx=outs[2], dA=grads[0], dB=grads[1])
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    for t in outs + grads:
        assert (t == 3).all()
    c["m_offsets"] = torch.tensor([0, 300, 400], dtype=torch.int32, device="cuda")
    c["adapter_ids"] = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    check_forward(fl, c)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite(value):
    """In one row of x, dy, base or dx_base they reach that row's outputs and its
    adapter's gradients, and nothing else changes by a bit."""
    import torch
    fl = lib()
    c = make(ROWS, LENGTHS, IDS, 3, 32, 4104, 4104)
    v = random_v(c)
    o0, v0 = apply(fl, c)
    g0 = backward(fl, c, v)
    rows = torch.ones(ROWS, dtype=torch.bool, device="cuda")

    def only(got, want, touched):
        keep = rows.clone()
        keep[touched] = False
        assert torch.equal(got[keep], want[keep])

    # row 699 ends segment 0, 2304 is after the last, 1000 is adapter 1's
    for r, who in ((699, 0), (1000, 1), (2304, None)):
        assert [i for lo, hi, i in segments(c) if lo <= r < hi] == ([who] if who is not None
                                                                   else [])
        d = dict(c, x=c["x"].clone(), dy=c["dy"].clone())
        d["x"][r, 77] = value
        d["dy"][r, 4103] = value
        o, w = apply(fl, d)
        dx, dA, dB = backward(fl, d, v)
        for got, want in ((o, o0), (w, v0), (dx, g0[0])):
            only(got, want, [r])
            assert torch.isfinite(got[r]).all() if who is None else (
                not torch.isfinite(got[r]).any())
        for got, want in ((dA, g0[1]), (dB, g0[2])):
            keep = [i for i in range(3) if i != who]
            assert torch.equal(got[keep], want[keep])
        if who is not None:
            assert not torch.isfinite(dA[who, :, 77]).any()
            assert not torch.isfinite(dB[who, :, 4103]).any()
        d = dict(c, base=c["base"].clone(), dx_base=c["dx_base"].clone())
        d["base"][r, 5] = value
        d["dx_base"][r, 6] = value
        o, w = apply(fl, d)
        dx, dA, dB = backward(fl, d, v)
        assert not torch.isfinite(o[r, 5]) and not torch.isfinite(dx[r, 6])
        o[r, 5], dx[r, 6] = o0[r, 5], g0[0][r, 6]
        for got, want in zip((o, w, dx, dA, dB), (o0, v0) + g0):
            assert torch.equal(got, want)
    assert fl.device_status() == 0


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,lengths,ids,R,K,N", [
    (70, [3, 0, 17, 16, 30], [1, 0, -1, 1, 0], 8, 72, 96),
    (ROWS, LENGTHS, IDS, 32, 264, 4104),
    (ROWS, LENGTHS, IDS, 32, 4104, 264),
])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_factors_that_are_not_finite(T, lengths, ids, R, K, N, xt, value):
    """An element of A reaches its rank of V and all of out in its adapter's rows,
    one of B its column of out and all of dx; other rows, columns and adapters are
    as before bit for bit."""
    import torch
    fl = lib()
    c = make(T, lengths, ids, 3, R, K, N, xt=xt)
    v = random_v(c)
    mine = torch.zeros(T, dtype=torch.bool, device="cuda")
    for lo, hi, i in segments(c):
        if i == 1:
            mine[lo:hi] = True
    o0, v0 = apply(fl, c)
    g0 = backward(fl, c, v)
    d = dict(c, A=c["A"].clone())
    d["A"][1, 5, 66] = value
    o, w = apply(fl, d)
    assert not torch.isfinite(w[mine, 5]).any() and not torch.isfinite(o[mine]).any()
    assert torch.equal(o[~mine], o0[~mine]) and torch.equal(w[~mine], v0[~mine])
    w[:, 5] = v0[:, 5]
    assert torch.equal(w, v0)
    dx, dA, dB = backward(fl, d, v)
    assert not torch.isfinite(dx[mine, 66]).any()
    dx[:, 66] = g0[0][:, 66]
    for a, b in zip((dx, dA, dB), g0):
        assert torch.equal(a, b)
    d = dict(c, B=c["B"].clone())
    d["B"][1, 5, 66] = value
    o, w = apply(fl, d)
    assert not torch.isfinite(o[mine, 66]).any() and torch.equal(w, v0)
    o[:, 66] = o0[:, 66]
    assert torch.equal(o, o0)
    dx, dA, dB = backward(fl, d, v)
    assert not torch.isfinite(dx[mine]).any() and not torch.isfinite(dA[1, 5]).any()
    assert torch.equal(dx[~mine], g0[0][~mine]) and torch.equal(dB, g0[2])
    dA[1, 5] = g0[1][1, 5]
    assert torch.equal(dA, g0[1])
    assert fl.device_status() == 0


@pytest.mark.parametrize("T,lengths", [(40, [20, 20]), (700, [300, 400])])
def test_fp32_beyond_bf16(T, lengths):
    """FP32's largest values are infinite to an adapter; BF16's are not."""
    import torch
    fl = lib()
    c = make(T, lengths, [0, 0], 1, 16, 264, 128, xt="float32")
    c["A"] *= 2.0 ** -20
    c["B"] *= 2.0 ** -120
    top = torch.finfo(torch.float32).max
    c["x"][3, 7] = top
    c["x"][4, 7] = -top
    c["x"][25, 8] = float(torch.finfo(torch.bfloat16).max)
    out, v = apply(fl, c)
    assert not torch.isfinite(v[3:5]).any()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[3:5] = False
    assert torch.isfinite(v[keep]).all() and torch.isfinite(out[keep].float()).all()
    want = c["x"][25].double() @ c["A"][0].double().t()
    assert ((v[25].double() - want).abs() <= 2.0 ** -20 * want.abs()).all()
