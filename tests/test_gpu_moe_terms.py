"""GPU: how many bits of FP32 x and of h the few-token expert layer keeps.

Both enter as four E4M3 terms under a scale that brings the group's largest
value into [128, 256): the first is off by half a step of 2^-3, each further one
by 2^-5 of what the one before left, so 2^-4-5-5-5 = 2^-19 of the value, and at
least 2^-27 of the group's largest (half of E4M3's smallest step, 2^-10, on the
second pair's scale of 2^-10, against 2^7).  With two terms it would be 2^-9.

A result that is rounded to BF16 hides that unless large products cancel, so the
first two tests make them cancel; the third counts the outputs that are not the
BF16 neighbour of the exact one."""

import math

import pytest

from _helpers import lib
from test_gpu_moe import make_layer

pytestmark = pytest.mark.gpu

TERMS = 2.0 ** -19
FLOOR = 2.0 ** -27
SUM = 2.0 ** -22      # of K max|a| max|b|, as in every FP8 product here
FP8 = "float8_e4m3fn"


def codes(values):
    """FP8 codes of exactly representable values, rows of 16 bytes or more."""
    import torch
    q = values.to(getattr(torch, FP8))
    assert torch.equal(q.double(), values.double())
    return q.view(torch.uint8).contiguous()


def exact(c):
    """y in 64 bits and the bound of its error before the BF16 rounding."""
    import torch
    x = c["x"].double()
    F = c["w2"].shape[2]
    ft = getattr(torch, FP8)
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    b = torch.zeros_like(y)
    for t in range(x.shape[0]):
        for j, e in enumerate(c["ids"][t].tolist()):
            W13 = c["w13"][e].view(ft).double() * c["scale13"][e].double()
            W2 = c["w2"][e].view(ft).double() * c["scale2"][e].double()
            top = x[t].abs().max()
            gu = W13 @ x[t]
            d = W13.abs() @ (TERMS * x[t].abs() + FLOOR * top)
            d = d + SUM * x.shape[1] * top * W13.abs().max()
            g, u, dg, du = gu[:F], gu[F:], d[:F], d[F:]
            act = g * torch.sigmoid(g)
            h = act * u
            # |silu'| < 1.13; the activation itself to 2^-18
            da = 1.13 * dg + 2.0 ** -18 * act.abs()
            dh = da * u.abs() + act.abs() * du + da * du
            htop = (h.abs() + dh).max()
            dy = W2.abs() @ (dh + TERMS * (h.abs() + dh) + FLOOR * htop)
            dy = dy + SUM * F * htop * W2.abs().max()
            w = c["weights"][t, j].double()
            y[t] += w * (W2 @ h)
            b[t] += w.abs() * dy
    return y, b


def check(fl, c, rounding_hides):
    import torch
    y = fl.moe_layer(**c)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    want, b = exact(c)
    # The bound has to be one that two terms would break.
    assert (b <= rounding_hides * want.abs()).all()
    err = (y.double() - want).abs()
    assert (err <= b + 2.0 ** -8 * (want.abs() + b)).all(), (err / want.abs()).max().item()


@pytest.mark.parametrize("T", [1, 16, 40])
def test_fp32_x_keeps_its_low_bits(T):
    """Neighbouring columns of x differ by 2^-7 and meet weights of opposite
    sign: what is left of a row's sum is 2^-7 of its products, which two terms
    of x would miss by 2^-2."""
    import torch
    fl = lib()
    D, F, E = 16, 16, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    x = 1 + torch.rand(T, D, generator=g, device="cuda")
    x[:, 1::2] = x[:, 0::2] * (1 - 2.0 ** -7)
    w = 2.0 ** torch.randint(-1, 1, (E, 2 * F, D), generator=g, device="cuda")
    w[:, :, 1::2] = -w[:, :, 0::2]
    w2 = 2.0 ** torch.randint(-3, 3, (E, D, F), generator=g, device="cuda")
    c = dict(x=x, ids=torch.arange(T, device="cuda").remainder(E).to(torch.int32)[:, None],
             weights=torch.ones(T, 1, device="cuda"), w13=codes(w), w2=codes(w2),
             scale13=torch.full((E,), 16.0, device="cuda"),
             scale2=torch.ones(E, device="cuda"))
    check(fl, c, 2.0 ** -4)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [1, 16, 40])
def test_h_keeps_its_low_bits(T, dtype):
    """Neighbouring rows of h differ by 2^-7 (their up rows do, through a second
    column) and meet weights of opposite sign."""
    import torch
    fl = lib()
    D, F, E = 16, 16, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.zeros(T, D, device="cuda", dtype=getattr(torch, dtype))
    x[:, :2] = 1
    w = torch.zeros(E, 2 * F, D, device="cuda")
    w[:, :, 0] = 1
    w[:, :F, 2] = 1
    w[:, F + 1::2, 1] = 2.0 ** -7
    w2 = 2.0 ** torch.randint(-1, 1, (E, D, F), generator=g, device="cuda")
    w2[:, :, 1::2] = -w2[:, :, 0::2]
    c = dict(x=x, ids=torch.arange(T, device="cuda").remainder(E).to(torch.int32)[:, None],
             weights=torch.ones(T, 1, device="cuda"), w13=codes(w), w2=codes(w2),
             scale13=torch.tensor([1.37, 0.83], device="cuda"),
             scale2=torch.ones(E, device="cuda"))
    check(fl, c, 2.0 ** -4)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [9, 60])
def test_outputs_are_rounded_once(T, dtype):
    """Independent relative errors of 2^-18 in the norm move an output over the
    middle between two BF16 numbers, 2^-8 or 2^-9 of it apart, in 2^-9 to 2^-8
    of all cases, and more often where y is small.  One in 50 is allowed; 8 bits
    of h alone make it one in 5."""
    import torch
    fl = lib()
    c = make_layer(T, 8, 2, 512, 384, dtype)
    y = fl.moe_layer(**c)
    want, _ = exact(c)
    assert (y != want.to(torch.bfloat16)).double().mean() <= 1 / 50
