"""GPU: the few-token expert layer where its blocks of h differ most, and what
it makes of values that are not finite."""

import pytest

from _helpers import lib
from test_gpu_moe import check_layer, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 16, 50])
def test_every_block_has_its_own_scale(T):
    """h of neighbouring 128-blocks differs by up to 2^12, so a sum under
    another block's scale is far off; bounds as in test_gpu_moe.py, and the same
    bits each time."""
    import torch
    fl = lib()
    F = 128 * 24
    c = make_layer(T, 4, 2, 64, F)
    g = torch.Generator(device="cuda").manual_seed(T)
    steps = torch.randint(-6, 7, (F // 128,), generator=g, device="cuda")
    up = c["w13"][:, F:].contiguous().view(torch.float8_e4m3fn).float()
    # codes near the middle of E4M3's range, so that 2^6 either way still fits
    up = torch.sign(up) * up.abs().clamp(1.0, 1.875)
    up = up.view(4, F // 128, 128, 64) * torch.exp2(steps)[None, :, None, None]
    c["w13"] = c["w13"].contiguous()
    c["w13"][:, F:] = up.view(4, F, 64).to(torch.float8_e4m3fn).view(torch.uint8)
    y = check_layer(fl, c)
    for _ in range(20):
        assert torch.equal(y, fl.moe_layer(**c))


def users(c, e):
    """Tokens that have expert e."""
    return (c["ids"] == e).any(1)


@pytest.mark.parametrize("T", [6, 40])
def test_weight_codes_that_are_not_finite(T):
    """An infinite or NaN E5M2 code of the gate or up weights reaches every
    output of its expert's tokens, one of the down weights their output of its
    row; nothing else changes by a bit."""
    import torch
    fl = lib()
    for code in (0x7C, 0xFC, 0x7F):
        c = make_layer(T, 5, 2, 200, 150, fmt="e5m2")
        y0 = fl.moe_layer(**c)
        hit = users(c, 3)
        assert hit.any() and not hit.all()
        for row in (17, 150 + 149):
            d = dict(c, w13=c["w13"].clone())
            d["w13"][3, row, 199] = code
            y = fl.moe_layer(**pad16(d))
            assert not torch.isfinite(y[hit].float()).any()
            assert torch.equal(y[~hit], y0[~hit])
        d = dict(c, w2=c["w2"].clone())
        d["w2"][3, 177, 149] = code
        y = fl.moe_layer(**pad16(d))
        assert not torch.isfinite(y[hit, 177].float()).any()
        y[:, 177] = y0[:, 177]
        assert torch.equal(y, y0)
    assert fl.device_status() == 0


def pad16(c):
    """Weights with rows of a multiple of 16 bytes."""
    import torch
    out = dict(c)
    for k in ("w13", "w2"):
        t = c[k]
        wide = torch.zeros((*t.shape[:2], (t.shape[2] + 15) // 16 * 16), dtype=torch.uint8,
                           device="cuda")
        wide[:, :, :t.shape[2]] = t
        out[k] = wide[:, :, :t.shape[2]]
    return out


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [6, 40])
def test_h_beyond_fp32(T, dtype):
    """Gate and up sums near 1e30 whose product is no FP32 number make NaN rows
    of the expert's tokens, and of no others."""
    import torch
    fl = lib()
    c = make_layer(T, 5, 2, 200, 150, dtype)
    y0 = fl.moe_layer(**c)
    hit = users(c, 2)
    assert hit.any() and not hit.all()
    c["scale13"][2] *= 1e30
    y = fl.moe_layer(**c)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.isnan(y[hit].float()).all()
    assert torch.equal(y[~hit], y0[~hit])
