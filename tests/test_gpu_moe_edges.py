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
