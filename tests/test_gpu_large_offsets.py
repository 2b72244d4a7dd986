"""GPU: rows, adapters and experts that begin more than 2^32 bytes, and 2^31
elements, after the first: every operand lies in a wide buffer of a few GB."""

import pytest

from _helpers import lib
from test_gpu_lora import check_backward, check_forward, make, random_v
from test_gpu_moe import check_layer, check_route, make_layer

pytestmark = pytest.mark.gpu


def far(t):
    """t with its rows (or matrices, if it has three dimensions) so far apart
    that the last begins after 2^31 elements."""
    import torch
    n = t.shape[0]
    step = ((1 << 31) // (n - 1) + 64) // 64 * 64
    flat = torch.empty(step * (n - 1) + t[0].numel() * 2, dtype=t.dtype, device="cuda")
    inner = (t.shape[2] + 16, 1) if t.dim() == 3 else (1,)
    v = flat.as_strided(t.shape, (step,) + inner)
    v.copy_(t)
    assert (n - 1) * step >= 1 << 31
    return v


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,lengths,R,K,N", [
    (40, [10, 0, 17, 12], 8, 128, 96),          # mma.sync in all kernels
    (300, [130, 0, 65, 100], 24, 264, 200),     # tcgen05 for V and the gradients
    (2305, [700, 100, 900, 605], 32, 72, 4104),     # and for out
    (2305, [700, 100, 900, 605], 32, 4104, 72),     # and for dx
])
def test_adapters(T, lengths, R, K, N, xt):
    import torch
    fl = lib()
    c = make(T, lengths, [0, 1, 2, -1], 3, R, K, N, xt=xt)
    v = random_v(c)
    names = ("x", "base", "A", "B")
    d = dict(c, **{k: far(c[k]) for k in names})
    out, vv = far(torch.zeros_like(c["base"])), far(torch.zeros_like(v))
    check_forward(fl, d, out=out, v=vv)
    del out, vv
    d = dict(c, **{k: far(c[k]) for k in ("x", "dy", "dx_base", "A", "B")})
    check_backward(fl, d, far(v), dx=far(torch.zeros_like(c["dx_base"])))
    del d
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [5, 60])
def test_layer(T, dtype):
    import torch
    fl = lib()
    c = make_layer(T, 3, 2, 96, 80, dtype)
    for k in ("w13", "w2"):
        t = c[k]
        step = (1 << 31) // 2 + 4096
        flat = torch.empty(2 * step + t[0].numel() * 2, dtype=torch.uint8, device="cuda")
        ld = (t.shape[2] + 31) // 16 * 16
        c[k] = flat.as_strided(t.shape, (step, ld, 1))
        c[k].copy_(t)
    c["x"] = far(c["x"])
    check_layer(fl, c, y=far(torch.zeros(T, 96, dtype=torch.bfloat16, device="cuda")))
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [20, 200])
def test_router(T, dtype):
    import torch
    fl = lib()
    z = far(torch.randn(T, 40, device="cuda").to(getattr(torch, dtype)))
    ids, w, offs, order = fl.moe_route(z, 4)
    near = fl.moe_route(z.contiguous(), 4)
    torch.cuda.synchronize()
    for a, b in zip((ids, w, offs, order), near):
        assert torch.equal(a, b)
    check_route(fl, z.contiguous(), 4, True)
    del z
    torch.cuda.empty_cache()
