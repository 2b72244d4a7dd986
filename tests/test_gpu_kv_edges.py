"""GPU: what the attention over the key/value cache makes of its limits: calls without
rows, sides without tokens, weights that underflow, V's scales and rows of any size.
Bounds are those of _kv.py."""

import math

import pytest

from _helpers import lib
from _kv import attend, check, close, fp8, make, reference

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
