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
