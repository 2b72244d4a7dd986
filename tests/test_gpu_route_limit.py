"""GPU: the router's 32-bit token numbers end at 2^31 - 2^16 pairs.

Near 2^31 a CTA's token range used to wrap around, and the last tokens kept
whatever their outputs held.  The first refused count is checked through the
library's entry, which refuses before it launches anything; the largest accepted
one is run, with a single expert."""

import pytest

from _helpers import lib

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 2 ** 16 - 1


def test_most_tokens():
    import torch
    fl = lib()
    z = torch.zeros((MOST, 1), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((MOST, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.full((MOST, 1), 7.0, device="cuda")
    fl.moe_route(z, 1, sort=False, ids=ids, weights=w)
    torch.cuda.synchronize()
    assert int(ids.max()) == 0 and int(ids.min()) == 0
    assert float(w.max()) == 1 and float(w.min()) == 1


@pytest.mark.parametrize("top_k", [1, 3])
def test_more_is_refused(top_k):
    import torch
    fl = lib()
    z = torch.zeros((4, 4), device="cuda")
    ids = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 3), device="cuda")
    with pytest.raises(fl.Fp8laError) as e:
        fl.fp8_moe_route(z.data_ptr(), 0, MOST // top_k + 1, 4, 4, top_k, 1, ids.data_ptr(),
                         w.data_ptr(), None, None, None, 0,
                         torch.cuda.current_stream().cuda_stream)
    assert e.value.status == fl.FP8LA_ERR_UNSUPPORTED
