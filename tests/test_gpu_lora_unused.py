"""GPU: adapters without rows get zero gradients, whatever stands in their
slots (factors and alpha of a slot that is not in use may never have been set)."""

import pytest

from _helpers import lib
from test_gpu_lora import make, random_v

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,lengths,ids,R,K,N", [
    (20, [5, 0, 15], [0, 1, 3], 8, 64, 72),             # 1 has an empty segment, 2 none
    (20, [5, 0, 15], [-1, 1, -1], 8, 64, 72),           # none of them has rows
    (700, [300, 0, 400], [0, 1, 3], 24, 264, 520),
    (2500, [1200, 0, 1300], [3, 1, 0], 32, 264, 4104),
])
def test_slots_without_rows(T, lengths, ids, R, K, N, xt):
    import torch
    fl = lib()
    c = make(T, lengths, ids, 4, R, K, N, xt=xt)
    v = random_v(c)
    fa = ("x", "A", "B", "alpha", "m_offsets", "adapter_ids")
    args = lambda c: (c["dy"], c["x"], v) + tuple(c[k] for k in fa[1:]) + (c["dx_base"],)
    want = fl.lora_apply(c["base"], *[c[k] for k in fa]) + fl.lora_backward(*args(c))
    used = {i for l, i in zip(lengths, ids) if l}
    for value in (float("nan"), float("inf")):
        d = {k: t.clone() for k, t in c.items()}
        for i in range(4):
            if i not in used:
                for k in ("A", "B", "alpha"):
                    d[k][i] = value
        got = fl.lora_apply(d["base"], *[d[k] for k in fa]) + fl.lora_backward(*args(d))
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for i in range(4):
            if i not in used:
                assert (got[3][i] == 0).all() and (got[4][i] == 0).all()
