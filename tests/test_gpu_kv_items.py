"""GPU: attention of many short pieces of work: several items a CTA, whose warps may get
ahead of each other.  Bounds are those of _kv.py."""

import pytest

from _helpers import lib
from _kv import attend, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q", ["bfloat16", "float32"])
@pytest.mark.parametrize("D", [64, 128])
def test_items_of_one_row_tile(D, q):
    """65 to 128 rows and 1 to 3 tiles of tokens an item, seven items a CTA: half of the
    warps that make weights have nothing to do but to bring rows that there are not."""
    import torch
    fl = lib()
    rows = [65 + (37 * i) % 64 for i in range(128)]
    lens = [n + (53 * i) % 173 for i, n in enumerate(rows)]
    c = make(lens, rows, 8, 1, D, 16, q)
    want, wl = check(fl, c, max_rows=128)
    for _ in range(20):
        out, lse = attend(fl, c, max_rows=128)
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("q", ["bfloat16", "float32"])
def test_items_of_one_and_two_row_tiles(q):
    """Both kinds in turn, with grouped heads and behind a prefix too."""
    import torch
    fl = lib()
    rows = [(65, 300, 100, 70, 257, 128, 90)[i % 7] for i in range(60)]
    lens = [n + (91 * i) % 150 for i, n in enumerate(rows)]
    check(fl, make(lens, rows, 8, 1, 64, 16, q), max_rows=300)
    few = [n // 8 for n in rows]
    check(fl, make([n + 5 * i for i, n in enumerate(few)], few, 4, 8, 128, 24, q, prefix=200),
          max_rows=max(few))
    # draft rows: 16 of them for 8 heads each are 128 rows
    c = make([16 + 3 * i for i in range(70)], [16] * 70, 8, 8, 128, 64, q)
    want, wl = check(fl, c, max_rows=16)
    for _ in range(20):
        out, lse = attend(fl, c, max_rows=16)
        assert torch.equal(out, want) and torch.equal(lse, wl)
