"""CPU checks: the router, the expert layer and the adapters refuse a pointer
that their kernels could not read or write element by element, before anything
is launched."""

import pytest

from test_abi_operators import P, layer, lib, lora, route  # noqa: F401

ALIGNMENT = -2


@pytest.mark.parametrize("kw", [
    dict(logits=P(258)), dict(dtype=1, logits=P(257)), dict(ids=P(257)), dict(w=P(258)),
    dict(offs=P(258)), dict(order=P(259)), dict(tokens=129, ws=P(258), nws=1 << 20),
])
def test_route(lib, kw):  # noqa: F811
    assert route(lib, **kw) == ALIGNMENT


@pytest.mark.parametrize("kw", [
    dict(ids=P(258)), dict(w=P(257)), dict(s13=P(258)), dict(s2=P(259)), dict(xt=0, x=P(258)),
])
def test_layer(lib, kw):  # noqa: F811
    assert layer(lib, **kw) == ALIGNMENT


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [dict(offs=P(258)), dict(ids=P(257))])
def test_lora(lib, kw, back):  # noqa: F811
    assert lora(lib, back, **kw) == ALIGNMENT
