"""GPU: the router and the few-token mixture-of-experts layer against their
definitions in 64 bits.

Bounds of the layer, from its roundings:
* an activation enters as two E4M3 terms: relative error at most 2^-9 (half a
  step of 2^-3, twice, the second on a remainder that is at most half of its
  binade), none for a BF16 value above 2^-15 of its K slice's largest, and an
  absolute error of at most 2^-22 of the slice's largest;
* h takes the same path, y is rounded once to BF16 (2^-8).
Elementwise the errors are propagated through |W| (worst case, with the
library's 2^-22 K max|a| max|b| for the FP32 accumulation).  That grows like K
where real errors grow like sqrt(K), so the norm is bounded too: independent
relative errors give at most themselves in the norm of the result, 2^-8 for y
and 2^-9 for each of x (if FP32) and h."""

import math

import numpy as np
import pytest

from _helpers import lib, to_dev

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": ("float8_e4m3fn", 448.0), "e5m2": ("float8_e5m2", 57344.0)}


# ------------------------------------------------------------------- router
def route_ref(z, k, renorm):
    """Selection and weights in 64 bits; z: numpy fp64 [T][E]."""
    T, E = z.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        nan = np.isnan(z[t])
        key = np.where(nan, np.inf, z[t])
        order = sorted(range(E), key=lambda e: (not nan[e], -key[e], e))
        chosen = [e for e in order[:k] if z[t, e] != -np.inf]
        if not chosen:
            continue
        ids[t, :len(chosen)] = chosen
        with np.errstate(all="ignore"):
            m = z[t, chosen[0]]
            p = np.exp(z[t] - m)
            s = p[chosen].sum() if renorm else p.sum()
            w[t, :len(chosen)] = p[chosen] / s
    return ids, w


def sort_ref(ids, E):
    flat = np.where(ids < 0, E, ids).reshape(-1)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    return np.searchsorted(np.sort(flat), np.arange(E + 1)).astype(np.int32), order


def check_route(fl, z, k, renorm, pad=0):
    import torch
    T, E = z.shape
    zd = torch.zeros((T, E + pad), dtype=z.dtype, device="cuda")
    zd[:, :E] = z
    ids, w, offs, order = fl.moe_route(zd[:, :E], k, renormalise=renorm)
    torch.cuda.synchronize()
    rid, rw = route_ref(z.double().cpu().numpy(), k, renorm)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    # expf, one sum of E terms and a division: a few units of 2^-24 each
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=(8 + E) * 2.0 ** -23, atol=1e-38)
    roffs, rorder = sort_ref(rid, E)
    np.testing.assert_array_equal(offs.cpu().numpy(), roffs)
    np.testing.assert_array_equal(order.cpu().numpy(), rorder)


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (3, 33, 5), (128, 64, 8), (129, 64, 8), (100, 1024, 16),
    (1000, 257, 3), (5000, 8, 2), (9001, 128, 1), (40000, 16, 16),
])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_route(T, E, k, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + E + k)
    z = torch.randn(T, E, generator=g, device="cuda").to(getattr(torch, dtype))
    check_route(lib(), z, k, True, pad=3)
    if T <= 1000:
        check_route(lib(), z, k, False)


def test_route_ties_masks_and_specials():
    import torch
    inf, nan = math.inf, math.nan
    rows = [
        [1, 1, 1, 1, 1, 1],              # ties: lowest indexes
        [-inf] * 6,                      # no expert at all
        [-inf, 2, -inf, -inf, 2, -inf],  # fewer than k left
        [0.0, -0.0, 0.0, -1, -1, -1],    # zeros of both signs tie
        [nan, 1, 2, 3, -inf, 0],         # NaN first, weights NaN
        [3, inf, 1, 0, -inf, 2],         # +inf: NaN weights
        [-3.4e38, -3.4e38, -inf, -inf, -inf, -3.4e38],   # the type's lowest as a mask
        [88, -88, 3e38, 0, 1, 2],
    ]
    z = torch.tensor(rows, dtype=torch.float32, device="cuda")
    for renorm in (True, False):
        check_route(lib(), z, 3, renorm)
    check_route(lib(), z.repeat(40, 1), 3, True)


def test_route_no_tokens_and_no_sort():
    import torch
    fl = lib()
    z = torch.zeros((0, 8), device="cuda")
    ids, w, offs, order = fl.moe_route(z, 2)
    assert ids.shape == (0, 2) and order.numel() == 0
    assert torch.equal(offs.cpu(), torch.zeros(9, dtype=torch.int32))
    z = torch.randn(5, 8, device="cuda")
    ids, w, offs, order = fl.moe_route(z, 2, sort=False)
    assert offs is None and order is None
    ids2, w2, _, _ = fl.moe_route(z, 2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


@pytest.mark.parametrize("T", [15, 16, 17, 32, 33, 47, 64, 65, 96, 113, 127, 128, 129])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (64, 8), (1024, 16)])
def test_route_one_launch(T, E, k):
    """Token counts around a CTA's and a cluster's, a fifth of the logits masked."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T * E + k)
    z = torch.randn(T, E, generator=g, device="cuda")
    z = z.masked_fill(torch.rand(T, E, generator=g, device="cuda") < 0.2, -math.inf)
    check_route(lib(), z, k, True)


def test_route_a_million_tokens_without_sort():
    """Only the sort limits tokens x top_k: 2^20 + 9 tokens with 16 of 16."""
    import torch
    fl = lib()
    T = (1 << 20) + 9
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(T, 16, generator=g, device="cuda")
    ids, w, offs, order = fl.moe_route(z, 16, sort=False)
    torch.cuda.synchronize()
    top, want = torch.sort(z, dim=1, descending=True, stable=True)
    assert offs is None and order is None
    assert torch.equal(ids.long(), want)
    p = torch.softmax(top.double(), 1)
    assert ((w.double() - p).abs() <= 24 * 2.0 ** -23 * p + 1e-38).all()


# -------------------------------------------------------------------- layer
def make_layer(T, E, k, D, F, dtype="bfloat16", fmt="e4m3", seed=0, ldpad=0):
    """Random weights as the quantiser leaves them, and a routing with
    distinct experts."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + T + E + D + F)

    def codes(rows, cols):
        ft, top = FP8[fmt]
        w = torch.randn(E, rows, cols, generator=g, device="cuda") * 0.05
        amax = w.abs().amax(dim=(1, 2))
        q = (w * (top / amax)[:, None, None]).to(getattr(torch, ft))
        ld = (cols + 15) // 16 * 16 + 16 * ldpad
        out = torch.full((E, rows, ld), 0x7F, dtype=torch.uint8, device="cuda")
        out[:, :, :cols] = q.view(torch.uint8)
        return out[:, :, :cols], (amax / top).contiguous()

    x = torch.randn(T, D, generator=g, device="cuda").to(getattr(torch, dtype))
    w13, s13 = codes(2 * F, D)
    w2, s2 = codes(D, F)
    z = torch.randn(T, E, generator=g, device="cuda")
    ids = z.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    w = torch.rand(T, k, generator=g, device="cuda")
    return dict(x=x, ids=ids, weights=w, w13=w13, scale13=s13, w2=w2, scale2=s2, fmt=fmt)


def layer_ref(c, activation):
    """(y, elementwise bound), fp64, and the bound in the norm."""
    import torch
    ft = getattr(torch, FP8[c["fmt"]][0])
    x, ids, w = c["x"].double(), c["ids"].cpu(), c["weights"].double()
    T, D = x.shape
    F = c["w2"].shape[2]
    u = 2.0 ** -9
    xr = u if c["x"].dtype == torch.float32 else 0.0
    y = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    b = torch.zeros_like(y)
    for e in range(c["w13"].shape[0]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        W13 = c["w13"][e].contiguous().view(ft).double() * c["scale13"][e].double()
        W2 = c["w2"][e].contiguous().view(ft).double() * c["scale2"][e].double()
        tok, we = tok.cuda(), w[tok, slot][:, None]
        xt = x[tok]
        top = xt.abs().amax(1, keepdim=True)
        gu = xt @ W13.t()
        dgu = (xt.abs() @ W13.abs().t() * xr + 2.0 ** -22 * top * W13.abs().sum(1)
               + 2.0 ** -22 * D * top * W13.abs().max())
        g, up, dg, du = gu[:, :F], gu[:, F:], dgu[:, :F], dgu[:, F:]
        if activation == "silu":
            act = g * torch.sigmoid(g)
        else:
            act = g / 2 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
        h = act * up
        # |act'| < 1.13 for both; the activation itself to 2^-18
        dact = 1.13 * dg + 2.0 ** -18 * (act.abs() + 2.0 ** -3 * (g.abs() < 8))
        dh = dact * up.abs() + act.abs() * du + dact * du
        htop = (h.abs() + dh).amax(1, keepdim=True)
        y.index_add_(0, tok, we * (h @ W2.t()))
        dy = ((dh + u * (h.abs() + dh)) @ W2.abs().t() + 2.0 ** -22 * htop * W2.abs().sum(1)
              + 2.0 ** -22 * F * htop * W2.abs().max())
        b.index_add_(0, tok, we.abs() * dy)
    # the last term: half of BF16's smallest number, where y underflows
    b = b + 2.0 ** -8 * (y.abs() + b) + 2.0 ** -134
    return y, b, 2.0 ** -8 + 2.0 ** -9 * (2 if xr else 1)


def check_layer(fl, c, activation="silu", **kw):
    import torch
    y = fl.moe_layer(activation=activation, **c, **kw)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ref, bound, rel = layer_ref(c, activation)
    err = (y.double() - ref).abs()
    assert torch.isfinite(y.float()).all()
    bad = ~(err <= bound)
    assert not bad.any(), "%d of %d outside the bound, worst ratio %g" % (
        bad.sum(), bad.numel(), (err / bound)[bad].max())
    floor = 2.0 ** -134 * math.sqrt(err.numel())
    assert err.norm() <= rel * ref.norm() + floor, (err.norm() / ref.norm()).item()
    return y


@pytest.mark.parametrize("T,E,k,D,F", [
    (1, 1, 1, 16, 16),
    (1, 8, 2, 256, 128),
    (1, 4, 2, 1024, 1024),          # few items: K is split in both kernels
    (1, 2, 1, 1, 1),
    (7, 10, 3, 1000, 1430),
    (16, 3, 2, 130, 70),            # tails in every dimension
    (16, 4, 4, 512, 2048),          # every token with every expert
    (17, 64, 8, 640, 200),
    (40, 2, 2, 384, 320),           # 40 tokens in one tile
    (100, 2, 1, 333, 517),
    (128, 4, 4, 256, 256),          # 128 tokens of one expert: two tiles
    (128, 1024, 16, 64, 48),        # the most pairs and experts
    (3, 5, 2, 4096, 64),
])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_layer(T, E, k, D, F, dtype):
    check_layer(lib(), make_layer(T, E, k, D, F, dtype))


@pytest.mark.parametrize("T", [2, 33])
def test_layer_e5m2_gelu_strided(T):
    """E5M2 weights with padded rows that hold NaN codes, strided x and y."""
    import torch
    c = make_layer(T, 6, 2, 200, 96, fmt="e5m2", ldpad=1)
    wide = torch.full((T, 211), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:203] = c["x"]
    c["x"] = wide[:, 3:203]
    out = torch.full((T, 205), 7.0, dtype=torch.bfloat16, device="cuda")
    check_layer(lib(), c, "gelu_tanh", y=out[:, :200])
    assert torch.all(out[:, 200:] == 7.0)


@pytest.mark.parametrize("T", [5, 50])
def test_layer_slots_without_expert_and_twice(T):
    """Slots with id -1 (their weight may be NaN), tokens without any expert
    (a zero row), one expert twice in a token."""
    import torch
    c = make_layer(T, 6, 3, 160, 144)
    ids, w = c["ids"], c["weights"]
    ids[0] = -1
    ids[1, 1] = -1
    w[1, 1] = float("nan")
    ids[2] = 4
    ids[3, 0] = -1
    ids[T - 1] = -1
    c2 = dict(c, weights=torch.where(ids < 0, torch.zeros_like(w), w))
    fl = lib()
    y = fl.moe_layer(**c)
    torch.cuda.synchronize()
    assert torch.all(y[0] == 0) and torch.all(y[T - 1] == 0)
    y2 = check_layer(fl, c2)
    assert torch.equal(y, y2)


def test_layer_bad_ids_write_nothing():
    import torch
    fl = lib()
    for T, bad in ((4, 9), (20, -2)):
        c = make_layer(T, 9, 2, 64, 64)
        c["ids"][T - 1, 1] = bad
        y = torch.full((T, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        fl.moe_layer(**c, y=y)
        assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
        assert torch.all(y == 5.0)
        c["ids"][T - 1, 1] = 0
        check_layer(fl, c, y=y)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T", [3, 30])
def test_layer_non_finite_tokens(value, T):
    """A token with a non-finite activation gets a NaN row; the others are
    as without it."""
    import torch
    fl = lib()
    c = make_layer(T, 4, 2, 300, 100)
    y0 = fl.moe_layer(**c).clone()
    c["x"][1, 177] = value
    y1 = fl.moe_layer(**c)
    torch.cuda.synchronize()
    assert torch.isnan(y1[1].float()).all()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y0[keep], y1[keep])


@pytest.mark.parametrize("magnitude", [1e-30, 1e-15, 1e-6, 1e6, 1e25])
def test_layer_magnitudes(magnitude):
    """x over a wide range (its square stays inside fp32's); one element far
    above the rest of its slice."""
    import torch
    c = make_layer(4, 3, 2, 600, 128, "float32")
    c["x"] *= magnitude
    c["x"][2, 7] *= 1e4
    # h grows like x^2: w2's scale brings y back into BF16's range
    c["scale2"] = (c["scale2"] / magnitude if magnitude > 1 else c["scale2"]).contiguous()
    if magnitude == 1e25:
        c["scale13"] = c["scale13"] * 1e-12
    check_layer(lib(), c)


def test_layer_is_deterministic_and_order_free():
    """The same call gives the same bits; a token's row does not depend on
    the other tokens of the batch."""
    import torch
    fl = lib()
    c = make_layer(60, 8, 2, 512, 384)
    y = fl.moe_layer(**c)
    for _ in range(5):
        assert torch.equal(y, fl.moe_layer(**c))
    perm = torch.randperm(60, device="cuda")
    c2 = dict(c, x=c["x"][perm].contiguous(), ids=c["ids"][perm].contiguous(),
              weights=c["weights"][perm].contiguous())
    assert torch.equal(y[perm], fl.moe_layer(**c2))


def test_layer_streams_graph_and_workspace():
    """On a side stream, captured in a graph, with the caller's workspace
    full of NaN."""
    import torch
    fl = lib()
    c = make_layer(9, 8, 2, 256, 192)
    want = fl.moe_layer(**c)
    ws = torch.full((fl.fp8_moe_layer_workspace_bytes(9, 2, 8, 256, 192),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    y = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fl.moe_layer(**c, y=y, workspace=ws)
    s.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.moe_layer(**c, y=y, workspace=ws)
        fl.moe_layer(**c, y=y, workspace=ws)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_back_to_back_layers_chain():
    """Each layer reads the one before it, with no wait between the calls."""
    import torch
    fl = lib()
    c = make_layer(8, 8, 2, 256, 192)
    x = c["x"]
    for _ in range(6):
        x = fl.moe_layer(**dict(c, x=x))
    torch.cuda.synchronize()
    x2 = c["x"]
    for _ in range(6):
        x2 = fl.moe_layer(**dict(c, x=x2))
        torch.cuda.synchronize()
    assert torch.equal(x, x2)


def test_router_feeds_layer_and_grouped_calls():
    """moe_route's order and m_offsets drive the grouped quantiser and GEMM;
    its ids and weights drive the layer."""
    import torch
    fl = lib()
    c = make_layer(96, 8, 2, 256, 128)
    z = torch.randn(96, 8, device="cuda")
    ids, w, offs, order = fl.moe_route(z, 2)
    c["ids"], c["weights"] = ids, w
    y = check_layer(fl, c)
    rows = c["x"].float()[(order // 2).long()].contiguous()
    q, _, s = fl.quantize_pertensor_grouped(rows, offs)
    gu = fl.grouped_gemm(offs, q, c["w13"], s, c["scale13"]).float()
    h = (torch.nn.functional.silu(gu[:, :128]) * gu[:, 128:]).contiguous()
    q, _, s = fl.quantize_pertensor_grouped(h, offs)
    part = fl.grouped_gemm(offs, q, c["w2"], s, c["scale2"]).float()
    out = torch.zeros(96, 256, device="cuda")
    out.index_add_(0, (order // 2).long(), part * w.reshape(-1)[order.long()][:, None])
    # the grouped path quantises activations to E4M3 (2^-4 relative) twice
    assert (out - y.float()).norm() <= 2 * 2.0 ** -4 * y.float().norm()


def test_refusals():
    import torch
    fl = lib()
    c = make_layer(4, 4, 2, 64, 64)

    def refuses(status, **kw):
        with pytest.raises(fl.Fp8laError) as e:
            fl.moe_layer(**dict(c, **kw))
        assert e.value.status == status

    big = make_layer(129, 4, 2, 64, 64)
    with pytest.raises(fl.Fp8laError) as e:
        fl.moe_layer(**big)
    assert e.value.status == fl.FP8LA_ERR_UNSUPPORTED
    refuses(fl.FP8LA_ERR_INVALID_ARG,
            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros((4, 128, 65), dtype=torch.uint8, device="cuda")[:, :, :64]
    refuses(fl.FP8LA_ERR_ALIGNMENT, w13=odd)
    with pytest.raises(fl.Fp8laError) as e:
        fl.moe_route(torch.zeros((2, 32), device="cuda"), 17)
    assert e.value.status == fl.FP8LA_ERR_UNSUPPORTED
    with pytest.raises(fl.Fp8laError) as e:
        fl.moe_route(torch.zeros((2, 4), device="cuda"), 5)
    assert e.value.status == fl.FP8LA_ERR_INVALID_ARG
