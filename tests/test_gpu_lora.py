"""GPU: low-rank adapters beside a shared projection, forward and backward,
against their definitions in 64 bits, and the gradients against differences.

Bounds.  BF16 products are exact in FP32.  An FP32 operand enters as two BF16
terms: relative error at most 2^-17 (half a step of 2^-7, twice, the second on
a remainder that is at most half of its binade); a sum of n products loses at most n 2^-23 of the sum of
magnitudes.  So, with |.| the sum of the magnitudes of the products:
  v    2^-17 |x||A| (FP32 x) + K 2^-23 |x||A|
  out  alpha times v's bound carried through |B|, plus 2^-16 of |v||B| and of
       the sum, plus the BF16 rounding 2^-8 |out|
  dA   dv's bound carried through |x|, plus the same for its own sum; dB alike
and in the norm, where independent errors do not add up like magnitudes: the
same relative terms against the norm of the result (for out: the rounding)."""

import math

import pytest

from _helpers import lib

pytestmark = pytest.mark.gpu

SPLIT = 2.0 ** -17
SUM = 2.0 ** -23


def make(T, lengths, ids, n, R, K, N, xt="bfloat16", seed=0, sigma=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + T + n + R + K + N)

    def normal(*shape, s=1.0, dt=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * s).to(dt)

    dt = getattr(torch, xt)
    offs = [0]
    for l in lengths:
        offs.append(offs[-1] + l)
    assert offs[-1] <= T and len(ids) == len(lengths)
    return dict(
        x=normal(T, K, dt=dt), dy=normal(T, N, dt=dt), base=normal(T, N),
        dx_base=normal(T, K), A=normal(n, R, K, s=K ** -0.5), B=normal(n, R, N, s=0.1),
        alpha=0.5 + torch.rand(n, generator=g, device="cuda"),
        m_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda"),
        adapter_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))


def segments(c):
    offs, ids = c["m_offsets"].tolist(), c["adapter_ids"].tolist()
    return [(lo, hi, i) for lo, hi, i in zip(offs, offs[1:], ids) if i >= 0 and hi > lo]


def forward_ref(c):
    import torch
    x, A, B = c["x"].double(), c["A"].double(), c["B"].double()
    K, R = A.shape[2], A.shape[1]
    split = SPLIT if c["x"].dtype == torch.float32 else 0.0
    v = torch.zeros(x.shape[0], R, dtype=torch.float64, device="cuda")
    vb, out = torch.zeros_like(v), c["base"].double()
    ob = torch.zeros_like(out)
    for lo, hi, i in segments(c):
        al = c["alpha"][i].double()
        v[lo:hi] = x[lo:hi] @ A[i].t()
        vb[lo:hi] = (split + K * SUM) * (x[lo:hi].abs() @ A[i].abs().t())
        out[lo:hi] += al * (v[lo:hi] @ B[i])
        mag = al * ((v[lo:hi].abs() + vb[lo:hi]) @ B[i].abs())
        ob[lo:hi] = al * (vb[lo:hi] @ B[i].abs()) + 2.0 ** -16 * mag
    ob += 2.0 ** -8 * (out.abs() + ob)
    return out, ob, v, vb


def check_forward(fl, c, **kw):
    import torch
    c = {k: c[k] for k in ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")}
    out, v = fl.lora_apply(**c, **kw)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rv, vb = forward_ref(c)
    assert ((v.double() - rv).abs() <= vb).all()
    assert ((out.double() - ro).abs() <= ob).all()
    K = c["x"].shape[1]
    assert (v.double() - rv).norm() <= (SPLIT + (K / 16 + 16) * SUM) * rv.norm()
    assert (out.double() - ro).norm() <= (2.0 ** -8 + 2.0 ** -15) * ro.norm()
    used = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
    for lo, hi, i in segments(c):
        used[lo:hi] = True
    assert torch.equal(out[~used], c["base"][~used])
    return out, v


def backward_ref(c, v):
    import torch
    x, dy, A, B = (c[k].double() for k in ("x", "dy", "A", "B"))
    n, R, K = A.shape
    N = B.shape[2]
    v = v.double()
    dx = c["dx_base"].double()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    dAb, dBb, dxb = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(dx)
    for lo, hi, i in segments(c):
        al, T = c["alpha"][i].double(), hi - lo
        dv = al * (dy[lo:hi] @ B[i].t())
        mag = al * (dy[lo:hi].abs() @ B[i].abs().t())
        dvb = (SPLIT + N * SUM) * mag
        dx[lo:hi] += dv @ A[i]
        dxb[lo:hi] = dvb @ A[i].abs() + 2.0 ** -16 * ((dv.abs() + dvb) @ A[i].abs())
        dA[i] += dv.t() @ x[lo:hi]
        dB[i] += al * (v[lo:hi].t() @ dy[lo:hi])
        each = SPLIT + c["x"].shape[0] * SUM
        dAb[i] += dvb.t() @ x[lo:hi].abs() + each * ((dv.abs() + dvb).t() @ x[lo:hi].abs())
        dBb[i] += al * each * (v[lo:hi].abs().t() @ dy[lo:hi].abs())
    dxb += 2.0 ** -8 * (dx.abs() + dxb)
    return (dx, dxb), (dA, dAb), (dB, dBb)


def check_backward(fl, c, v, **kw):
    import torch
    d = {k: c[k] for k in ("dy", "x", "A", "B", "alpha", "m_offsets", "adapter_ids", "dx_base")}
    got = fl.lora_backward(v=v, **d, **kw)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for name, g, (r, b), rel in zip(("dx", "dA", "dB"), got, backward_ref(c, v),
                                    (2.0 ** -8 + 2.0 ** -15, 2.0 ** -15, 2.0 ** -15)):
        assert ((g.double() - r).abs() <= b).all(), name
        assert (g.double() - r).norm() <= rel * r.norm(), name
    return got


def random_v(c):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    return torch.randn(c["x"].shape[0], c["A"].shape[1], generator=g, device="cuda")


CASES = [
    # T, lengths, ids, n, R, K, N
    (1, [1], [0], 1, 1, 1, 1),
    (1, [1], [1], 2, 16, 256, 512),
    (8, [1] * 8, [3, 1, 0, 2, 7, 6, 5, 4], 8, 16, 1024, 768),
    (13, [1] * 9, [0, -1, 0, 1, 1, -1, 2, 0, 0], 3, 8, 200, 136),    # rows after the last
    (70, [3, 0, 17, 16, 30], [1, 0, -1, 1, 0], 2, 24, 333, 517),     # odd widths, empty, bare
    (333, [100, 1, 0, 200, 20], [0, 2, 2, 1, 2], 3, 64, 1000, 1001),
    (257, [257], [0], 1, 33, 96, 2048),
    (200, [64, 65, 63], [0, 1, 0], 2, 128, 512, 640),
    (40, [1] * 40, [i % 3 for i in range(40)], 3, 100, 448, 72),
    (2048, [512, 1024, 512], [1, 0, 1], 2, 16, 512, 1024),
    (1024, [1] * 1000, [(7 * i) % 11 - 1 for i in range(1000)], 10, 4, 64, 64),
    (100, [], [], 1, 8, 64, 64),                                     # no segment at all
    (700, [130, 63, 1, 64, 300, 129], [0, 1, 0, 2, 1, 0], 3, 32, 640, 1096),
    (900, [257, 0, 500, 100], [1, 0, -1, 1], 2, 64, 8, 2056),
    (600, [17, 583], [0, 0], 1, 128, 1992, 264),
    (5000, [1500, 2100, 1400], [0, 1, 0], 2, 48, 264, 520),          # long sums over rows
    (300, [299], [0], 1, 20, 8192, 64),                              # long sums over K
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
def test_forward(case, xt):
    check_forward(lib(), make(*case, xt=xt))


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
def test_backward(case, xt):
    c = make(*case, xt=xt)
    check_backward(lib(), c, random_v(c))


@pytest.mark.parametrize("off", [1, 4])
def test_strided_and_misaligned(off):
    """Rows and factors inside wider tensors full of NaN, at bases that rule
    out 16-byte accesses (off = 1) or leave them to some tensors."""
    import torch
    fl = lib()
    c = make(90, [40, 50], [1, 0], 2, 20, 208, 304)
    v = random_v(c)

    def inside(t, fill=float("nan")):
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 12), fill, dtype=t.dtype, device="cuda")
        part = wide[..., off:off + t.shape[-1]]
        part.copy_(t)
        return part

    d = {k: inside(t) if t.dtype == torch.bfloat16 else t for k, t in c.items()}
    out = inside(torch.zeros_like(c["base"]), 7.0)
    vv = inside(torch.zeros_like(v), 7.0)
    o1, v1 = check_forward(fl, d, out=out, v=vv)
    o2, v2 = check_forward(fl, c)
    assert torch.equal(o1, o2) and torch.equal(v1, v2)
    assert (out._base[:, :off] == 7).all() and (out._base[:, off + 304:] == 7).all()
    assert (vv._base[:, :off] == 7).all() and (vv._base[:, off + 20:] == 7).all()
    g1 = check_backward(fl, d, inside(v))
    g2 = check_backward(fl, c, v)
    for a, b in zip(g1, g2):
        assert torch.equal(a, b)


def test_in_place():
    import torch
    fl = lib()
    c = make(150, [70, 80], [0, -1], 1, 16, 128, 600)
    out, v = check_forward(fl, c)
    base = c["base"].clone()
    o2, _ = fl.lora_apply(base, c["x"], c["A"], c["B"], c["alpha"], c["m_offsets"],
                          c["adapter_ids"], out=base)
    assert o2 is base and torch.equal(base, out)
    dx, _, _ = check_backward(fl, c, v)
    dxb = c["dx_base"].clone()
    fl.lora_backward(c["dy"], c["x"], v, c["A"], c["B"], c["alpha"], c["m_offsets"],
                     c["adapter_ids"], dxb, dx=dxb)
    assert torch.equal(dxb, dx)


def test_mixed_types_in_backward():
    """dy FP32 beside x BF16, and the other way round."""
    import torch
    fl = lib()
    for keys in (("dy",), ("x",)):
        c = make(140, [60, 80], [0, 1], 2, 12, 160, 96)
        for k in keys:
            c[k] = c[k].float() * 1.2345
        check_backward(fl, c, random_v(c))


def test_non_finite_stays_in_its_rows():
    """A NaN or infinity in one request's rows reaches that request's outputs
    and its adapter's gradients, no others."""
    import torch
    fl = lib()
    for xt, more in (("bfloat16", 0), ("float32", 0), ("bfloat16", 400)):
        c = make(60 + more, [20, 25, 15, more], [0, 1, -1, 0], 2, 16, 192, 256, xt=xt)
        out, v = fl.lora_apply(c["base"], c["x"], c["A"], c["B"], c["alpha"], c["m_offsets"],
                               c["adapter_ids"])
        c["x"][22, 5] = float("nan")
        c["x"][23, 6] = float("inf")
        c["x"][50, 7] = float("nan")     # no adapter there
        c["dy"][22, 9] = float("nan")
        o2, v2 = fl.lora_apply(c["base"], c["x"], c["A"], c["B"], c["alpha"], c["m_offsets"],
                               c["adapter_ids"])
        assert torch.isnan(o2[22].float()).all() and torch.isnan(v2[22]).all()
        assert not torch.isfinite(v2[23]).any()
        keep = [t for t in range(60 + more) if t not in (22, 23)]
        assert torch.equal(out[keep], o2[keep]) and torch.equal(v[keep], v2[keep])
        dx, dA, dB = fl.lora_backward(c["dy"], c["x"], v, c["A"], c["B"], c["alpha"],
                                      c["m_offsets"], c["adapter_ids"], c["dx_base"])
        assert torch.isfinite(dA[0]).all() and torch.isfinite(dB[0]).all()
        assert torch.isnan(dA[1]).any() and torch.isnan(dB[1, :, 9]).all()
        assert torch.isnan(dx[22].float()).all()
        keep = [t for t in range(60 + more) if t != 22]
        assert torch.isfinite(dx[keep].float()).all()


def test_gradients_against_differences():
    """Directional differences of L = <G, out(x, A, B)>, linear in each of x,
    A and B: half of L(p + e) - L(p - e) is the derivative along e, up to the
    outputs' BF16 rounding, 2^-8 |G||out| at most for each evaluation (the
    norm of it, since the roundings are independent)."""
    import torch
    fl = lib()
    c = make(96, [40, 16, 30], [1, 0, 1], 2, 16, 320, 256)
    c["base"].zero_()
    c["dx_base"].zero_()
    G = c["dy"]
    keys = ("x", "A", "B")

    def L(d):
        out, v = fl.lora_apply(c["base"], d["x"], d["A"], d["B"], c["alpha"], c["m_offsets"],
                               c["adapter_ids"])
        return out.double(), v

    p = {k: c[k] for k in keys}
    out, v = L(p)
    dx, dA, dB = fl.lora_backward(G, c["x"], v, c["A"], c["B"], c["alpha"], c["m_offsets"],
                                  c["adapter_ids"], c["dx_base"])
    for k, grad in zip(keys, (dx, dA, dB)):
        # powers of two times p: p + e and p - e are BF16 numbers
        sign = (torch.randint(0, 2, p[k].shape, device="cuda") * 2 - 1).to(torch.bfloat16)
        e = torch.where(sign > 0, p[k], -0.5 * p[k])
        plus, _ = L(dict(p, **{k: (p[k].double() + e.double()).to(torch.bfloat16)}))
        minus, _ = L(dict(p, **{k: (p[k].double() - e.double()).to(torch.bfloat16)}))
        e = ((p[k].double() + e.double()).to(torch.bfloat16).double()
             - (p[k].double() - e.double()).to(torch.bfloat16).double()) / 2
        diff = (G.double() * (plus - minus)).sum() / 2
        want = (grad.double() * e).sum()
        noise = 2.0 ** -8 * ((G.double() * plus).norm() + (G.double() * minus).norm()) / 2
        if k == "x":     # dx itself is rounded to BF16
            noise = noise + 2.0 ** -8 * (grad.double() * e).norm()
        assert (diff - want).abs() <= 2 * noise, k


def test_repeatable_graph_and_streams():
    import torch
    fl = lib()
    c = make(300, [100, 0, 150, 50], [1, 0, 0, 1], 2, 32, 640, 384)
    fa = [c[k] for k in ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")]
    out, v = fl.lora_apply(*fa)
    ba = [c["dy"], c["x"], v] + [c[k] for k in ("A", "B", "alpha", "m_offsets", "adapter_ids",
                                                "dx_base")]
    want = (out, v) + fl.lora_backward(*ba)
    for _ in range(3):
        got = fl.lora_apply(*fa) + fl.lora_backward(*ba)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    mine = [torch.zeros_like(t) for t in want]
    w2 = torch.full((fl.fp8la_lora_workspace_bytes(300, 32),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fl.lora_apply(*fa, out=mine[0], v=mine[1])
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.lora_apply(*fa, out=mine[0], v=mine[1])
        ba[2] = mine[1]
        fl.lora_backward(*ba, dx=mine[2], dA=mine[3], dB=mine[4], workspace=w2)
    for _ in range(2):
        for m in mine:
            m.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, mine))


@pytest.mark.parametrize("offs,ids", [
    ([0, 30, 20], [0, 1]),      # decreasing
    ([1, 30, 40], [0, 1]),      # does not start at 0
    ([0, 30, 61], [0, 1]),      # past the last row
    ([0, 30, 40], [0, 2]),      # no such adapter
    ([0, 30, 40], [-2, 1]),
])
def test_bad_segments_write_nothing(offs, ids):
    import torch
    fl = lib()
    c = make(60, [30, 10], [0, 1], 2, 16, 128, 128)
    v = random_v(c)
    c["m_offsets"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    c["adapter_ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    out = torch.full_like(c["base"], 3.0)
    v2 = torch.full_like(v, 3.0)
    fa = [c[k] for k in ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")]
    fl.lora_apply(*fa, out=out, v=v2)
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert (out == 3).all() and (v2 == 3).all()
    dx = torch.full_like(c["dx_base"], 3.0)
    dA = torch.full((2, 16, 128), 3.0, device="cuda")
    dB = torch.full((2, 16, 128), 3.0, device="cuda")
    fl.lora_backward(c["dy"], c["x"], v, c["A"], c["B"], c["alpha"], c["m_offsets"],
                     c["adapter_ids"], c["dx_base"], dx=dx, dA=dA, dB=dB)
    assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
    assert (dx == 3).all() and (dA == 3).all() and (dB == 3).all()


def test_no_rows():
    import torch
    fl = lib()
    c = make(0, [0, 0], [0, 1], 2, 8, 64, 32)
    out, v = fl.lora_apply(c["base"], c["x"], c["A"], c["B"], c["alpha"], c["m_offsets"],
                           c["adapter_ids"])
    assert out.shape == (0, 32) and v.shape == (0, 8)
    dx, dA, dB = fl.lora_backward(c["dy"], c["x"], v, c["A"], c["B"], c["alpha"],
                                  c["m_offsets"], c["adapter_ids"], c["dx_base"])
    torch.cuda.synchronize()
    assert (dA == 0).all() and (dB == 0).all()


def test_refusals():
    import torch
    fl = lib()
    c = make(20, [20], [0], 1, 129, 64, 64)
    fa = [c[k] for k in ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")]
    with pytest.raises(fl.Fp8laError) as e:
        fl.lora_apply(*fa)
    assert e.value.status == fl.FP8LA_ERR_UNSUPPORTED
    c = make(20, [20], [0], 1, 16, 64, 64)
    fa = [c[k] for k in ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")]
    with pytest.raises(fl.Fp8laError) as e:
        fl.lora_backward(c["dy"], c["x"], random_v(c), *fa[2:], c["dx_base"],
                         workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fl.FP8LA_ERR_INVALID_ARG
    with pytest.raises(AssertionError):
        fl.lora_apply(*fa[:2], c["A"].float(), *fa[3:])


# ----------------------------------------- where one kernel hands over to another
@pytest.mark.parametrize("R", [4, 16, 17, 32, 64, 128])
@pytest.mark.parametrize("T,lengths,n", [
    (1, [1], 1),                                # a single row
    (7, [7], 1),
    (8, [1] * 8, 8),                            # one row each
    (31, [3, 0, 17, 11], 2),
    (64, [2] * 32, 3),
    (255, [1] * 200 + [55], 4),
    (256, [1] * 256, 5),                        # many short segments
    (300, [15] * 20, 3),
])
def test_short_segments_aligned(T, lengths, n, R):
    """Rows that TMA can read, from a single one up: every kernel's smallest
    tiles, with neighbours' rows beside each segment's."""
    ids = [i % (n + 1) - (i % (n + 1) == n) * (n + 1) for i in range(len(lengths))]
    c = make(T, lengths, ids, n, R, 264, 328, xt="bfloat16")
    check_forward(lib(), c)
    check_backward(lib(), c, random_v(c))


@pytest.mark.parametrize("R", [16, 17, 32, 64, 65])
@pytest.mark.parametrize("T,lengths", [
    (2047, [1000, 1047]),
    (2048, [2048]),
    (2305, [700, 1, 900, 127, 300, 201]),       # rows after the last, tiles cut short
    (2500, [39] * 64),                          # too short for the widest tiles
])
def test_many_rows_and_columns(T, lengths, R):
    """Both sides of the sizes from which the widest tiles are used."""
    ids = [i % 3 - (i % 3 == 2) * 3 for i in range(len(lengths))]
    c = make(T, lengths, ids, 2, R, 72, 4104, xt="bfloat16")
    check_forward(lib(), c)


@pytest.mark.parametrize("ld", [1 << 13, 1 << 45])
def test_single_row_of_any_stride(ld):
    """The stride of a single row or adapter is never used."""
    import torch
    fl = lib()
    T, n, R, K, N = 1, 1, 1, 256, 512
    c = make(T, [1], [0], n, R, K, N, xt="bfloat16")
    v = random_v(c)
    (want, wv), wb = check_forward(fl, c), check_backward(fl, c, v)
    P = {k: t.data_ptr() for k, t in c.items()}
    out, dx = torch.empty_like(c["base"]), torch.empty_like(c["dx_base"])
    gv, dA, dB = torch.empty_like(wv), torch.empty_like(wb[1]), torch.empty_like(wb[2])
    ws = torch.empty(fl.fp8la_lora_workspace_bytes(T, R), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    fl.fp8la_lora_apply(P["base"], ld, P["x"], 1, ld, T, P["A"], ld, ld, P["B"], ld, ld,
                        P["alpha"], n, R, K, N, 1, P["m_offsets"], P["adapter_ids"],
                        out.data_ptr(), ld, gv.data_ptr(), ld, s)
    fl.fp8la_lora_backward(P["dy"], 1, ld, P["x"], 1, ld, v.data_ptr(), ld, T, P["A"], ld, ld,
                           P["B"], ld, ld, P["alpha"], n, R, K, N, 1, P["m_offsets"],
                           P["adapter_ids"], P["dx_base"], ld, dx.data_ptr(), ld, dA.data_ptr(),
                           dB.data_ptr(), ws.data_ptr(), ws.numel(), s)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for g, w in zip((out, gv, dx, dA, dB), (want, wv, *wb)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("R", [8, 17, 48, 128])
@pytest.mark.parametrize("T,lengths,K", [
    (128, [128], 64),
    (130, [1] * 130, 100),                      # one row each, K short of a stage
    (300, [15] * 20, 264),
    (1000, [400, 129, 0, 471], 1996),
])
def test_fp32_rows_aligned(T, lengths, K, R):
    """FP32 rows that TMA can read, K ending inside a stage."""
    ids = [i % 3 - (i % 3 == 2) * 3 for i in range(len(lengths))]
    c = make(T, lengths, ids, 2, R, K, 328, xt="float32")
    check_forward(lib(), c)
    check_backward(lib(), c, random_v(c))


@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_non_finite_rows_stay_their_own(xt, value):
    """A non-finite input makes its own row of V and out non-finite, no other."""
    import torch
    fl = lib()
    c = make(300, [170, 130], [1, 0], 2, 24, 264, 328, xt=xt)
    names = ("base", "x", "A", "B", "alpha", "m_offsets", "adapter_ids")
    out0, v0 = fl.lora_apply(*[c[k] for k in names])
    c["x"][131, 77] = value
    c["x"][299, 263] = value
    out, v = fl.lora_apply(*[c[k] for k in names])
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[131, 299]] = False
    assert torch.equal(v[keep], v0[keep]) and torch.equal(out[keep], out0[keep])
    assert not torch.isfinite(v[~keep]).any() and not torch.isfinite(out[~keep]).any()
