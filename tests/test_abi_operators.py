"""CPU checks of the router's, the expert layer's and the adapters' entry
points: sizes of their workspaces, and refusals before anything is launched."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from precision_linear_algebra_gb300 import build
    import precision_linear_algebra_gb300 as fl
    build.build()
    return fl.load()


P = ctypes.c_void_p
A = P(256)      # an aligned address that is never read


def route(lib, **kw):
    a = dict(logits=A, dtype=0, tokens=4, experts=8, ld=8, k=2, renorm=1, ids=A, w=A, offs=A,
             order=A, ws=None, nws=0)
    a.update(kw)
    return lib.fp8_moe_route(a["logits"], a["dtype"], a["tokens"], a["experts"], a["ld"], a["k"],
                             a["renorm"], a["ids"], a["w"], a["offs"], a["order"], a["ws"],
                             a["nws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -1), (dict(tokens=-1), -1), (dict(experts=0), -1), (dict(k=0), -1),
    (dict(k=9), -1), (dict(ld=7), -1), (dict(logits=None), -1), (dict(ids=None), -1),
    (dict(w=None), -1), (dict(offs=None), -1), (dict(order=None), -1),
    (dict(experts=1025, ld=1025), -3), (dict(experts=32, ld=32, k=17), -3),
    (dict(tokens=129), -1),                       # a sort of this size needs a workspace
    (dict(tokens=129, ws=A, nws=8), -1),
    (dict(tokens=2 ** 31), -3),
    (dict(tokens=0, offs=None, order=None), 0),   # nothing to do
])
def test_route_refusals(lib, kw, status):
    assert route(lib, **kw) == status


def test_route_workspace(lib):
    f = lib.fp8_moe_route_workspace_bytes
    assert f(-1, 8) == -1 and f(8, 0) == -1 and f(8, 1025) == -1
    assert f(128, 1024) == 0 and f(129, 8) > 0
    assert f(1 << 20, 1024) <= 256 * 1025 * 4


def layer(lib, **kw):
    a = dict(x=A, xt=1, T=4, D=64, ldx=64, ids=A, w=A, k=2, E=4, w13=A, ld13=64, st13=96 * 64,
             s13=A, w2=A, ld2=48, st2=64 * 48, s2=A, F=48, fmt=0, act=0, y=A, ldy=64, ws=A,
             nws=1 << 40)
    a.update(kw)
    return lib.fp8_moe_layer(a["x"], a["xt"], a["T"], a["D"], a["ldx"], a["ids"], a["w"], a["k"],
                             a["E"], a["w13"], a["ld13"], a["st13"], a["s13"], a["w2"], a["ld2"],
                             a["st2"], a["s2"], a["F"], a["fmt"], a["act"], a["y"], a["ldy"],
                             a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), -1), (dict(fmt=2), -1), (dict(act=2), -1), (dict(T=-1), -1), (dict(D=0), -1),
    (dict(F=0), -1), (dict(k=0), -1), (dict(E=0), -1), (dict(ldx=63), -1), (dict(ldy=63), -1),
    (dict(ld13=63), -1), (dict(ld2=47), -1), (dict(st13=96 * 64 - 16), -1),
    (dict(st2=64 * 48 - 16), -1), (dict(x=None), -1), (dict(ids=None), -1), (dict(y=None), -1),
    (dict(ws=None), -1), (dict(nws=100), -1), (dict(T=129), -3), (dict(k=17), -3),
    (dict(E=1025), -3), (dict(D=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21, ld13=1 << 21), -3),
    (dict(w13=P(264)), -2), (dict(w2=P(257)), -2), (dict(ld13=72, st13=96 * 80), -2),
    (dict(st13=96 * 64 + 8), -2), (dict(x=P(257)), -2), (dict(y=P(257)), -2),
    (dict(ws=P(264)), -2), (dict(T=0), 0),
])
def test_layer_refusals(lib, kw, status):
    assert layer(lib, **kw) == status


def test_layer_workspace(lib):
    f = lib.fp8_moe_layer_workspace_bytes
    assert f(-1, 2, 8, 64, 64) == -1 and f(4, 0, 8, 64, 64) == -1 and f(4, 2, 8, 0, 64) == -1
    assert f(129, 2, 8, 64, 64) == -3 and f(4, 17, 32, 64, 64) == -3
    # codes of x and h and the pairs' sums, at least
    assert f(16, 2, 8, 4096, 14336) >= 32 * (2 * 4096 + 2 * 14336 + 4 * 4096)


def lora(lib, back=False, **kw):
    a = dict(base=A, ldb_=64, x=A, xt=1, ldx=32, T=10, A=A, lda=32, sa=8 * 32, B=A, ldb=64,
             sb=8 * 64, alpha=A, n=2, R=8, K=32, N=64, S=3, offs=A, ids=A, out=A, ldo=64, v=A,
             ldv=8, dy=A, dyt=1, lddy=64, dxb=A, lddxb=32, dx=A, lddx=32, dA=A, dB=A, ws=A,
             nws=1 << 40)
    a.update(kw)
    if back:
        return lib.fp8la_lora_backward(
            a["dy"], a["dyt"], a["lddy"], a["x"], a["xt"], a["ldx"], a["v"], a["ldv"], a["T"],
            a["A"], a["lda"], a["sa"], a["B"], a["ldb"], a["sb"], a["alpha"], a["n"], a["R"],
            a["K"], a["N"], a["S"], a["offs"], a["ids"], a["dxb"], a["lddxb"], a["dx"], a["lddx"],
            a["dA"], a["dB"], a["ws"], a["nws"], None)
    return lib.fp8la_lora_apply(
        a["base"], a["ldb_"], a["x"], a["xt"], a["ldx"], a["T"], a["A"], a["lda"], a["sa"],
        a["B"], a["ldb"], a["sb"], a["alpha"], a["n"], a["R"], a["K"], a["N"], a["S"], a["offs"],
        a["ids"], a["out"], a["ldo"], a["v"], a["ldv"], None)


COMMON = [
    (dict(xt=2), -1), (dict(T=-1), -1), (dict(S=-1), -1), (dict(n=0), -1), (dict(R=0), -1),
    (dict(K=0), -1), (dict(N=0), -1), (dict(ldx=31), -1), (dict(ldv=7), -1), (dict(lda=31), -1),
    (dict(ldb=63), -1), (dict(sa=8 * 32 - 1), -1), (dict(sb=8 * 64 - 1), -1), (dict(x=None), -1),
    (dict(A=None), -1), (dict(B=None), -1), (dict(alpha=None), -1), (dict(offs=None), -1),
    (dict(ids=None), -1), (dict(v=None), -1), (dict(R=129, ldv=129), -3), (dict(S=1025), -3),
    (dict(T=(1 << 19) + 1), -3), (dict(n=65536), -3), (dict(K=(1 << 22) + 1), -3),
    (dict(x=P(257)), -2), (dict(A=P(257)), -2), (dict(B=P(259)), -2), (dict(v=P(258)), -2),
    (dict(alpha=P(258)), -2),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(base=None), -1), (dict(out=None), -1), (dict(ldb_=63), -1), (dict(ldo=63), -1),
    (dict(base=P(257)), -2), (dict(out=P(257)), -2), (dict(T=0), 0),
])
def test_lora_apply_refusals(lib, kw, status):
    assert lora(lib, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dyt=7), -1), (dict(dy=None), -1), (dict(dxb=None), -1), (dict(dx=None), -1),
    (dict(dA=None), -1), (dict(dB=None), -1), (dict(lddy=63), -1), (dict(lddxb=31), -1),
    (dict(lddx=31), -1), (dict(ws=None), -1), (dict(nws=10), -1), (dict(dy=P(257)), -2),
    (dict(dx=P(257)), -2), (dict(dxb=P(257)), -2), (dict(dA=P(258)), -2), (dict(dB=P(258)), -2),
    (dict(ws=P(264)), -2),
])
def test_lora_backward_refusals(lib, kw, status):
    assert lora(lib, True, **kw) == status


def test_lora_workspace(lib):
    f = lib.fp8la_lora_workspace_bytes
    assert f(-1, 8) == -1 and f(10, 0) == -1 and f(10, 129) == -3
    assert f(100, 13) == 100 * 16 * 4


def test_no_cpu_fallback_without_a_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: this checks the GPU-less behaviour")
    import precision_linear_algebra_gb300 as fl
    z = torch.zeros((2, 4))
    ids = torch.full((2, 1), 7, dtype=torch.int32)
    w = torch.zeros((2, 1))
    with pytest.raises(fl.Fp8laError) as e:
        fl.fp8_moe_route(z.data_ptr(), 0, 2, 4, 4, 1, 1, ids.data_ptr(), w.data_ptr(), None, None,
                         None, 0, None)
    assert e.value.status == fl.FP8LA_ERR_UNSUPPORTED
    assert torch.all(ids == 7)
