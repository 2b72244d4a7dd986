"""CPU checks of the key/value cache's entry points: sizes of the workspace, and
refusals before anything is launched."""

import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def lib():
    from precision_linear_algebra_gb300 import build
    build.build()
    import precision_linear_algebra_gb300 as fl
    return fl.load()


P = ctypes.c_void_p
A = 256         # an aligned address that is never read


def cache(**kw):
    import precision_linear_algebra_gb300 as fl
    a = dict(k=A, v=A, k_scale=A, v_scale=A, num_pages=6, page_size=16, kv_heads=2, head_dim=64,
             format=0, page_stride=2048, head_stride=1024, token_stride=64, scale_page_stride=32,
             scale_head_stride=16, scale_token_stride=1)
    a.update(kw)
    return fl.fp8la_kv_cache(**a)


CACHE = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
    (dict(format=2), -1), (dict(num_pages=0), -1), (dict(page_size=0), -1),
    (dict(kv_heads=0), -1), (dict(head_dim=0), -1), (dict(token_stride=48), -1),
    (dict(head_stride=48), -1), (dict(page_stride=48), -1), (dict(scale_token_stride=0), -1),
    (dict(scale_head_stride=-16), -1), (dict(scale_page_stride=0), -1),
    (dict(head_dim=72), -3), (dict(head_dim=272), -3), (dict(kv_heads=1025), -3),
    (dict(num_pages=2 ** 31), -3), (dict(page_size=2 ** 30 + 1), -3),
    (dict(k=A + 8), -2), (dict(v=A + 1), -2), (dict(k_scale=A + 2), -2),
    (dict(v_scale=A + 1), -2), (dict(token_stride=72), -2), (dict(head_stride=1032), -2),
    (dict(page_stride=2056), -2),
]
ROWS = [
    (dict(T=-1), -1), (dict(S=-1), -1), (dict(pages=-1), -1), (dict(ldt=2), -1),
    (dict(offs=None), -1), (dict(lens=None), -1), (dict(table=None), -1), (dict(S=1025), -3),
    (dict(T=2 ** 31), -3), (dict(pages=2 ** 31, ldt=2 ** 31), -3), (dict(offs=A + 2), -2),
    (dict(lens=A + 2), -2), (dict(table=A + 2), -2), (dict(S=0), 0),
]


def copy(lib, read, **kw):
    a = dict(k=A, ldk=128, ldkh=64, v=A, ldv=128, ldvh=64, dtype=0, T=5, S=3, offs=A, lens=A,
             table=A, ldt=3, pages=3, cache=cache())
    a.update(kw)
    f = lib.fp8_kv_read if read else lib.fp8_kv_append
    c = a["cache"]
    return f(a["k"], a["ldk"], a["ldkh"], a["v"], a["ldv"], a["ldvh"], a["dtype"], a["T"], a["S"],
             a["offs"], a["lens"], a["table"], a["ldt"], a["pages"],
             None if c is None else ctypes.addressof(c), None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(dtype=2), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(ldk=-1), -1),
    (dict(ldvh=-64), -1), (dict(k=A + 2), -2), (dict(v=A + 1), -2), (dict(k=A + 1, dtype=1), -2),
    (dict(T=2 ** 30, ldk=2 ** 10), -3), (dict(cache=None), -1), (dict(T=0), 0),
])
def test_copy_refusals(lib, read, kw, status):
    if "T" in kw and kw["T"] == 2 ** 30:
        kw = dict(kw, cache=cache(kv_heads=8, head_dim=256, token_stride=256, head_stride=4096,
                                  page_stride=32768), ldkh=256, ldvh=256, ldk=2048, ldv=2048)
    assert copy(lib, read, **kw) == status


@pytest.mark.parametrize("kw", [dict(ldk=64), dict(ldk=127), dict(ldkh=63), dict(ldv=0),
                                dict(ldvh=0)])
def test_read_refuses_overlapping_rows(lib, kw):
    assert copy(lib, True, **kw) == -1


@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_refusals(lib, kw, status):
    assert copy(lib, False, cache=cache(**kw)) == status
    assert copy(lib, True, cache=cache(**kw)) == status
    assert attention(lib, cache=cache(**kw), Hq=max(1, kw.get("kv_heads", 2))) == status


def attention(lib, **kw):
    a = dict(q=A, dtype=1, ldq=512, ldqh=64, Hq=8, T=5, S=3, offs=A, lens=A, table=A, ldt=3,
             pages=3, most=5, ptable=None, ppages=0, plen=None, cache=cache(), scale=0.125,
             causal=1, out=A, ldo=512, ldoh=64, lse=A, ldl=8, ws=A, nws=1 << 40)
    a.update(kw)
    c = a["cache"]
    return lib.fp8_kv_attention(
        a["q"], a["dtype"], a["ldq"], a["ldqh"], a["Hq"], a["T"], a["S"], a["offs"], a["lens"],
        a["table"], a["ldt"], a["pages"], a["most"], a["ptable"], a["ppages"], a["plen"],
        None if c is None else ctypes.addressof(c), a["scale"], a["causal"], a["out"], a["ldo"],
        a["ldoh"], a["lse"], a["ldl"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(nws=100), -1),
    (dict(dtype=3), -1), (dict(Hq=0), -1), (dict(Hq=7), -1), (dict(most=-1), -1),
    (dict(ldq=-1), -1), (dict(ldqh=-64), -1), (dict(ldo=511), -1), (dict(ldoh=63), -1),
    (dict(ldl=7), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(ppages=-1), -1), (dict(ppages=2, plen=A), -1), (dict(ppages=2, ptable=A), -1),
    (dict(cache=None), -1), (dict(T=2 ** 28), -3), (dict(T=1, Hq=65538), -3), (dict(q=A + 1), -2),
    (dict(q=A + 2, dtype=0), -2), (dict(out=A + 1), -2), (dict(lse=A + 2), -2),
    (dict(ws=A + 8), -2), (dict(ptable=A + 2, ppages=2, plen=A), -2),
    (dict(ptable=A, ppages=2, plen=A + 1), -2), (dict(T=0), 0),
])
def test_attention_refusals(lib, kw, status):
    assert attention(lib, **kw) == status


def test_attention_workspace(lib):
    f = lib.fp8_kv_attention_workspace_bytes
    assert f(-1, 8, 64, 0) == -1 and f(4, 0, 64, 0) == -1 and f(4, 8, 0, 0) == -1
    assert f(4, 8, 72, 0) == -3 and f(4, 8, 272, 0) == -3 and f(2 ** 28, 8, 64, 0) == -3
    assert f(4, 8, 64, 0) > 0
    assert f(1, 65536, 64, 0) > 0 and f(1, 65538, 64, 0) == -3 and f(2 ** 62, 4, 64, 0) == -3
    # the prefix's results of every row
    assert f(1000, 8, 64, 1) - f(1000, 8, 64, 0) >= 1000 * 8 * 65 * 4


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    import precision_linear_algebra_gb300 as fl
    codes = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    scales = torch.ones(4, 2, 16)
    with pytest.raises(AssertionError):
        fl.KVCache(codes, codes.clone(), scales, scales.clone())


def test_no_cpu_fallback_without_a_gpu(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: this checks the GPU-less behaviour")
    assert copy(lib, False) in (-3, -4)
    assert copy(lib, True) in (-3, -4)
    assert attention(lib) in (-3, -4)
