"""GPU: the key/value cache as a program uses it: a prompt in pieces, decoding steps
captured and replayed for growing sequences, several streams, caches and rows beyond
2^31 elements.  Bounds are those of _kv.py."""

import math

import pytest

from _helpers import lib
from _kv import attend, check, close, fp8, make, reference

pytestmark = pytest.mark.gpu


def empty(fl, S, most, H, D, page, fmt="e4m3", seed=0):
    """A cache for S sequences of up to `most` tokens, all of it NaN."""
    import torch
    width = -(-most // page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = fl.kv_cache(S * width, H, page, D, fmt)
    for t in (cache.k, cache.v):
        t.fill_(0x7F)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(math.nan)
    table = torch.randperm(S * width, generator=g, device="cuda").to(torch.int32).view(S, width)
    return cache, table


def whole(fl, c, cache, table, q, lens, rows, H, G, D, page, fmt):
    """reference() of sequences `lens` whose last `rows` are q."""
    import torch
    d = dict(H=H, G=G, D=D, page=page, fmt=fmt, lens=lens, rows=rows, prefix=0, table=table,
             prefix_table=table[0, :0], cache=cache, q=q, T=q.shape[0])
    return reference(d)


@pytest.mark.parametrize("fmt,page,q_type", [("e4m3", 16, "bfloat16"), ("e5m2", 24, "float32")])
def test_prompt_in_pieces_and_decoding(fmt, page, q_type):
    """Prompts of different lengths are appended and attended to piece by piece, then
    decoded token by token; every step against 64 bits on what the cache holds."""
    import torch
    fl = lib()
    S, H, G, D = 3, 2, 4, 64
    cache, table = empty(fl, S, 400, H, D, page, fmt)
    g = torch.Generator(device="cuda").manual_seed(5)
    dt = getattr(torch, q_type)
    lens = [0] * S
    for rows in ([130, 1, 70], [100, 64, 0], [1, 1, 1], [2, 1, 0], [1, 1, 1]):
        T = sum(rows)
        qkv = torch.randn(T, (G + 2) * H, D, generator=g, device="cuda").to(dt)
        offs = torch.tensor([0, rows[0], rows[0] + rows[1], T], dtype=torch.int32, device="cuda")
        lens = [a + b for a, b in zip(lens, rows)]
        kvl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q, k, v = qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
        fl.kv_append(k, v, cache, offs, kvl, table)
        out, lse = fl.kv_attention(q, cache, offs, kvl, table, max_rows=max(rows))
        k2, v2 = fl.kv_read(cache, offs, kvl, table, T, dtype=torch.float32)
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        # half a step of the format: 2^-4 or 2^-3 of a value, or of its smallest normal
        step, least = (2.0 ** -4, 2.0 ** -6 / 448) if fmt == "e4m3" else (2.0 ** -3, 2.0 ** -14 / 57344)
        for x, y in ((k, k2), (v, v2)):
            x = x.float()
            amax = x.abs().amax(-1, keepdim=True)
            assert ((x - y).abs() <= step * torch.maximum(x.abs(), least * amax) * (1 + 1e-5)).all()
        ro, ob, rl, lb = whole(fl, None, cache, table, q, lens, rows, H, G, D, page, fmt)
        assert close(out, ro, ob) and close(lse, rl, lb)


def test_captured_step_is_replayed_for_longer_sequences():
    """One captured append and attention; lengths, pages and rows change between
    replays, in place."""
    import torch
    fl = lib()
    S, H, G, D, page = 4, 2, 4, 128, 16
    cache, table = empty(fl, S, 700, H, D, page)
    q = torch.zeros(S, G * H, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(S, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    offs = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    kvl = torch.ones(S, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    lse = torch.zeros(S, G * H, device="cuda")

    def step():
        fl.kv_append(k, v, cache, offs, kvl, table)
        fl.kv_attention(q, cache, offs, kvl, table, max_rows=1, out=out, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [0, 0, 0, 0]
    kvl.zero_()
    for fill in ((600, 5, 0, 33), (0, 1, 0, 0), (0, 0, 0, 0)):
        # longer histories, written outside the graph
        if any(fill):
            T = sum(fill)
            o = torch.tensor([0, fill[0], fill[0] + fill[1], fill[0] + fill[1], T],
                             dtype=torch.int32, device="cuda")
            lens = [a + b for a, b in zip(lens, fill)]
            x = torch.randn(2, T, H, D, generator=g, device="cuda")
            fl.kv_append(x[0], x[1], cache, o, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         table)
        lens = [n + 1 for n in lens]
        kvl.copy_(torch.tensor(lens, dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        ro, ob, rl, lb = whole(fl, None, cache, table, q, lens, [1] * S, H, G, D, page, "e4m3")
        assert close(out, ro, ob) and close(lse, rl, lb)


def test_two_streams():
    """Calls on two streams at once, each with its own workspace and cache."""
    import torch
    fl = lib()
    cases = [make((900, 40), (1, 1), 2, 4, 128, 64, seed=1),
             make((300, 70), (300, 70), 2, 4, 64, 16, seed=2, prefix=100)]
    want = [attend(fl, c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(attend(fl, c))
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_two_graphs_share_a_workspace():
    import torch
    fl = lib()
    cases = [make((900, 40), (1, 1), 2, 4, 128, 64, seed=1), make((300,), (40,), 2, 4, 64, 16, seed=2)]
    want = [attend(fl, c) for c in cases]
    need = max(fl.fp8_kv_attention_workspace_bytes(c["T"], c["H"] * c["G"], c["D"], False)
               for c in cases)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(attend(fl, c, workspace=ws))
        graphs.append(g)
    for i in (0, 1, 0, 0, 1):
        ws.fill_(0xFF)
        for t in got[i]:
            t.fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


@pytest.mark.parametrize("rows,D", [(1, 128), (100, 128), (1, 256)])
def test_pages_beyond_2_31_elements(rows, D):
    """A cache of 5 GB: sequences in its last pages, for every call."""
    import torch
    fl = lib()
    H, G, page = 2, 2, 16
    P = 5 * 2 ** 30 // (H * page * D)
    k = torch.empty((P, H, page, D), dtype=torch.uint8, device="cuda")
    ks = torch.empty((P, H, page), device="cuda")
    cache = fl.KVCache(k, k, ks, ks)           # V is K, as nothing is written twice here
    n = rows + 50
    pages = -(-n // page)
    table = torch.arange(P - 1, P - 1 - pages, -1, dtype=torch.int32, device="cuda").view(1, -1)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(n, H, D, generator=g, device="cuda")
    offs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kvl = torch.tensor([n], dtype=torch.int32, device="cuda")
    fl.kv_append(x, x, cache, offs, kvl, table)
    back, _ = fl.kv_read(cache, offs, kvl, table, n, dtype=torch.float32)
    amax = x.abs().amax(-1, keepdim=True)
    assert ((back - x).abs() <= 2.0 ** -4 * torch.maximum(x.abs(), amax * 2.0 ** -6 / 448) * (1 + 1e-5)).all()
    q = torch.randn(rows, H * G, D, generator=g, device="cuda").to(torch.bfloat16)
    offs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out, lse = fl.kv_attention(q, cache, offs, kvl, table)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    ro, ob, rl, lb = whole(fl, None, cache, table, q, [n], [rows], H, G, D, page, "e4m3")
    assert close(out, ro, ob) and close(lse, rl, lb)


@pytest.mark.parametrize("prefix", [False, True])
def test_rows_beyond_2_31_elements(prefix):
    """The last rows of q and out lie behind 2^31 elements, with short sequences."""
    import torch
    fl = lib()
    H, G, D, page, S = 2, 32, 128, 16, 270
    each = 1000                                # rows of a sequence; 270000 * 64 * 128 > 2^31
    T = S * each
    cache, table = empty(fl, S, 40, H, D, page)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(2, S * 40, H, D, generator=g, device="cuda")
    n40 = torch.full((S,), 40, dtype=torch.int32, device="cuda")
    fl.kv_append(x[0], x[1], cache, torch.arange(S + 1, dtype=torch.int32, device="cuda") * 40, n40,
                 table)
    q = torch.zeros(T, H * G, D, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(each, H * G, D, generator=g, device="cuda").to(torch.bfloat16)
    q[-each:] = last
    offs = torch.arange(S + 1, dtype=torch.int32, device="cuda") * each
    kw = {}
    if prefix:
        kw = dict(prefix_table=table[3].contiguous(),
                  prefix_len=torch.tensor([20], dtype=torch.int32, device="cuda"))
    out, lse = fl.kv_attention(q, cache, offs, n40, table, max_rows=each, causal=False, **kw)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    d = dict(H=H, G=G, D=D, page=page, fmt="e4m3", lens=[40], rows=[each], prefix=20 * prefix,
             table=table[-1:], prefix_table=table[3], cache=cache, q=last, T=each)
    ro, ob, rl, lb = reference(d, causal=False)
    assert close(out[-each:], ro, ob) and close(lse[-each:], rl, lb)


def test_rows_before_the_begin_see_the_prefix():
    fl = lib()
    c = make((3, 0), (7, 2), 2, 2, 64, 4, prefix=9)
    check(fl, c)
    c = make((3, 0), (90, 80), 2, 2, 128, 4, prefix=9)
    check(fl, c)


def test_one_head_and_many():
    """A single K/V head for many query heads, and each its own."""
    fl = lib()
    check(fl, make((700, 3), (1, 2), 1, 71, 64, 16), max_rows=2)
    check(fl, make((150, 90), (1, 3), 40, 1, 64, 16), max_rows=3)
    check(fl, make((260,), (9,), 1, 64, 128, 32))


def test_lse_is_optional():
    import torch
    fl = lib()
    c = make((90, 4), (1, 2), 2, 4, 64, 16)
    want, _ = attend(fl, c)
    out = torch.zeros_like(want)
    ws = torch.empty(fl.fp8_kv_attention_workspace_bytes(3, 8, 64, 0), dtype=torch.uint8, device="cuda")
    fl.fp8_kv_attention(c["q"].data_ptr(), fl.FP8LA_TYPE_BF16, 512, 64, 8, 3, 2, c["offs"].data_ptr(),
                        c["kv_lens"].data_ptr(), c["table"].data_ptr(), c["table"].stride(0),
                        c["table"].shape[1], 3, None, 0, None, c["cache"].ref, 0.125, 1,
                        out.data_ptr(), 512, 64, None, 0, ws.data_ptr(), ws.numel(),
                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert fl.device_status() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("rows", [2, 70])
def test_workspace_of_any_16_byte_alignment(rows):
    """Sequences shared by several CTAs, whose partial results go through it."""
    import torch
    fl = lib()
    c = make((3000, 2000), (rows, rows), 2, 4, 64, 16, prefix=100)
    want, wl = check(fl, c)
    need = fl.fp8_kv_attention_workspace_bytes(c["T"], 8, 64, 1)
    ws = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
    for at in (16, 48, 240):
        got, gl = attend(fl, c, workspace=ws[at:at + need])
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        assert torch.equal(got, want) and torch.equal(gl, wl)
        assert torch.all(ws[:at] == 0x7F) and torch.all(ws[at + need:] == 0x7F)
        ws.fill_(0x7F)


@pytest.mark.parametrize("rows", [1, 70])
def test_lengths_whose_tiles_would_pass_2_31(rows):
    """2^31 - 4096 tokens is the most; the page table's row has room for more."""
    import torch
    fl = lib()
    page, pages = 2 ** 16, 2 ** 15
    cache = fl.kv_cache(1, 1, page, 16)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    kvl = torch.tensor([2 ** 31 - 4095], dtype=torch.int32, device="cuda")
    x = torch.ones(rows, 1, 16, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 5.0)
    for call in (lambda: fl.kv_append(x, x, cache, offs, kvl, table),
                 lambda: fl.kv_read(cache, offs, kvl, table, rows, k=out, v=out.clone()),
                 lambda: fl.kv_attention(x, cache, offs, kvl, table, out=out),
                 lambda: fl.kv_attention(x, cache, offs, torch.ones_like(kvl), table, out=out,
                                         prefix_table=table[0], prefix_len=kvl)):
        call()
        torch.cuda.synchronize()
        assert fl.device_status() == fl.FP8LA_ERR_DEVICE_ARG
        assert torch.all(out == 5.0) and torch.all(cache.k == 0)
    kvl -= 1
    fl.kv_append(x, x, cache, offs, kvl, table)
    fl.kv_read(cache, offs, kvl, table, rows, k=out, v=out.clone())
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    # 1 and 1 / 448 are off by 2^-24 each, BF16's rounding takes that away
    assert torch.all(out == 1.0) and (cache.k != 0).any(-1).sum() == rows


@pytest.mark.parametrize("rows", [1, 70])
def test_strides_of_dimensions_of_one_element_address_nothing(rows):
    import torch
    fl = lib()
    c = make((30,), (min(rows, 20),), 1, 8, 64, 32, spare=0)
    want, wl = check(fl, c)
    for stride in (1 << 62, -17):
        s = c["cache"].struct
        assert s.num_pages == 1 and s.kv_heads == 1
        s.page_stride = s.head_stride = s.scale_page_stride = s.scale_head_stride = stride
        got, gl = attend(fl, c)
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_host_tensors_are_refused():
    import torch
    fl = lib()
    c = make((30, 20), (2, 1), 2, 4, 64, 16, prefix=20)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache, seqs = c["cache"], (c["offs"], c["kv_lens"], c["table"])
    out, lse = attend(fl, c)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def refused(f, args, at, kw={}):
        args, kw = list(args), dict(kw)
        if isinstance(at, int):
            args[at] = args[at].cpu()
        else:
            kw[at] = kw[at].cpu()
        with pytest.raises(AssertionError):
            f(*args, **kw)

    for at in (0, 1, 3, 4, 5):
        refused(fl.kv_append, (x, x, cache, *seqs), at)
    for at in (1, 2, 3, "k", "v"):
        refused(fl.kv_read, (cache, *seqs, 3), at, dict(k=x.clone(), v=x.clone()))
    kw = dict(prefix_table=c["prefix_table"], prefix_len=c["prefix_len"], out=out, lse=lse,
              workspace=ws)
    for at in (0, 2, 3, 4, *kw):
        refused(fl.kv_attention, (c["q"], cache, *seqs), at, kw)
    codes = [cache.k, cache.v, cache.k_scale, cache.v_scale]
    for at in range(4):
        refused(fl.KVCache, codes, at)
    with pytest.raises(AssertionError):  # a prefix without its length
        fl.kv_attention(c["q"], cache, *seqs, prefix_table=c["prefix_table"])
    torch.cuda.synchronize()
    assert fl.device_status() == 0


def test_calls_in_a_row_share_a_workspace():
    """Short and long segments in one call, behind a prefix and without one, decoding
    steps and a prompt, queued one behind the other: each as when it is alone."""
    import torch
    fl = lib()
    problems = [make((900, 300, 40, 1200), (200, 1, 3, 130), 2, 4, 64, 16),
                make((90, 0, 40, 35, 7), (1, 0, 3, 33, 1), 2, 4, 64, 16, prefix=700),
                make((900, 300, 40, 1200), (150, 1, 3, 1), 2, 4, 64, 16, prefix=300),
                make((5000, 3000), (1, 2), 2, 4, 64, 16),
                make((400,), (400,), 2, 4, 64, 16)]
    want = []
    for c in problems:
        out, lse = attend(fl, c)
        torch.cuda.synchronize()
        want.append((out, lse))
    ws = torch.empty(max(fl.fp8_kv_attention_workspace_bytes(c["T"], 8, 64, 1) for c in problems),
                     dtype=torch.uint8, device="cuda")
    order = torch.randperm(60, generator=torch.Generator().manual_seed(3)) % len(problems)
    got = [(i, attend(fl, problems[i], workspace=ws)) for i in order.tolist()]
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_captured_calls_in_a_row():
    """The same in one graph, whose launches overlap as far as they do on a stream."""
    import torch
    fl = lib()
    problems = [make((900, 300, 40, 1200), (200, 1, 3, 130), 2, 4, 64, 16),
                make((90, 0, 40, 35, 7), (1, 0, 3, 33, 1), 2, 4, 64, 16, prefix=700),
                make((2000, 300), (1, 1), 2, 4, 64, 24, prefix=40),
                make((5000, 3000), (1, 2), 2, 4, 64, 16, q="float32")]
    want = [attend(fl, c) for c in problems]
    need = max(fl.fp8_kv_attention_workspace_bytes(c["T"], 8, 64, 1) for c in problems)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [attend(fl, c, workspace=ws) for c in problems * 3]
    for _ in range(8):
        for out, lse in got:
            out.fill_(5.0)
            lse.fill_(5.0)
        ws.fill_(0x7F)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert fl.device_status() == 0
        for (out, lse), (a, b) in zip(got, want * 3):
            assert torch.equal(out, a) and torch.equal(lse, b)


@pytest.mark.parametrize("rows", [1, 40])
def test_sequences_without_pages_of_their_own(rows):
    """A page table without columns: only the prefix is there."""
    import torch
    fl = lib()
    c = make((0, 0, 0), (rows, 1, 0), 2, 4, 64, 16, prefix=333)
    c["table"] = c["table"][:, :0].contiguous()
    want, wl, *_ = check(fl, c)
    assert torch.isfinite(wl).all()
    # without the prefix there is nothing at all
    out, lse = fl.kv_attention(c["q"], c["cache"], c["offs"], c["kv_lens"], c["table"])
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


def test_broadcast_rows():
    """One row for all heads (stride 0): each head has the same codes and result."""
    import torch
    fl = lib()
    H, D, T = 4, 64, 37
    cache, table = empty(fl, 1, T, H, D, 16)
    offs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    x = torch.randn(T, 1, D, device="cuda").to(torch.bfloat16)
    k = x.expand(T, H, D)
    fl.kv_append(k, k, cache, offs, offs[1:], table)
    out, lse = fl.kv_attention(x.expand(T, 2 * H, D), cache, offs, offs[1:], table)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    assert torch.equal(out, out[:, :1].expand_as(out)) and torch.isfinite(lse).all()
    assert torch.equal(lse, lse[:, :1].expand_as(lse))
