"""GB300 (sm_103a) FP8 E4M3 quantize + scaled GEMM library: Python binding.

The compute lives in ``libfp8la.so`` (CUDA C++ with inline PTX, built from
``csrc/`` by ``build.py``); its C ABI is ``include/fp8la.h``.  This module
only marshals arguments: it loads the library with ctypes, exposes each C
entry point under the same name (``fp8_quantize_pertensor``, ``fp8_gemm``,
``fp8_gemm_blockscaled_32x32``, ``fp8_grouped_gemm``, ...) taking raw
integers for pointers, and adds thin torch-tensor wrappers (``quantize_*``,
``gemm*``) that allocate outputs with torch and pass ``data_ptr()`` and the
current CUDA stream.  There is no fallback: if the library cannot be loaded
or a call fails, an exception is raised.
"""

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libfp8la.so")

FP8LA_OK = 0
FP8LA_ERR_INVALID_ARG = -1
FP8LA_ERR_ALIGNMENT = -2
FP8LA_ERR_UNSUPPORTED = -3
FP8LA_ERR_CUDA = -4
FP8LA_ERR_DEVICE_TIMEOUT = -5
FP8LA_ERR_DEVICE_ARG = -6
FP8LA_FORMAT_E4M3 = 0
FP8LA_FORMAT_E5M2 = 1
FP8LA_TYPE_F32 = 0
FP8LA_TYPE_BF16 = 1
FP8LA_ACT_SILU = 0
FP8LA_ACT_GELU_TANH = 1
_ACTIVATIONS = {"silu": FP8LA_ACT_SILU, "gelu_tanh": FP8LA_ACT_GELU_TANH}
_FORMATS = {"e4m3": FP8LA_FORMAT_E4M3, "e5m2": FP8LA_FORMAT_E5M2}

# (name, restype, argtypes) of every entry point in include/fp8la.h.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_S = ctypes.c_int
SIGNATURES = [
    ("fp8_quantize_pertensor", _S, [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _P]),
    ("fp8_quantize_pertensor_ex", _S, [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _I32, _P]),
    ("fp8_quantize_pertensor_delayed", _S,
     [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _I32, _P]),
    ("fp8_quantize_blockwise_32x32", _S, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    ("fp8_quantize_pertensor_grouped", _S,
     [_P, _I32, _P, _I64, _I64, _I64, _P, _I64, _P, _P, _P]),
    ("fp8_gemm", _S, [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _P]),
    ("fp8_gemm_ex", _S, [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _I32, _I32, _P]),
    ("fp8_gemm_blockscaled_32x32", _S,
     [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    ("fp8_grouped_gemm", _S,
     [_I32, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _P, _P, _P]),
    ("fp8_moe_route_workspace_bytes", _I64, [_I64, _I32]),
    ("fp8_moe_route", _S,
     [_P, _I32, _I64, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _P, _I64, _P]),
    ("fp8_moe_layer_workspace_bytes", _I64, [_I64, _I32, _I32, _I64, _I64]),
    ("fp8_moe_layer", _S,
     [_P, _I32, _I64, _I64, _I64, _P, _P, _I32, _I32, _P, _I64, _I64, _P, _P, _I64, _I64, _P,
      _I64, _I32, _I32, _P, _I64, _P, _I64, _P]),
    ("fp8la_lora_apply", _S,
     [_P, _I64, _P, _I32, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I32, _I32, _I64,
      _I64, _I32, _P, _P, _P, _I64, _P, _I64, _P]),
    ("fp8la_lora_workspace_bytes", _I64, [_I64, _I32]),
    ("fp8la_lora_backward", _S,
     [_P, _I32, _I64, _P, _I32, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I32,
      _I32, _I64, _I64, _I32, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P]),
    ("fp8_get_device_status", _S, [_P]),
    ("fp8la_set_wait_timeout_ns", _S, [_I64]),
    ("fp8la_diag_gemm_withheld_arrival", _S, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P]),
    ("fp8la_diag_withheld_arrival", _S,
     [_I32, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    ("fp8la_set_gemm_variant", _S, [_I32]),
    ("fp8la_status_string", ctypes.c_char_p, [_S]),
    ("fp8la_version", _S, []),
]

_lib = None


class Fp8laError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, status_string(status), status))


def load(path=None):
    """Load libfp8la.so (build it first with build.build()); raise if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            "libfp8la.so is not built (%s); run `python -m "
            "precision_linear_algebra_gb300.build`" % p)
    lib = ctypes.CDLL(p)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def status_string(status):
    try:
        return load().fp8la_status_string(status).decode()
    except Exception:
        return "status %d" % status


def _call(name, *args):
    st = getattr(load(), name)(*args)
    if st != FP8LA_OK:
        raise Fp8laError(st, name)
    return st


# --------------------------------------------------- raw C-ABI entry points
def fp8_quantize_pertensor(x, rows, cols, ldx, q, ldq, amax_out, scale_out, stream):
    return _call("fp8_quantize_pertensor", x, rows, cols, ldx, q, ldq, amax_out,
                 scale_out, stream)


def fp8_quantize_pertensor_delayed(x, rows, cols, ldx, q, ldq, amax_prev, amax_out, scale_out,
                                   fmt, stream):
    return _call("fp8_quantize_pertensor_delayed", x, rows, cols, ldx, q, ldq, amax_prev,
                 amax_out, scale_out, fmt, stream)


def fp8_quantize_pertensor_ex(x, rows, cols, ldx, q, ldq, amax_out, scale_out, fmt, stream):
    return _call("fp8_quantize_pertensor_ex", x, rows, cols, ldx, q, ldq, amax_out,
                 scale_out, fmt, stream)


def fp8_gemm_ex(A, lda, B, ldb, C, ldc, M, N, K, scale_a, scale_b, a_fmt, b_fmt, stream):
    return _call("fp8_gemm_ex", A, lda, B, ldb, C, ldc, M, N, K, scale_a, scale_b,
                 a_fmt, b_fmt, stream)


def fp8_quantize_blockwise_32x32(x, rows, cols, ldx, q, ldq, scales, ld_scales, stream):
    return _call("fp8_quantize_blockwise_32x32", x, rows, cols, ldx, q, ldq,
                 scales, ld_scales, stream)


def fp8_quantize_pertensor_grouped(x, num_groups, m_offsets, rows_capacity, cols, ldx, q, ldq,
                                   amax_out, scale_out, stream):
    return _call("fp8_quantize_pertensor_grouped", x, num_groups, m_offsets, rows_capacity,
                 cols, ldx, q, ldq, amax_out, scale_out, stream)


def fp8_gemm(A, lda, B, ldb, C, ldc, M, N, K, scale_a, scale_b, stream):
    return _call("fp8_gemm", A, lda, B, ldb, C, ldc, M, N, K, scale_a, scale_b, stream)


def fp8_gemm_blockscaled_32x32(A, lda, B, ldb, C, ldc, M, N, K, sa, ld_sa, sb,
                               ld_sb, stream):
    return _call("fp8_gemm_blockscaled_32x32", A, lda, B, ldb, C, ldc, M, N, K,
                 sa, ld_sa, sb, ld_sb, stream)


def fp8_grouped_gemm(num_groups, m_offsets, m_capacity, A, lda, B, ldb,
                     b_group_stride, C, ldc, N, K, scale_a, scale_b, stream):
    return _call("fp8_grouped_gemm", num_groups, m_offsets, m_capacity, A, lda,
                 B, ldb, b_group_stride, C, ldc, N, K, scale_a, scale_b, stream)


def _bytes(name, *args):
    n = getattr(load(), name)(*args)
    if n < 0:
        raise Fp8laError(n, name)
    return n


def fp8_moe_route_workspace_bytes(tokens, num_experts):
    return _bytes("fp8_moe_route_workspace_bytes", tokens, num_experts)


def fp8_moe_route(logits, dtype, tokens, num_experts, ld, top_k, renormalise, ids, weights,
                  m_offsets, order, workspace, workspace_bytes, stream):
    return _call("fp8_moe_route", logits, dtype, tokens, num_experts, ld, top_k, renormalise,
                 ids, weights, m_offsets, order, workspace, workspace_bytes, stream)


def fp8_moe_layer_workspace_bytes(tokens, top_k, num_experts, D, F):
    return _bytes("fp8_moe_layer_workspace_bytes", tokens, top_k, num_experts, D, F)


def fp8_moe_layer(x, x_dtype, tokens, D, ldx, ids, weights, top_k, num_experts, w13, ld13,
                  expert_stride13, scale13, w2, ld2, expert_stride2, scale2, F, fmt, activation,
                  y, ldy, workspace, workspace_bytes, stream):
    return _call("fp8_moe_layer", x, x_dtype, tokens, D, ldx, ids, weights, top_k, num_experts,
                 w13, ld13, expert_stride13, scale13, w2, ld2, expert_stride2, scale2, F, fmt,
                 activation, y, ldy, workspace, workspace_bytes, stream)


def fp8la_lora_apply(base, ld_base, x, x_dtype, ldx, rows, A, lda, stride_a, B, ldb, stride_b,
                     alpha, num_adapters, rank, K, N, num_segments, m_offsets, adapter_ids, out,
                     ld_out, v, ldv, stream):
    return _call("fp8la_lora_apply", base, ld_base, x, x_dtype, ldx, rows, A, lda, stride_a, B,
                 ldb, stride_b, alpha, num_adapters, rank, K, N, num_segments, m_offsets,
                 adapter_ids, out, ld_out, v, ldv, stream)


def fp8la_lora_workspace_bytes(rows, rank):
    return _bytes("fp8la_lora_workspace_bytes", rows, rank)


def fp8la_lora_backward(dy, dy_dtype, ld_dy, x, x_dtype, ldx, v, ldv, rows, A, lda, stride_a, B,
                        ldb, stride_b, alpha, num_adapters, rank, K, N, num_segments, m_offsets,
                        adapter_ids, dx_base, ld_dx_base, dx, ld_dx, dA, dB, workspace,
                        workspace_bytes, stream):
    return _call("fp8la_lora_backward", dy, dy_dtype, ld_dy, x, x_dtype, ldx, v, ldv, rows, A,
                 lda, stride_a, B, ldb, stride_b, alpha, num_adapters, rank, K, N, num_segments,
                 m_offsets, adapter_ids, dx_base, ld_dx_base, dx, ld_dx, dA, dB, workspace,
                 workspace_bytes, stream)


def fp8_get_device_status(stream):
    """Sync `stream`, read and clear the device status word; return it."""
    return load().fp8_get_device_status(stream)


def fp8la_set_wait_timeout_ns(ns):
    return _call("fp8la_set_wait_timeout_ns", int(ns))


def fp8la_diag_gemm_withheld_arrival(A, lda, B, ldb, C, ldc, scale_a, scale_b, stream):
    return _call("fp8la_diag_gemm_withheld_arrival", A, lda, B, ldb, C, ldc,
                 scale_a, scale_b, stream)


FP8LA_DIAG_KERNEL_PAIR = 1
FP8LA_DIAG_KERNEL_BLOCK32 = 2


def fp8la_diag_withheld_arrival(kernel, A, lda, B, ldb, C, ldc, M, N, K, scale_a, ld_sa,
                                scale_b, ld_sb, stream):
    return _call("fp8la_diag_withheld_arrival", kernel, A, lda, B, ldb, C, ldc, M, N, K,
                 scale_a, ld_sa, scale_b, ld_sb, stream)


def fp8la_set_gemm_variant(variant):
    """0 = by shape, 1 = single-CTA kernel, 2 = CTA-pair kernel, 3 = single-CTA
    kernel with 128 x 128 tiles, 4 = two CTA pairs per cluster sharing A."""
    return _call("fp8la_set_gemm_variant", int(variant))


def fp8la_version():
    return load().fp8la_version()


# ------------------------------------------------------ torch conveniences
def _stream():
    """The current stream's handle, without building a torch.cuda.Stream (3 us
    of the 4 us that a small launch takes)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _ld(t):
    """Leading dimension of a row-major 2-D tensor.  A single-row tensor's
    row stride is meaningless (torch keeps whatever it was given, even 0), so
    its row length is used."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _ld_tma(t):
    """As _ld, for an FP8 GEMM operand, whose row stride goes into a TMA
    descriptor (a multiple of 16 bytes even when there is one row: the
    stride of a single row never addresses memory, so the row length
    rounded up to 16 is passed)."""
    return t.stride(0) if t.shape[0] > 1 else (max(t.shape[1], 1) + 15) // 16 * 16


def _ld_scales(t):
    """As _ld, for a block-scale grid, whose row stride the GEMM reads by TMA
    (a multiple of 4 floats even when there is one row)."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 3) // 4 * 4


def quantize_pertensor(x, q=None, amax=None, scale=None, fmt="e4m3"):
    """x: fp32 CUDA [rows][cols] (row stride may exceed cols).

    Returns (q uint8 [rows][cols], amax fp32 [1], scale fp32 [1]), all on
    x's device; nothing is synchronised.  fmt: "e4m3" or "e5m2".
    """
    import torch
    assert x.dtype == torch.float32 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    amax = torch.empty(1, dtype=torch.float32, device=x.device) if amax is None else amax
    scale = torch.empty(1, dtype=torch.float32, device=x.device) if scale is None else scale
    fp8_quantize_pertensor_ex(_ptr(x), rows, cols, _ld(x), _ptr(q), _ld(q),
                              _ptr(amax), _ptr(scale), _FORMATS[fmt], _stream())
    return q, amax, scale


def quantize_pertensor_delayed(x, amax_prev, q=None, amax=None, scale=None, fmt="e4m3"):
    """One-pass quantisation with the scale of a carried-over amax.

    x: fp32 CUDA [rows][cols]; amax_prev: fp32 CUDA tensor holding one value
    (e.g. the amax this call returned at the previous step).  Returns
    (q uint8 [rows][cols], amax fp32 [1] of x, scale fp32 [1] of the codes);
    amax must not share storage with amax_prev.
    """
    import torch
    assert x.dtype == torch.float32 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    amax = torch.empty(1, dtype=torch.float32, device=x.device) if amax is None else amax
    scale = torch.empty(1, dtype=torch.float32, device=x.device) if scale is None else scale
    fp8_quantize_pertensor_delayed(_ptr(x), rows, cols, _ld(x), _ptr(q), _ld(q),
                                   _ptr(amax_prev), _ptr(amax), _ptr(scale),
                                   _FORMATS[fmt], _stream())
    return q, amax, scale


def quantize_blockwise_32x32(x, q=None, scales=None):
    """x: fp32 CUDA [rows][cols] -> (q uint8, scales fp32 [ceil(r/32)][ceil(c/32)])."""
    import torch
    assert x.dtype == torch.float32 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        # leading dimension rounded up to 4 floats, as the block-scaled GEMM
        # reads scale grids with TMA (16-byte rows)
        tc = (cols + 31) // 32
        scales = torch.empty(((rows + 31) // 32, (tc + 3) // 4 * 4),
                             dtype=torch.float32, device=x.device)[:, :tc]
    fp8_quantize_blockwise_32x32(_ptr(x), rows, cols, _ld(x), _ptr(q), _ld(q),
                                 _ptr(scales), _ld(scales), _stream())
    return q, scales


def quantize_pertensor_grouped(x, m_offsets, q=None, amax=None, scale=None):
    """x: fp32 CUDA [rows_capacity][cols]; m_offsets: int32 CUDA [E+1].

    Group e (rows m_offsets[e] .. m_offsets[e+1]-1) is quantised with its own
    per-tensor amax and scale.  Returns (q uint8 [rows_capacity][cols],
    amax fp32 [E], scale fp32 [E]); nothing is synchronised.
    """
    import torch
    assert x.dtype == torch.float32 and x.dim() == 2 and x.stride(1) == 1
    assert m_offsets.dtype == torch.int32 and m_offsets.dim() == 1
    rows, cols = x.shape
    E = m_offsets.numel() - 1
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    amax = torch.empty(E, dtype=torch.float32, device=x.device) if amax is None else amax
    scale = torch.empty(E, dtype=torch.float32, device=x.device) if scale is None else scale
    fp8_quantize_pertensor_grouped(_ptr(x), E, _ptr(m_offsets), rows, cols, _ld(x), _ptr(q),
                                   _ld(q), _ptr(amax), _ptr(scale), _stream())
    return q, amax, scale


def gemm(A, B, scale_a, scale_b, C=None, a_fmt="e4m3", b_fmt="e4m3"):
    """A uint8 [M][K], B uint8 [N][K] (K-major), scales fp32 [1] -> C bf16 [M][N].

    a_fmt, b_fmt: "e4m3" (default, fp8_gemm) or "e5m2" (fp8_gemm_ex)."""
    import torch
    M, K = A.shape
    N = B.shape[0]
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    if a_fmt == "e4m3" and b_fmt == "e4m3":
        fp8_gemm(_ptr(A), _ld_tma(A), _ptr(B), _ld_tma(B), _ptr(C), _ld(C),
                 M, N, K, _ptr(scale_a), _ptr(scale_b), _stream())
    else:
        fp8_gemm_ex(_ptr(A), _ld_tma(A), _ptr(B), _ld_tma(B), _ptr(C), _ld(C),
                    M, N, K, _ptr(scale_a), _ptr(scale_b), _FORMATS[a_fmt],
                    _FORMATS[b_fmt], _stream())
    return C


def gemm_blockscaled_32x32(A, B, sa, sb, C=None):
    """Block-scaled GEMM; sa [ceil(M/32)][ceil(K/32)], sb [ceil(N/32)][ceil(K/32)]."""
    import torch
    M, K = A.shape
    N = B.shape[0]
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    fp8_gemm_blockscaled_32x32(_ptr(A), _ld_tma(A), _ptr(B), _ld_tma(B), _ptr(C),
                               _ld(C), M, N, K, _ptr(sa), _ld_scales(sa),
                               _ptr(sb), _ld_scales(sb), _stream())
    return C


def grouped_gemm(m_offsets, A, B, scale_a, scale_b, C=None):
    """m_offsets int32 [E+1] (device); A [cap][K]; B [E][N][K]; scales [E]."""
    import torch
    E = B.shape[0]
    cap, K = A.shape
    N = B.shape[1]
    if C is None:
        C = torch.empty((cap, N), dtype=torch.bfloat16, device=A.device)
    ldb = B.stride(1) if N > 1 else (max(K, 1) + 15) // 16 * 16
    bstride = B.stride(0) if E > 1 else N * ldb
    fp8_grouped_gemm(E, _ptr(m_offsets), cap, _ptr(A), _ld_tma(A), _ptr(B),
                     ldb, bstride, _ptr(C), _ld(C), N, K,
                     _ptr(scale_a), _ptr(scale_b), _stream())
    return C


# The calls below run in the microseconds of a decoding step, so they look at
# each tensor's shape and strides once and pass them straight to the library.
# A tensor of the host is refused here: its pointer would reach a kernel.
def _rows(t, rows, cols, dtype=None):
    """Row stride of a CUDA [rows][cols] tensor whose rows are contiguous."""
    assert t.is_cuda and t.shape == (rows, cols) and (dtype is None or t.dtype is dtype)
    s0, s1 = t.stride()
    assert s1 == 1 or cols == 1
    return s0 if rows > 1 else max(cols, 1)


def _dense(t, shape, dtype):
    assert t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _type(t):
    import torch
    dt = t.dtype
    if dt is torch.bfloat16:
        return FP8LA_TYPE_BF16
    assert dt is torch.float32
    return FP8LA_TYPE_F32


def _workspace(workspace, need, device):
    """(pointer, bytes, tensor): the caller's workspace, or a fresh one."""
    import torch
    if need == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    assert workspace.is_cuda and workspace.is_contiguous()
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def moe_route(logits, top_k, renormalise=True, sort=True, ids=None, weights=None,
              m_offsets=None, order=None, workspace=None):
    """logits: fp32 or bf16 CUDA [T][E] (row stride may exceed E).

    Returns (ids int32 [T][top_k], weights fp32 [T][top_k], m_offsets int32
    [E+1], order int32 [T*top_k]); the last two, the pairs sorted by expert,
    are None with sort=False.  Ties go to the lowest index; a slot without an
    expert (all other logits -inf) has id -1 and weight 0.  Nothing is
    synchronised.
    """
    import torch
    T, E = logits.shape
    dev = logits.device
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    else:
        _dense(ids, (T, top_k), torch.int32)
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    else:
        _dense(weights, (T, top_k), torch.float32)
    po = pr = pw = ws = None
    nbytes = 0
    if sort:
        if m_offsets is None:
            m_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        else:
            _dense(m_offsets, (E + 1,), torch.int32)
        if order is None:
            order = torch.empty(T * top_k, dtype=torch.int32, device=dev)
        else:
            _dense(order, (T * top_k,), torch.int32)
        po, pr = m_offsets.data_ptr(), order.data_ptr()
        pw, nbytes, ws = _workspace(workspace, fp8_moe_route_workspace_bytes(T, E), dev)
    else:
        m_offsets = order = None
    _call("fp8_moe_route", logits.data_ptr(), _type(logits), T, E, _rows(logits, T, E), top_k,
          renormalise, ids.data_ptr(), weights.data_ptr(), po, pr, pw, nbytes, _stream())
    return ids, weights, m_offsets, order


def moe_layer(x, ids, weights, w13, scale13, w2, scale2, y=None, workspace=None, fmt="e4m3",
              activation="silu"):
    """Mixture-of-experts layer for up to 128 tokens: x fp32 or bf16 CUDA
    [T][D], ids int32 and weights fp32 [T][top_k] -> y bf16 [T][D].

    w13 uint8 [E][2F][D] (gate rows, then up rows) and w2 uint8 [E][D][F] are
    codes of fmt ("e4m3" or "e5m2") with row strides that are multiples of
    16; scale13, scale2 fp32 [E].  activation: "silu" or "gelu_tanh".
    Nothing is synchronised.
    """
    import torch
    T, D = x.shape
    E, _, F = w2.shape
    top_k = ids.shape[1]
    assert w13.shape == (E, 2 * F, D) and w2.shape[1] == D
    assert w13.dtype is torch.uint8 and w2.dtype is torch.uint8
    assert w13.is_cuda and w2.is_cuda
    e13, ld13, one13 = w13.stride()
    e2, ld2, one2 = w2.stride()
    assert (one13 == 1 or D == 1) and (one2 == 1 or F == 1)
    _dense(ids, (T, top_k), torch.int32)
    _dense(weights, (T, top_k), torch.float32)
    _dense(scale13, (E,), torch.float32)
    _dense(scale2, (E,), torch.float32)
    if y is None:
        y, ldy = torch.empty((T, D), dtype=torch.bfloat16, device=x.device), D
    else:
        ldy = _rows(y, T, D, torch.bfloat16)
    pw, nbytes, ws = _workspace(workspace, fp8_moe_layer_workspace_bytes(T, top_k, E, D, F),
                                x.device)
    _call("fp8_moe_layer", x.data_ptr(), _type(x), T, D, _rows(x, T, D), ids.data_ptr(),
          weights.data_ptr(), top_k, E, w13.data_ptr(), ld13, e13, scale13.data_ptr(),
          w2.data_ptr(), ld2, e2, scale2.data_ptr(), F, _FORMATS[fmt],
          _ACTIVATIONS[activation], y.data_ptr(), ldy, pw, nbytes, _stream())
    return y


def _adapters(A, B, alpha, m_offsets, adapter_ids, N):
    """Sizes and strides of a set of adapters and its segments."""
    import torch
    n, R, K = A.shape
    assert A.dtype is torch.bfloat16 and B.dtype is torch.bfloat16 and B.shape == (n, R, N)
    assert A.is_cuda and B.is_cuda
    sa, lda, onea = A.stride()
    sb, ldb, oneb = B.stride()
    assert (onea == 1 or K == 1) and (oneb == 1 or N == 1)
    _dense(alpha, (n,), torch.float32)
    S = adapter_ids.numel()
    _dense(adapter_ids, (S,), torch.int32)
    _dense(m_offsets, (S + 1,), torch.int32)
    return n, R, K, S, lda, sa, ldb, sb


def lora_apply(base, x, A, B, alpha, m_offsets, adapter_ids, out=None, v=None):
    """Adds each request's low-rank adapter to a shared projection's output.

    base bf16 [T][N] (e.g. from gemm), x fp32 or bf16 [T][K], A bf16 [n][R][K],
    B bf16 [n][R][N], alpha fp32 [n]; segment s, the rows m_offsets[s] ..
    m_offsets[s+1]-1 (int32 [S+1]), uses adapter adapter_ids[s] (int32 [S],
    -1: none).  Returns (out bf16 [T][N] = base + alpha v B, v fp32 [T][R] =
    x A^T); out may be base.  All CUDA; nothing is synchronised.
    """
    import torch
    T, N = base.shape
    n, R, K, S, lda, sa, ldb, sb = _adapters(A, B, alpha, m_offsets, adapter_ids, N)
    if out is None:
        out, ldo = torch.empty((T, N), dtype=torch.bfloat16, device=x.device), N
    else:
        ldo = _rows(out, T, N, torch.bfloat16)
    if v is None:
        v, ldv = torch.empty((T, R), dtype=torch.float32, device=x.device), R
    else:
        ldv = _rows(v, T, R, torch.float32)
    _call("fp8la_lora_apply", base.data_ptr(), _rows(base, T, N, torch.bfloat16), x.data_ptr(),
          _type(x), _rows(x, T, K), T, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb,
          alpha.data_ptr(), n, R, K, N, S, m_offsets.data_ptr(), adapter_ids.data_ptr(),
          out.data_ptr(), ldo, v.data_ptr(), ldv, _stream())
    return out, v


def lora_backward(dy, x, v, A, B, alpha, m_offsets, adapter_ids, dx_base, dx=None, dA=None,
                  dB=None, workspace=None):
    """Backward pass of lora_apply.

    dy fp32 or bf16 [T][N], v as lora_apply returned it, dx_base bf16 [T][K]
    the shared projection's gradient with respect to x.  Returns (dx bf16
    [T][K] = dx_base + dv A, dA fp32 [n][R][K], dB fp32 [n][R][N]); dx may be
    dx_base.  All CUDA; nothing is synchronised.
    """
    import torch
    T, N = dy.shape
    n, R, K, S, lda, sa, ldb, sb = _adapters(A, B, alpha, m_offsets, adapter_ids, N)
    dev = x.device
    if dx is None:
        dx, lddx = torch.empty((T, K), dtype=torch.bfloat16, device=dev), K
    else:
        lddx = _rows(dx, T, K, torch.bfloat16)
    if dA is None:
        dA = torch.empty((n, R, K), dtype=torch.float32, device=dev)
    else:
        _dense(dA, (n, R, K), torch.float32)
    if dB is None:
        dB = torch.empty((n, R, N), dtype=torch.float32, device=dev)
    else:
        _dense(dB, (n, R, N), torch.float32)
    pw, nbytes, ws = _workspace(workspace, fp8la_lora_workspace_bytes(T, R), dev)
    _call("fp8la_lora_backward", dy.data_ptr(), _type(dy), _rows(dy, T, N), x.data_ptr(),
          _type(x), _rows(x, T, K), v.data_ptr(), _rows(v, T, R, torch.float32), T,
          A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, alpha.data_ptr(), n, R, K, N, S,
          m_offsets.data_ptr(), adapter_ids.data_ptr(), dx_base.data_ptr(),
          _rows(dx_base, T, K, torch.bfloat16), dx.data_ptr(), lddx, dA.data_ptr(),
          dB.data_ptr(), pw, nbytes, _stream())
    return dx, dA, dB


def device_status():
    return fp8_get_device_status(_stream())
