"""Per-token NVFP4 quantization and block-scaled W4A4 GEMM on MI355X (gfx950).

Thin Python binding over the C ABI of ``libnvfp4.so`` (declared in
``include/nvfp4.h``).  Every step of the path runs in the library's HIP
kernels; this module only checks tensor metadata, allocates outputs with
torch and passes device pointers plus torch's current stream.  There is no
CPU fallback: if the library is missing or the device is not gfx950 the
calls raise.

Functions keep the C names:

  nvfp4_quantize_rows(x, amax_in=None)            -> (q, sb, s)
  nvfp4_quantize_weight(w, amax_in=None)          -> (q, sb, s, amax)
  nvfp4_gemm(a, b)                                -> y
  nvfp4_grouped_gemm(a, offsets, b, row_index=None, m_total=None) -> y
  nvfp4_grouped_gemm_swiglu(a, offsets, b, row_index=None, m_total=None) -> (h, amax)
  nvfp4_bf16_grouped_gemm(x, offsets, w, row_index=None)          -> y
  nvfp4_bf16_grouped_dgrad(dy, offsets, w)                        -> dx
  nvfp4_bf16_grouped_wgrad(dy, x, offsets, row_index=None, add=None) -> dw
  nvfp4_residual_norm(x, residual, norm_weight, ...)              -> {"residual", "h", ...}
  nvfp4_residual_norm_backward(x, residual, norm_weight, dh, d_residual, ...) -> {"dx", ...}
  nvfp4_moe_combine(y, slot_of, weights=None)                     -> out
  nvfp4_moe_combine_backward(dout, y, slot_of, weights=None)      -> {"dy", "d_weights"}
  nvfp4_clip_grad_norm(grads, max_norm, out=None)                 -> norm

(The codec self-test hooks live in the test-only ``selftest`` submodule over
``libnvfp4_selftest.so``.)

Layouts (all row-major): x bf16 [rows, k]; q uint8 [rows, k/2] with element
2i in the low nibble; sb uint8 [rows, k/16] (E4M3 codes); s float32 [rows]
(per-token) or [groups] (weights); a GEMM operand is the tuple (q, sb, s).
"""
import bisect
import contextlib
import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
PRODUCT_LIB_PATH = os.path.join(_HERE, "libnvfp4.so")
# the checked build: the same library with device-side preconditions
# (finite inputs and scales, no NaN scale codes, non-decreasing offsets)
# validated before every call's work; it synchronizes the host on each call
CHECKED_LIB_PATH = os.path.join(_HERE, "libnvfp4_checked.so")
# NVFP4_CHECKED=1 in the environment makes the binding load the checked build
LIB_PATH = CHECKED_LIB_PATH if os.environ.get("NVFP4_CHECKED", "0") not in ("", "0") else PRODUCT_LIB_PATH

SUCCESS = 0
ERROR_PRECONDITION = 6
_lib = None
_loaded = {}


class NVFP4Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (fn, status_string(status), status))


def load(path):
    """Load one build of the library (libnvfp4.so or libnvfp4_checked.so,
    built in-tree by ``__graft_entry__.build()``) with its C signatures."""
    if path in _loaded:
        return _loaded[path]
    if not os.path.exists(path):
        raise RuntimeError("%s is not built: run __graft_entry__.build() "
                           "(or python -m nvfp4_token_quantization_amd.build)" % os.path.basename(path))
    L = ctypes.CDLL(path)
    P, I64 = ctypes.c_void_p, ctypes.c_int64
    L.nvfp4_version.restype = ctypes.c_int
    L.nvfp4_status_string.argtypes = [ctypes.c_int]
    L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_quantize_rows.argtypes = [P, I64, I64, P, P, P, P, P]
    L.nvfp4_quantize_weight.argtypes = [P, I64, I64, I64, P, P, P, P, P, P]
    L.nvfp4_gemm.argtypes = [P, P, P, I64, P, P, P, I64, I64, P, P]
    L.nvfp4_grouped_gemm.argtypes = [P, P, P, I64, P, I64, P, I64, P, P, P, I64, I64, P, P]
    L.nvfp4_grouped_gemm_swiglu.argtypes = [P, P, P, I64, P, I64, P, I64, P, P, P, I64, I64,
                                            P, P, P]
    L.nvfp4_swiglu_quantize_rows.argtypes = [P, I64, I64, P, P, P, P, P, P]
    L.nvfp4_moe_route.argtypes = [P, I64, I64, I64, P, P, P, P, P]
    L.nvfp4_dequantize_rows.argtypes = [P, P, P, I64, I64, I64, P, P]
    L.nvfp4_mxfp8_quantize_rows.argtypes = [P, I64, I64, P, P, P]
    L.nvfp4_mxfp8_gemm.argtypes = [P, P, I64, P, P, I64, I64, P, P]
    L.nvfp4_mxfp8_grouped_gemm.argtypes = [P, P, I64, P, I64, P, I64, P, P, I64, I64, P, P]
    I32, F32 = ctypes.c_int, ctypes.c_float
    L.nvfp4_bf16_grouped_gemm.argtypes = [P, I64, P, I64, P, I64, P, I64, I64, P, I32, P]
    L.nvfp4_bf16_grouped_dgrad.argtypes = [P, I64, P, I64, P, I64, I64, P, I32, P]
    L.nvfp4_bf16_grouped_wgrad.argtypes = [P, I64, P, I64, P, P, I64, I64, I64, P, P, I32, P]
    L.nvfp4_residual_norm.argtypes = [P, I32, P, I32, P, P, I32, P, I32, I64, I64, F32, F32,
                                      P, P, P, P, P, P, P]
    L.nvfp4_residual_norm_backward.argtypes = [P, I32, P, I32, P, P, I32, P, I32, P, P, I64, I64, F32,
                                               F32, P, I32, P, P, P, P, P, I64, P]
    L.nvfp4_moe_combine.argtypes = [P, I32, I64, P, P, I64, I64, I64, P, I32, P]
    L.nvfp4_moe_combine_backward.argtypes = [P, I32, P, I32, I64, P, P, I64, I64, I64, P, I32, P, P]
    L.nvfp4_clip_grad_norm.argtypes = [P, P, P, P, I64, F32, P, P, I64, P]
    L.nvfp4_residual_norm_backward_workspace.argtypes = [I64, I64]
    L.nvfp4_residual_norm_backward_workspace.restype = I64
    L.nvfp4_clip_grad_norm_workspace.argtypes = [I64]
    L.nvfp4_clip_grad_norm_workspace.restype = I64
    for f in ("nvfp4_bf16_grouped_gemm", "nvfp4_bf16_grouped_dgrad", "nvfp4_bf16_grouped_wgrad",
              "nvfp4_residual_norm", "nvfp4_residual_norm_backward", "nvfp4_moe_combine",
              "nvfp4_moe_combine_backward", "nvfp4_clip_grad_norm"):
        getattr(L, f).restype = ctypes.c_int
    for f in ("nvfp4_quantize_rows", "nvfp4_quantize_weight", "nvfp4_gemm",
              "nvfp4_swiglu_quantize_rows", "nvfp4_moe_route", "nvfp4_dequantize_rows",
              "nvfp4_mxfp8_quantize_rows", "nvfp4_mxfp8_gemm", "nvfp4_mxfp8_grouped_gemm",
              "nvfp4_grouped_gemm", "nvfp4_grouped_gemm_swiglu"):
        getattr(L, f).restype = ctypes.c_int
    _loaded[path] = L
    return L


def lib():
    """The library every call goes through: LIB_PATH (the product build
    unless NVFP4_CHECKED is set)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def version():
    return lib().nvfp4_version()


def status_string(status):
    return lib().nvfp4_status_string(int(status)).decode()


def _check(fn, status):
    if status != SUCCESS:
        raise NVFP4Error(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without building a Stream object (1.8 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(dev.index))
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dev(t, name, dtypes, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU (got %s)" % (name, t.device))
    if t.dtype not in dtypes:
        raise TypeError("%s must have dtype in %s (got %s)" % (name, dtypes, t.dtype))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims (got %s)" % (name, ndim, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _out(t, name, shape, dtype, device):
    """Check a caller-supplied output tensor: the kernels write exactly
    `shape` elements of `dtype` through its pointer, so anything else (a
    smaller or strided buffer, another device) is refused."""
    _dev(t, name, (dtype,))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s (got %s)" % (name, device, t.device))
    return t


def _out_rows(t, name, min_rows, cols, dtype, device):
    """Output of a grouped GEMM: [rows >= min_rows, cols]; the kernels write
    only rows below offsets[groups] <= min_rows, so a taller buffer is fine."""
    _dev(t, name, (dtype,), 2)
    if t.shape[0] < min_rows or t.shape[1] != cols:
        raise ValueError("%s must have shape (>= %d, %d) (got %s)" % (name, min_rows, cols, tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s (got %s)" % (name, device, t.device))
    return t


def _same_device(device, *named):
    for name, t in named:
        if t is not None and t.device != device:
            raise ValueError("%s must be on %s (got %s)" % (name, device, t.device))


def nvfp4_quantize_rows(x, amax_in=None, out=None):
    """Per-token NVFP4 of bf16 rows x [rows, k] (k % 16 == 0).

    amax_in: optional float32 [rows], the producer's row amax (amax reuse).
    out: optional preallocated (q, sb, s).  Returns (q, sb, s).
    """
    _dev(x, "x", _BF16, 2)
    rows, k = x.shape
    dev = x.device
    if out is None:
        q = torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
        sb = torch.empty((rows, k // 16), dtype=torch.uint8, device=dev)
        s = torch.empty((rows,), dtype=torch.float32, device=dev)
    else:
        q, sb, s = out
        _out(q, "out q", (rows, k // 2), torch.uint8, dev)
        _out(sb, "out sb", (rows, k // 16), torch.uint8, dev)
        _out(s, "out s", (rows,), torch.float32, dev)
    if amax_in is not None:
        _dev(amax_in, "amax_in", (torch.float32,), 1)
        if amax_in.numel() != rows:
            raise ValueError("amax_in must have one entry per row")
        _same_device(dev, ("amax_in", amax_in))
    st = lib().nvfp4_quantize_rows(_ptr(x), rows, k, _ptr(amax_in), _ptr(q), _ptr(sb), _ptr(s),
                                   _stream(dev))
    _check("nvfp4_quantize_rows", st)
    return q, sb, s


def nvfp4_swiglu_quantize_rows(gate_up, want_h=False, want_amax=False, quantize=True, out=None):
    """SwiGLU of a fused fp32 gate|up block [rows, 2f] (gate in columns
    [0, f), up in [f, 2f)) fused with per-token NVFP4 of its bf16 output.

    Returns a dict with the requested outputs: "h" (bf16 [rows, f]), "amax"
    (float32 [rows]) and "q", "sb", "s" when quantize is true.  `out` may hold
    preallocated tensors under the same keys.
    """
    _dev(gate_up, "gate_up", (torch.float32,), 2)
    rows, f2 = gate_up.shape
    if f2 % 2:
        raise ValueError("gate_up must have an even number of columns")
    f = f2 // 2
    dev = gate_up.device
    out = dict(out or {})
    res = {}
    want = []
    if want_h:
        want.append(("h", (rows, f), torch.bfloat16))
    if want_amax:
        want.append(("amax", (rows,), torch.float32))
    if quantize:
        want += [("q", (rows, f // 2), torch.uint8), ("sb", (rows, f // 16), torch.uint8),
                 ("s", (rows,), torch.float32)]
    for key, shape, dt in want:
        t = out.get(key, None)
        res[key] = torch.empty(shape, dtype=dt, device=dev) if t is None else \
            _out(t, "out " + key, shape, dt, dev)
    st = lib().nvfp4_swiglu_quantize_rows(_ptr(gate_up), rows, f, _ptr(res.get("h")),
                                          _ptr(res.get("amax")), _ptr(res.get("q")),
                                          _ptr(res.get("sb")), _ptr(res.get("s")), _stream(dev))
    _check("nvfp4_swiglu_quantize_rows", st)
    return res


def nvfp4_dequantize_rows(q, sb, s, rows_per_scale=1, out=None):
    """bf16 dequantization of NVFP4 rows: q [rows, k/2] (or [groups, rows,
    k/2]), sb matching, s float32 with one entry per rows_per_scale rows.
    Returns bf16 [rows, k] (same leading shape as q)."""
    _dev(q, "q", (torch.uint8,))
    _dev(sb, "sb", (torch.uint8,))
    _dev(s, "s", (torch.float32,))
    k = q.shape[-1] * 2
    rows = q.numel() // max(q.shape[-1], 1) if q.shape[-1] else int(np.prod(q.shape[:-1]))
    if sb.numel() != rows * (k // 16):
        raise ValueError("sb must hold k/16 scale codes per row")
    if s.numel() * rows_per_scale < rows:
        raise ValueError("s must hold one outer scale per rows_per_scale rows")
    _same_device(q.device, ("sb", sb), ("s", s))
    shape = tuple(q.shape[:-1]) + (k,)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    else:
        _out(out, "out", shape, torch.bfloat16, q.device)
    st = lib().nvfp4_dequantize_rows(_ptr(q), _ptr(sb), _ptr(s), rows, k, int(rows_per_scale),
                                     _ptr(out), _stream(q.device))
    _check("nvfp4_dequantize_rows", st)
    return out


def nvfp4_mxfp8_quantize_rows(x, out=None):
    """MXFP8 of bf16 rows x [rows, k] (k % 32 == 0): returns (q uint8 [rows,
    k] E4M3 codes, sc uint8 [rows, k/32] E8M0 codes)."""
    _dev(x, "x", _BF16, 2)
    rows, k = x.shape
    if out is None:
        q = torch.empty((rows, k), dtype=torch.uint8, device=x.device)
        sc = torch.empty((rows, k // 32), dtype=torch.uint8, device=x.device)
    else:
        q, sc = out
        _out(q, "out q", (rows, k), torch.uint8, x.device)
        _out(sc, "out sc", (rows, k // 32), torch.uint8, x.device)
    st = lib().nvfp4_mxfp8_quantize_rows(_ptr(x), rows, k, _ptr(q), _ptr(sc), _stream(x.device))
    _check("nvfp4_mxfp8_quantize_rows", st)
    return q, sc


def nvfp4_mxfp8_gemm(a, b, out=None):
    """Y = deq(A) . deq(B)^T for MXFP8 operands a = (q [m, k], sc [m, k/32]),
    b = (q [n, k], sc [n, k/32]); fp32 [m, n]."""
    aq, asc = _mx_operand(a, "a", 2)
    bq, bsc = _mx_operand(b, "b", 2)
    m, k = aq.shape
    n = bq.shape[0]
    if bq.shape[1] != k:
        raise ValueError("A and B must have the same k")
    _same_device(aq.device, ("b.q", bq))
    y = _out(out, "out", (m, n), torch.float32, aq.device) if out is not None else \
        torch.empty((m, n), dtype=torch.float32, device=aq.device)
    st = lib().nvfp4_mxfp8_gemm(_ptr(aq), _ptr(asc), m, _ptr(bq), _ptr(bsc), n, k, _ptr(y),
                                _stream(aq.device))
    _check("nvfp4_mxfp8_gemm", st)
    return y


def nvfp4_mxfp8_grouped_gemm(a, offsets, b, row_index=None, m_total=None, out=None):
    """Grouped MXFP8 GEMM: a = (q [a_rows, k], sc [a_rows, k/32]); offsets
    int32 [groups+1] on the device; b = (q [groups, n, k], sc [groups, n,
    k/32]); row_index optional int32 [m_total]."""
    aq, asc = _mx_operand(a, "a", 2)
    bq, bsc = _mx_operand(b, "b", 3)
    _dev(offsets, "offsets", (torch.int32,), 1)
    groups, n, k = bq.shape[0], bq.shape[1], bq.shape[2]
    if aq.shape[1] != k:
        raise ValueError("A and B must have the same k")
    if offsets.numel() != groups + 1:
        raise ValueError("offsets must have groups + 1 entries")
    m_total = _grouped_rows(aq.shape[0], row_index, m_total)
    _same_device(aq.device, ("b.q", bq), ("offsets", offsets), ("row_index", row_index))
    y = _out_rows(out, "out", m_total, n, torch.float32, aq.device) if out is not None else \
        torch.empty((m_total, n), dtype=torch.float32, device=aq.device)
    st = lib().nvfp4_mxfp8_grouped_gemm(_ptr(aq), _ptr(asc), aq.shape[0], _ptr(row_index), m_total,
                                        _ptr(offsets), groups, _ptr(bq), _ptr(bsc), n, k, _ptr(y),
                                        _stream(aq.device))
    _check("nvfp4_mxfp8_grouped_gemm", st)
    return y


def nvfp4_moe_route(logits, topk, out=None):
    """Top-k routing of fp32 logits [tokens, experts] into the contiguous
    per-expert layout on the device.  Returns a dict of int32 tensors:
    experts [tokens, topk], offsets [experts+1], row_index [tokens*topk],
    slot_of [tokens, topk]."""
    _dev(logits, "logits", (torch.float32,), 2)
    T, E = logits.shape
    dev = logits.device
    out = dict(out or {})
    i32 = torch.int32
    res = {}
    for key, shape in (("experts", (T, topk)), ("offsets", (E + 1,)), ("row_index", (T * topk,)),
                       ("slot_of", (T, topk))):
        t = out.get(key, None)
        res[key] = torch.empty(shape, dtype=i32, device=dev) if t is None else \
            _out(t, "out " + key, shape, i32, dev)
    st = lib().nvfp4_moe_route(_ptr(logits), T, E, int(topk), _ptr(res["experts"]),
                               _ptr(res["offsets"]), _ptr(res["row_index"]), _ptr(res["slot_of"]),
                               _stream(dev))
    _check("nvfp4_moe_route", st)
    return res


def nvfp4_quantize_weight(w, amax_in=None, out=None):
    """Per-tensor (groups == 1) or per-expert NVFP4 of bf16 w [groups, rows, k].

    Returns (q [groups, rows, k/2], sb [groups, rows, k/16], s [groups],
    amax [groups]).
    """
    _dev(w, "w", _BF16, 3)
    g, r, k = w.shape
    dev = w.device
    if out is None:
        q = torch.empty((g, r, k // 2), dtype=torch.uint8, device=dev)
        sb = torch.empty((g, r, k // 16), dtype=torch.uint8, device=dev)
        s = torch.empty((g,), dtype=torch.float32, device=dev)
        amax = torch.empty((g,), dtype=torch.float32, device=dev)
    else:
        q, sb, s, amax = out
        _out(q, "out q", (g, r, k // 2), torch.uint8, dev)
        _out(sb, "out sb", (g, r, k // 16), torch.uint8, dev)
        _out(s, "out s", (g,), torch.float32, dev)
        _out(amax, "out amax", (g,), torch.float32, dev)
    if amax_in is not None:
        _dev(amax_in, "amax_in", (torch.float32,), 1)
        if amax_in.numel() != g:
            raise ValueError("amax_in must have one entry per group")
        _same_device(dev, ("amax_in", amax_in))
    st = lib().nvfp4_quantize_weight(_ptr(w), g, r, k, _ptr(amax_in), _ptr(amax), _ptr(q),
                                     _ptr(sb), _ptr(s), _stream(dev))
    _check("nvfp4_quantize_weight", st)
    return q, sb, s, amax


def _operand(t, name, ndim, scales):
    """Check an NVFP4 operand (q, sb, s): q [..., k/2] and sb [..., k/16]
    with the same leading shape (ndim dims), s with `scales` entries, all on
    one device."""
    q, sb, s = t
    _dev(q, name + ".q", (torch.uint8,), ndim)
    _dev(sb, name + ".sb", (torch.uint8,), ndim)
    _dev(s, name + ".s", (torch.float32,))
    if tuple(sb.shape[:-1]) != tuple(q.shape[:-1]) or sb.shape[-1] * 8 != q.shape[-1]:
        raise ValueError("%s.sb must be %s + [k/16] for %s.q of shape %s (got %s)" % (
            name, tuple(q.shape[:-1]), name, tuple(q.shape), tuple(sb.shape)))
    if s.numel() != scales:
        raise ValueError("%s.s must have %d entries (got %d)" % (name, scales, s.numel()))
    _same_device(q.device, (name + ".sb", sb), (name + ".s", s))
    return q, sb, s


def _mx_operand(t, name, ndim):
    """Check an MXFP8 operand (q [..., k], sc [..., k/32])."""
    q, sc = t
    _dev(q, name + ".q", (torch.uint8,), ndim)
    _dev(sc, name + ".sc", (torch.uint8,), ndim)
    if tuple(sc.shape[:-1]) != tuple(q.shape[:-1]) or sc.shape[-1] * 32 != q.shape[-1]:
        raise ValueError("%s.sc must be %s + [k/32] for %s.q of shape %s (got %s)" % (
            name, tuple(q.shape[:-1]), name, tuple(q.shape), tuple(sc.shape)))
    _same_device(q.device, (name + ".sc", sc))
    return q, sc


def _grouped_rows(a_rows, row_index, m_total):
    """Output rows of a grouped GEMM: m_total, else len(row_index), else
    a_rows; checks row_index covers them (or, without it, that A does)."""
    if row_index is not None:
        _dev(row_index, "row_index", (torch.int32,), 1)
        if m_total is None:
            m_total = row_index.numel()
        elif row_index.numel() < m_total:
            raise ValueError("row_index must have m_total entries")
    elif m_total is None:
        m_total = a_rows
    elif m_total > a_rows:
        raise ValueError("without row_index, A must have at least m_total rows")
    return int(m_total)


def nvfp4_gemm(a, b, out=None):
    """Y = deq(A) . deq(B)^T, fp32 [m, n].  a = (q [m, k/2], sb [m, k/16],
    s [m]); b = (q [n, k/2], sb [n, k/16], s [1])."""
    aq = a[0]
    m = aq.shape[0]
    aq, asb, as_ = _operand(a, "a", 2, m)
    bq = b[0]
    if bq.dim() == 3 and bq.shape[0] == 1:  # a per-tensor weight from nvfp4_quantize_weight
        b = (bq[0], b[1][0] if b[1].dim() == 3 else b[1], b[2])
    bq, bsb, bs = _operand(b, "b", 2, 1)
    n = bq.shape[0]
    k = aq.shape[-1] * 2
    if bq.shape[-1] * 2 != k:
        raise ValueError("A and B must have the same k")
    dev = aq.device
    _same_device(dev, ("b.q", bq))
    y = torch.empty((m, n), dtype=torch.float32, device=dev) if out is None else \
        _out(out, "out", (m, n), torch.float32, dev)
    st = lib().nvfp4_gemm(_ptr(aq), _ptr(asb), _ptr(as_), m, _ptr(bq), _ptr(bsb), _ptr(bs), n, k,
                          _ptr(y), _stream(dev))
    _check("nvfp4_gemm", st)
    return y


def nvfp4_grouped_gemm(a, offsets, b, row_index=None, m_total=None, out=None):
    """Grouped GEMM over a contiguous per-expert layout.

    a = (q [a_rows, k/2], sb [a_rows, k/16], s [a_rows]);
    offsets int32 [groups+1] (device); b = (q [groups, n, k/2],
    sb [groups, n, k/16], s [groups]); row_index optional int32 [m_total].
    m_total defaults to len(row_index) or a_rows (the host never reads
    offsets).  Rows at or past offsets[groups] of the output are not written.
    """
    aq, asb, as_ = _operand(a, "a", 2, a[0].shape[0] if a[0].dim() == 2 else -1)
    if b[0].dim() != 3:
        raise ValueError("b.q must be [groups, n, k/2]")
    bq, bsb, bs = _operand(b, "b", 3, b[0].shape[0])
    _dev(offsets, "offsets", (torch.int32,), 1)
    groups, n, k = bq.shape[0], bq.shape[1], bq.shape[2] * 2
    if aq.shape[1] * 2 != k:
        raise ValueError("A and B must have the same k")
    if offsets.numel() != groups + 1:
        raise ValueError("offsets must have groups + 1 entries")
    a_rows = aq.shape[0]
    m_total = _grouped_rows(a_rows, row_index, m_total)
    dev = aq.device
    _same_device(dev, ("b.q", bq), ("offsets", offsets), ("row_index", row_index))
    y = torch.empty((m_total, n), dtype=torch.float32, device=dev) if out is None else \
        _out_rows(out, "out", m_total, n, torch.float32, dev)
    st = lib().nvfp4_grouped_gemm(_ptr(aq), _ptr(asb), _ptr(as_), a_rows, _ptr(row_index),
                                  m_total, _ptr(offsets), groups, _ptr(bq), _ptr(bsb), _ptr(bs),
                                  n, k, _ptr(y), _stream(dev))
    _check("nvfp4_grouped_gemm", st)
    return y


def nvfp4_grouped_gemm_swiglu(a, offsets, b, row_index=None, m_total=None, out=None):
    """Grouped up-projection with SwiGLU in the epilogue.

    a, offsets, row_index, m_total as nvfp4_grouped_gemm; b = the fused
    gate|up weight (q [groups, 2f, k/2], sb [groups, 2f, k/16], s [groups]),
    gate rows first.  Returns (h bf16 [m_total, f], amax float32 [m_total]):
    H = silu(gate) * up of the GEMM output and its row amax (the amax_in of
    the requantize).  out: optional preallocated (h, amax).  k must be a
    positive multiple of 256.
    """
    aq, asb, as_ = _operand(a, "a", 2, a[0].shape[0] if a[0].dim() == 2 else -1)
    if b[0].dim() != 3:
        raise ValueError("b.q must be [groups, 2f, k/2]")
    bq, bsb, bs = _operand(b, "b", 3, b[0].shape[0])
    _dev(offsets, "offsets", (torch.int32,), 1)
    groups, n2, k = bq.shape[0], bq.shape[1], bq.shape[2] * 2
    if n2 % 2:
        raise ValueError("b must have an even number of rows per expert (gate, then up)")
    f = n2 // 2
    if aq.shape[1] * 2 != k:
        raise ValueError("A and B must have the same k")
    if offsets.numel() != groups + 1:
        raise ValueError("offsets must have groups + 1 entries")
    a_rows = aq.shape[0]
    m_total = _grouped_rows(a_rows, row_index, m_total)
    dev = aq.device
    _same_device(dev, ("b.q", bq), ("offsets", offsets), ("row_index", row_index))
    if out is None:
        h = torch.empty((m_total, f), dtype=torch.bfloat16, device=dev)
        amax = torch.empty((m_total,), dtype=torch.float32, device=dev)
    else:
        h = _out_rows(out[0], "out.h", m_total, f, torch.bfloat16, dev)
        amax = out[1]
        _dev(amax, "out.amax", (torch.float32,), 1)
        if amax.numel() < m_total or amax.device != dev:
            raise ValueError("out.amax must have at least m_total entries on %s" % dev)
    st = lib().nvfp4_grouped_gemm_swiglu(_ptr(aq), _ptr(asb), _ptr(as_), a_rows, _ptr(row_index),
                                         m_total, _ptr(offsets), groups, _ptr(bq), _ptr(bsb),
                                         _ptr(bs), f, k, _ptr(h), _ptr(amax), _stream(dev))
    _check("nvfp4_grouped_gemm_swiglu", st)
    return h, amax


_TYPES = {torch.float32: 0, torch.bfloat16: 1}  # NVFP4_TYPE_*
_FLOATS = (torch.float32, torch.bfloat16)


_HERE_ALREADY = contextlib.nullcontext()


def _on(dev):
    """The tensors' device as the current one for a call's launches (entering
    it costs microseconds, so only where it is not current already)."""
    return _HERE_ALREADY if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _type(t):
    return 0 if t is None else _TYPES[t.dtype]


def _out_dtype(dtype):
    if dtype not in _TYPES:
        raise TypeError("an output dtype is torch.float32 or torch.bfloat16 (got %s)" % dtype)
    return dtype


def _no_overlap(out, name, *inputs):
    """An output that shares memory with an input would be read while it is
    written, one that shares it with another output written twice."""
    if out is None or out.numel() == 0:
        return
    lo, hi = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t in inputs:
        if t is not None and t.numel() and t.data_ptr() < hi and lo < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError("%s must not overlap an input or another output" % name)


def _given(out, *keys):
    """The preallocated outputs of a call that takes them by name: a name it
    does not know would be a tensor that is silently never written."""
    out = out or {}
    for key in out:
        if key not in keys:
            raise ValueError("out may hold %s (got %r)" % (", ".join(keys), key))
    return out


def _experts(offsets, groups, dev):
    _dev(offsets, "offsets", (torch.int32,), 1)
    if offsets.numel() != groups + 1:
        raise ValueError("offsets must have groups + 1 entries")
    _same_device(dev, ("offsets", offsets))


def nvfp4_bf16_grouped_gemm(x, offsets, w, row_index=None, m_total=None, out=None, out_dtype=torch.float32):
    """bf16 product grouped by expert: Y[i] = X[r(i)] W_e^T for the rows i of
    expert e, r(i) = row_index[i] or i.

    x bf16 [a_rows, k]; offsets int32 [groups+1] (device); w bf16 [groups, n,
    k]; row_index optional int32 [m_total] (indices outside x are zero rows).
    m_total as for nvfp4_grouped_gemm.  Returns [m_total, n] of out_dtype
    (float32 or bfloat16); rows that no expert owns are not written.
    n % 8 == 0, k % 8 == 0.
    """
    _dev(x, "x", (torch.bfloat16,), 2)
    _dev(w, "w", (torch.bfloat16,), 3)
    groups, n, k = w.shape
    if x.shape[1] != k:
        raise ValueError("x and w must have the same k")
    dev = x.device
    _experts(offsets, groups, dev)
    m_total = _grouped_rows(x.shape[0], row_index, m_total)
    _same_device(dev, ("w", w), ("row_index", row_index))
    if out is None:
        out = torch.empty((m_total, n), dtype=_out_dtype(out_dtype), device=dev)
    else:
        _out_rows(out, "out", m_total, n, _out_dtype(out.dtype), dev)
        _no_overlap(out, "out", x, w, offsets, row_index)
    with _on(dev):
        st = lib().nvfp4_bf16_grouped_gemm(_ptr(x), x.shape[0], _ptr(row_index), m_total, _ptr(offsets), groups,
                                           _ptr(w), n, k, _ptr(out), _type(out), _stream(dev))
    _check("nvfp4_bf16_grouped_gemm", st)
    return out


def nvfp4_bf16_grouped_dgrad(dy, offsets, w, m_total=None, out=None, out_dtype=torch.float32):
    """Data gradient of the grouped product: dX[i] = dY[i] W_e for the rows i
    of expert e.  dy bf16 [m_total, n], w bf16 [groups, n, k] (as
    nvfp4_dequantize_rows writes it in the dequantized backward mode); returns
    the routed rows' gradients [m_total, k] of out_dtype.  A token's own
    gradient is their sum, nvfp4_moe_combine(dx, slot_of)."""
    _dev(dy, "dy", (torch.bfloat16,), 2)
    _dev(w, "w", (torch.bfloat16,), 3)
    groups, n, k = w.shape
    if dy.shape[1] != n:
        raise ValueError("dy and w must have the same n")
    dev = dy.device
    _experts(offsets, groups, dev)
    m_total = _grouped_rows(dy.shape[0], None, m_total)
    _same_device(dev, ("w", w))
    if out is None:
        out = torch.empty((m_total, k), dtype=_out_dtype(out_dtype), device=dev)
    else:
        _out_rows(out, "out", m_total, k, _out_dtype(out.dtype), dev)
        _no_overlap(out, "out", dy, w, offsets)
    with _on(dev):
        st = lib().nvfp4_bf16_grouped_dgrad(_ptr(dy), m_total, _ptr(offsets), groups, _ptr(w), n, k, _ptr(out),
                                            _type(out), _stream(dev))
    _check("nvfp4_bf16_grouped_dgrad", st)
    return out


def nvfp4_bf16_grouped_wgrad(dy, x, offsets, row_index=None, add=None, out=None, out_dtype=torch.float32):
    """Weight gradient of the grouped product: dW_e = add_e + the sum over
    expert e's rows i of dY[i]^T X[r(i)].

    dy bf16 [m_total, n]; x bf16 [a_rows, k]; row_index optional int32
    [m_total]; add optional [groups, n, k] of the output's dtype, which may be
    `out` itself (gradients of several microbatches added up in place).
    Returns [groups, n, k]: zeros (or add) for an expert without rows.
    """
    _dev(dy, "dy", (torch.bfloat16,), 2)
    _dev(x, "x", (torch.bfloat16,), 2)
    _dev(offsets, "offsets", (torch.int32,), 1)
    groups = offsets.numel() - 1
    if groups < 1:
        raise ValueError("offsets must have groups + 1 entries, groups >= 1")
    m_total, n = dy.shape
    k = x.shape[1]
    dev = dy.device
    _grouped_rows(x.shape[0], row_index, m_total)
    _same_device(dev, ("x", x), ("offsets", offsets), ("row_index", row_index), ("add", add))
    shape = (groups, n, k)
    if add is not None:
        _dev(add, "add", _FLOATS, 3)
        if tuple(add.shape) != shape:
            raise ValueError("add must have shape %s (got %s)" % (shape, tuple(add.shape)))
    if out is None:
        out = torch.empty(shape, dtype=_out_dtype(out_dtype) if add is None else add.dtype, device=dev)
    else:
        _out(out, "out", shape, _out_dtype(out.dtype), dev)
        _no_overlap(out, "out", dy, x, offsets, row_index)
    if add is not None:
        if add.dtype != out.dtype:
            raise TypeError("add must have the output's dtype %s (got %s)" % (out.dtype, add.dtype))
        if add.data_ptr() != out.data_ptr():
            _no_overlap(out, "out", add)
    with _on(dev):
        st = lib().nvfp4_bf16_grouped_wgrad(_ptr(dy), m_total, _ptr(x), x.shape[0], _ptr(row_index), _ptr(offsets),
                                            groups, n, k, _ptr(add), _ptr(out), _type(out), _stream(dev))
    _check("nvfp4_bf16_grouped_wgrad", st)
    return out


def _norm_params(dev, rows, d, post_weight, gate, norm_weight):
    """Check the parameters of the residual norms (one dtype, [d]; the gate
    [d] or [rows, d]); returns (param dtype, gate is per row)."""
    dtype = None
    for name, t in (("post_weight", post_weight), ("gate", gate), ("norm_weight", norm_weight)):
        if t is None:
            continue
        _dev(t, name, _FLOATS)
        if t.shape != (d,) and not (t is gate and t.shape == (rows, d)):
            raise ValueError("%s must have shape (%d,)%s (got %s)" % (
                name, d, " or (%d, %d)" % (rows, d) if t is gate else "", tuple(t.shape)))
        if dtype is not None and t.dtype != dtype:
            raise TypeError("post_weight, gate and norm_weight must have one dtype (got %s and %s)" % (dtype, t.dtype))
        dtype = t.dtype
        if t.device != dev:
            raise ValueError("%s must be on %s (got %s)" % (name, dev, t.device))
    return dtype or torch.float32, gate is not None and gate.dim() == 2


def _like(t, name, ref, dtypes=None):
    _dev(t, name, dtypes or (ref.dtype,), 2)
    if t.shape != ref.shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(ref.shape), tuple(t.shape)))
    _same_device(ref.device, (name, t))


def nvfp4_residual_norm(x, residual=None, norm_weight=None, post_weight=None, gate=None, scale=1.0, eps=1e-6,
                        want_h=True, want_amax=False, quantize=False, residual_dtype=None, out=None):
    """The norms after and before a block with its gate and residual:

      n = x / sqrt(mean(x^2) + eps) * post_weight   (n = x without it)
      r' = residual + scale * gate * n
      h = r' / sqrt(mean(r'^2) + eps) * norm_weight, bf16

    x [rows, d] float32 or bfloat16; residual [rows, d] (None: zeros, and r'
    has residual_dtype, bfloat16 unless given); post_weight and norm_weight
    [d], gate [d] or [rows, d], of one dtype.  Returns a dict: "residual" (r',
    in the residual's dtype) and, with norm_weight, "h" (want_h), "amax"
    (want_amax: float32 [rows], max |h|) and "q", "sb", "s" (quantize: as
    nvfp4_quantize_rows(h)).  `out` may hold preallocated tensors under the
    same keys (those not asked for are left as they are); its "residual" may be
    `residual` itself.
    """
    _dev(x, "x", _FLOATS, 2)
    rows, d = x.shape
    dev = x.device
    ptype, gate_rows = _norm_params(dev, rows, d, post_weight, gate, norm_weight)
    if residual is not None:
        _like(residual, "residual", x, _FLOATS)
        if residual_dtype not in (None, residual.dtype):
            raise TypeError("residual_dtype must be the residual's own dtype")
        rdt = residual.dtype
    else:
        rdt = _out_dtype(residual_dtype or torch.bfloat16)
    if norm_weight is None:
        if want_amax or quantize:
            raise ValueError("amax and the quantized rows need norm_weight")
        want_h = False
    want = [("residual", (rows, d), rdt)]
    if want_h:
        want.append(("h", (rows, d), torch.bfloat16))
    if want_amax:
        want.append(("amax", (rows,), torch.float32))
    if quantize:
        want += [("q", (rows, d // 2), torch.uint8), ("sb", (rows, d // 16), torch.uint8),
                 ("s", (rows,), torch.float32)]
    out = _given(out, "residual", "h", "amax", "q", "sb", "s")
    res = {}
    for key, shape, dt in want:
        t = out.get(key)
        if t is None:
            res[key] = torch.empty(shape, dtype=dt, device=dev)
            continue
        res[key] = _out(t, "out " + key, shape, dt, dev)
        same = key == "residual" and residual is not None and t.data_ptr() == residual.data_ptr()
        _no_overlap(t, "out " + key, x, None if same else residual, post_weight, gate, norm_weight,
                    *[o for k, o in res.items() if k != key])
    g = res.get
    with _on(dev):
        st = lib().nvfp4_residual_norm(_ptr(x), _type(x), _ptr(residual), _TYPES[rdt], _ptr(post_weight), _ptr(gate),
                                       int(gate_rows), _ptr(norm_weight), _TYPES[ptype], rows, d, float(scale),
                                       float(eps), _ptr(res["residual"]), _ptr(g("h")), _ptr(g("amax")), _ptr(g("q")),
                                       _ptr(g("sb")), _ptr(g("s")), _stream(dev))
    _check("nvfp4_residual_norm", st)
    return res


def nvfp4_residual_norm_backward(x, residual, norm_weight=None, dh=None, d_residual=None, post_weight=None, gate=None,
                                 scale=1.0, eps=1e-6, dx_dtype=torch.bfloat16, out=None, workspace=None):
    """Backward pass of nvfp4_residual_norm.

    x: the block output; residual: the stored new residual r' (not the one
    that went in); dh bf16 [rows, d] and d_residual (residual's dtype), the
    gradients of h and of r' (either may be None).  Returns a dict: "dx"
    (dx_dtype), "d_residual" (gradient of the residual that went in), and for
    the parameters given "d_post_weight", "d_norm_weight" (float32 [d]) and
    "d_gate" (float32 [d], or [rows, d] of the gate's dtype).  `out` may hold
    preallocated tensors under these keys (those of parameters not given are
    left as they are); its "d_residual" may be `d_residual` itself.
    workspace: optional uint8 tensor of at least
    nvfp4_residual_norm_backward_workspace(rows, d) bytes.
    """
    _dev(x, "x", _FLOATS, 2)
    rows, d = x.shape
    dev = x.device
    ptype, gate_rows = _norm_params(dev, rows, d, post_weight, gate, norm_weight)
    _like(residual, "residual", x, _FLOATS)
    if dh is None and d_residual is None:
        raise ValueError("dh or d_residual must be given")
    if dh is not None:
        if norm_weight is None:
            raise ValueError("dh needs norm_weight")
        _like(dh, "dh", x, (torch.bfloat16,))
    if d_residual is not None:
        _like(d_residual, "d_residual", residual)
    want = [("dx", (rows, d), _out_dtype(dx_dtype)), ("d_residual", (rows, d), residual.dtype)]
    if post_weight is not None:
        want.append(("d_post_weight", (d,), torch.float32))
    if gate is not None:
        want.append(("d_gate", (rows, d), gate.dtype) if gate_rows else ("d_gate", (d,), torch.float32))
    if norm_weight is not None:
        want.append(("d_norm_weight", (d,), torch.float32))
    out = _given(out, "dx", "d_residual", "d_post_weight", "d_gate", "d_norm_weight")
    res = {}
    for key, shape, dt in want:
        t = out.get(key)
        if t is None:
            res[key] = torch.empty(shape, dtype=dt, device=dev)
            continue
        res[key] = _out(t, "out " + key, shape, dt, dev)
        same = key == "d_residual" and d_residual is not None and t.data_ptr() == d_residual.data_ptr()
        _no_overlap(t, "out " + key, x, residual, dh, None if same else d_residual, post_weight, gate, norm_weight,
                    *[o for k, o in res.items() if k != key])
    g = res.get
    if workspace is None:
        with _on(dev):
            need = lib().nvfp4_residual_norm_backward_workspace(rows, d)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    else:
        _dev(workspace, "workspace", (torch.uint8,), 1)
        _same_device(dev, ("workspace", workspace))
        _no_overlap(workspace, "workspace", x, residual, dh, d_residual, post_weight, gate, norm_weight, *res.values())
    with _on(dev):
        st = lib().nvfp4_residual_norm_backward(
            _ptr(x), _type(x), _ptr(residual), _type(residual), _ptr(post_weight), _ptr(gate), int(gate_rows),
            _ptr(norm_weight), _TYPES[ptype], _ptr(dh), _ptr(d_residual), rows, d, float(scale), float(eps),
            _ptr(res["dx"]), _TYPES[dx_dtype], _ptr(res["d_residual"]), _ptr(g("d_post_weight")), _ptr(g("d_gate")),
            _ptr(g("d_norm_weight")), _ptr(workspace), workspace.numel(), _stream(dev))
    _check("nvfp4_residual_norm_backward", st)
    return res


def _slots(slot_of, weights, dev):
    _dev(slot_of, "slot_of", (torch.int32,), 2)
    _same_device(dev, ("slot_of", slot_of), ("weights", weights))
    if weights is not None:
        _dev(weights, "weights", (torch.float32,), 2)
        if weights.shape != slot_of.shape:
            raise ValueError("weights must have slot_of's shape %s (got %s)" % (tuple(slot_of.shape),
                                                                              tuple(weights.shape)))
    return slot_of.shape


def nvfp4_moe_combine(y, slot_of, weights=None, out=None, out_dtype=torch.bfloat16):
    """A token's sum over its experts' rows: out[t] = sum_j weights[t, j] *
    y[slot_of[t, j]].  y [rows, d] float32 or bfloat16; slot_of int32 [tokens,
    topk] as nvfp4_moe_route writes it (a slot outside y adds nothing);
    weights optional float32 [tokens, topk].  Returns [tokens, d]."""
    _dev(y, "y", _FLOATS, 2)
    dev = y.device
    tokens, topk = _slots(slot_of, weights, dev)
    d = y.shape[1]
    if out is None:
        out = torch.empty((tokens, d), dtype=_out_dtype(out_dtype), device=dev)
    else:
        _out(out, "out", (tokens, d), _out_dtype(out.dtype), dev)
        _no_overlap(out, "out", y, slot_of, weights)
    with _on(dev):
        st = lib().nvfp4_moe_combine(_ptr(y), _type(y), y.shape[0], _ptr(slot_of), _ptr(weights), tokens, topk, d,
                                     _ptr(out), _type(out), _stream(dev))
    _check("nvfp4_moe_combine", st)
    return out


def nvfp4_moe_combine_backward(dout, y, slot_of, weights=None, dy_dtype=torch.bfloat16, out=None):
    """Backward pass of nvfp4_moe_combine: "dy" [rows, d] (dy[slot_of[t, j]] =
    weights[t, j] * dout[t]; rows that no slot names are not written) and,
    with weights, "d_weights" [tokens, topk].  No row may be named twice.
    `out` may hold preallocated tensors under these keys ("d_weights" is left
    as it is without weights)."""
    _dev(y, "y", _FLOATS, 2)
    dev = y.device
    tokens, topk = _slots(slot_of, weights, dev)
    d = y.shape[1]
    _dev(dout, "dout", _FLOATS, 2)
    if tuple(dout.shape) != (tokens, d):
        raise ValueError("dout must have shape (%d, %d) (got %s)" % (tokens, d, tuple(dout.shape)))
    _same_device(dev, ("dout", dout))
    out = _given(out, "dy", "d_weights")
    dy = out.get("dy")
    if dy is None:
        dy = torch.empty(tuple(y.shape), dtype=_out_dtype(dy_dtype), device=dev)
    else:
        _out(dy, "out dy", tuple(y.shape), _out_dtype(dy.dtype), dev)
        _no_overlap(dy, "out dy", dout, y, slot_of, weights)
    res = {"dy": dy}
    if weights is not None:
        dw = out.get("d_weights")
        if dw is None:
            dw = torch.empty((tokens, topk), dtype=torch.float32, device=dev)
        else:
            _out(dw, "out d_weights", (tokens, topk), torch.float32, dev)
            _no_overlap(dw, "out d_weights", dout, y, slot_of, weights, dy)
        res["d_weights"] = dw
    with _on(dev):
        st = lib().nvfp4_moe_combine_backward(_ptr(dout), _type(dout), _ptr(y), _type(y), y.shape[0], _ptr(slot_of),
                                              _ptr(weights), tokens, topk, d, _ptr(dy), _type(dy),
                                              _ptr(res.get("d_weights")), _stream(dev))
    _check("nvfp4_moe_combine_backward", st)
    return res


def nvfp4_clip_grad_norm(grads, max_norm, out=None, norm_only=False, workspace=None):
    """Global norm of gradient tensors (float32 and bfloat16, any shapes, one
    device) and clipping by it: g *= min(1, max_norm / (norm + 1e-6)).

    Clips in place (no tensor may then be listed twice), into the tensors of
    `out` (same shapes and dtypes) when given, or not at all with norm_only.
    Returns the norm as a float32 scalar tensor on the device; the host never
    waits.  workspace: optional uint8 tensor of at least
    nvfp4_clip_grad_norm_workspace(len(grads)) bytes.
    """
    grads = list(grads)
    n = len(grads)
    if n == 0:
        raise ValueError("grads must hold at least one tensor")
    dev = grads[0].device if isinstance(grads[0], torch.Tensor) else None
    types, counts, ptrs = [], [], []
    for t in grads:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _TYPES and t.is_contiguous()):
            _dev(t, "a gradient", _FLOATS)  # raises
        if t.device != dev:
            raise ValueError("every gradient must be on %s (got %s)" % (dev, t.device))
        types.append(_TYPES[t.dtype])
        counts.append(t.numel())
        ptrs.append(t.data_ptr())
    outs = ptrs
    if norm_only:
        if out is not None:
            raise ValueError("norm_only takes no out")
        outs = None
    elif out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError("out must have one tensor per gradient")
        outs = []
        for t, g in zip(out, grads):
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == g.dtype and t.is_contiguous()):
                _dev(t, "an out tensor", (g.dtype,))  # raises
            if t.shape != g.shape or t.device != dev:
                raise ValueError("an out tensor must have its gradient's shape %s on %s (got %s on %s)" % (
                    tuple(g.shape), dev, tuple(t.shape), t.device))
            outs.append(t.data_ptr())
    if outs is not None:
        _disjoint(ptrs, outs, [c * (2 if k else 4) for c, k in zip(counts, types)])
        outs = (ctypes.c_void_p * n)(*outs)
    ptrs = (ctypes.c_void_p * n)(*ptrs)
    counts = (ctypes.c_int64 * n)(*counts)
    types = (ctypes.c_int32 * n)(*types)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty((lib().nvfp4_clip_grad_norm_workspace(n),), dtype=torch.uint8, device=dev)
    else:
        _dev(workspace, "workspace", (torch.uint8,), 1)
        _same_device(dev, ("workspace", workspace))
        _no_overlap(workspace, "workspace", *grads, *(out or ()))
    with _on(dev):
        st = lib().nvfp4_clip_grad_norm(ptrs, outs, counts, types, n, float(max_norm), _ptr(norm), _ptr(workspace),
                                        workspace.numel(), _stream(dev))
    _check("nvfp4_clip_grad_norm", st)
    return norm


def _disjoint(grads, outs, sizes):
    """No output may share memory with another output or another gradient: it
    would be read, or scaled twice, after it was written.  grads and outs:
    addresses, outs[i] of the same size in bytes as grads[i]."""
    spans = sorted((p, p + size, i) for i, (p, size) in enumerate(zip(outs, sizes)) if size)
    end = 0
    for lo, hi, i in spans:
        if lo < end:
            raise ValueError("the tensors that are written must not overlap (tensor %d)" % i)
        end = hi
    if outs is grads:
        return
    starts = [s[0] for s in spans]
    for i, (lo, size) in enumerate(zip(grads, sizes)):
        k = bisect.bisect_left(starts, lo + size) - 1  # the last output that starts below the gradient's end
        if size and k >= 0 and spans[k][1] > lo and (spans[k][0] != lo or spans[k][2] != i):
            raise ValueError("out must not overlap another gradient (tensor %d)" % i)
