"""Bi-Level Routing Attention (BiFormer) forward on B200, sm_100a.

A thin ctypes binding over the C ABI of ``libbra_b200.so`` (declared in
``include/bra.h``).  Every step of the path runs in the library's CUDA
kernels; this module only turns torch tensors into pointers and sizes and
turns status codes into exceptions.  There is no CPU fallback: if the
library is missing the import of the binding fails.

Entry points (same names as the C ABI):

    bra_workspace_bytes(shape)
    bra_route(shape, q, k, idx, workspace, stream=None)
    bra_attend(shape, q, k, v, idx, o, workspace, stream=None)
    bra_forward(shape, q, k, v, o, idx, workspace, stream=None)
    bra_device_status(shape, workspace, stream=None)

the operators around the attention in a conditioned block, whose shapes
come from their tensors (``cross_shape_for``, ``rotary_shape_for``):

    bra_cross_attend(shape, q, k, v, kv_len, kv_mask, o, lse, workspace, stream=None)
    bra_cross_attend_backward(shape, q, k, v, kv_len, kv_mask, o, lse, grad_o,
                              dq, dk, dv, workspace, stream=None)
    bra_rotary(shape, q, k, pos, inv_freq, q_out, k_out, stream=None)
    bra_dropout_add(x, residual, p, rng, y, unit=1, stream=None)

and a convenience wrapper ``forward(q, k, v, heads, S, topk)`` that
allocates the outputs and workspace with torch and returns ``(o, idx)``.
"""
from __future__ import annotations

import ctypes
import os
import warnings

__all__ = [
    "BraError", "BraShape", "shape_for", "bra_workspace_bytes", "bra_route", "bra_attend",
    "bra_forward", "bra_device_status", "bra_status_string", "forward", "library_path",
    "bra_route_noalloc", "bra_lce", "bra_selftest_bounded_wait", "bra_attend_backward",
    "bra_qkv_project", "bra_forward_qkv", "bra_forward_lce", "EXPORTED_SYMBOLS",
    "BraCrossShape", "cross_shape_for", "bra_cross_workspace_bytes", "bra_cross_attend",
    "bra_cross_attend_backward", "bra_cross_device_status", "cross_attention",
    "BraRotaryShape", "rotary_shape_for", "bra_rotary", "bra_dropout_add",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
# BRA_LIBRARY selects another build of the same library, e.g. the debug build
# libbra_b200_debug.so (output-index checks in the attention kernels).
library_path = os.environ.get("BRA_LIBRARY") or os.path.join(_HERE, "libbra_b200.so")
debug_library_path = os.path.join(_HERE, "libbra_b200_debug.so")

(BRA_OK, BRA_ERR_INVALID_ARG, BRA_ERR_UNSUPPORTED, BRA_ERR_CUDA, BRA_ERR_TIMEOUT, BRA_ERR_BAD_ROUTE,
 BRA_ERR_BOUNDS) = range(7)
BRA_DTYPE_F32, BRA_DTYPE_BF16 = 0, 1

EXPORTED_SYMBOLS = ("bra_workspace_bytes", "bra_route", "bra_attend", "bra_forward",
                    "bra_device_status", "bra_status_string", "bra_version", "bra_route_noalloc",
                    "bra_lce", "bra_selftest_bounded_wait", "bra_attend_backward", "bra_qkv_project",
                    "bra_forward_qkv", "bra_forward_lce", "bra_cross_workspace_bytes", "bra_cross_attend",
                    "bra_cross_attend_backward", "bra_cross_device_status", "bra_rotary", "bra_dropout_add")
NOALLOC_MAX_MEANS = 1 << 20  # BRA_NOALLOC_MAX_MEANS


class BraShape(ctypes.Structure):
    """Mirror of ``bra_shape``."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int), ("C", ctypes.c_int),
                ("heads", ctypes.c_int), ("S", ctypes.c_int), ("topk", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class BraCrossShape(ctypes.Structure):
    """Mirror of ``bra_cross_shape``."""
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "Lq", "Lk", "heads", "kv_heads", "d", "dtype")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("q_row", "q_batch", "k_row", "k_batch", "v_row", "v_batch")])


class BraRotaryShape(ctypes.Structure):
    """Mirror of ``bra_rotary_shape``."""
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "T", "H", "W", "heads", "kv_heads", "d")]
                + [("pairs", ctypes.c_int * 3)]
                + [(n, ctypes.c_int) for n in ("interleaved", "inverse", "dtype")]
                + [(n, ctypes.c_int64) for n in ("pos_batch", "q_row", "q_batch", "k_row", "k_batch", "qo_row",
                                                 "qo_batch", "ko_row", "ko_batch")])


class BraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bra_status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(library_path):
        raise ImportError(
            f"{library_path} is not built; run `python dynamic_sparse_attention_bra_b200/build.py`")
    lib = ctypes.CDLL(library_path)
    vp, sp = ctypes.c_void_p, ctypes.POINTER(BraShape)
    lib.bra_workspace_bytes.argtypes = [sp]
    lib.bra_workspace_bytes.restype = ctypes.c_size_t
    lib.bra_route.argtypes = [sp, vp, vp, vp, vp, vp]
    lib.bra_attend.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp]
    lib.bra_forward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp]
    lib.bra_lce.argtypes = [sp, vp, vp, vp, vp, vp]
    lib.bra_forward_lce.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.bra_selftest_bounded_wait.argtypes = [sp, vp, ctypes.c_uint, ctypes.c_int, vp]
    lib.bra_attend_backward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.bra_qkv_project.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.bra_forward_qkv.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.bra_device_status.argtypes = [sp, vp, vp]
    lib.bra_route_noalloc.argtypes = [sp, vp, vp, vp, vp]
    lib.bra_route_noalloc.restype = ctypes.c_int
    for f in (lib.bra_route, lib.bra_attend, lib.bra_forward, lib.bra_device_status):
        f.restype = ctypes.c_int
    cp, rp = ctypes.POINTER(BraCrossShape), ctypes.POINTER(BraRotaryShape)
    lib.bra_cross_workspace_bytes.argtypes = [cp]
    lib.bra_cross_workspace_bytes.restype = ctypes.c_size_t
    lib.bra_cross_attend.argtypes = [cp] + [vp] * 9
    lib.bra_cross_attend_backward.argtypes = [cp] + [vp] * 13
    lib.bra_cross_device_status.argtypes = [cp, vp, vp]
    lib.bra_rotary.argtypes = [rp] + [vp] * 7
    lib.bra_dropout_add.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_double] + [vp] * 5
    for f in (lib.bra_cross_attend, lib.bra_cross_attend_backward, lib.bra_cross_device_status, lib.bra_rotary,
              lib.bra_dropout_add):
        f.restype = ctypes.c_int
    lib.bra_status_string.argtypes = [ctypes.c_int]
    lib.bra_status_string.restype = ctypes.c_char_p
    lib.bra_version.argtypes = []
    lib.bra_version.restype = ctypes.c_int
    return lib


_lib = _load()


def bra_status_string(status: int) -> str:
    return _lib.bra_status_string(status).decode()


def shape_for(B: int, H: int, W: int, C: int, heads: int, S: int, topk: int, dtype) -> BraShape:
    """``bra_shape`` for a problem; ``dtype`` is a torch dtype or "f32"/"bf16"."""
    name = str(dtype)
    code = BRA_DTYPE_BF16 if "bf16" in name or "bfloat16" in name else BRA_DTYPE_F32
    return BraShape(B, H, W, C, heads, S, topk, code)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status: int, where: str):
    if status != BRA_OK:
        raise BraError(status, where)


def bra_workspace_bytes(shape: BraShape) -> int:
    return int(_lib.bra_workspace_bytes(ctypes.byref(shape)))


def bra_route(shape: BraShape, q, k, idx, workspace, stream=None) -> None:
    _check(_lib.bra_route(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(idx), _ptr(workspace),
                          _stream(stream)), "bra_route")


def bra_attend(shape: BraShape, q, k, v, idx, o, workspace, stream=None) -> None:
    _check(_lib.bra_attend(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(o),
                           _ptr(workspace), _stream(stream)), "bra_attend")


def bra_forward(shape: BraShape, q, k, v, o, idx, workspace, stream=None) -> None:
    _check(_lib.bra_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(idx),
                            _ptr(workspace), _stream(stream)), "bra_forward")


def bra_attend_backward(shape: BraShape, q, k, v, idx, grad_o, dq, dk, dv, workspace, stream=None) -> None:
    """dQ, dK, dV (fp32 tensors, overwritten) of bra_attend for the fixed routing ``idx``."""
    _check(_lib.bra_attend_backward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(grad_o),
                                    _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), _stream(stream)),
           "bra_attend_backward")


def bra_qkv_project(shape: BraShape, x, w_qkv, b_qkv, q, k, v, q_r, k_r, workspace, stream=None) -> None:
    """[q | k | v] = x w_qkv^T (+ b_qkv) in bf16 and the fp32 region means q_r, k_r of q and k."""
    _check(_lib.bra_qkv_project(ctypes.byref(shape), _ptr(x), _ptr(w_qkv), _ptr(b_qkv) if b_qkv is not None else None,
                                _ptr(q), _ptr(k), _ptr(v), _ptr(q_r), _ptr(k_r), _ptr(workspace), _stream(stream)),
           "bra_qkv_project")


def bra_forward_qkv(shape: BraShape, x, w_qkv, b_qkv, q, k, v, o, idx, workspace, stream=None) -> None:
    """The path from the feature map x: projection with region means, routing, attention."""
    _check(_lib.bra_forward_qkv(ctypes.byref(shape), _ptr(x), _ptr(w_qkv), _ptr(b_qkv) if b_qkv is not None else None,
                                _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(idx), _ptr(workspace), _stream(stream)),
           "bra_forward_qkv")


def bra_selftest_bounded_wait(shape: BraShape, workspace, tries: int, arrive: bool, stream=None) -> None:
    """Launch the bounded-wait self-test kernel (see include/bra.h); read the
    outcome with bra_device_status."""
    _check(_lib.bra_selftest_bounded_wait(ctypes.byref(shape), _ptr(workspace), tries, 1 if arrive else 0,
                                          _stream(stream)), "bra_selftest_bounded_wait")


def bra_lce(shape: BraShape, v, weight, bias, o, stream=None) -> None:
    """o += bias + 5x5 depthwise filter of v (weight fp32 [C, 5, 5], bias fp32 [C] or None)."""
    _check(_lib.bra_lce(ctypes.byref(shape), _ptr(v), _ptr(weight), _ptr(bias) if bias is not None else None,
                        _ptr(o), _stream(stream)), "bra_lce")


def bra_forward_lce(shape: BraShape, q, k, v, weight, bias, o, idx, workspace, stream=None) -> None:
    """Routing, attention and the local context term (weight [C,5,5] fp32, bias [C] or None) in one call."""
    _check(_lib.bra_forward_lce(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(weight),
                                _ptr(bias) if bias is not None else None, _ptr(o), _ptr(idx), _ptr(workspace),
                                _stream(stream)), "bra_forward_lce")


def bra_route_noalloc(shape: BraShape, q, k, idx, stream=None) -> None:
    """bra_route with the library's own fixed scratch: for callers that cannot
    allocate device memory (see include/bra.h for the size limit and the
    rule that overlapping calls race)."""
    _check(_lib.bra_route_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(idx), _stream(stream)),
           "bra_route_noalloc")


def bra_device_status(shape: BraShape, workspace, stream=None) -> int:
    """Synchronises the stream; returns (and clears) the device status code."""
    return int(_lib.bra_device_status(ctypes.byref(shape), _ptr(workspace), _stream(stream)))


def _check_tensor(t, name: str, dtype, numel: int):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and t.dtype == dtype
            and t.numel() == numel):
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of {numel} elements")


def forward(q, k, v, heads: int, S: int, topk: int, stream=None):
    """O, I^r for channels-last q, k, v [B, H, W, C] (float32 or bfloat16).

    Allocates O [B, H, W, C], I^r int32 [B, heads, S*S, topk] and a zeroed
    workspace with torch on q's device, then runs ``bra_forward``."""
    import torch
    B, H, W, C = q.shape
    shape = shape_for(B, H, W, C, heads, S, topk, q.dtype)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, name, q.dtype, B * H * W * C)
    nbytes = bra_workspace_bytes(shape)
    if nbytes == 0:
        raise BraError(BRA_ERR_INVALID_ARG, "forward")
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    idx = torch.empty((B, heads, S * S, topk), dtype=torch.int32, device=q.device)
    bra_forward(shape, q, k, v, o, idx, ws, stream)
    return o, idx


# ---- operators around the attention: shapes and strides come from tensors ----

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BRA_DTYPE_BF16
    if t.dtype == torch.float32:
        return BRA_DTYPE_F32
    raise ValueError(f"expected a bfloat16 or float32 tensor, got {t.dtype}")


def _token_strides(t, name: str, width: int):
    """(B, L, row step, entry step) in elements of tokens [B, L, width], or of
    a contiguous map [B, H, W, width] (or [B, T, H, W, width])."""
    if t.ndim != 3:
        if t.ndim < 3 or t.shape[-1] != width or not t.is_contiguous():
            raise ValueError(f"{name}: expected [B, L, {width}] or a contiguous map, got {tuple(t.shape)}")
        B, L = t.shape[0], 1
        for n in t.shape[1:-1]:
            L *= n
        return B, L, width, L * width
    B, L, w = t.shape
    sb, sl, se = t.stride()
    if w != width or (se != 1 and w > 1):
        raise ValueError(f"{name}: expected [B, L, {width}] with consecutive elements, got {tuple(t.shape)}, "
                         f"strides {t.stride()}")
    row = sl if L > 1 else width  # a step that is never taken is the dense one
    return B, L, row, sb if B > 1 else L * row


def _same_tokens(t, name, width, B, L, row, batch, dtype, dev: int):
    """``t`` is what the shape says: its size, steps, type and device."""
    if t.dtype is dtype and t.get_device() == dev:
        if t.dim() == 3:
            size, step = t.shape, t.stride()
            if (size[0] == B and size[1] == L and size[2] == width and step[2] == 1 and (L <= 1 or step[1] == row)
                    and (B <= 1 or step[0] == batch)):
                return
        elif _token_strides(t, name, width) == (B, L, row, batch):
            return
    raise ValueError(f"{name}: {t.dtype} of {tuple(t.shape)}, strides {t.stride()}, on {t.device} is not what the "
                     f"shape says ({dtype} of [{B}, {L}, {width}], steps {batch}, {row}, on cuda:{dev})")


def _dense(t, name, dtype, numel, dev: int) -> bool:
    """``t`` is contiguous with ``numel`` elements or more; whether it has just these."""
    n = t.numel()
    if t.dtype is not dtype or t.get_device() != dev or n < numel or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {numel} elements on cuda:{dev}, got "
                         f"{t.dtype} of {tuple(t.shape)} on {t.device}")
    return n == numel


def _entries(t, name, count: int, entry: int):
    """A larger ``t`` has entries of the shape's ``entry`` elements, where there is more than one."""
    if count > 1 and entry and t.dim() > 1 and t.numel() != t.shape[0] * entry:
        raise ValueError(f"{name}: the entries of {tuple(t.shape)} do not have the shape's {entry} elements")


def _cuda_device(t, where: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{where}: expected CUDA tensors, got one on {t.device}")
    return t.get_device()


def _current_stream(dev: int) -> int:
    """The handle of ``dev``'s current stream.  The direct query, where this torch has
    it, costs a tenth of a microsecond; a stream object two."""
    import torch
    direct = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return direct(dev) if direct is not None else torch.cuda.current_stream(dev).cuda_stream


_query_device = None


def _current_device() -> int:
    """torch.cuda.current_device(), by the direct query where this torch has it."""
    global _query_device
    if _query_device is None:
        import torch
        _query_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _query_device()


def _call(where: str, fn, dev: int, stream, *args):
    """``fn(*args, stream)`` with device ``dev`` current; None is its current stream."""
    if stream is None:
        raw = _current_stream(dev)
    else:
        raw = stream if isinstance(stream, int) else stream.cuda_stream
    if dev == _current_device():
        status = fn(*args, raw)
    else:
        import torch
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != BRA_OK:
        raise BraError(status, where)


def _torch_dtype(code: int):
    import torch
    return torch.bfloat16 if code == BRA_DTYPE_BF16 else torch.float32


def cross_shape_for(q, k, v, heads: int, kv_heads: int | None = None, scale: float | None = None) -> BraCrossShape:
    """``bra_cross_shape`` of q [B, Lq, heads * d] (or a contiguous map) and k, v
    [B, Lk, kv_heads * d]; the three may be slices or (in B) expanded views.
    ``scale`` defaults to 1 / sqrt(d)."""
    kv_heads = heads if kv_heads is None else kv_heads
    dtype = _dtype_code(q)
    wq = q.shape[-1]
    if heads < 1 or kv_heads < 1 or wq % heads:
        raise ValueError(f"{heads} heads do not divide {wq} channels")
    d = wq // heads
    B, Lq, q_row, q_batch = _token_strides(q, "q", wq)
    Bk, Lk, k_row, k_batch = _token_strides(k, "k", kv_heads * d)
    Bv, Lv, v_row, v_batch = _token_strides(v, "v", kv_heads * d)
    if (Bk, Bv) != (B, B) or Lk != Lv or _dtype_code(k) != dtype or _dtype_code(v) != dtype:
        raise ValueError("q, k and v disagree in batch, length or type")
    return BraCrossShape(B, Lq, Lk, heads, kv_heads, d, dtype, d ** -0.5 if scale is None else scale, q_row, q_batch,
                         k_row, k_batch, v_row, v_batch)


def _cross_inputs(s, q, k, v, kv_len, kv_mask, workspace):
    import torch
    dev, dtype = _cuda_device(q, "cross attention"), _torch_dtype(s.dtype)
    B, Lk, wk = s.B, s.Lk, s.kv_heads * s.d
    _same_tokens(q, "q", s.heads * s.d, B, s.Lq, s.q_row, s.q_batch, dtype, dev)
    _same_tokens(k, "k", wk, B, Lk, s.k_row, s.k_batch, dtype, dev)
    _same_tokens(v, "v", wk, B, Lk, s.v_row, s.v_batch, dtype, dev)
    if kv_len is not None:
        _dense(kv_len, "kv_len", torch.int32, s.B, dev)
    if kv_mask is not None:
        if kv_mask.dtype == torch.bool:
            kv_mask = kv_mask.view(torch.uint8)
        _dense(kv_mask, "kv_mask", torch.uint8, B * Lk, dev) or _entries(kv_mask, "kv_mask", B, Lk)
    _dense(workspace, "workspace", torch.uint8, _cross_workspace_bytes_on(s, dev), dev)
    return dev, kv_mask


def _dense_log_sums(lse, s, dev: int):
    import torch
    each = s.heads * s.Lq
    _dense(lse, "lse", torch.float32, s.B * each, dev) or _entries(lse, "lse", s.B * s.heads, each)


def _cross_workspace_bytes_on(shape, dev: int) -> int:
    """The size for device ``dev``, by whose number of SMs its kernels split their work."""
    if dev == _current_device():
        return bra_cross_workspace_bytes(shape)
    import torch
    with torch.cuda.device(dev):
        return bra_cross_workspace_bytes(shape)


def bra_cross_workspace_bytes(shape: BraCrossShape) -> int:
    """Bytes of workspace that ``shape`` needs on the current device."""
    return int(_lib.bra_cross_workspace_bytes(ctypes.byref(shape)))


def bra_cross_attend(shape: BraCrossShape, q, k, v, kv_len, kv_mask, o, lse, workspace, stream=None) -> None:
    """o [B, Lq, heads * d] (and lse fp32 [B, heads, Lq], or None) of q over the
    states k, v; kv_len int32 [B] and kv_mask uint8 or bool [B, Lk], or None,
    say which states are valid.  ``workspace``: bra_cross_workspace_bytes(shape)
    bytes of uint8, zeroed once.  Outputs and masks may be larger (more entries, flat
    memory), not with longer entries: those lie elsewhere."""
    import torch
    s = shape
    dev, kv_mask = _cross_inputs(s, q, k, v, kv_len, kv_mask, workspace)
    each = s.Lq * s.heads * s.d
    _dense(o, "o", q.dtype, s.B * each, dev) or _entries(o, "o", s.B, each)
    if lse is not None:
        _dense_log_sums(lse, s, dev)
    _call("bra_cross_attend", _lib.bra_cross_attend, dev, stream, ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v),
          _ptr(kv_len), _ptr(kv_mask), _ptr(o), _ptr(lse), _ptr(workspace))


def bra_cross_attend_backward(shape: BraCrossShape, q, k, v, kv_len, kv_mask, o, lse, grad_o, dq, dk, dv, workspace,
                              stream=None) -> None:
    """dq, dk, dv (dense, of q's type, overwritten) for the gradient grad_o of
    bra_cross_attend's o; o and lse as it wrote them."""
    import torch
    s = shape
    dev, kv_mask = _cross_inputs(s, q, k, v, kv_len, kv_mask, workspace)
    nq, nk = s.Lq * s.heads * s.d, s.Lk * s.kv_heads * s.d
    for t, name, n in ((o, "o", nq), (grad_o, "grad_o", nq), (dq, "dq", nq), (dk, "dk", nk), (dv, "dv", nk)):
        _dense(t, name, q.dtype, s.B * n, dev) or _entries(t, name, s.B, n)
    _dense_log_sums(lse, s, dev)
    _call("bra_cross_attend_backward", _lib.bra_cross_attend_backward, dev, stream, ctypes.byref(s), _ptr(q), _ptr(k),
          _ptr(v), _ptr(kv_len), _ptr(kv_mask), _ptr(o), _ptr(lse), _ptr(grad_o), _ptr(dq), _ptr(dk), _ptr(dv),
          _ptr(workspace))


def bra_cross_device_status(shape: BraCrossShape, workspace, stream=None) -> int:
    """Synchronises the stream (None: the workspace's device's current one);
    returns (and clears) the device status code."""
    import torch
    dev = _cuda_device(workspace, "cross attention")
    raw = _current_stream(dev) if stream is None else _stream(stream)
    with torch.cuda.device(dev):
        return int(_lib.bra_cross_device_status(ctypes.byref(shape), _ptr(workspace), raw))


def cross_attention(q, k, v, heads: int, kv_heads: int | None = None, kv_len=None, kv_mask=None,
                    scale: float | None = None, stream=None):
    """(o, lse) of q [B, Lq, heads * d] over the states k, v [B, Lk, kv_heads * d].

    Allocates o, lse and a zeroed workspace with torch on q's device (as
    ``stream``'s, where one is given: what is freed is not used again before the
    kernels end), then runs ``bra_cross_attend``.  The results carry no autograd
    graph (a warning says so where an input asks for gradients): those come from
    ``bra_cross_attend_backward`` with this o and lse."""
    import torch
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        warnings.warn("cross_attention returns o and lse without an autograd graph; the gradients of q, k and v are "
                      "bra_cross_attend_backward's", stacklevel=2)
    shape = cross_shape_for(q, k, v, heads, kv_heads, scale)
    nbytes = _cross_workspace_bytes_on(shape, _cuda_device(q, "cross attention"))
    if nbytes == 0:
        raise BraError(BRA_ERR_INVALID_ARG if shape.d in (32, 64, 128) else BRA_ERR_UNSUPPORTED, "cross_attention")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=q.device)
    with torch.cuda.stream(stream):  # None: as it is
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty((shape.B, heads, shape.Lq), dtype=torch.float32, device=q.device)
        bra_cross_attend(shape, q, k, v, kv_len, kv_mask, o, lse, ws, stream)
    return o, lse


def rotary_shape_for(q, k, heads: int, kv_heads: int, pairs, grid=None, pos=None, interleaved: bool = False,
                     inverse: bool = False, q_out=None, k_out=None) -> BraRotaryShape:
    """``bra_rotary_shape`` of q [B, L, heads * d] and k [B, L, kv_heads * d] (or
    None).  ``pairs``: rotation pairs of (time, height, width).  ``grid``: (T,
    H, W) of the L tokens, or None for a sequence (time runs over L).  ``pos``:
    the positions int32 [B, L, 3] (or [1, L, 3], shared) that the calls will be
    given, if any.  ``q_out``, ``k_out``: outputs that are not dense."""
    wq = q.shape[-1]
    if heads < 1 or wq % heads:
        raise ValueError(f"{heads} heads do not divide {wq} channels")
    d = wq // heads
    B, L, q_row, q_batch = _token_strides(q, "q", wq)
    T, H, W = (L, 1, 1) if grid is None else grid
    if T * H * W != L:
        raise ValueError(f"a grid of {T} x {H} x {W} has no {L} tokens")
    k_row = k_batch = ko_row = ko_batch = 0
    qo_row, qo_batch = wq, L * wq
    if q_out is not None:
        qo_row, qo_batch = _token_strides(q_out, "q_out", wq)[2:]
    if k is not None:
        wk = kv_heads * d
        Bk, Lk, k_row, k_batch = _token_strides(k, "k", wk)
        if (Bk, Lk) != (B, L) or _dtype_code(k) != _dtype_code(q):
            raise ValueError("q and k disagree in batch, length or type")
        ko_row, ko_batch = wk, L * wk
        if k_out is not None:
            ko_row, ko_batch = _token_strides(k_out, "k_out", wk)[2:]
    pos_batch = L * 3 if pos is not None and pos.shape[0] > 1 else 0
    return BraRotaryShape(B, T, H, W, heads, kv_heads if k is not None else 0, d, tuple(pairs), int(interleaved),
                          int(inverse), _dtype_code(q), pos_batch, q_row, q_batch, k_row, k_batch, qo_row, qo_batch,
                          ko_row, ko_batch)


def _check_positions(pos, B: int, L: int, step: int):
    """``pos`` has its entries where ``step`` (0: shared) finds them; a tensor that is merely
    large enough would turn entries by another's positions."""
    n = pos.numel()
    if B <= 1 or n == (B * step if step else L * 3):
        return
    if step:
        fine = pos.dim() < 3 or n == pos.shape[0] * step
    else:
        fine = pos.shape[0] == 1 or (pos.dim() < 3 and n < B * L * 3)
    if not fine:
        raise ValueError(f"pos: {tuple(pos.shape)} is not what the shape says ({B} entries of {L} tokens, "
                         f"{f'{step} elements apart' if step else 'sharing their positions'}); "
                         "rotary_shape_for takes the positions that the calls will be given")


def bra_rotary(shape: BraRotaryShape, q, k, pos, inv_freq, q_out, k_out, stream=None) -> None:
    """q_out, k_out = q, k turned by their positions: pos int32 [B or 1, L, 3]
    (time, height, width), or None for the shape's grid; inv_freq fp32, one for
    each pair.  k and k_out may both be None."""
    import torch
    s, dev = shape, _cuda_device(q, "rotary positions")
    dtype, B = _torch_dtype(s.dtype), s.B
    L, wq, wk = s.T * s.H * s.W, s.heads * s.d, s.kv_heads * s.d
    _same_tokens(q, "q", wq, B, L, s.q_row, s.q_batch, dtype, dev)
    _same_tokens(q_out, "q_out", wq, B, L, s.qo_row, s.qo_batch, dtype, dev)
    if (k is None) != (k_out is None) or (k is None) != (s.kv_heads == 0):
        raise ValueError("k, k_out and the shape's kv_heads go together")
    if k is not None:
        _same_tokens(k, "k", wk, B, L, s.k_row, s.k_batch, dtype, dev)
        _same_tokens(k_out, "k_out", wk, B, L, s.ko_row, s.ko_batch, dtype, dev)
    if pos is not None:
        _check_positions(pos, B, L, s.pos_batch)
        _dense(pos, "pos", torch.int32, (B - 1) * s.pos_batch + L * 3 if B else 0, dev)
    _dense(inv_freq, "inv_freq", torch.float32, sum(s.pairs), dev)
    _call("bra_rotary", _lib.bra_rotary, dev, stream, ctypes.byref(s), _ptr(q), _ptr(k), _ptr(pos), _ptr(inv_freq),
          _ptr(q_out), _ptr(k_out))


def bra_dropout_add(x, residual, p: float, rng, y, unit: int = 1, stream=None) -> None:
    """y = residual + (keep ? x / (1 - p) : 0), ``unit`` consecutive elements
    sharing a draw (see include/bra.h); residual may be None, rng is an int64
    (or uint64) tensor {seed, offset} on x's device.  The gradient of x is the
    same call on the gradient of y, without a residual."""
    import torch
    n, dev = x.numel(), _cuda_device(x, "dropout")
    dtype = _dtype_code(x)
    for t, name in ((x, "x"), (residual, "residual"), (y, "y")):
        if t is not None and not _dense(t, name, x.dtype, n, dev) and x.dim() > 1 and n:
            _entries(t, name, x.shape[0], n // x.shape[0])
    _dense(rng, "rng", torch.uint64 if rng.dtype == torch.uint64 else torch.int64, 2, dev)
    _call("bra_dropout_add", _lib.bra_dropout_add, dev, stream, dtype, n, unit, p, _ptr(rng), _ptr(x), _ptr(residual),
          _ptr(y))
