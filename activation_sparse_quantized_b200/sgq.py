"""Thin ctypes binding to libsgq.so (include/sgq.h). Argument marshalling only.

Each ``sgq_*`` function here has the name and argument order of the C entry
point; torch tensors are passed as device pointers (``data_ptr()``), the
stream defaults to torch's current stream, and a nonzero return code raises
``SgqError``. Every step of the computation runs in the CUDA library; there
is no fallback. If ``libsgq.so`` is missing the first call raises.

``alloc_*`` helpers only allocate correctly sized torch tensors (device
memory is plumbing, not part of the path).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsgq.so")

SGQ_ACT_SILU = 0
SGQ_ACT_RELU = 1
SGQ_STATUS_NONFINITE_W = 1
SGQ_STATUS_BAD_INDEX = 2
SGQ_STATUS_BAD_COUNT = 4
SGQ_STATUS_TIMEOUT = 8
SGQ_MAX_BATCH = 16
SGQ_STATUS_NO_PAGES = 16
SGQ_NOALLOC_MAX_N = 65536
SGQ_TYPE_BF16 = 0
SGQ_TYPE_F32 = 1
SGQ_TYPE_E4M3 = 2
SGQ_MAX_REQUESTS = 8192

EXPORTS = (
    "sgq_packed_sizes", "sgq_pack", "sgq_select", "sgq_gemv_workspace_bytes", "sgq_gemv",
    "sgq_gemv_thresh", "sgq_gemv_dense", "sgq_glu", "sgq_status_string", "sgq_last_cuda_error",
    "sgq_layout_version", "sgq_gemv_thresh_noalloc", "sgq_gemv_glu", "sgq_gemv_glu_thresh",
    "sgq_gemv_glu_dense", "sgq_select_mask", "sgq_gemv_mask", "sgq_packed_sizes_nm",
    "sgq_pack_nm", "sgq_gemv_nm", "sgq_gemv_nm_thresh", "sgq_gemv_acc", "sgq_gemv_thresh_acc",
    "sgq_ffn_workspace_bytes", "sgq_ffn", "sgq_read_status", "sgq_debug_gemv_withhold",
    "sgq_gemv_thresh_batch", "sgq_gemv_glu_thresh_batch", "sgq_cache_plan", "sgq_cache_write",
    "sgq_tree_attn_workspace_bytes", "sgq_tree_attn", "sgq_residual_norm",
    "sgq_debug_tree_attn_withhold",
)


class SgqError(RuntimeError):
    def __init__(self, fn, code, lib):
        msg = lib.sgq_status_string(code).decode()
        if code == -8:
            msg += f" (cudaError {lib.sgq_last_cuda_error()})"
        super().__init__(f"{fn}: {msg} [{code}]")
        self.code = code


_lib = None
_lock = threading.Lock()


def _open(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"libsgq.so not found at {path}: build it with "
            "`python -m activation_sparse_quantized_b200.build` (there is no CPU fallback)")
    return _declare(ctypes.CDLL(path))


def load(path: str = LIB_PATH):
    """Load libsgq.so (raises if it has not been built)."""
    global _lib
    if path is LIB_PATH and _lib is not None:
        return _lib
    if path != LIB_PATH:
        return _open(path)
    with _lock:
        if _lib is None:
            _lib = _open(path)
    return _lib


def _declare(lib):
    P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    L = ctypes.c_longlong
    sig = {
        "sgq_packed_sizes": ([I, I, I, ctypes.POINTER(Z), ctypes.POINTER(Z)], I),
        "sgq_pack": ([P, I, I, I, P, P, P, P], I),
        "sgq_select": ([P, I, I, P, P, P, P], I),
        "sgq_gemv_workspace_bytes": ([I, I, I], Z),
        "sgq_gemv": ([P, P, I, I, I, P, I, P, P, P, P, P, Z, P, P], I),
        "sgq_debug_gemv_withhold": ([P, P, I, I, I, P, I, P, P, P, P, P, Z, P, P], I),
        "sgq_gemv_thresh": ([P, P, I, I, I, P, F, P, P, P, Z, P, P], I),
        "sgq_gemv_thresh_batch": ([P, P, I, I, I, P, I, P, P, P, P, Z, P, P], I),
        "sgq_gemv_glu_thresh_batch": ([P, P, I, I, I, P, I, P, I, P, P, P, Z, P, P], I),
        "sgq_gemv_dense": ([P, P, I, I, I, P, I, P, P, P, Z, P, P], I),
        "sgq_gemv_thresh_noalloc": ([P, P, I, I, I, P, F, P, P, P, P], I),
        "sgq_glu": ([P, P, P, I, I, I, P], I),
        "sgq_gemv_glu": ([P, P, I, I, I, P, I, P, P, I, P, P, P, Z, P, P], I),
        "sgq_gemv_glu_thresh": ([P, P, I, I, I, P, F, I, P, P, P, Z, P, P], I),
        "sgq_gemv_glu_dense": ([P, P, I, I, I, P, I, I, P, P, P, Z, P, P], I),
        "sgq_select_mask": ([P, I, I, P, P, P, P], I),
        "sgq_gemv_mask": ([P, P, I, I, I, P, I, P, P, P, P, Z, P, P], I),
        "sgq_packed_sizes_nm": ([I, I, I, ctypes.POINTER(Z), ctypes.POINTER(Z),
                                 ctypes.POINTER(Z)], I),
        "sgq_pack_nm": ([P, I, I, I, P, P, P, P, P], I),
        "sgq_gemv_nm": ([P, P, P, I, I, I, P, P, P, P, P, P, Z, P, P], I),
        "sgq_gemv_nm_thresh": ([P, P, P, I, I, I, P, F, P, P, P, Z, P, P], I),
        "sgq_gemv_acc": ([P, P, I, I, I, P, I, P, P, P, P, P], I),
        "sgq_gemv_thresh_acc": ([P, P, I, I, I, P, F, P, P, P], I),
        "sgq_ffn_workspace_bytes": ([I, I], Z),
        "sgq_read_status": ([P, P, I, P], I),
        "sgq_ffn": ([P, P, P, P, I, I, I, P, F, I, F, P, P, P, P, Z, P, P], I),
        "sgq_cache_plan": ([P, P, I, I, I, P, I, P, P, P, P, P, P, I, P, P, P, P, P, P], I),
        "sgq_cache_write": ([P, L, P, L, P, L, I, P, I, P, P, I, P, P, L, P, P, P], I),
        "sgq_tree_attn_workspace_bytes": ([I, I, I, I, I], Z),
        "sgq_tree_attn": ([P, L, I, I, I, P, P, P, I, P, P, I, F, P, L, P, P, Z, P, P], I),
        "sgq_debug_tree_attn_withhold": ([P, L, I, I, I, P, P, P, I, P, P, I, F, P, L, P, P, Z, P, P], I),
        "sgq_residual_norm": ([P, L, I, P, P, L, F, P, L, I, P, L, P, I, F, P, L, I, I, F, P], I),
        "sgq_status_string": ([I], ctypes.c_char_p),
        "sgq_last_cuda_error": ([], I),
        "sgq_layout_version": ([], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current device and its current stream's handle, by torch's own short way where
# this torch has it (building a Stream object takes 3 us).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream, dev=None):
    if stream is None:
        return _current_stream(torch.cuda.current_device() if dev is None else dev)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise SgqError(fn, rc, load())


# --------------------------------------------------------------------------
# The C entry points, one to one.
# --------------------------------------------------------------------------

def sgq_read_status(status, clear=True, stream=None) -> int:
    """The SGQ_STATUS_* bits of a device status word (synchronises the stream
    to return the value; the C call itself only enqueues the copy)."""
    out = ctypes.c_int32(0)
    _check("sgq_read_status", load().sgq_read_status(_ptr(status), ctypes.byref(out),
                                                     1 if clear else 0, _stream(stream)))
    (stream or torch.cuda.current_stream()).synchronize()
    return out.value


def sgq_layout_version() -> int:
    return load().sgq_layout_version()


def sgq_packed_sizes(N: int, K: int, group: int):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check("sgq_packed_sizes", load().sgq_packed_sizes(N, K, group, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def sgq_pack(W, N, K, group, qweight, sz, status=None, stream=None):
    _check("sgq_pack", load().sgq_pack(_ptr(W), N, K, group, _ptr(qweight), _ptr(sz),
                                       _ptr(status), _stream(stream)))


def sgq_select(x, B, K, t_host, idx, count, stream=None):
    t = (ctypes.c_float * B)(*[float(v) for v in t_host])
    _check("sgq_select", load().sgq_select(_ptr(x), B, K, t, _ptr(idx), _ptr(count),
                                           _stream(stream)))


def sgq_select_mask(x, B, K, t_host, mask, count=None, stream=None):
    t = (ctypes.c_float * B)(*[float(v) for v in t_host])
    _check("sgq_select_mask", load().sgq_select_mask(_ptr(x), B, K, t, _ptr(mask), _ptr(count),
                                                     _stream(stream)))


def sgq_gemv_mask(qweight, sz, N, K, group, x, B, mask, y, y_f32, workspace, status=None,
                  stream=None):
    _check("sgq_gemv_mask", load().sgq_gemv_mask(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), B, _ptr(mask), _ptr(y), _ptr(y_f32),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_packed_sizes_nm(N: int, K: int, group: int):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check("sgq_packed_sizes_nm", load().sgq_packed_sizes_nm(
        N, K, group, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def sgq_pack_nm(W, N, K, group, qweight, keep, sz, status=None, stream=None):
    _check("sgq_pack_nm", load().sgq_pack_nm(_ptr(W), N, K, group, _ptr(qweight), _ptr(keep),
                                             _ptr(sz), _ptr(status), _stream(stream)))


def sgq_gemv_nm(qweight, keep, sz, N, K, group, x, idx, count, y, y_f32, workspace, status=None,
                stream=None):
    _check("sgq_gemv_nm", load().sgq_gemv_nm(
        _ptr(qweight), _ptr(keep), _ptr(sz), N, K, group, _ptr(x), _ptr(idx), _ptr(count),
        _ptr(y), _ptr(y_f32), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))


def sgq_gemv_nm_thresh(qweight, keep, sz, N, K, group, x, t, y, y_f32, workspace, status=None,
                       stream=None):
    _check("sgq_gemv_nm_thresh", load().sgq_gemv_nm_thresh(
        _ptr(qweight), _ptr(keep), _ptr(sz), N, K, group, _ptr(x), float(t), _ptr(y),
        _ptr(y_f32), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))


def sgq_gemv_acc(qweight, sz, N, K, group, x, B, idx, count, y_acc, status=None, stream=None):
    """y_acc (fp32 [B][N]) += the sparse GEMV; one kernel, no workspace."""
    _check("sgq_gemv_acc", load().sgq_gemv_acc(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), B, _ptr(idx), _ptr(count), _ptr(y_acc),
        _ptr(status), _stream(stream)))


def sgq_gemv_thresh_acc(qweight, sz, N, K, group, x, t, y_acc, status=None, stream=None):
    _check("sgq_gemv_thresh_acc", load().sgq_gemv_thresh_acc(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), float(t), _ptr(y_acc), _ptr(status),
        _stream(stream)))


def sgq_gemv_workspace_bytes(N: int, K: int, B: int) -> int:
    return load().sgq_gemv_workspace_bytes(N, K, B)


def sgq_gemv(qweight, sz, N, K, group, x, B, idx, count, y, y_f32, workspace, status=None,
             stream=None):
    _check("sgq_gemv", load().sgq_gemv(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), B, _ptr(idx), _ptr(count), _ptr(y),
        _ptr(y_f32), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_debug_gemv_withhold(qweight, sz, N, K, group, x, B, idx, count, y, y_f32, workspace,
                            status, stream=None):
    """Test hook: sgq_gemv (B = 9..16) whose last group run is never released,
    so the kernel's bounded waits run out and set SGQ_STATUS_TIMEOUT."""
    _check("sgq_debug_gemv_withhold", load().sgq_debug_gemv_withhold(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), B, _ptr(idx), _ptr(count), _ptr(y),
        _ptr(y_f32), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_gemv_thresh(qweight, sz, N, K, group, x, t, y, y_f32, workspace, status=None,
                    stream=None):
    _check("sgq_gemv_thresh", load().sgq_gemv_thresh(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), float(t), _ptr(y), _ptr(y_f32),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_gemv_thresh_batch(qweight, sz, N, K, group, x, B, t_host, y, y_f32, workspace,
                          status=None, stream=None):
    t = (ctypes.c_float * B)(*[float(v) for v in t_host])
    _check("sgq_gemv_thresh_batch", load().sgq_gemv_thresh_batch(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), B, t, _ptr(y), _ptr(y_f32),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_gemv_thresh_noalloc(qweight, sz, N, K, group, x, t, y, y_f32, status=None, stream=None):
    """sgq_gemv_thresh with the library's fixed scratch instead of a workspace
    (for callers that cannot allocate); N <= SGQ_NOALLOC_MAX_N."""
    _check("sgq_gemv_thresh_noalloc", load().sgq_gemv_thresh_noalloc(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), float(t), _ptr(y), _ptr(y_f32),
        _ptr(status), _stream(stream)))


def sgq_gemv_dense(qweight, sz, N, K, group, x, B, y, y_f32, workspace, status=None,
                   stream=None):
    _check("sgq_gemv_dense", load().sgq_gemv_dense(
        _ptr(qweight), _ptr(sz), N, K, group, _ptr(x), B, _ptr(y), _ptr(y_f32), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)))


def sgq_gemv_glu(qweight, sz, I, K, group, x, B, idx, count, act, h, h_f32, workspace,
                 status=None, stream=None):
    """Fused gate + up + act over the stacked [W_g; W_u] weights (packed with N = 2I)."""
    _check("sgq_gemv_glu", load().sgq_gemv_glu(
        _ptr(qweight), _ptr(sz), I, K, group, _ptr(x), B, _ptr(idx), _ptr(count), act, _ptr(h),
        _ptr(h_f32), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))


def sgq_gemv_glu_thresh(qweight, sz, I, K, group, x, t, act, h, h_f32, workspace, status=None,
                        stream=None):
    _check("sgq_gemv_glu_thresh", load().sgq_gemv_glu_thresh(
        _ptr(qweight), _ptr(sz), I, K, group, _ptr(x), float(t), act, _ptr(h), _ptr(h_f32),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_gemv_glu_thresh_batch(qweight, sz, I, K, group, x, B, t_host, act, h, h_f32, workspace,
                              status=None, stream=None):
    t = (ctypes.c_float * B)(*[float(v) for v in t_host])
    _check("sgq_gemv_glu_thresh_batch", load().sgq_gemv_glu_thresh_batch(
        _ptr(qweight), _ptr(sz), I, K, group, _ptr(x), B, t, act, _ptr(h), _ptr(h_f32),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_gemv_glu_dense(qweight, sz, I, K, group, x, B, act, h, h_f32, workspace, status=None,
                       stream=None):
    _check("sgq_gemv_glu_dense", load().sgq_gemv_glu_dense(
        _ptr(qweight), _ptr(sz), I, K, group, _ptr(x), B, act, _ptr(h), _ptr(h_f32),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))


def sgq_ffn_workspace_bytes(H: int, I: int) -> int:
    return load().sgq_ffn_workspace_bytes(H, I)


def sgq_ffn(qweight_gu, sz_gu, qweight_d, sz_d, H, I, group, x, t_in, act, t_h, y, y_f32,
            h_out, workspace, status=None, stream=None):
    """The batch-1 decode FFN in three kernels (gate/up GEMV, down GEMV with the
    GLU and the selection of h in its prologue, epilogue)."""
    _check("sgq_ffn", load().sgq_ffn(
        _ptr(qweight_gu), _ptr(sz_gu), _ptr(qweight_d), _ptr(sz_d), H, I, group, _ptr(x),
        float(t_in), act, float(t_h), _ptr(y), _ptr(y_f32), _ptr(h_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)))


def alloc_ffn_workspace(H, I, device="cuda"):
    return torch.zeros(sgq_ffn_workspace_bytes(H, I) // 4, dtype=torch.int32, device=device)


def sgq_glu(gate, up, h, B, I, act, stream=None):
    _check("sgq_glu", load().sgq_glu(_ptr(gate), _ptr(up), _ptr(h), B, I, act, _stream(stream)))


# --------------------------------------------------------------------------
# The step around the projections: cache plan and store, tree attention, norm.
# These wrappers check what the C ABI cannot see of a tensor: its element type,
# that it lies on the current device, that it is dense (rows: along a row), and
# that it holds what the sizes say is read or written.
# --------------------------------------------------------------------------

_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
_FLOATS = {torch.bfloat16: SGQ_TYPE_BF16, torch.float32: SGQ_TYPE_F32}
_OF_TYPE = (torch.bfloat16, torch.float32)  # by SGQ_TYPE_*
_CACHES = {torch.bfloat16: SGQ_TYPE_BF16, torch.float8_e4m3fn: SGQ_TYPE_E4M3}


def _dev(name, t, dtype, dev):
    """The address of a tensor of the type on device ``dev`` (None passes)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: element type {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected the current device, cuda:{dev}")
    return t.data_ptr()


def _dense(name, t, dtype, dev, need):
    """The address of a dense tensor of at least ``need`` elements (None passes)."""
    at = _dev(name, t, dtype, dev)
    if t is not None:
        if t.numel() < need:
            raise ValueError(f"{name}: {t.numel()} elements, expected {need} at least")
        if not t.is_contiguous():
            raise ValueError(f"{name}: strides {t.stride()} of {tuple(t.shape)} are not dense")
    return at


def _rows(name, t, dtype, dev, rows, ld, width):
    """The address of ``rows`` rows of ``width`` elements, ``ld`` apart, which may be a view of
    wider ones (None passes)."""
    at = _dev(name, t, dtype, dev)
    if t is None:
        return at
    need = (rows - 1) * ld + width
    if t.numel() >= need and t.is_contiguous():
        return at
    side = 1  # elements side by side so far, from the last dimension on
    for n, stride in zip(reversed(t.shape), reversed(t.stride())):
        if n > 1 and side < width and stride == side:
            side *= n
        elif n > 1:  # the rows
            if stride != ld and (side < width or rows > 1 and ld):
                raise ValueError(f"{name}: strides {t.stride()} of {tuple(t.shape)} are not those of dense rows, {ld} apart")
            break
    held = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if held < need:
        raise ValueError(f"{name}: {held} elements, expected {rows} rows of {width}, {ld} apart")
    return at


_fast = None


def _addresses(dev, names, tensors, types, sizes):
    """The addresses of several tensors, each as from _dense (its size is a number) or from
    _rows (rows, ld, width); by the module csrc/tensors.cpp in a tenth of the time, and here
    where something is wrong, to say what (or where that module has not been built)."""
    global _fast
    if _fast is None:
        try:
            from ._tensors import addresses as _fast
        except ImportError:
            _fast = lambda *a: None  # noqa: E731
    at = _fast(dev, tensors, types, sizes)
    if at is None:
        at = [_rows(name, t, dtype, dev, *n) if isinstance(n, tuple) else _dense(name, t, dtype, dev, n)
              for name, t, dtype, n in zip(names, tensors, types, sizes)]
    return at


def _float_type(name, t):
    """The C ABI's type of a bf16 or fp32 tensor."""
    if t.dtype not in _FLOATS:
        raise TypeError(f"{name}: element type {t.dtype}, expected bfloat16 or float32")
    return _FLOATS[t.dtype]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int),
                ("page", ctypes.c_int), ("num_pages", ctypes.c_int), ("heads", ctypes.c_int),
                ("dim", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("slot_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Cache:
    """The ``sgq_cache`` that describes a paged cache held in two tensors.

    ``k`` and ``v`` are [num_pages, page, heads, dim] in bf16 or float8_e4m3fn,
    contiguous along dim and with the same strides; any order of the other
    dimensions is taken from the strides (heads before slots:
    ``buf.transpose(1, 2)`` of a [num_pages, heads, page, dim] buffer). The
    tensors are kept alive by this object.
    """

    def __init__(self, k, v, k_scale=1.0, v_scale=1.0):
        if k.dim() != 4 or v.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("Cache: k and v must be [num_pages, page, heads, dim] alike")
        if k.dtype not in _CACHES:
            raise TypeError(f"Cache: element type {k.dtype}, expected bfloat16 or float8_e4m3fn")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("Cache: k and v must be contiguous along dim")
        if k.get_device() != v.get_device():
            raise ValueError("Cache: k and v must be on one device")
        # a dimension of one entry is never stepped over, whatever its stride says
        strides, other = (tuple(s if n > 1 else t.shape[3] for s, n in zip(t.stride(), t.shape)) for t in (k, v))
        if strides != other:
            raise ValueError("Cache: k and v must have the same strides")
        self.k, self.v = k, v
        self.device = k.get_device()
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), _CACHES[k.dtype], k.shape[1],
                                   k.shape[0], k.shape[2], k.shape[3], *strides[:3], float(k_scale),
                                   float(v_scale))
        self.ptr = ctypes.addressof(self.struct)

    def on(self, dev):
        if self.device != dev:
            raise ValueError(f"cache: on device {self.device}, expected the current device, cuda:{dev}")
        return self.ptr


_PLAN = ("lens", "news", "table", "held", "held_out", "free_pages", "free_count", "free_count_out", "depth", "cu_new",
         "slots", "pos", "req", "status")
_PLAN_TYPES = (_I32,) * 10 + (_I64,) + (_I32,) * 3


def sgq_cache_plan(lens, news, R, page, num_pages, table, table_ld, held, held_out, free_pages,
                   free_count, free_count_out, depth, max_tokens, cu_new, slots, pos, req,
                   status=None, stream=None):
    """Block tables, slots and positions of the requests' new tokens, on the GPU."""
    d = _current_device()
    # (of depth as many are read as there are new tokens, which the device alone knows)
    (lens, news, table, held, held_out, free_pages, free_count, free_count_out, depth, cu_new, slots, pos, req,
     status) = _addresses(
        d, _PLAN, (lens, news, table, held, held_out, free_pages, free_count, free_count_out, depth, cu_new, slots, pos,
                   req, status), _PLAN_TYPES,
        (R, R, (R, table_ld, table_ld), R, R, num_pages, 1, 1, 0, R + 1, max_tokens, max_tokens, max_tokens, 1))
    _check("sgq_cache_plan", load().sgq_cache_plan(
        lens, news, R, page, num_pages, table, table_ld, held, held_out, free_pages, free_count, free_count_out, depth,
        max_tokens, cu_new, slots, pos, req, status, _stream(stream, d)))


_WRITE = ("q", "k", "v", "n_tokens", "pos", "rope", "slots", "q_out", "status")
_WRITE_TYPES = (_BF16, _BF16, _BF16, _I32, _I32, _F32, _I64, _BF16, _I32)


def sgq_cache_write(q, ld_q, k, ld_k, v, ld_v, T, n_tokens, Hq, pos, rope, rope_len, slots,
                    q_out, ld_qo, cache, status=None, stream=None):
    """Rotate q and k by position; q to q_out, k and v into their slots of ``cache`` (a Cache)."""
    d = _current_device()
    dim = cache.struct.dim
    kv = cache.struct.heads * dim
    q, k, v, n_tokens, pos, rope, slots, q_out, status = _addresses(
        d, _WRITE, (q, k, v, n_tokens, pos, rope, slots, q_out, status), _WRITE_TYPES,
        ((T, ld_q, Hq * dim), (T, ld_k, kv), (T, ld_v, kv), 1, 0 if rope is None else T, rope_len * dim, T,
         (T, ld_qo, Hq * dim), 1))
    _check("sgq_cache_write", load().sgq_cache_write(
        q, ld_q, k, ld_k, v, ld_v, T, n_tokens, Hq, pos, rope, rope_len, slots, q_out, ld_qo, cache.on(d), status,
        _stream(stream, d)))


def sgq_tree_attn_workspace_bytes(T: int, R: int, Hq: int, Hkv: int, D: int) -> int:
    return load().sgq_tree_attn_workspace_bytes(T, R, Hq, Hkv, D)


def sgq_tree_attn(q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache, tree, tree_words,
                  scale, out, ld_out, lse, workspace, status=None, stream=None):
    """Attention of each request's new tokens over its pages of ``cache`` (a Cache)."""
    _tree_attn("sgq_tree_attn", q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache, tree,
               tree_words, scale, out, ld_out, lse, workspace, status, stream)


def sgq_debug_tree_attn_withhold(q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache, tree,
                                 tree_words, scale, out, ld_out, lse, workspace, status,
                                 stream=None):
    """Test hook: sgq_tree_attn whose scores are never passed on, so the
    kernel's bounded waits run out and set SGQ_STATUS_TIMEOUT."""
    _tree_attn("sgq_debug_tree_attn_withhold", q, ld_q, T, R, Hq, lens, cu_new, table, table_ld,
               cache, tree, tree_words, scale, out, ld_out, lse, workspace, status, stream)


_ATTN = ("q", "lens", "cu_new", "table", "tree", "out", "lse", "workspace", "status")
_ATTN_TYPES = (_BF16, _I32, _I32, _I32, _I32, _BF16, _F32, _I32, _I32)
_ATTN_TYPES_U32 = (_BF16, _I32, _I32, _I32, torch.uint32, _BF16, _F32, _I32, _I32)


def _tree_attn(name, q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache, tree, tree_words,
               scale, out, ld_out, lse, workspace, status, stream):
    d = _current_device()
    width, ws_bytes = Hq * cache.struct.dim, 0 if workspace is None else workspace.nbytes
    q, lens, cu_new, table, tree, out, lse, workspace, status = _addresses(
        d, _ATTN, (q, lens, cu_new, table, tree, out, lse, workspace, status),
        _ATTN_TYPES_U32 if tree is not None and tree.dtype is torch.uint32 else _ATTN_TYPES,
        ((T, ld_q, width), R, R + 1, (R, table_ld, table_ld), (T, tree_words, tree_words), (T, ld_out, width), T * Hq, 0, 1))
    _check(name, getattr(load(), name)(
        q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache.on(d), tree, tree_words, scale, out, ld_out, lse, workspace,
        ws_bytes, status, _stream(stream, d)))


_NORM = ("a", "w_post", "gate", "resid", "resid_out", "w_pre", "x")


def sgq_residual_norm(a, ld_a, w_post, gate, ld_gate, scale, resid, ld_r, resid_out, ld_ro,
                      w_pre, w_offset, x, ld_x, B, H, eps, stream=None):
    """The norms around a block with its gate and scaled residual; the element
    types of the C entry point (a_type, r_type, w_type) are the tensors' own."""
    d = _current_device()
    w = w_pre if w_pre is not None else w_post if w_post is not None else gate
    at = SGQ_TYPE_F32 if a is None else _float_type("a", a)
    rt = SGQ_TYPE_F32 if resid is None else _float_type("resid", resid)
    wt = SGQ_TYPE_F32 if w is None else _float_type("w_pre, w_post and gate", w)
    r, ws = _OF_TYPE[rt], _OF_TYPE[wt]
    a, w_post, gate, resid, resid_out, w_pre, x = _addresses(
        d, _NORM, (a, w_post, gate, resid, resid_out, w_pre, x), (_OF_TYPE[at], ws, ws, r, r, ws, _BF16),
        ((B, ld_a, H), H, (B, ld_gate, H), (B, ld_r, H), (B, ld_ro, H), H, (B, ld_x, H)))
    _check("sgq_residual_norm", load().sgq_residual_norm(
        a, ld_a, at, w_post, gate, ld_gate, scale, resid, ld_r, rt, resid_out, ld_ro, w_pre, wt, w_offset, x, ld_x, B, H,
        eps, _stream(stream, d)))


# --------------------------------------------------------------------------
# Allocation helpers (torch device memory; plumbing only).
# --------------------------------------------------------------------------

def alloc_packed(N, K, group, device="cuda"):
    qb, sb = sgq_packed_sizes(N, K, group)
    return (torch.empty(qb, dtype=torch.uint8, device=device),
            torch.empty(sb // 4, dtype=torch.int32, device=device))


def alloc_workspace(N, K, B, device="cuda"):
    nbytes = sgq_gemv_workspace_bytes(N, K, B)
    return torch.zeros(nbytes // 4, dtype=torch.int32, device=device)


def alloc_packed_nm(N, K, group, device="cuda"):
    """(qweight u8, keep u8, sz int32) buffers of the 2:4 layout."""
    qb, kb, sb = sgq_packed_sizes_nm(N, K, group)
    return (torch.empty(qb, dtype=torch.uint8, device=device),
            torch.empty(kb, dtype=torch.uint8, device=device),
            torch.empty(sb // 4, dtype=torch.int32, device=device))


def alloc_mask(K, device="cuda"):
    """uint32 words for a K-channel bitmask (int32 tensor; bits are what matter)."""
    return torch.zeros((K + 31) // 32, dtype=torch.int32, device=device)


def alloc_select(K, device="cuda"):
    return (torch.empty(K, dtype=torch.int32, device=device),
            torch.zeros(1, dtype=torch.int32, device=device))


def alloc_tree_attn_workspace(T, R, Hq, Hkv, D, device="cuda"):
    return torch.empty(sgq_tree_attn_workspace_bytes(T, R, Hq, Hkv, D) // 4, dtype=torch.int32,
                       device=device)
