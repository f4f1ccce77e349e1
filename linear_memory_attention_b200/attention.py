"""ctypes binding of liblard_attn (the C ABI declared in include/lard_attn.h):
cross attention and attention over a shared prefix.

Argument marshalling only, as in ``lard``: every step of the computation runs in the
library's kernels, and importing this module fails loudly if the library has not been
built.  Functions with the C names take the caller's buffers:
    lard_cross_attn_fwd(q, k, v, tau, out, lse, k_len=None, workspace=None, stream=None,
                        rest=None)
    lard_cross_attn_bwd(q, k, v, tau, out, lse, dout, dq, dk, dv, k_len=None,
                        workspace=None, stream=None, rest=None)
    lard_prefix_attn(q, kp, vp, ks, vs, s_len, tau, out, lse, workspace=None, stream=None)
    lard_cross_attn_fwd_workspace_bytes(q, k), lard_cross_attn_bwd_workspace_bytes(q, k),
    lard_prefix_attn_workspace_bytes(q, kp, ks) -> bytes
    lard_attn_device_status(stream=None) -> fault bits (raises on timeout)
and two that allocate what they return (and the workspace):
    cross_attention(q, k, v, tau, k_len=None, dout=None, stream=None)
    prefix_attention(q, kp, vp, ks, vs, s_len, tau, stream=None)
stream is a torch stream or a raw handle of the inputs' GPU; None: its current one.
Tensors are torch tensors on one GPU, bf16 or fp32, [B, H, rows, d] by shape; in memory
any batch, head and row strides that are multiples of 16 bytes, the last dimension
contiguous (so x.transpose(1, 2) of a [B, rows, H, d] tensor is taken as it is).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from .lard import LARD_DTYPE_BF16, LARD_DTYPE_FP32, LARD_OK, LardError, _gpu_of

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblard_attn.so")

EXPORTS = ("lard_cross_attn_fwd_workspace_bytes", "lard_cross_attn_bwd_workspace_bytes",
           "lard_cross_attn_fwd", "lard_cross_attn_bwd", "lard_prefix_attn_workspace_bytes",
           "lard_prefix_attn", "lard_attn_device_status")

# struct lard_cross_attn and lard_prefix_attn_args, packed in one go: seven ints and a
# float, then 8-byte fields (a view is a pointer and three strides).
_CROSS = struct.Struct("7if" + "4q" * 3 + "q" + "4q" + "q" + "4q" * 5)
_PREFIX = struct.Struct("8if4x" + "4q" * 5 + "q" + "4q" + "q")
_NO_VIEW = (0, 0, 0, 0)
_NO_GRADS = _NO_VIEW * 4


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"liblard_attn.so is not built ({LIB_PATH}); build it with "
            "`python -m linear_memory_attention_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    vp = ctypes.c_void_p
    for name in EXPORTS:
        f = getattr(lib, name)
        if name.endswith("_workspace_bytes"):
            f.restype, f.argtypes = ctypes.c_size_t, [vp]
        elif name == "lard_attn_device_status":
            f.restype, f.argtypes = ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_uint)]
        else:
            f.restype, f.argtypes = ctypes.c_int, [vp, vp, ctypes.c_size_t, vp]
    return lib


_lib = _load()


def _current_stream(device: int) -> int:
    if device < 0:
        raise ValueError("tensors must be on a GPU")
    return _raw_stream(device)


# torch.cuda.current_stream builds a Stream object, which costs more than the C call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return LARD_DTYPE_BF16
    if t.dtype == torch.float32:
        return LARD_DTYPE_FP32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _refuse(t, shape, dtype, q, name):
    """The reason why t is not such a tensor."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != q.device:
        raise ValueError(f"{name}: on {t.device}, q on {q.device}")
    raise ValueError(f"{name}: must be contiguous (its last dimension, where views are taken)")


def _view(t, shape, q, name):
    """The fields of a lard_attn_view of t [B, H, rows, d], which must have this shape and q's
    dtype and device."""
    if t.shape != shape or t.dtype is not q.dtype or t.get_device() != q.get_device():
        _refuse(t, shape, q.dtype, q, name)
    batch, head, row, one = t.stride()
    if one != 1:
        _refuse(t, shape, q.dtype, q, name)
    return t.data_ptr(), batch, head, row


def _shared(t, shape, q, name):
    """The fields of a lard_attn_view of t [H, rows, d], one block for all sequences."""
    if t.shape != shape or t.dtype is not q.dtype or t.get_device() != q.get_device():
        _refuse(t, shape, q.dtype, q, name)
    head, row, one = t.stride()
    if one != 1:
        _refuse(t, shape, q.dtype, q, name)
    return t.data_ptr(), 0, head, row


def _flat(t, shape, dtype, q, name):
    """The address of a contiguous tensor of this shape and dtype on q's device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != q.get_device() or not t.is_contiguous():
        _refuse(t, shape, dtype, q, name)
    return t.data_ptr()


def _workspace(ws, need, q):
    """(address, bytes) of the workspace to pass."""
    if ws is None:
        if need:
            raise ValueError(f"workspace: {need} bytes needed")
        return None, 0
    if ws.device != q.device or not ws.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the inputs' device")
    size = ws.numel() * ws.element_size()
    if size < need:
        raise ValueError(f"workspace: {size} bytes, {need} needed")
    return ws.data_ptr(), size


def _handle(stream, q):
    """The CUDA stream to enqueue on: the given one, or the current one of q's GPU."""
    if stream is None:
        return _current_stream(q.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(fn, name, args, ws, need, q, stream):
    at, size = _workspace(ws, need, q)
    st = fn(args, at, size, _handle(stream, q))
    if st != LARD_OK:
        raise LardError(st, name)


def _cross_sizes(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be [B, H, rows, d]")
    B, Hq, n, d = q.shape
    _, Hkv, m, _ = k.shape
    return _dtype(q), B, Hq, Hkv, n, m, d


def _cross_bytes(fn, sizes):
    return fn(_CROSS.pack(*sizes, 1.0, *_NO_VIEW * 3, 0, *_NO_VIEW, 0, *_NO_GRADS, *_NO_VIEW))


def lard_cross_attn_fwd_workspace_bytes(q, k) -> int:
    """Bytes of workspace lard_cross_attn_fwd needs for queries q over keys k."""
    return _cross_bytes(_lib.lard_cross_attn_fwd_workspace_bytes, _cross_sizes(q, k))


def lard_cross_attn_bwd_workspace_bytes(q, k) -> int:
    """Bytes of workspace lard_cross_attn_bwd needs for queries q over keys k."""
    return _cross_bytes(_lib.lard_cross_attn_bwd_workspace_bytes, _cross_sizes(q, k))


def _cross_args(q, k, v, tau, k_len, out, lse, grads=None, rest=None):
    sizes = _cross_sizes(q, k)
    _, B, Hq, Hkv, n, m, d = sizes
    qs, ks = (B, Hq, n, d), (B, Hkv, m, d)
    grad_views = _NO_GRADS
    if grads is not None:
        dout, dq, dk, dv = grads
        grad_views = (*_view(dout, qs, q, "dout"), *_view(dq, qs, q, "dq"), *_view(dk, ks, q, "dk"),
                      *_view(dv, ks, q, "dv"))
    return _CROSS.pack(*sizes, tau, *_view(q, qs, q, "q"), *_view(k, ks, q, "k"), *_view(v, ks, q, "v"),
                       0 if k_len is None else _flat(k_len, (B,), torch.int32, q, "k_len"),
                       *_view(out, qs, q, "out"), _flat(lse, (B, Hq, n), torch.float32, q, "lse"), *grad_views,
                       *(_NO_VIEW if rest is None else _view(rest, qs, q, "rest")))


def lard_cross_attn_fwd(q, k, v, tau, out, lse, k_len=None, workspace=None, stream=None, rest=None):
    """Cross attention: writes out [B, Hq, n, d] and lse [B, Hq, n] (fp32) of queries q
    [B, Hq, n, d] over k, v [B, Hkv, m, d], of which sequence b has k_len[b] rows (int32).  rest (bf16, like out):
    takes what rounding left of out, for the backward pass."""
    args = _cross_args(q, k, v, tau, k_len, out, lse, None, rest)
    need = _lib.lard_cross_attn_fwd_workspace_bytes(args)
    _call(_lib.lard_cross_attn_fwd, "lard_cross_attn_fwd", args, workspace, need, q, stream)


def lard_cross_attn_bwd(q, k, v, tau, out, lse, dout, dq, dk, dv, k_len=None, workspace=None, stream=None,
                        rest=None):
    """Gradients of cross attention: writes dq, dk and dv for the upstream gradient dout, given
    out, lse and (where it was taken) rest of lard_cross_attn_fwd on the same inputs."""
    args = _cross_args(q, k, v, tau, k_len, out, lse, (dout, dq, dk, dv), rest)
    need = _lib.lard_cross_attn_bwd_workspace_bytes(args)
    _call(_lib.lard_cross_attn_bwd, "lard_cross_attn_bwd", args, workspace, need, q, stream)


def _prefix_sizes(q, kp, ks):
    if q.dim() != 4 or (kp is not None and kp.dim() != 3) or (ks is not None and ks.dim() != 4):
        raise ValueError("q, ks and vs must be [B, H, rows, d], kp and vp [H, rows, d]")
    if kp is None and ks is None:
        raise ValueError("a shared prefix (kp, vp), rows of each sequence's own (ks, vs), or both")
    B, Hq, n, d = q.shape
    return (_dtype(q), B, Hq, kp.shape[0] if ks is None else ks.shape[1], n, 0 if kp is None else kp.shape[1],
            0 if ks is None else ks.shape[2], d)


def lard_prefix_attn_workspace_bytes(q, kp, ks) -> int:
    """Bytes of workspace lard_prefix_attn needs for these shapes."""
    return _lib.lard_prefix_attn_workspace_bytes(
        _PREFIX.pack(*_prefix_sizes(q, kp, ks), 1.0, *_NO_VIEW * 5, 0, *_NO_VIEW, 0))


def _prefix_args(q, kp, vp, ks, vs, s_len, tau, out, lse):
    if (kp is None) != (vp is None) or (ks is None) != (vs is None):
        raise ValueError("keys and values are given together")
    if (vp is not None and vp.dim() != 3) or (vs is not None and vs.dim() != 4):
        raise ValueError("vp must be [H, rows, d], vs [B, H, rows, d]")
    sizes = _prefix_sizes(q, kp, ks)
    _, B, Hq, Hkv, n, P, S, d = sizes
    views = _NO_VIEW * 2 if kp is None else (*_shared(kp, (Hkv, P, d), q, "kp"), *_shared(vp, (Hkv, P, d), q, "vp"))
    own = _NO_VIEW * 2 if ks is None else (*_view(ks, (B, Hkv, S, d), q, "ks"), *_view(vs, (B, Hkv, S, d), q, "vs"))
    return _PREFIX.pack(*sizes, tau, *_view(q, q.shape, q, "q"), *views, *own,
                        0 if s_len is None else _flat(s_len, (B,), torch.int32, q, "s_len"),
                        *_view(out, q.shape, q, "out"), _flat(lse, (B, Hq, n), torch.float32, q, "lse"))


def lard_prefix_attn(q, kp, vp, ks, vs, s_len, tau, out, lse, workspace=None, stream=None):
    """Attention of the n newest rows q [B, Hq, n, d] of B sequences over the rows that all share
    (kp, vp [Hkv, P, d], or None) and their own (ks, vs [B, Hkv, S, d], or None), of which sequence
    b has s_len[b] (int32; None: all S), the newest among them: writes out and lse."""
    args = _prefix_args(q, kp, vp, ks, vs, s_len, tau, out, lse)
    need = _lib.lard_prefix_attn_workspace_bytes(args)
    _call(_lib.lard_prefix_attn, "lard_prefix_attn", args, workspace, need, q, stream)


def _on(stream, q):
    """A context in which what is allocated on q's GPU belongs to the given stream.  A raw handle
    is one of q's GPU, which need not be the current one."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=q.device)
    return torch.cuda.stream(stream)


def _bytes(need, q):
    return torch.empty_strided((need,), (1,), device=q.device, dtype=torch.uint8) if need else None


def _outputs(q):
    """out in q's layout, lse [B, Hq, n]."""
    B, Hq, n, _ = q.shape
    return torch.empty_like(q), torch.empty_strided((B, Hq, n), (Hq * n, n, 1), device=q.device, dtype=torch.float32)


def cross_attention(q, k, v, tau, k_len=None, dout=None, stream=None):
    """Allocate the outputs and run cross attention, and its gradients if dout is given.

    Returns a dict with out (q's dtype and layout), lse [B, Hq, n] and, with dout, dq, dk, dv.
    """
    if stream is not None:
        with _on(stream, q):
            return _cross_attention(q, k, v, tau, k_len, dout, stream)
    return _cross_attention(q, k, v, tau, k_len, dout, None)


def _cross_attention(q, k, v, tau, k_len, dout, stream):
    if q.dim() != 4:
        raise ValueError("q must be [B, H, rows, d]")
    out, lse = _outputs(q)
    grads = None if dout is None else (dout, torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    rest = torch.empty_like(q) if grads is not None and q.dtype is torch.bfloat16 else None
    args = _cross_args(q, k, v, tau, k_len, out, lse, grads, rest)
    need = _lib.lard_cross_attn_fwd_workspace_bytes(args)
    _call(_lib.lard_cross_attn_fwd, "lard_cross_attn_fwd", args, _bytes(need, q), need, q, stream)
    got = {"out": out, "lse": lse}
    if grads is not None:
        need = _lib.lard_cross_attn_bwd_workspace_bytes(args)
        _call(_lib.lard_cross_attn_bwd, "lard_cross_attn_bwd", args, _bytes(need, q), need, q, stream)
        got["dq"], got["dk"], got["dv"] = grads[1:]
    return got


def prefix_attention(q, kp, vp, ks, vs, s_len, tau, stream=None):
    """Allocate the outputs and run lard_prefix_attn: returns a dict with out and lse."""
    if stream is not None:
        with _on(stream, q):
            return _prefix_attention(q, kp, vp, ks, vs, s_len, tau, stream)
    return _prefix_attention(q, kp, vp, ks, vs, s_len, tau, None)


def _prefix_attention(q, kp, vp, ks, vs, s_len, tau, stream):
    if q.dim() != 4:
        raise ValueError("q must be [B, H, rows, d]")
    out, lse = _outputs(q)
    args = _prefix_args(q, kp, vp, ks, vs, s_len, tau, out, lse)
    need = _lib.lard_prefix_attn_workspace_bytes(args)
    _call(_lib.lard_prefix_attn, "lard_prefix_attn", args, _bytes(need, q), need, q, stream)
    return {"out": out, "lse": lse}


def lard_attn_device_status(stream=None) -> int:
    """Synchronise the stream and check the kernels' fault word on its GPU; raises on a
    timed-out wait."""
    bits = ctypes.c_uint(0)
    with _gpu_of(stream):
        handle = torch.cuda.current_stream().cuda_stream if stream is None else _handle(stream, None)
        st = _lib.lard_attn_device_status(handle, ctypes.byref(bits))
    if st != LARD_OK:
        err = LardError(st, f"lard_attn_device_status (fault bits 0x{bits.value:x})")
        err.fault_bits = bits.value
        raise err
    return bits.value
