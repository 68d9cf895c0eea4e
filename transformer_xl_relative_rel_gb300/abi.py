"""ctypes binding of libtxl (the C ABI in include/txl.h).

Argument marshalling only: the functions take torch tensors that already live
on the GPU, check their shapes, dtypes and layouts, and pass raw device
pointers and sizes to the library.  Every step of the computation runs in the
library's CUDA kernels; there is no CPU path.  If ``libtxl.so`` is missing the
first call raises ``TxlError``.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

TXL_F32 = 0
TXL_BF16 = 1

_STATUS = {0: "TXL_OK", 1: "TXL_ERR_INVALID", 2: "TXL_ERR_UNSUPPORTED", 3: "TXL_ERR_CUDA",
           4: "TXL_ERR_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libtxl.so"
_lib: Optional[ctypes.CDLL] = None

#: every symbol include/txl.h declares (checked by the host-side tests)
EXPORTS = ("txl_rel_attn_fwd", "txl_mem_update", "txl_check", "txl_status_string",
           "txl_last_cuda_error", "txl_version", "txl_shutdown", "txl_rel_attn_fwd_noalloc",
           "txl_rel_attn_fwd_ring", "txl_ring_append", "txl_rel_attn_fwd_padded", "txl_project_heads",
           "txl_project_qkv", "txl_project_qkv_cells", "txl_rel_table", "txl_rel_attn_bwd", "txl_rel_attn_bwd_workspace", "txl_rel_attn_fwd_lse", "txl_rel_attn_fwd_mem", "txl_rel_attn_fwd_mem_cells", "txl_rel_attn_fwd_plan", "txl_selftest_wait",
           "txl_softmax_xent_workspace", "txl_softmax_xent_fwd", "txl_softmax_xent_bwd",
           "txl_distill_workspace", "txl_distill_fwd", "txl_distill_bwd",
           "txl_embed_fwd", "txl_embed_bwd_workspace", "txl_embed_bwd",
           "txl_layer_norm_fwd", "txl_layer_norm_bwd_workspace", "txl_layer_norm_bwd",
           "txl_grad_norm_workspace", "txl_grad_norm", "txl_adamw_step")


class _AdamwTensor(ctypes.Structure):
    """txl_adamw_tensor"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("param", "master", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                                "exp_avg_sq_scale")] +
                [("size", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("param_dtype", ctypes.c_int),
                 ("grad_dtype", ctypes.c_int)])


# an _AdamwTensor's fields, without the padding behind them: packed at once, in
# half the time that assigning them takes
_ADAMW_FIELDS = struct.Struct("@7Pqfii")


class _AdamwOptions(ctypes.Structure):
    """txl_adamw_options"""
    _fields_ = [("lr", ctypes.c_float), ("eps", ctypes.c_float), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("step", ctypes.c_int64), ("lr_device", ctypes.c_void_p), ("step_device", ctypes.c_void_p),
                ("grad_scale", ctypes.c_void_p), ("seed", ctypes.c_uint64)]


class TxlError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS.get(status, status)}")


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load_library() -> ctypes.CDLL:
    """Load libtxl.so from the package directory (built by ``_build.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise TxlError(3, f"{path} not built (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.txl_rel_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp]
    lib.txl_rel_attn_fwd.restype = i
    lib.txl_rel_attn_fwd_lse.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp]
    lib.txl_rel_attn_fwd_lse.restype = i
    ip = ctypes.POINTER(ctypes.c_int)
    lib.txl_rel_attn_fwd_plan.argtypes = [i, i, i, i, i, i, ip, ip]
    lib.txl_rel_attn_fwd_plan.restype = i
    lib.txl_rel_attn_fwd_mem.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, i, vp]
    lib.txl_rel_attn_fwd_mem.restype = i
    pp = ctypes.POINTER(vp)
    lib.txl_rel_attn_fwd_mem_cells.argtypes = [i, pp, pp, pp, pp, pp, pp, i, i, i, i, i, i, pp, pp, pp, i, vp]
    lib.txl_rel_attn_fwd_mem_cells.restype = i
    lib.txl_rel_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp]
    lib.txl_rel_attn_fwd_noalloc.restype = i
    lib.txl_rel_attn_fwd_ring.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp]
    lib.txl_rel_attn_fwd_ring.restype = i
    lib.txl_ring_append.argtypes = [vp, vp, i, i, i, i, i, vp]
    lib.txl_ring_append.restype = i
    lib.txl_rel_attn_fwd_padded.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp]
    lib.txl_rel_attn_fwd_padded.restype = i
    lib.txl_project_heads.argtypes = [vp, vp, vp, i, i, i, i, i, i, vp]
    lib.txl_project_heads.restype = i
    lib.txl_project_qkv.argtypes = [vp, i, i, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.txl_project_qkv.restype = i
    pp = ctypes.POINTER(ctypes.c_void_p)
    lib.txl_project_qkv_cells.argtypes = [i, pp, pp, pp, pp, pp, pp, pp, i, i, i, i, i, i, i, vp]
    lib.txl_project_qkv_cells.restype = i
    lib.txl_rel_table.argtypes = [vp, vp, i, i, i, i, i, i, vp]
    lib.txl_rel_table.restype = i
    lib.txl_rel_attn_bwd_workspace.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
    lib.txl_rel_attn_bwd_workspace.restype = i
    lib.txl_rel_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                     vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.txl_rel_attn_bwd.restype = i
    sz, f = ctypes.c_size_t, ctypes.c_float
    lib.txl_softmax_xent_workspace.argtypes = [i, i, i, i, i, ctypes.POINTER(sz)]
    lib.txl_softmax_xent_workspace.restype = i
    lib.txl_softmax_xent_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, vp, vp, sz, vp]
    lib.txl_softmax_xent_fwd.restype = i
    lib.txl_softmax_xent_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, vp, vp, vp, vp, sz, vp]
    lib.txl_softmax_xent_bwd.restype = i
    lib.txl_distill_workspace.argtypes = [i, i, i, i, i, i, ctypes.POINTER(sz)]
    lib.txl_distill_workspace.restype = i
    lib.txl_distill_fwd.argtypes = [vp, vp, vp, vp, vp, i, f, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.txl_distill_fwd.restype = i
    lib.txl_distill_bwd.argtypes = [vp, vp, vp, vp, vp, i, f, vp, vp, i, i, i, i, i, vp, vp, vp, vp, sz, vp]
    lib.txl_distill_bwd.restype = i
    szp, tp = ctypes.POINTER(sz), ctypes.POINTER(_AdamwTensor)
    lib.txl_embed_fwd.argtypes = [vp, vp, f, i, i, i, i, vp, vp]
    lib.txl_embed_bwd_workspace.argtypes = [i, i, i, i, szp]
    lib.txl_embed_bwd.argtypes = [vp, vp, f, i, i, i, i, i, vp, vp, sz, vp]
    lib.txl_layer_norm_fwd.argtypes = [vp, vp, vp, vp, f, i, i, i, vp, vp, vp, vp, vp]
    lib.txl_layer_norm_bwd_workspace.argtypes = [i, i, i, szp]
    lib.txl_layer_norm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, vp, vp, vp, vp, sz, vp]
    lib.txl_grad_norm_workspace.argtypes = [i, tp, szp]
    lib.txl_grad_norm.argtypes = [i, tp, f, vp, vp, vp, sz, vp]
    lib.txl_adamw_step.argtypes = [i, tp, ctypes.POINTER(_AdamwOptions), vp]
    for name in ("txl_embed_fwd", "txl_embed_bwd_workspace", "txl_embed_bwd", "txl_layer_norm_fwd",
                 "txl_layer_norm_bwd_workspace", "txl_layer_norm_bwd", "txl_grad_norm_workspace", "txl_grad_norm",
                 "txl_adamw_step"):
        getattr(lib, name).restype = i
    lib.txl_mem_update.argtypes = [vp, vp, i, i, i, i, i, vp]
    lib.txl_mem_update.restype = i
    lib.txl_selftest_wait.argtypes = [ctypes.c_uint, vp]
    lib.txl_selftest_wait.restype = i
    lib.txl_check.argtypes = [vp]
    lib.txl_check.restype = i
    lib.txl_status_string.argtypes = [i]
    lib.txl_status_string.restype = ctypes.c_char_p
    lib.txl_last_cuda_error.argtypes = []
    lib.txl_last_cuda_error.restype = i
    lib.txl_version.argtypes = []
    lib.txl_version.restype = i
    lib.txl_shutdown.argtypes = []
    lib.txl_shutdown.restype = None
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().txl_status_string(int(status)).decode()


def _raise(st: int, what: str):
    if st != 0:
        lib = load_library()
        msg = f"{what} ({lib.txl_status_string(st).decode()}"
        if st == 3:
            msg += f", cuda error {lib.txl_last_cuda_error()}"
        raise TxlError(st, msg + ")")


def _stream_ptr(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return TXL_F32
    if t.dtype == torch.bfloat16:
        return TXL_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t) -> Optional[int]:
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _check_attn(q, k, v, r, u_bias, v_bias, mem_len, out):
    import torch
    L, B, H, D = q.shape
    T = mem_len + L
    for name, t, shp in (("k", k, (T, B, H, D)), ("v", v, (T, B, H, D)), ("r", r, (T, H, D))):
        if tuple(t.shape) != shp:
            raise ValueError(f"{name} must be {list(shp)}, got {list(t.shape)}")
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    for name, t in (("u_bias", u_bias), ("v_bias", v_bias)):
        if t is not None and (tuple(t.shape) != (H, D) or t.dtype != torch.float32):
            raise ValueError(f"{name} must be float32 [{H}, {D}] or None")
    if out is not None and (tuple(out.shape) != (L, B, H, D) or out.dtype != q.dtype):
        raise ValueError("out must be a contiguous tensor shaped and typed like q")
    for t in (q, k, v, r, u_bias, v_bias, out):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if out is None:
        out = torch.empty_like(q)
    return out


def rel_attn_fwd(q, k, v, r, u_bias, v_bias, mem_len: int, out=None, stream=None, lse=None):
    """Relative attention of one layer (Transformer-XL Section 3.3).

    q: [L, B, H, D]; k, v: [M+L, B, H, D]; r: [M+L, H, D] (reversed table);
    u_bias, v_bias: [H, D] float32, or None to drop that bias term (both
    None: Shaw et al.'s form, terms (a) + (b) only); all CUDA, contiguous,
    same dtype (float32 or bfloat16) except the biases.  Returns ``out``
    [L, B, H, D].  ``lse`` (bfloat16 inputs only): a contiguous float32 CUDA
    tensor [B, H, L] that receives each query row's log-sum-exp of its
    scaled scores (txl_rel_attn_fwd_lse), to hand to ``rel_attn_bwd``.
    """
    import torch
    L, B, H, D = q.shape
    out = _check_attn(q, k, v, r, u_bias, v_bias, mem_len, out)
    if lse is None:
        st = load_library().txl_rel_attn_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias),
            B, mem_len, L, H, D, _dtype_code(q), _ptr(out), _stream_ptr(stream))
        _raise(st, "txl_rel_attn_fwd")
        return out
    if tuple(lse.shape) != (B, H, L) or lse.dtype != torch.float32 or not lse.is_cuda \
            or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 CUDA tensor [{B}, {H}, {L}]")
    st = load_library().txl_rel_attn_fwd_lse(
        _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias),
        B, mem_len, L, H, D, _dtype_code(q), _ptr(out), _ptr(lse), _stream_ptr(stream))
    _raise(st, "txl_rel_attn_fwd_lse")
    return out


def rel_attn_fwd_plan(batch: int, mem_len: int, seg_len: int, heads: int, d_head: int,
                      dtype_code: int) -> tuple:
    """(key splits, kernel launches) of a txl_rel_attn_fwd call of this shape."""
    sp, nl = ctypes.c_int(0), ctypes.c_int(0)
    st = load_library().txl_rel_attn_fwd_plan(batch, mem_len, seg_len, heads, d_head, dtype_code,
                                              ctypes.byref(sp), ctypes.byref(nl))
    _raise(st, "txl_rel_attn_fwd_plan")
    return int(sp.value), int(nl.value)


def rel_attn_fwd_mem(q, k, v, r, u_bias, v_bias, mem_len: int, mem_next, ext_ctx, out=None, stream=None):
    """``rel_attn_fwd`` and ``mem_update`` of one layer in one call
    (txl_rel_attn_fwd_mem): returns ``out``; ``mem_next`` receives the newest
    ``mem_len`` rows of ``ext_ctx`` [M+L, B, d_model] (same dtype as q)."""
    L, B, H, D = q.shape
    out = _check_attn(q, k, v, r, u_bias, v_bias, mem_len, out)
    if ext_ctx.dim() != 3 or ext_ctx.shape[0] != mem_len + L or ext_ctx.shape[1] != B:
        raise ValueError(f"ext_ctx must be [{mem_len + L}, {B}, d_model]")
    dm = ext_ctx.shape[2]
    for name, t in (("ext_ctx", ext_ctx), ("mem_next", mem_next)):
        if t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor typed like q")
    if mem_next.numel() < mem_len * B * dm:
        raise ValueError(f"mem_next must hold at least [{mem_len}, {B}, {dm}]")
    st = load_library().txl_rel_attn_fwd_mem(
        _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias),
        B, mem_len, L, H, D, _dtype_code(q), _ptr(out), _ptr(mem_next), _ptr(ext_ctx), dm, _stream_ptr(stream))
    _raise(st, "txl_rel_attn_fwd_mem")
    return out


def rel_attn_fwd_mem_cells(qs, ks, vs, rs, us, ws, mem_len: int, mem_nexts, ext_ctxs, outs=None, stream=None):
    """Several independent ``rel_attn_fwd_mem`` calls of one shape
    (txl_rel_attn_fwd_mem_cells): lists of equal length, call c taking
    qs[c] .. ext_ctxs[c] (``us``/``ws`` may be None, or hold None entries).
    Returns the list of outputs."""
    n = len(qs)
    lists = [ks, vs, rs, mem_nexts, ext_ctxs] + [x for x in (us, ws, outs) if x is not None]
    if any(len(x) != n for x in lists):
        raise ValueError("the calls' lists must have the same length")
    if n == 0:
        return []
    L, B, H, D = qs[0].shape
    dm = ext_ctxs[0].shape[2] if ext_ctxs[0].dim() == 3 else -1
    for c in range(n):
        if tuple(qs[c].shape) != (L, B, H, D) or qs[c].dtype != qs[0].dtype:
            raise ValueError("every call's q must have the first call's shape and dtype")
        if tuple(ext_ctxs[c].shape) != (mem_len + L, B, dm):
            raise ValueError(f"ext_ctx must be [{mem_len + L}, {B}, {dm}] in every call")
    res = []
    for c in range(n):
        u = None if us is None else us[c]
        w = None if ws is None else ws[c]
        out = _check_attn(qs[c], ks[c], vs[c], rs[c], u, w, mem_len, None if outs is None else outs[c])
        ext, nxt = ext_ctxs[c], mem_nexts[c]
        for name, t in (("ext_ctx", ext), ("mem_next", nxt)):
            if t.dtype != qs[0].dtype or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor typed like q")
        if nxt.numel() < mem_len * B * dm:
            raise ValueError(f"mem_next must hold at least [{mem_len}, {B}, {dm}]")
        res.append(out)
    arr = lambda ts: (ctypes.c_void_p * n)(*[_ptr(t) for t in ts])
    st = load_library().txl_rel_attn_fwd_mem_cells(
        n, arr(qs), arr(ks), arr(vs), arr(rs), None if us is None else arr(us), None if ws is None else arr(ws),
        B, mem_len, L, H, D, _dtype_code(qs[0]), arr(res), arr(mem_nexts), arr(ext_ctxs), dm, _stream_ptr(stream))
    _raise(st, "txl_rel_attn_fwd_mem_cells")
    return res


def rel_attn_bwd_workspace_bytes(batch: int, mem_len: int, seg_len: int, heads: int, d_head: int,
                                 dtype_code: int) -> int:
    """Workspace bytes txl_rel_attn_bwd needs for this shape."""
    n = ctypes.c_size_t(0)
    st = load_library().txl_rel_attn_bwd_workspace(batch, mem_len, seg_len, heads, d_head, dtype_code,
                                                   ctypes.byref(n))
    _raise(st, "txl_rel_attn_bwd_workspace")
    return int(n.value)


def rel_attn_bwd(q, k, v, r, u_bias, v_bias, dout, mem_len: int, workspace=None, grads=None,
                 bias_grads: bool = True, stream=None, out=None, lse=None):
    """Gradients of ``rel_attn_fwd`` for the output gradient ``dout`` (shaped
    like q).  Returns a dict ``dq, dk, dv, dr`` (shaped and typed like q, k,
    v, r) and ``du, dw`` (float32 [H, D]; None when ``bias_grads`` is False).
    ``workspace``: a CUDA uint8 tensor of at least
    ``rel_attn_bwd_workspace_bytes`` bytes (allocated when None); ``grads``:
    preallocated outputs with the same keys.  ``out``, ``lse``: the forward's
    output and row log-sum-exp from ``rel_attn_fwd(..., lse=...)`` on the
    same inputs (both or neither); given, the backward skips its own
    forward."""
    import torch
    L, B, H, D = q.shape
    _check_attn(q, k, v, r, u_bias, v_bias, mem_len, q)
    if tuple(dout.shape) != (L, B, H, D) or dout.dtype != q.dtype or not dout.is_cuda \
            or not dout.is_contiguous():
        raise ValueError("dout must be a contiguous CUDA tensor shaped and typed like q")
    if grads is None:
        grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                     dr=torch.empty_like(r))
        if bias_grads:
            grads["du"] = torch.empty((H, D), dtype=torch.float32, device=q.device)
            grads["dw"] = torch.empty((H, D), dtype=torch.float32, device=q.device)
    grads.setdefault("du", None)
    grads.setdefault("dw", None)
    if (out is None) != (lse is None):
        raise ValueError("out and lse come together or not at all")
    if out is not None:
        if tuple(out.shape) != (L, B, H, D) or out.dtype != q.dtype or not out.is_cuda \
                or not out.is_contiguous():
            raise ValueError("out must be a contiguous CUDA tensor shaped and typed like q")
        if tuple(lse.shape) != (B, H, L) or lse.dtype != torch.float32 or not lse.is_cuda \
                or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 CUDA tensor [{B}, {H}, {L}]")
    nbytes = rel_attn_bwd_workspace_bytes(B, mem_len, L, H, D, _dtype_code(q))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace must hold {nbytes} bytes")
    st = load_library().txl_rel_attn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias), _ptr(dout), _ptr(out), _ptr(lse),
        B, mem_len, L, H, D, _dtype_code(q),
        _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dr"]),
        _ptr(grads["du"]), _ptr(grads["dw"]), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _raise(st, "txl_rel_attn_bwd")
    return grads


def rel_attn_fwd_ring(q, k, v, r, u_bias, v_bias, mem_len: int, kv_start: int, out=None, stream=None):
    """rel_attn_fwd with k, v stored as a ring of M+L rows: the context's key j
    (0 = oldest memory row) is at row (kv_start + j) mod (M+L)."""
    L, B, H, D = q.shape
    out = _check_attn(q, k, v, r, u_bias, v_bias, mem_len, out)
    st = load_library().txl_rel_attn_fwd_ring(
        _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias),
        B, mem_len, L, H, D, int(kv_start), _dtype_code(q), _ptr(out), _stream_ptr(stream))
    _raise(st, "txl_rel_attn_fwd_ring")
    return out


def rel_attn_fwd_padded(q, k, v, r, u_bias, v_bias, mem_len: int, d_head: int, out=None, stream=None):
    """rel_attn_fwd on head vectors padded to q.shape[-1] elements (zeros past
    ``d_head``), as project_heads / rel_table write them."""
    L, B, H, Dp = q.shape
    out = _check_attn(q, k, v, r, u_bias, v_bias, mem_len, out)
    st = load_library().txl_rel_attn_fwd_padded(
        _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias),
        B, mem_len, L, H, int(d_head), Dp, _dtype_code(q), _ptr(out), _stream_ptr(stream))
    _raise(st, "txl_rel_attn_fwd_padded")
    return out


def project_heads(x, w, heads: int, d_head: int, d_pad: int, out=None, stream=None):
    """y[..., heads, d_pad] = x[..., d_in] @ w.T with ``w`` the paper's
    [heads*d_head, d_in] projection (torch.nn.Linear's weight layout);
    padding columns d_head.. are zero.  x: [*lead, d_in]; returns
    [*lead, heads, d_pad]."""
    import torch
    lead = tuple(x.shape[:-1])
    d_in = x.shape[-1]
    rows = 1
    for n in lead:
        rows *= n
    if tuple(w.shape) != (heads * d_head, d_in) or w.dtype != x.dtype:
        raise ValueError(f"w must be [{heads * d_head}, {d_in}] of x's dtype")
    if out is not None and (tuple(out.shape) != lead + (heads, d_pad) or out.dtype != x.dtype):
        raise ValueError(f"out must be {list(lead + (heads, d_pad))} of x's dtype")
    for t in (x, w, out):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")
    if out is None:
        out = torch.empty(*lead, heads, d_pad, dtype=x.dtype, device=x.device)
    st = load_library().txl_project_heads(_ptr(x), _ptr(w), _ptr(out), rows, d_in, heads, d_head, d_pad,
                                          _dtype_code(x), _stream_ptr(stream))
    _raise(st, "txl_project_heads")
    return out


def _qkv_prepare(x, w_q, w_k, w_v, heads, d_head, d_pad, q_from, q, k, v):
    """project_qkv's argument checks; returns its (q, k, v) outputs, allocated where not given."""
    import torch
    T = x.shape[0]
    rest = tuple(x.shape[1:-1])
    d_in = x.shape[-1]
    per = 1
    for n in rest:
        per *= n
    if not 0 <= q_from <= T:
        raise ValueError(f"q_from must lie in [0, {T}]")
    for name, w in (("w_q", w_q), ("w_k", w_k), ("w_v", w_v)):
        if w is None and name != "w_q":
            raise ValueError(f"{name} is required")
        if w is not None and (tuple(w.shape) != (heads * d_head, d_in) or w.dtype != x.dtype):
            raise ValueError(f"{name} must be [{heads * d_head}, {d_in}] of x's dtype")
    if w_q is None and q is not None:
        raise ValueError("q is given without w_q")
    shapes = {"q": (T - q_from,) + rest + (heads, d_pad), "k": (T,) + rest + (heads, d_pad),
              "v": (T,) + rest + (heads, d_pad)}
    outs = {"q": q, "k": k, "v": v}
    for name, t in outs.items():
        if t is not None and (tuple(t.shape) != shapes[name] or t.dtype != x.dtype):
            raise ValueError(f"{name} must be {list(shapes[name])} of x's dtype")
    for t in (x, w_q, w_k, w_v, q, k, v):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")
    for name in ("k", "v") + (("q",) if w_q is not None else ()):
        if outs[name] is None:
            outs[name] = torch.empty(*shapes[name], dtype=x.dtype, device=x.device)
    return outs["q"], outs["k"], outs["v"]


def project_qkv(x, w_q, w_k, w_v, heads: int, d_head: int, d_pad: int, q_from: int = 0,
                q=None, k=None, v=None, stream=None):
    """A layer's q, k, v projections of one extended context: k = x @ w_k.T
    and v = x @ w_v.T over all of x's leading positions, q = x[q_from:] @
    w_q.T (the segment's own positions; ``w_q=None`` skips q).  x: [T, *rest,
    d_in]; outputs [T or T - q_from, *rest, heads, d_pad], as project_heads
    writes them.  Returns (q, k, v)."""
    T = x.shape[0]
    d_in = x.shape[-1]
    per = 1
    for n in x.shape[1:-1]:
        per *= n
    q, k, v = _qkv_prepare(x, w_q, w_k, w_v, heads, d_head, d_pad, q_from, q, k, v)
    outs = {"q": q, "k": k, "v": v}
    # no q rows (q_from == T): the library is asked for k and v only
    wq_arg = w_q if (w_q is not None and q_from < T) else None
    st = load_library().txl_project_qkv(
        _ptr(x), T * per, d_in, _ptr(wq_arg), _ptr(w_k), _ptr(w_v), _ptr(outs["q"]) if wq_arg is not None else None,
        _ptr(outs["k"]), _ptr(outs["v"]), q_from * per, heads, d_head, d_pad, _dtype_code(x), _stream_ptr(stream))
    _raise(st, "txl_project_qkv")
    return outs["q"], outs["k"], outs["v"]


def project_qkv_cells(xs, wqs, wks, wvs, heads: int, d_head: int, d_pad: int, q_from: int = 0,
                      qs=None, ks=None, vs=None, stream=None):
    """project_qkv for several layer calls of one shape at once (lists of
    equal length: the cells' extended contexts, their weights and, if given,
    their outputs); ``wqs=None`` skips q.  Returns (qs, ks, vs) lists."""
    n = len(xs)
    if not (len(wks) == len(wvs) == n and (wqs is None or len(wqs) == n)):
        raise ValueError("the cells' lists must have the same length")
    if n == 0:
        return [], [], []
    T = xs[0].shape[0]
    shape = tuple(xs[0].shape)
    for x in xs:
        if tuple(x.shape) != shape or x.dtype != xs[0].dtype:
            raise ValueError("every cell's x must have the first cell's shape and dtype")
    res = {"q": [], "k": [], "v": []}
    for c in range(n):
        # per cell, the single-cell binding's checks and allocations (no call)
        q1, k1, v1 = _qkv_prepare(xs[c], None if wqs is None else wqs[c], wks[c], wvs[c], heads, d_head, d_pad,
                                  q_from, None if qs is None else qs[c], None if ks is None else ks[c],
                                  None if vs is None else vs[c])
        res["q"].append(q1)
        res["k"].append(k1)
        res["v"].append(v1)
    per = 1
    for d in shape[1:-1]:
        per *= d
    with_q = wqs is not None and q_from < T
    arr = lambda ts: (ctypes.c_void_p * n)(*[_ptr(t) for t in ts])
    st = load_library().txl_project_qkv_cells(
        n, arr(xs), arr(wqs) if with_q else None, arr(wks), arr(wvs), arr(res["q"]) if with_q else None,
        arr(res["k"]), arr(res["v"]), T * per, shape[-1], q_from * per, heads, d_head, d_pad, _dtype_code(xs[0]),
        _stream_ptr(stream))
    _raise(st, "txl_project_qkv_cells")
    return (res["q"] if wqs is not None else None), res["k"], res["v"]


def rel_table(w_r, klen: int, heads: int, d_head: int, d_pad: int, out=None, stream=None):
    """Appendix B's reversed projected table [klen, heads, d_pad] from W_kR in
    the paper's layout [heads*d_head, d_model] and the sinusoid of the
    relative distance."""
    import torch
    if w_r.dim() != 2 or w_r.shape[0] != heads * d_head or not w_r.is_cuda or not w_r.is_contiguous():
        raise ValueError(f"w_r must be a contiguous CUDA [{heads * d_head}, d_model] tensor")
    d_model = w_r.shape[1]
    if out is None:
        out = torch.empty(klen, heads, d_pad, dtype=w_r.dtype, device=w_r.device)
    st = load_library().txl_rel_table(_ptr(w_r), _ptr(out), klen, d_model, heads, d_head, d_pad,
                                      _dtype_code(w_r), _stream_ptr(stream))
    _raise(st, "txl_rel_table")
    return out


def ring_append(ring, rows, start: int, stream=None):
    """Write ``rows`` [n, ...] into ``ring`` [ring_len, ...] at rows
    (start + i) mod ring_len; returns the next start, (start + n) mod ring_len."""
    n = rows.shape[0]
    ring_len = ring.shape[0]
    if tuple(rows.shape[1:]) != tuple(ring.shape[1:]) or rows.dtype != ring.dtype:
        raise ValueError("rows must match the ring's row shape and dtype")
    for t in (ring, rows):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    row_elems = ring[0].numel() if ring_len else 0
    st = load_library().txl_ring_append(_ptr(ring), _ptr(rows), ring_len, n, row_elems, int(start),
                                        _dtype_code(ring), _stream_ptr(stream))
    _raise(st, "txl_ring_append")
    return (start + n) % ring_len if ring_len else 0


def rel_attn_fwd_noalloc(q, k, v, r, u_bias, v_bias, mem_len: int, out, stream=None):
    """The same call through txl_rel_attn_fwd_noalloc, for callers that may not
    allocate device memory: ``out`` must be given, and the library allocates
    nothing (its split-key scratch is a fixed array in the library).  The
    arguments are checked exactly as ``rel_attn_fwd`` checks them."""
    if out is None:
        raise ValueError("out must be given: this entry point allocates nothing")
    L, B, H, D = q.shape
    _check_attn(q, k, v, r, u_bias, v_bias, mem_len, out)
    code = _dtype_code(q)
    st = load_library().txl_rel_attn_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(u_bias), _ptr(v_bias),
        B, mem_len, L, H, D, code, _ptr(out), _stream_ptr(stream))
    _raise(st, "txl_rel_attn_fwd_noalloc")
    return out


def rel_attn_fwd_raw(q_ptr, k_ptr, v_ptr, r_ptr, u_ptr, w_ptr, batch, mem_len, seg_len,
                     heads, d_head, dtype_code, out_ptr, stream_ptr) -> int:
    """The C entry point with raw integers (for host-side argument tests)."""
    return load_library().txl_rel_attn_fwd(q_ptr, k_ptr, v_ptr, r_ptr, u_ptr, w_ptr, batch,
                                           mem_len, seg_len, heads, d_head, dtype_code,
                                           out_ptr, stream_ptr)


def mem_update(mem_next, ext_ctx, mem_len: int, stream=None):
    """Memory rollover (Section 3.2): mem_next[:M] = newest M rows of ext_ctx.

    ext_ctx: [M+L, B, d_model]; mem_next: [>= M, B, d_model]; same dtype.
    """
    T, B, dm = ext_ctx.shape
    L = T - mem_len
    if L < 0:
        raise ValueError("mem_len larger than the extended context")
    if mem_next.dim() != 3 or mem_next.shape[0] < mem_len or tuple(mem_next.shape[1:]) != (B, dm):
        raise ValueError(f"mem_next must be [>= {mem_len}, {B}, {dm}]")
    if mem_next.dtype != ext_ctx.dtype:
        raise TypeError("mem_next and ext_ctx dtypes differ")
    for t in (mem_next, ext_ctx):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    st = load_library().txl_mem_update(_ptr(mem_next), _ptr(ext_ctx), B, mem_len, L, dm,
                                       _dtype_code(ext_ctx), _stream_ptr(stream))
    _raise(st, "txl_mem_update")
    return mem_next


def mem_update_raw(dst_ptr, src_ptr, batch, mem_len, seg_len, d_model, dtype_code,
                   stream_ptr) -> int:
    return load_library().txl_mem_update(dst_ptr, src_ptr, batch, mem_len, seg_len, d_model,
                                         dtype_code, stream_ptr)


def _loss_sizes(what: str, *sizes: int):
    """Refuses sizes that a C int does not hold (ctypes would pass their low
    32 bits); the library refuses the others that are too large."""
    if max(sizes) > 0x7fffffff:
        _raise(2, what)


def softmax_xent_workspace_bytes(rows: int, d_model: int, vocab: int, dtype_code: int,
                                 backward: bool = False) -> int:
    """Workspace bytes of ``softmax_xent_fwd`` (or, with ``backward``, of
    ``softmax_xent_bwd``, which then suffices for both)."""
    n = ctypes.c_size_t(0)
    _loss_sizes("txl_softmax_xent_workspace", rows, d_model, vocab)
    st = load_library().txl_softmax_xent_workspace(rows, d_model, vocab, dtype_code, int(bool(backward)),
                                                   ctypes.byref(n))
    _raise(st, "txl_softmax_xent_workspace")
    return int(n.value)


def distill_workspace_bytes(rows: int, d_model: int, vocab: int, top_k: int, dtype_code: int,
                            backward: bool = False) -> int:
    """Workspace bytes of ``distill_fwd`` (or, with ``backward``, of
    ``distill_bwd``, which then suffices for both)."""
    n = ctypes.c_size_t(0)
    _loss_sizes("txl_distill_workspace", rows, d_model, vocab, top_k)
    st = load_library().txl_distill_workspace(rows, d_model, vocab, top_k, dtype_code, int(bool(backward)),
                                              ctypes.byref(n))
    _raise(st, "txl_distill_workspace")
    return int(n.value)


class _Call:
    """The checks that the calls over rows share, and where their own tensors
    are made: on the tensors' device and, with ``stream`` given, in that
    stream's order (so that a workspace freed at return is reused only behind
    the call)."""

    def __init__(self, first, stream):
        self.dev = first.get_device()
        self.stream = stream
        self.placed = first.is_contiguous()

    def arg(self, name, t, shape, dtype):
        """A tensor argument's pointer (None stays None)."""
        if t is None:
            return None
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != self.dev or not t.is_contiguous():
            self.placed = False
        return t.data_ptr()

    def on_device(self):
        """After every argument given: all of them contiguous, on one CUDA device."""
        if self.dev < 0 or not self.placed:
            raise ValueError("all tensors must be contiguous CUDA tensors on one device")
        if self.stream is not None and self.stream.device_index != self.dev:
            raise ValueError("stream must belong to the tensors' device")

    def make(self, shape, dtype):
        import torch
        device = torch.device("cuda", self.dev)
        if self.stream is not None:
            with torch.cuda.stream(self.stream):
                return torch.empty(shape, dtype=dtype, device=device)
        return torch.empty(shape, dtype=dtype, device=device)

    def launch(self, fn, *args):
        """fn(*args, stream) with the tensors' device current; its status"""
        import torch
        stream = self.stream.cuda_stream if self.stream is not None else torch._C._cuda_getCurrentRawStream(self.dev)
        if torch._C._cuda_getDevice() == self.dev:
            return fn(*args, stream)
        with torch.cuda.device(self.dev):
            return fn(*args, stream)

    def run(self, fn, what, need, workspace, *args):
        """Calls fn(*args, workspace, its bytes, stream); need() is the workspace's size."""
        import torch
        if workspace is None:
            workspace = self.make((need(),), torch.uint8)
        elif workspace.get_device() != self.dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the other tensors' device")
        nbytes = workspace.nbytes
        st = self.launch(fn, *args, workspace.data_ptr(), nbytes)
        if st == 1 and nbytes < need():
            raise ValueError(f"workspace must hold {need()} bytes")
        _raise(st, what)


class _LossCall(_Call):
    """An output-layer loss: h's rows, and the weights."""

    def __init__(self, h, w, stream):
        shape, w_shape = h.shape, w.shape
        if len(w_shape) != 2 or not shape or w_shape[1] != shape[-1] or w.dtype != h.dtype:
            raise ValueError("w must be [vocab, d_model] with h's last dimension and dtype")
        self.lead = shape[:-1]
        self.rows = self.lead.numel()
        self.vocab, self.d = w_shape
        if (self.rows | self.vocab | self.d) >> 31:
            _loss_sizes("output-layer loss", self.rows, self.vocab, self.d)
        self.code = _dtype_code(h)
        _Call.__init__(self, h, stream)
        self.h = h
        self.placed = self.placed and w.is_contiguous() and w.get_device() == self.dev

    def gradients(self, grads, w, bias, weight_grads):
        """The dict of a backward's outputs (given tensors used, absent ones made) and their pointers."""
        import torch
        grads = {} if grads is None else dict(grads)
        given = [self.arg("dh", grads.get("dh"), self.h.shape, self.h.dtype)]
        if weight_grads:
            given.append(self.arg("dw", grads.get("dw"), w.shape, w.dtype))
            given.append(self.arg("db", grads.get("db"), (self.vocab,), torch.float32))
        self.on_device()
        if given[0] is None:
            grads["dh"] = self.make(self.h.shape, self.h.dtype)
        if not weight_grads:
            grads["dw"] = grads["db"] = None
            return grads, (grads["dh"].data_ptr(), None, None)
        if given[1] is None:
            grads["dw"] = self.make(w.shape, w.dtype)
        if given[2] is None:
            grads["db"] = self.make((self.vocab,), torch.float32) if bias is not None else None
        return grads, (grads["dh"].data_ptr(), grads["dw"].data_ptr(),
                       grads["db"].data_ptr() if grads["db"] is not None else None)


def softmax_xent_fwd(h, w, target, bias=None, loss=None, lse=None, workspace=None, stream=None):
    """Cross entropy of the output layer z = h @ w.T + bias without its logits
    (txl_softmax_xent_fwd).

    h: [*lead, d_model] hidden states; w: [vocab, d_model] (torch.nn.Linear's
    and Embedding's layout), h's dtype (float32 or bfloat16); target: [*lead]
    int64 (a label outside [0, vocab), such as -100, is a padding row: loss
    0); bias: [vocab] float32 or None; all CUDA, contiguous.  Returns
    (loss, lse), float32 [*lead]: the rows' losses (no reduction) and
    log-sum-exps, the latter for ``softmax_xent_bwd``.  ``workspace``: a CUDA
    tensor of at least ``softmax_xent_workspace_bytes`` bytes, not shared with
    a call that may run at the same time (allocated when None)."""
    import torch
    c = _LossCall(h, w, stream)
    y = c.arg("target", target, c.lead, torch.int64)
    b = c.arg("bias", bias, (c.vocab,), torch.float32)
    c.arg("loss", loss, c.lead, torch.float32)
    c.arg("lse", lse, c.lead, torch.float32)
    c.on_device()
    loss = c.make(c.lead, torch.float32) if loss is None else loss
    lse = c.make(c.lead, torch.float32) if lse is None else lse
    c.run(load_library().txl_softmax_xent_fwd, "txl_softmax_xent_fwd",
          lambda: softmax_xent_workspace_bytes(c.rows, c.d, c.vocab, c.code), workspace, h.data_ptr(), w.data_ptr(), b,
          y, c.rows, c.d, c.vocab, c.code, loss.data_ptr(), lse.data_ptr())
    return loss, lse


def softmax_xent_bwd(h, w, target, lse, dloss, bias=None, grads=None, weight_grads: bool = True, workspace=None,
                     stream=None):
    """Gradients of ``(dloss * loss).sum()`` of one ``softmax_xent_fwd`` call
    (txl_softmax_xent_bwd): a dict ``dh`` (like h), ``dw`` (like w) and ``db``
    (float32 [vocab]; None without a bias).  ``lse``: the forward's; ``dloss``:
    float32 [*lead] (1 / tokens for a mean).  ``weight_grads=False`` skips dw
    and db (a frozen output layer).  ``grads``: preallocated outputs with the
    same keys; ``workspace`` as the forward's, of
    ``softmax_xent_workspace_bytes(..., backward=True)`` bytes."""
    import torch
    c = _LossCall(h, w, stream)
    y = c.arg("target", target, c.lead, torch.int64)
    b = c.arg("bias", bias, (c.vocab,), torch.float32)
    s = c.arg("lse", lse, c.lead, torch.float32)
    g = c.arg("dloss", dloss, c.lead, torch.float32)
    grads, out = c.gradients(grads, w, bias, weight_grads)
    c.run(load_library().txl_softmax_xent_bwd, "txl_softmax_xent_bwd",
          lambda: softmax_xent_workspace_bytes(c.rows, c.d, c.vocab, c.code, backward=True), workspace, h.data_ptr(),
          w.data_ptr(), b, y, s, g, c.rows, c.d, c.vocab, c.code, *out)
    return grads


def _teacher(c, teacher_idx, teacher_logits):
    """(top_k, pointers of the indices and logits, the logits' type code)"""
    import torch
    shape = teacher_idx.shape
    if shape[:-1] != c.lead or len(shape) != len(c.lead) + 1:
        raise ValueError(f"teacher_idx must be {list(c.lead)} + [top_k]")
    _loss_sizes("output-layer loss", shape[-1])
    if teacher_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"teacher_logits must be float32 or bfloat16, got {teacher_logits.dtype}")
    e = c.arg("teacher_idx", teacher_idx, shape, torch.int64)
    y = c.arg("teacher_logits", teacher_logits, shape, teacher_logits.dtype)
    return shape[-1], e, y, _dtype_code(teacher_logits)


def distill_fwd(h, w, teacher_idx, teacher_logits, temperature: float = 1.0, bias=None, loss=None, lse=None,
                workspace=None, stream=None):
    """Distillation loss of the output layer against a teacher's kept logits
    (txl_distill_fwd): per row temperature^2 times the KL divergence from the
    teacher's softmax over its kept entries to the student's softmax over the
    vocabulary, both at ``temperature`` (2^-63 to 2^63).

    teacher_idx: [*lead, top_k] int64, teacher_logits: [*lead, top_k] float32
    or bfloat16 (``torch.topk``'s outputs; entries with an index outside
    [0, vocab) or a logit of -inf are left out, a row without entries is a
    padding row: loss 0).  Everything else as ``softmax_xent_fwd``.  Returns
    (loss, lse); lse is the student's at ``temperature``."""
    import torch
    c = _LossCall(h, w, stream)
    k, e, y, t_code = _teacher(c, teacher_idx, teacher_logits)
    b = c.arg("bias", bias, (c.vocab,), torch.float32)
    c.arg("loss", loss, c.lead, torch.float32)
    c.arg("lse", lse, c.lead, torch.float32)
    c.on_device()
    loss = c.make(c.lead, torch.float32) if loss is None else loss
    lse = c.make(c.lead, torch.float32) if lse is None else lse
    c.run(load_library().txl_distill_fwd, "txl_distill_fwd",
          lambda: distill_workspace_bytes(c.rows, c.d, c.vocab, k, c.code), workspace, h.data_ptr(), w.data_ptr(), b, e,
          y, t_code, temperature, c.rows, c.d, c.vocab, k, c.code, loss.data_ptr(), lse.data_ptr())
    return loss, lse


def distill_bwd(h, w, teacher_idx, teacher_logits, lse, dloss, temperature: float = 1.0, bias=None, grads=None,
                weight_grads: bool = True, workspace=None, stream=None):
    """Gradients of ``(dloss * loss).sum()`` of one ``distill_fwd`` call
    (txl_distill_bwd), as ``softmax_xent_bwd`` returns them."""
    import torch
    c = _LossCall(h, w, stream)
    k, e, y, t_code = _teacher(c, teacher_idx, teacher_logits)
    b = c.arg("bias", bias, (c.vocab,), torch.float32)
    s = c.arg("lse", lse, c.lead, torch.float32)
    g = c.arg("dloss", dloss, c.lead, torch.float32)
    grads, out = c.gradients(grads, w, bias, weight_grads)
    c.run(load_library().txl_distill_bwd, "txl_distill_bwd",
          lambda: distill_workspace_bytes(c.rows, c.d, c.vocab, k, c.code, backward=True), workspace, h.data_ptr(),
          w.data_ptr(), b, e, y, t_code, temperature, s, g, c.rows, c.d, c.vocab, k, c.code, *out)
    return grads


def embed_bwd_workspace_bytes(rows: int, d_model: int, vocab: int, dtype_code: int) -> int:
    """Workspace bytes of ``embed_bwd``."""
    n = ctypes.c_size_t(0)
    _loss_sizes("txl_embed_bwd_workspace", rows, d_model, vocab)
    _raise(load_library().txl_embed_bwd_workspace(rows, d_model, vocab, dtype_code, ctypes.byref(n)),
           "txl_embed_bwd_workspace")
    return int(n.value)


def embed_fwd(tokens, table, scale: float = 1.0, out=None, stream=None):
    """The token embedding: out[..., :] = scale * table[tokens], rows of zeros
    for tokens outside [0, vocab) (txl_embed_fwd).

    tokens: [*lead] int64; table: [vocab, d_model] float32 or bfloat16; both
    CUDA, contiguous.  Returns out [*lead, d_model] of the table's dtype."""
    import torch
    if table.dim() != 2:
        raise ValueError("table must be [vocab, d_model]")
    vocab, d = table.shape
    c = _Call(table, stream)
    lead = tokens.shape
    rows = lead.numel()
    if (rows | vocab | d) >> 31:
        _loss_sizes("txl_embed_fwd", rows, vocab, d)
    code = _dtype_code(table)
    t = c.arg("tokens", tokens, lead, torch.int64)
    shape = lead + (d,)
    c.arg("out", out, shape, table.dtype)
    c.on_device()
    out = c.make(shape, table.dtype) if out is None else out
    _raise(c.launch(load_library().txl_embed_fwd, t, table.data_ptr(), scale, rows, d, vocab, code, out.data_ptr()),
           "txl_embed_fwd")
    return out


def embed_bwd(tokens, dout, dtable=None, scale: float = 1.0, accumulate: bool = False, vocab: Optional[int] = None,
              workspace=None, stream=None):
    """The table's gradient of one ``embed_fwd`` call (txl_embed_bwd):
    dtable[t] = scale * the sum of dout's rows with token t.

    dout: [*lead, d_model]; dtable: [vocab, d_model] of dout's dtype (made when
    None, with ``vocab`` given).  ``accumulate=True`` adds to dtable instead of
    overwriting it (a table tied to the output layer: the ``dw`` of its
    losses).  ``workspace``: a CUDA tensor of at least
    ``embed_bwd_workspace_bytes`` bytes, not shared with a call that may run at
    the same time (made when None).  Returns dtable."""
    import torch
    if not dout.dim():
        raise ValueError("dout must be [*lead, d_model]")
    lead, d = dout.shape[:-1], dout.shape[-1]
    if dtable is None:
        if vocab is None or accumulate:
            raise ValueError("without dtable, vocab is required (and there is nothing to accumulate to)")
    elif dtable.dim() != 2 or (vocab is not None and vocab != dtable.shape[0]):
        raise ValueError("dtable must be [vocab, d_model]")
    else:
        vocab = dtable.shape[0]
    rows = lead.numel()
    if (rows | vocab | d) >> 31:
        _loss_sizes("txl_embed_bwd", rows, vocab, d)
    c = _Call(dout, stream)
    code = _dtype_code(dout)
    t = c.arg("tokens", tokens, lead, torch.int64)
    c.arg("dtable", dtable, (vocab, d), dout.dtype)
    c.on_device()
    dtable = c.make((vocab, d), dout.dtype) if dtable is None else dtable
    c.run(load_library().txl_embed_bwd, "txl_embed_bwd", lambda: embed_bwd_workspace_bytes(rows, d, vocab, code),
          workspace, t, dout.data_ptr(), scale, rows, d, vocab, code, 1 if accumulate else 0, dtable.data_ptr())
    return dtable


def layer_norm_bwd_workspace_bytes(rows: int, d_model: int, dtype_code: int) -> int:
    """Workspace bytes of ``layer_norm_bwd``."""
    n = ctypes.c_size_t(0)
    _loss_sizes("txl_layer_norm_bwd_workspace", rows, d_model)
    _raise(load_library().txl_layer_norm_bwd_workspace(rows, d_model, dtype_code, ctypes.byref(n)),
           "txl_layer_norm_bwd_workspace")
    return int(n.value)


def _norm_sizes(x, what):
    """(shape, lead, rows, d) of a layer norm's x"""
    shape = tuple(x.shape)
    if not shape:
        raise ValueError("x must be [*lead, d_model]")
    lead, d = shape[:-1], shape[-1]
    rows = 1
    for n in lead:
        rows *= n
    if (rows | d) >> 31:
        _loss_sizes(what, rows, d)
    return shape, lead, rows, d


def layer_norm_fwd(x, gamma=None, beta=None, residual=None, eps: float = 1e-5, y=None, sum=None, mean=None, rstd=None,
                   stream=None):
    """Layer norm of x + residual over the last dimension (txl_layer_norm_fwd).

    x, residual: [*lead, d_model] float32 or bfloat16 (residual may be None);
    gamma, beta: [d_model] float32 or None (1, 0); all CUDA, contiguous.
    ``sum``: a tensor like x that receives x + residual (for the next
    residual), rounded to x's dtype, and is normalised as rounded.  Returns
    (y, mean, rstd): y like x, the others float32 [*lead], for
    ``layer_norm_bwd``."""
    import torch
    shape, lead, rows, d = _norm_sizes(x, "txl_layer_norm_fwd")
    c = _Call(x, stream)
    code, dt, f32 = _dtype_code(x), x.dtype, torch.float32
    r = c.arg("residual", residual, shape, dt)
    g = c.arg("gamma", gamma, (d,), f32)
    b = c.arg("beta", beta, (d,), f32)
    c.arg("y", y, shape, dt)
    kept = c.arg("sum", sum, shape, dt)
    c.arg("mean", mean, lead, f32)
    c.arg("rstd", rstd, lead, f32)
    c.on_device()
    y = c.make(shape, dt) if y is None else y
    mean = c.make(lead, f32) if mean is None else mean
    rstd = c.make(lead, f32) if rstd is None else rstd
    _raise(c.launch(load_library().txl_layer_norm_fwd, x.data_ptr(), r, g, b, eps, rows, d, code, y.data_ptr(), kept,
                    mean.data_ptr(), rstd.data_ptr()), "txl_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, gamma=None, residual=None, dsum=None, grads=None, weight_grads: bool = True,
                   workspace=None, stream=None):
    """Gradients of one ``layer_norm_fwd`` call (txl_layer_norm_bwd): a dict
    ``dx`` (like x; the gradient of x and of the residual alike) and
    ``dgamma``, ``dbeta`` (float32 [d_model]; None with ``weight_grads=False``).

    x, residual: the forward's; or the ``sum`` it kept as x, and no residual.
    mean, rstd: the forward's.  ``dsum``: the gradient of the kept sum by its
    other path, added to dx, or None.  ``grads``: preallocated outputs with the
    same keys; ``workspace``: of ``layer_norm_bwd_workspace_bytes`` bytes, as
    ``embed_bwd``'s."""
    import torch
    shape, lead, rows, d = _norm_sizes(x, "txl_layer_norm_bwd")
    c = _Call(x, stream)
    code, dt, f32 = _dtype_code(x), x.dtype, torch.float32
    given = c.arg("dy", dy, shape, dt)
    r = c.arg("residual", residual, shape, dt)
    o = c.arg("dsum", dsum, shape, dt)
    g = c.arg("gamma", gamma, (d,), f32)
    m = c.arg("mean", mean, lead, f32)
    v = c.arg("rstd", rstd, lead, f32)
    grads = {} if grads is None else dict(grads)
    c.arg("dx", grads.get("dx"), shape, dt)
    if weight_grads:
        c.arg("dgamma", grads.get("dgamma"), (d,), f32)
        c.arg("dbeta", grads.get("dbeta"), (d,), f32)
    c.on_device()
    if grads.get("dx") is None:
        grads["dx"] = c.make(shape, dt)
    for name in ("dgamma", "dbeta"):
        if not weight_grads:
            grads[name] = None
        elif grads.get(name) is None:
            grads[name] = c.make((d,), f32)
    dg, db = grads["dgamma"], grads["dbeta"]
    args = (given, x.data_ptr(), r, o, g, m, v, rows, d, code, grads["dx"].data_ptr(),
            dg.data_ptr() if weight_grads else None, db.data_ptr() if weight_grads else None)
    if weight_grads:
        c.run(load_library().txl_layer_norm_bwd, "txl_layer_norm_bwd",
              lambda: layer_norm_bwd_workspace_bytes(rows, d, code), workspace, *args)
    else:
        _raise(c.launch(load_library().txl_layer_norm_bwd, *args, None, 0), "txl_layer_norm_bwd")
    return grads


class AdamwTensors:
    """The tensors of an optimiser step, checked and laid out once: lists of
    equal length of contiguous tensors on one CUDA device, one entry per
    weight, for ``adamw_step`` and ``grad_norm``.

    params: float32 or bfloat16; grads: float32 or bfloat16, shaped alike;
    masters: float32 weights of which the bfloat16 params are rounded copies
    (None, or None entries: the step acts on the param itself).
    exp_avgs, exp_avg_sqs: the moments, float32 (zeros at first), or 8 bits:
    ``torch.float8_e4m3fn`` with exp_avg_scales, exp_avg_sq_scales, float32
    [ceil(elements / 256)] (all zeros at first; exp_avg_sqs then holds square
    roots); these lists may mix both, with None for float32 moments' scales.
    weight_decay: a number, or one per tensor.

    The object keeps the tensors' memory, and steps act on it: a weight or
    gradient moved elsewhere wants a new one (gradients stay where they are
    when the backward calls write them by their ``grads=`` or ``dtable``).
    Making one takes the host some 2 to 3 us per tensor, more than a step may:
    it is made once."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, masters=None, exp_avg_scales=None, exp_avg_sq_scales=None,
                 weight_decay=0.0):
        import torch
        n = len(params)
        none = [None] * n
        lists = dict(params=params, grads=grads, exp_avgs=exp_avgs, exp_avg_sqs=exp_avg_sqs, masters=masters or none,
                     exp_avg_scales=exp_avg_scales or none, exp_avg_sq_scales=exp_avg_sq_scales or none)
        lists = {name: list(x) for name, x in lists.items()}
        single = lambda x: ctypes.c_float(x).value       # (infinity past its range: the step refuses that)
        decay = [single(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [single(float(x)) for x in weight_decay]
        for name, x in list(lists.items()) + [("weight_decay", decay)]:
            if len(x) != n:
                raise ValueError(f"{name} must have an entry per param ({n}), got {len(x)}")
        array, entry = (_AdamwTensor * max(n, 1))(), ctypes.sizeof(_AdamwTensor)
        kept = []       # storages, not tensors: one whose ``data`` is replaced lets go of its storage
        dev = params[0].get_device() if n else None
        f32, e4m3 = torch.float32, torch.float8_e4m3fn
        codes = {f32: TXL_F32, torch.bfloat16: TXL_BF16}
        for k, (p, g, m, v, w, ms, vs, wd) in enumerate(zip(*lists.values(), decay)):
            shape, size = p.shape, p.numel()
            if g.shape != shape or m.shape != shape or v.shape != shape or (w is not None and w.shape != shape):
                raise ValueError(f"tensor {k}: grad, master and moments must be {list(shape)}")
            code, g_code = codes.get(p.dtype), codes.get(g.dtype)
            if code is None or g_code is None:
                raise TypeError(f"tensor {k}: unsupported dtype {p.dtype}, {g.dtype} (float32 or bfloat16)")
            if w is not None and (w.dtype is not f32 or code == TXL_F32):
                raise TypeError(f"tensor {k}: a master is float32 beside a bfloat16 param")
            state = f32 if ms is None else e4m3
            if (ms is None) != (vs is None) or m.dtype is not state or v.dtype is not state:
                raise TypeError(f"tensor {k}: moments are float32 without scales, or float8_e4m3fn with both")
            if ms is not None:
                blocks = ((size + 255) // 256,)
                if ms.shape != blocks or vs.shape != blocks or ms.dtype is not f32 or vs.dtype is not f32:
                    raise ValueError(f"tensor {k}: scales must be float32 {list(blocks)}")
            for x in (p, g, m, v, w, ms, vs):
                if x is None:
                    continue
                if x.get_device() != dev or not x.is_contiguous():
                    dev = -1
                kept.append(x.untyped_storage())
            if dev < 0:
                raise ValueError("all tensors must be contiguous CUDA tensors on one device")
            if size:
                _ADAMW_FIELDS.pack_into(array, k * entry, p.data_ptr(), 0 if w is None else w.data_ptr(), g.data_ptr(),
                                        m.data_ptr(), v.data_ptr(), 0 if ms is None else ms.data_ptr(),
                                        0 if ms is None else vs.data_ptr(), size, wd, code, g_code)
            else:
                _ADAMW_FIELDS.pack_into(array, k * entry, 0, 0, 0, 0, 0, 0, 0, 0, wd, code, g_code)
        self._array, self._dev, self._count, self._kept = array, dev, n, kept

    def __len__(self):
        return self._count


class _ListCall(_Call):
    """A call over an ``AdamwTensors``."""

    def __init__(self, tensors, stream):
        import torch
        if not isinstance(tensors, AdamwTensors):
            raise TypeError("tensors must be an AdamwTensors")
        self.dev = torch.cuda.current_device() if tensors._dev is None else tensors._dev
        self.stream, self.placed = stream, True


def grad_norm_workspace_bytes(tensors) -> int:
    """Workspace bytes of ``grad_norm``."""
    n = ctypes.c_size_t(0)
    _raise(load_library().txl_grad_norm_workspace(tensors._count, tensors._array, ctypes.byref(n)),
           "txl_grad_norm_workspace")
    return int(n.value)


def grad_norm(tensors, max_norm: float, norm=None, clip=None, workspace=None, stream=None):
    """The norm of all gradients of an ``AdamwTensors`` together and the
    factor min(1, max_norm / norm) that clips them (NaN where the norm is not
    finite), both float32 [1] on the device (txl_grad_norm): (norm, clip).
    ``workspace``: of ``grad_norm_workspace_bytes`` bytes, as ``embed_bwd``'s."""
    import torch
    c = _ListCall(tensors, stream)
    c.arg("norm", norm, (1,), torch.float32)
    c.arg("clip", clip, (1,), torch.float32)
    c.on_device()
    norm = c.make((1,), torch.float32) if norm is None else norm
    clip = c.make((1,), torch.float32) if clip is None else clip
    c.run(load_library().txl_grad_norm, "txl_grad_norm", lambda: grad_norm_workspace_bytes(tensors), workspace,
          tensors._count, tensors._array, max_norm, norm.data_ptr(), clip.data_ptr())
    return norm, clip


def adamw_step(tensors, lr, step, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, grad_scale=None,
               seed: int = 0, stream=None) -> None:
    """One AdamW step over an ``AdamwTensors``, in place (txl_adamw_step).

    lr: a number, or a float32 [1] CUDA tensor; step: the step's number (1 at
    first), or an int64 [1] CUDA tensor: tensors are read when the kernel runs,
    so a captured step can be replayed with other values.  grad_scale: a
    float32 [1] CUDA tensor that multiplies the gradients (``grad_norm``'s
    clip), or None; one that is not finite leaves everything as it is.  seed:
    of the 8-bit moments' stochastic rounding."""
    import torch
    c = _ListCall(tensors, stream)
    o = _AdamwOptions()
    o.beta1, o.beta2, o.eps, o.seed = beta1, beta2, eps, seed & 0xffffffffffffffff
    if isinstance(lr, torch.Tensor):
        o.lr_device = c.arg("lr", lr, (1,), torch.float32)
    else:
        o.lr = lr
    if isinstance(step, torch.Tensor):
        o.step_device = c.arg("step", step, (1,), torch.int64)
    elif not 1 <= step < 2 ** 63:
        raise ValueError(f"step must be at least 1, got {step}")
    else:
        o.step = step
    o.grad_scale = c.arg("grad_scale", grad_scale, (1,), torch.float32)
    c.on_device()
    _raise(c.launch(load_library().txl_adamw_step, tensors._count, tensors._array, ctypes.byref(o)), "txl_adamw_step")


def selftest_wait(limit_us: int, stream=None) -> None:
    """Launch the bounded-wait self test (txl_selftest_wait): a wait that runs
    out after ``limit_us`` microseconds; the next ``check`` raises
    TXL_ERR_TIMEOUT."""
    _raise(load_library().txl_selftest_wait(int(limit_us), _stream_ptr(stream)), "txl_selftest_wait")


def check(stream=None) -> None:
    """Synchronise the stream and raise if a kernel reported an error."""
    _raise(load_library().txl_check(_stream_ptr(stream)), "txl_check")
