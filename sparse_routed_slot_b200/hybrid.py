"""Python binding of the operators beside the mixer (include/rsm.h): window attention, attention over
a paged cache, and the block norms, on torch CUDA tensors.

Like api.py this layer only marshals arguments; the work runs in the library's kernels on the current
stream of the tensors' device. All tensors are contiguous and on one device.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .api import _DTYPES, gradient

_NO_SIZE = ctypes.c_size_t(-1).value
_ACTS = {"silu": _lib.RSM_ACT_SILU, "sigmoid": _lib.RSM_ACT_SIGMOID}
_INT_MAX = 2**31 - 1
_ref = ctypes.byref

# A single-token step is a few microseconds on the device, so the checks below are written to cost little
# where they find nothing: one test per tensor, and the words only for one that fails.


def _fault(t, name, dtype, shape, index):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return f"{name} must be a CUDA tensor"
    if not t.is_contiguous():
        return f"{name} must be contiguous"
    if t.dtype != dtype:
        return f"{name} must be {dtype}, got {t.dtype}"
    if tuple(t.shape) != tuple(shape):
        return f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}"
    return f"{name} must be on cuda:{index}, got {t.device}"


def _ptr(t, name, dtype, shape, index):
    """The address of a contiguous tensor of that type, shape and device; None for None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape and
            t.is_contiguous()):
        raise ValueError(_fault(t, name, dtype, shape, index))
    return t.data_ptr()


def _given(t, name, dtype, shape, index):
    """_ptr of a tensor that has to be there."""
    if t is None:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _ptr(t, name, dtype, shape, index)


def _first(t, name, dims):
    """(type, shape, device index) of the tensor that the others have to agree with."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dims and t.dim() != len(dims):
        raise ValueError(f"{name} must be [{','.join(dims)}], got {tuple(t.shape)}")
    _ints(t, name)
    return t.dtype, t.shape, t.get_device()


def _ints(t, name):
    """Refuses sizes that are no C ints (the library takes them as such)."""
    if t.numel() > _INT_MAX and max(t.shape) > _INT_MAX:
        raise ValueError(f"{name} has a size of 2^31 or more: {tuple(t.shape)}")


def _run(fn, args, index, size_fn=None, workspace=None):
    """A library call on the device's current stream, with that device current. With size_fn it gets a
    workspace: the caller's (a uint8 tensor) where that is large enough, else a new one of torch's."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _run(fn, args, index, size_fn, workspace)
    if size_fn is not None:
        need = size_fn(_ref(args))
        if need == _NO_SIZE:
            _lib.check(fn(_ref(args), None))  # raises with the reason
        if need:
            if workspace is None or workspace.numel() < need:
                workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index))
            args.workspace = _given(workspace, "workspace", torch.uint8, workspace.shape, index)
            args.workspace_bytes = workspace.numel()
    status = fn(_ref(args), torch._C._cuda_getCurrentRawStream(index))
    if status:
        _lib.check(status)


def _scale(scale, D):
    return 1.0 / math.sqrt(D) if scale is None and D else float(scale or 0.0)


def _int(x):
    """A C int; past its range the largest one, which is as good as no limit, or one below zero, which is refused."""
    return max(min(int(x), _INT_MAX), -_INT_MAX)


# ------------------------------------------------------------------------------ window attention
def _window_args(cls, q, k, v, window, sinks, scale, validate):
    dtype, shape, index = _first(q, "q", "BTHD")
    B, T, H, D = shape
    _, kshape, _ = _first(k, "k", ("B", "T", "Hkv", "D"))
    Hkv = kshape[2]
    kshape = torch.Size((B, T, Hkv, D))
    a = cls(B, T, H, Hkv, D, _int(window), _int(sinks), _DTYPES[dtype], _scale(scale, D), _ptr(q, "q", dtype, shape, index),
            _ptr(k, "k", dtype, kshape, index), _given(v, "v", dtype, kshape, index))
    if validate:
        a.flags = _lib.RSM_FLAG_VALIDATE
    return a, dtype, shape, kshape, index


def window_forward(q, k, v, window: int, sinks: int = 0, scale=None, *, lse: bool = False, low: bool = False,
                   validate: bool = False, out=None):
    """Causal attention over the last `window` keys and the first `sinks`. q [B,T,H,D]; k, v
    [B,T,Hkv,D] with Hkv dividing H; float32 or bfloat16. scale defaults to 1/sqrt(D).

    Returns dict(o [B,T,H,D] in q's dtype, lse [B,T,H] fp32 or None, low like o or None: with `low`, what
    rounding left of a bfloat16 o, for window_backward). `out` may supply preallocated tensors under the
    same keys."""
    a, dtype, shape, _, index = _window_args(_lib.WindowArgs, q, k, v, window, sinks, scale, validate)
    o = ls = lo = None
    if out:
        o, ls, lo = out.get("o"), out.get("lse"), out.get("low")
    if o is None:
        o = torch.empty_like(q)
    if ls is None and lse:
        ls = torch.empty(shape[:3], dtype=torch.float32, device=q.device)
    if lo is None and low and dtype is torch.bfloat16:
        lo = torch.empty_like(q)
    a.o, a.lse = _ptr(o, "o", dtype, shape, index), _ptr(ls, "lse", torch.float32, shape[:3], index)
    a.o_low = _ptr(lo, "low", dtype, shape, index)
    _run(_lib.load().rsm_window_forward, a, index)
    return {"o": o, "lse": ls, "low": lo}


def window_backward(q, k, v, o, lse, dO, window: int, sinks: int = 0, scale=None, *, low=None,
                    need=(True, True, True), validate: bool = False, out=None, workspace=None):
    """Gradients of window_forward: its inputs, its o, lse and (if kept) low, and dO [B,T,H,D] in q's dtype.
    Returns dict(dq, dk, dv) in q's dtype (None where `need` says so)."""
    a, dtype, shape, kshape, index = _window_args(_lib.WindowBackwardArgs, q, k, v, window, sinks, scale, validate)
    a.o, a.dO = _given(o, "o", dtype, shape, index), _given(dO, "dO", dtype, shape, index)
    a.lse = _given(lse, "lse", torch.float32, shape[:3], index)
    a.o_low = _ptr(low, "low", dtype, shape, index)
    got = {}
    for name, like, size, wanted in zip(("dq", "dk", "dv"), (q, k, v), (shape, kshape, kshape), need):
        g = None
        if wanted:
            g = out.get(name) if out else None
            if g is None:
                g = torch.empty_like(like)
            setattr(a, name, _ptr(g, name, dtype, size, index))
        got[name] = g
    L = _lib.load()
    _run(L.rsm_window_backward, a, index, L.rsm_window_backward_workspace_size, workspace)
    return got


class WindowFunction(torch.autograd.Function):
    """Window attention as an autograd function: apply(q, k, v, window, sinks=0, scale=None) -> o.

    Recording a training step into a CUDA graph follows torch's own rule for every autograd function: no
    eager graph of the same leaves may be alive during the capture (torch then touches their old stream from
    its backward thread, which fails the capture and can end the process). window_forward and
    window_backward, called directly, carry no such state."""

    @staticmethod
    def forward(ctx, q, k, v, window, sinks=0, scale=None):
        r = window_forward(q, k, v, window, sinks, scale, lse=True, low=True)
        ctx.save_for_backward(q, k, v, r["o"], r["lse"], r["low"])
        ctx.how = (window, sinks, scale)
        return r["o"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        q, k, v, o, lse, low = ctx.saved_tensors
        g = window_backward(q, k, v, o, lse, gradient(dO), *ctx.how, low=low, need=ctx.needs_input_grad[:3])
        return g["dq"], g["dk"], g["dv"], None, None, None


# ------------------------------------------------------------------------------- paged attention
_CACHE = ("pages", "page_size", "Hkv", "D")


def paged_append(k, v, k_cache, v_cache, page_table, cu_q, kv_len) -> None:
    """Writes the new tokens' keys and values (k, v [N,Hkv,D]; sequence b's are rows cu_q[b] ..
    cu_q[b+1]-1) to places kv_len[b] - n_b .. kv_len[b] - 1 of the caches [pages, page_size, Hkv, D],
    in place. page_table int32 [B, width], cu_q int32 [B+1], kv_len int32 [B] (new tokens included)."""
    dtype, shape, index = _first(k, "k", ("N", "Hkv", "D"))
    cshape = _first(k_cache, "k_cache", _CACHE)[1]
    pages, page, Hkv, D = cshape
    N = shape[0]
    B, width = _table(page_table)
    shape = torch.Size((N, Hkv, D))
    a = _lib.PagedAppendArgs(B, N, Hkv, D, pages, page, width, _DTYPES[dtype], _ptr(k, "k", dtype, shape, index),
                             _given(v, "v", dtype, shape, index), _ptr(k_cache, "k_cache", dtype, cshape, index),
                             _given(v_cache, "v_cache", dtype, cshape, index), *_places(page_table, cu_q, kv_len, B, width, index))
    _run(_lib.load().rsm_paged_append, a, index)


def _table(page_table):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a CUDA tensor [B, width]")
    _ints(page_table, "page_table")
    return page_table.shape


def _places(page_table, cu_q, kv_len, B, width, index):
    i32 = torch.int32
    return (_ptr(page_table, "page_table", i32, page_table.shape, index), _given(cu_q, "cu_q", i32, torch.Size((B + 1,)), index),
            _given(kv_len, "kv_len", i32, torch.Size((B,)), index))


def paged_forward(q, k_cache, v_cache, page_table, cu_q, kv_len, max_q: int, *, window: int = 0, sinks: int = 0,
                  scale=None, lse: bool = False, validate: bool = False, out=None, workspace=None):
    """Attention of the new tokens q [N,H,D] over the cache, which holds their keys and values already
    (paged_append). No sequence has more than `max_q` new tokens; 1 is a generation step. window = 0
    sees every earlier place, else the last `window` and the first `sinks`.

    Returns dict(o [N,H,D] in q's dtype, lse [N,H] fp32 or None); a row that sees nothing gets zeros.
    device_status() reports pages and lengths outside the cache. Pages that nothing sees are not looked up:
    behind a window they may have been given back."""
    dtype, shape, index = _first(q, "q", "NHD")
    cshape = _first(k_cache, "k_cache", _CACHE)[1]
    pages, page, Hkv, D = cshape
    N, H, _ = shape
    B, width = _table(page_table)
    qp = _ptr(q, "q", dtype, torch.Size((N, H, D)), index)
    o = ls = None
    if out:
        o, ls = out.get("o"), out.get("lse")
    if o is None:
        o = torch.empty_like(q)
    if ls is None and lse:
        ls = torch.empty(N, H, dtype=torch.float32, device=q.device)
    a = _lib.PagedArgs(B, N, _int(max_q), H, Hkv, D, pages, page, width, _int(window), _int(sinks), _DTYPES[dtype],
                       _scale(scale, D), qp, _ptr(k_cache, "k_cache", dtype, cshape, index),
                       _given(v_cache, "v_cache", dtype, cshape, index), *_places(page_table, cu_q, kv_len, B, width, index),
                       _ptr(o, "o", dtype, shape, index), _ptr(ls, "lse", torch.float32, shape[:2], index))
    if validate:
        a.flags = _lib.RSM_FLAG_VALIDATE
    L = _lib.load()
    _run(L.rsm_paged_forward, a, index, L.rsm_paged_workspace_size, workspace)
    return {"o": o, "lse": ls}


# ----------------------------------------------------------------------------------- block norms
def _norm_args(cls, y, gate, residual, w_post, w_pre, act, scale, eps):
    dtype, shape, index = _first(residual, "residual", None)
    if not shape:
        raise ValueError("residual must have at least one dimension")
    d = shape[-1]
    ty = _first(y, "y", None)[0]
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    w = torch.Size((d,))
    a = cls(residual.numel() // d if d else 0, d, _DTYPES[ty], _DTYPES[dtype], code, float(scale), float(eps),
            _ptr(y, "y", ty, shape, index), _ptr(gate, "gate", dtype, shape, index),
            _ptr(residual, "residual", dtype, shape, index), _given(w_post, "w_post", torch.float32, w, index),
            _ptr(w_pre, "w_pre", torch.float32, w, index))
    return a, dtype, shape, index


def block_norm_forward(y, gate, residual, w_post, w_pre=None, *, act: str = "silu", scale: float = 1.0,
                       eps: float = 1e-6, out=None):
    """h = residual + scale rmsnorm(y) w_post act(gate) and x = rmsnorm(h) w_pre over the last axis d.
    y is float32 or of residual's dtype; gate may be None; w_post, w_pre are float32 [d]; without w_pre
    there is no x. Returns dict(h, x) in residual's dtype. `out` may supply them."""
    a, dtype, shape, index = _norm_args(_lib.BlockNormArgs, y, gate, residual, w_post, w_pre, act, scale, eps)
    h = x = None
    if out:
        h, x = out.get("h"), out.get("x")
    if h is None:
        h = torch.empty_like(residual)
    if w_pre is None:
        x = None
    elif x is None:
        x = torch.empty_like(residual)
    a.h, a.x = _ptr(h, "h", dtype, shape, index), _ptr(x, "x", dtype, shape, index)
    _run(_lib.load().rsm_block_norm_forward, a, index)
    return {"h": h, "x": x}


def block_norm_backward(y, gate, residual, w_post, w_pre=None, dh=None, dx=None, *, act: str = "silu",
                        scale: float = 1.0, eps: float = 1e-6, need=(True, True, True, True, True), out=None,
                        workspace=None):
    """Gradients of block_norm_forward from dh and dx (residual's dtype; None = zero). Returns dict(dy,
    dgate, dresidual, dw_post, dw_pre), None where there is no input or `need` says so."""
    a, dtype, shape, index = _norm_args(_lib.BlockNormBackwardArgs, y, gate, residual, w_post, w_pre, act, scale, eps)
    a.dh, a.dx = _ptr(dh, "dh", dtype, shape, index), _ptr(dx, "dx", dtype, shape, index)
    got = {}
    for name, like, wanted in zip(("dy", "dgate", "dresidual", "dw_post", "dw_pre"), (y, gate, residual, w_post, w_pre),
                                  need):
        g = None
        if wanted and like is not None:
            g = out.get(name) if out else None
            if g is None:
                g = torch.empty_like(like)
            setattr(a, name, _ptr(g, name, like.dtype, like.shape, index))
        got[name] = g
    L = _lib.load()
    _run(L.rsm_block_norm_backward, a, index, L.rsm_block_norm_backward_workspace_size, workspace)
    return got


class BlockNormFunction(torch.autograd.Function):
    """The block norms as an autograd function: apply(y, gate, residual, w_post, w_pre, act="silu",
    scale=1.0, eps=1e-6) -> (h, x). Capturing it into a CUDA graph: see WindowFunction."""

    @staticmethod
    def forward(ctx, y, gate, residual, w_post, w_pre, act="silu", scale=1.0, eps=1e-6):
        r = block_norm_forward(y, gate, residual, w_post, w_pre, act=act, scale=scale, eps=eps)
        ctx.save_for_backward(y, gate, residual, w_post, w_pre)
        ctx.how = dict(act=act, scale=scale, eps=eps)
        ctx.set_materialize_grads(False)
        return r["h"], r["x"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dx):
        g = block_norm_backward(*ctx.saved_tensors, dh=gradient(dh), dx=gradient(dx), need=ctx.needs_input_grad[:5], **ctx.how)
        return g["dy"], g["dgate"], g["dresidual"], g["dw_post"], g["dw_pre"], None, None, None
