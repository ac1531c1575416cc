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
from .api import _DTYPES, _need, _stream

_NO_SIZE = ctypes.c_size_t(-1).value
_ACTS = {"silu": _lib.RSM_ACT_SILU, "sigmoid": _lib.RSM_ACT_SIGMOID}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
    return _DTYPES[t.dtype]


def _call(fn, args, dev):
    """Runs a library call on the device's current stream, with that device current."""
    if dev.index == torch.cuda.current_device():
        _lib.check(fn(ctypes.byref(args), _stream(dev)))
    else:
        with torch.cuda.device(dev):
            _lib.check(fn(ctypes.byref(args), _stream(dev)))


def _workspace(size_fn, fn, args, dev, workspace):
    """Fills args.workspace: the caller's (a uint8 tensor) where it is large enough, else a new one.
    Returns the tensor, which has to live until the call is queued."""
    if dev.index == torch.cuda.current_device():
        need = size_fn(ctypes.byref(args))
    else:
        with torch.cuda.device(dev):
            need = size_fn(ctypes.byref(args))
    if need == _NO_SIZE:
        _lib.check(fn(ctypes.byref(args), None))  # raises with the reason
    if need:
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _need(workspace, "workspace", torch.uint8)
            _same_device(dev, workspace=workspace)
        args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return workspace


def _fill(a, **kw):
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def _scale(scale, D):
    return 1.0 / math.sqrt(D) if scale is None else float(scale)


# ------------------------------------------------------------------------------ window attention
def _window_args(a, q, k, v, window, sinks, scale, validate):
    dt = _dtype(q, "q")
    _need(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must be [B,T,H,D], got {tuple(q.shape)}")
    B, T, H, D = q.shape
    _need(k, "k", q.dtype)
    if k.dim() != 4:
        raise ValueError(f"k must be [B,T,Hkv,D], got {tuple(k.shape)}")
    Hkv = k.shape[2]
    _need(k, "k", shape=(B, T, Hkv, D))
    _need(v, "v", q.dtype, (B, T, Hkv, D))
    _same_device(q.device, k=k, v=v)
    # a window longer than the sequence is the whole sequence; the C int holds no more than 2^31 - 1
    return _fill(a, B=B, T=T, H=H, Hkv=Hkv, D=D, window=min(int(window), 2**31 - 1), sinks=min(int(sinks), 2**31 - 1),
                 dtype=dt, scale=_scale(scale, D), q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(),
                 flags=_lib.RSM_FLAG_VALIDATE if validate else 0)


def window_forward(q, k, v, window: int, sinks: int = 0, scale=None, *, lse: bool = False, validate: bool = False,
                   out=None):
    """Causal attention over the last `window` keys and the first `sinks`. q [B,T,H,D]; k, v
    [B,T,Hkv,D] with Hkv dividing H; float32 or bfloat16. scale defaults to 1/sqrt(D).

    Returns dict(o [B,T,H,D] in q's dtype, lse [B,T,H] fp32 or None). `out` may supply preallocated
    tensors under the same keys."""
    a = _window_args(_lib.WindowArgs(), q, k, v, window, sinks, scale, validate)
    out = out or {}
    o, ls = out.get("o"), out.get("lse")
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, q.shape)
    if ls is not None:
        _need(ls, "lse", torch.float32, q.shape[:3])
    elif lse:
        ls = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    _same_device(q.device, o=o, lse=ls)
    a.o, a.lse = o.data_ptr(), _ptr(ls)
    _call(_lib.load().rsm_window_forward, a, q.device)
    return {"o": o, "lse": ls}


def window_backward(q, k, v, o, lse, dO, window: int, sinks: int = 0, scale=None, *, need=(True, True, True),
                    validate: bool = False, out=None, workspace=None):
    """Gradients of window_forward: its inputs, its o and lse, and dO [B,T,H,D] in q's dtype.
    Returns dict(dq, dk, dv) in q's dtype (None where `need` says so)."""
    a = _window_args(_lib.WindowBackwardArgs(), q, k, v, window, sinks, scale, validate)
    _need(o, "o", q.dtype, q.shape)
    _need(lse, "lse", torch.float32, q.shape[:3])
    _need(dO, "dO", q.dtype, q.shape)
    out = dict(out or {})
    for name, like, wanted in zip(("dq", "dk", "dv"), (q, k, v), need):
        if not wanted:
            out[name] = None
            continue
        if out.get(name) is None:
            out[name] = torch.empty_like(like)
        _need(out[name], name, like.dtype, like.shape)
        setattr(a, name, out[name].data_ptr())
    _same_device(q.device, o=o, lse=lse, dO=dO, **out)
    a.o, a.lse, a.dO = o.data_ptr(), lse.data_ptr(), dO.data_ptr()
    L = _lib.load()
    ws = _workspace(L.rsm_window_backward_workspace_size, L.rsm_window_backward, a, q.device, workspace)
    _call(L.rsm_window_backward, a, q.device)
    del ws
    return out


class WindowFunction(torch.autograd.Function):
    """Window attention as an autograd function: apply(q, k, v, window, sinks=0, scale=None) -> o.

    Recording a training step into a CUDA graph follows torch's own rule: no graph of the same
    leaves built outside the capture may be alive meanwhile, or the capture fails. window_forward and
    window_backward carry no such state."""

    @staticmethod
    def forward(ctx, q, k, v, window, sinks=0, scale=None):
        r = window_forward(q, k, v, window, sinks, scale, lse=True)
        ctx.save_for_backward(q, k, v, r["o"], r["lse"])
        ctx.how = (window, sinks, scale)
        return r["o"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        q, k, v, o, lse = ctx.saved_tensors
        g = window_backward(q, k, v, o, lse, dO.contiguous(), *ctx.how, need=ctx.needs_input_grad[:3])
        return g["dq"], g["dk"], g["dv"], None, None, None


# ------------------------------------------------------------------------------- paged attention
def _cache_args(a, new, k_cache, v_cache, page_table, cu_q, kv_len):
    _need(k_cache, "k_cache", new.dtype)
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be [pages, page_size, Hkv, D], got {tuple(k_cache.shape)}")
    pages, page, Hkv, D = k_cache.shape
    _need(v_cache, "v_cache", new.dtype, k_cache.shape)
    _need(page_table, "page_table", torch.int32)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [B, width], got {tuple(page_table.shape)}")
    B = page_table.shape[0]
    _need(cu_q, "cu_q", torch.int32, (B + 1,))
    _need(kv_len, "kv_len", torch.int32, (B,))
    _same_device(new.device, k_cache=k_cache, v_cache=v_cache, page_table=page_table, cu_q=cu_q, kv_len=kv_len)
    return _fill(a, B=B, N=new.shape[0], Hkv=Hkv, D=D, num_pages=pages, page_size=page, table_width=page_table.shape[1],
                 dtype=_dtype(new, "q or k"), k_cache=k_cache.data_ptr(), v_cache=v_cache.data_ptr(),
                 page_table=page_table.data_ptr(), cu_q=cu_q.data_ptr(), kv_len=kv_len.data_ptr())


def paged_append(k, v, k_cache, v_cache, page_table, cu_q, kv_len) -> None:
    """Writes the new tokens' keys and values (k, v [N,Hkv,D]; sequence b's are rows cu_q[b] ..
    cu_q[b+1]-1) to places kv_len[b] - n_b .. kv_len[b] - 1 of the caches [pages, page_size, Hkv, D],
    in place. page_table int32 [B, width], cu_q int32 [B+1], kv_len int32 [B] (new tokens included)."""
    _dtype(k, "k")
    _need(k, "k")
    a = _cache_args(_lib.PagedAppendArgs(), k, k_cache, v_cache, page_table, cu_q, kv_len)
    _need(k, "k", shape=(k.shape[0], a.Hkv, a.D))
    _need(v, "v", k.dtype, k.shape)
    _same_device(k.device, v=v)
    a.k, a.v = k.data_ptr(), v.data_ptr()
    _call(_lib.load().rsm_paged_append, a, k.device)


def paged_forward(q, k_cache, v_cache, page_table, cu_q, kv_len, max_q: int, *, window: int = 0, sinks: int = 0,
                  scale=None, lse: bool = False, validate: bool = False, out=None, workspace=None):
    """Attention of the new tokens q [N,H,D] over the cache, which holds their keys and values already
    (paged_append). No sequence has more than `max_q` new tokens; 1 is a generation step. window = 0
    sees every earlier place, else the last `window` and the first `sinks`.

    Returns dict(o [N,H,D] in q's dtype, lse [N,H] fp32 or None); a row that sees nothing gets zeros.
    device_status() reports pages and lengths outside the cache."""
    _dtype(q, "q")
    _need(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [N,H,D], got {tuple(q.shape)}")
    a = _cache_args(_lib.PagedArgs(), q, k_cache, v_cache, page_table, cu_q, kv_len)
    N, H, D = q.shape
    _need(q, "q", shape=(N, H, a.D))
    out = out or {}
    o, ls = out.get("o"), out.get("lse")
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, "o", q.dtype, q.shape)
    if ls is not None:
        _need(ls, "lse", torch.float32, (N, H))
    elif lse:
        ls = torch.empty(N, H, dtype=torch.float32, device=q.device)
    _same_device(q.device, o=o, lse=ls)
    _fill(a, max_q=int(max_q), H=H, window=min(int(window), 2**31 - 1), sinks=min(int(sinks), 2**31 - 1),
          scale=_scale(scale, D), q=q.data_ptr(), o=o.data_ptr(), lse=_ptr(ls),
          flags=_lib.RSM_FLAG_VALIDATE if validate else 0)
    L = _lib.load()
    ws = _workspace(L.rsm_paged_workspace_size, L.rsm_paged_forward, a, q.device, workspace)
    _call(L.rsm_paged_forward, a, q.device)
    del ws
    return {"o": o, "lse": ls}


# ----------------------------------------------------------------------------------- block norms
def _norm_args(a, y, gate, residual, w_post, w_pre, act, scale, eps):
    dt = _dtype(residual, "residual")
    _need(residual, "residual")
    if residual.dim() < 1:
        raise ValueError("residual must have at least one dimension")
    d = residual.shape[-1]
    ty = _dtype(y, "y")
    _need(y, "y", shape=residual.shape)
    if gate is not None:
        _need(gate, "gate", residual.dtype, residual.shape)
    _need(w_post, "w_post", torch.float32, (d,))
    if w_pre is not None:
        _need(w_pre, "w_pre", torch.float32, (d,))
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    _same_device(residual.device, y=y, gate=gate, w_post=w_post, w_pre=w_pre)
    return _fill(a, rows=residual.numel() // d if d else 0, d=d, y_dtype=ty, dtype=dt, act=_ACTS[act],
                 scale=float(scale), eps=float(eps), y=y.data_ptr(), gate=_ptr(gate), residual=residual.data_ptr(),
                 w_post=w_post.data_ptr(), w_pre=_ptr(w_pre))


def block_norm_forward(y, gate, residual, w_post, w_pre=None, *, act: str = "silu", scale: float = 1.0,
                       eps: float = 1e-6, out=None):
    """h = residual + scale rmsnorm(y) w_post act(gate) and x = rmsnorm(h) w_pre over the last axis d.
    y is float32 or of residual's dtype; gate may be None; w_post, w_pre are float32 [d]; without w_pre
    there is no x. Returns dict(h, x) in residual's dtype. `out` may supply them."""
    a = _norm_args(_lib.BlockNormArgs(), y, gate, residual, w_post, w_pre, act, scale, eps)
    out = out or {}
    h, x = out.get("h"), out.get("x")
    if h is None:
        h = torch.empty_like(residual)
    else:
        _need(h, "h", residual.dtype, residual.shape)
    if w_pre is None:
        x = None
    elif x is None:
        x = torch.empty_like(residual)
    else:
        _need(x, "x", residual.dtype, residual.shape)
    _same_device(residual.device, h=h, x=x)
    a.h, a.x = h.data_ptr(), _ptr(x)
    _call(_lib.load().rsm_block_norm_forward, a, residual.device)
    return {"h": h, "x": x}


def block_norm_backward(y, gate, residual, w_post, w_pre=None, dh=None, dx=None, *, act: str = "silu",
                        scale: float = 1.0, eps: float = 1e-6, need=(True, True, True, True, True), out=None,
                        workspace=None):
    """Gradients of block_norm_forward from dh and dx (residual's dtype; None = zero). Returns dict(dy,
    dgate, dresidual, dw_post, dw_pre), None where there is no input or `need` says so."""
    a = _norm_args(_lib.BlockNormBackwardArgs(), y, gate, residual, w_post, w_pre, act, scale, eps)
    for name, t in (("dh", dh), ("dx", dx)):
        if t is not None:
            _need(t, name, residual.dtype, residual.shape)
            setattr(a, name, t.data_ptr())
    out = dict(out or {})
    for name, like, wanted in zip(("dy", "dgate", "dresidual", "dw_post", "dw_pre"), (y, gate, residual, w_post, w_pre),
                                  need):
        if not wanted or like is None:
            out[name] = None
            continue
        if out.get(name) is None:
            out[name] = torch.empty_like(like)
        _need(out[name], name, like.dtype, like.shape)
        setattr(a, name, out[name].data_ptr())
    _same_device(residual.device, dh=dh, dx=dx, **out)
    L = _lib.load()
    ws = _workspace(L.rsm_block_norm_backward_workspace_size, L.rsm_block_norm_backward, a, residual.device, workspace)
    _call(L.rsm_block_norm_backward, a, residual.device)
    del ws
    return out


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
        g = block_norm_backward(*ctx.saved_tensors, dh=None if dh is None else dh.contiguous(),
                                dx=None if dx is None else dx.contiguous(), need=ctx.needs_input_grad[:5], **ctx.how)
        return g["dy"], g["dgate"], g["dresidual"], g["dw_post"], g["dw_pre"], None, None, None
