"""Binding of the layer operators (include/mgs_layers.h): linear attention with a
decay per head, the root-mean-square norm with the residual's addition, and the
global gradient norm with clipping.

As in the package's other functions, each carries the name of the C entry point
that it calls and only marshals arguments; there is no fallback path.
"""
from __future__ import annotations

import ctypes

from ._lib import LinattnDesc, check, load

__all__ = [
    "mgs_linattn_workspace_size", "mgs_linattn_fwd", "mgs_linattn_bwd", "mgs_linattn_step",
    "mgs_rmsnorm_fwd", "mgs_rmsnorm_fwd_fp8", "mgs_rmsnorm_workspace_size", "mgs_rmsnorm_bwd",
    "mgs_clip_norm_workspace_size", "mgs_clip_norm",
]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _dtype(dtype):
    import torch
    if dtype is torch.bfloat16:
        return 1
    if dtype is torch.float32:
        return 0
    raise TypeError(f"elements must be float32 or bfloat16, got {dtype}")


DENSE, LAST, ANY = 0, 1, 2   # what of a tensor has to be contiguous: all of it, its last dimension, nothing


def _tensor(name, t, shape, dtype, device, dense=DENSE):
    """Raises unless t is what it should be; the tests are few while it is."""
    if (t is not None and t.dtype is dtype and t.device == device and t.is_cuda and t.shape == shape and
            (t.is_contiguous() if dense == DENSE else dense == ANY or t.stride(-1) == 1 or t.shape[-1] <= 1)):
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor (no CPU path exists)")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous" + ("" if dense == DENSE else " in its last dimension"))


def _out(name, t, shape, dtype, device):
    import torch
    if t is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    _tensor(name, t, shape, dtype, device)
    return t


def _scratch(ws, nbytes, device):
    """ws, or a new workspace of nbytes() bytes (the operators here need no zero-fill)."""
    import torch
    if ws is None:
        return torch.empty(max(nbytes(), 256), dtype=torch.uint8, device=device)
    _tensor("ws", ws, ws.shape, torch.uint8, device)
    return ws


# ------------------------------------------------------- linear attention

_NONE = (0, 0, 0)   # strides that are not read


def _step_strides(t):
    st = t.stride()
    return st[0], 0, st[1]


def mgs_linattn_workspace_size(B, T, H, Hk, dk, dv, dtype=None, backward=False):
    """Bytes, with backward=True enough for the forward and the backward; dtype (the inputs') defaults to float32."""
    import torch
    out = ctypes.c_size_t(0)
    d = LinattnDesc(B, T, H, Hk, dk, dv, _dtype(dtype or torch.float32), 0, 1.0)
    check(load().mgs_linattn_workspace_size(ctypes.byref(d), int(bool(backward)), ctypes.byref(out)),
          "mgs_linattn_workspace_size")
    return int(out.value)


def _attn_inputs(q, k, v, g, S0, lengths):
    """Checks the inputs of a whole-sequence call; (B, T, H, Hk, dk, dv), per-head decay?"""
    import torch
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k must be (B,T,Hk,dk) and v (B,T,H,dv)")
    (B, T, H, dv), (Hk, dk), dev = v.shape, q.shape[2:], v.device
    _tensor("v", v, (B, T, H, dv), v.dtype, dev, dense=LAST)
    _tensor("q", q, (B, T, Hk, dk), v.dtype, dev, dense=LAST)
    _tensor("k", k, (B, T, Hk, dk), v.dtype, dev, dense=LAST)
    per_head = g is not None and g.dim() == 1
    _tensor("g", g, (H,) if per_head else (B, T, H), torch.float32, dev, dense=DENSE if per_head else ANY)
    if S0 is not None:
        _tensor("S0", S0, (B, H, dv, dk), torch.float32, dev)
    if lengths is not None:
        _tensor("lengths", lengths, (B,), torch.int32, dev)
    return (B, T, H, Hk, dk, dv), per_head


def mgs_linattn_fwd(q, k, v, g, S0=None, lengths=None, scale=1.0, o=None, ST=None, ws=None, want_state=True,
                    stream=None):
    """(o (B,T,H,dv), S_T (B,H,dv,dk) or None, ws) of S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t
    per sequence and head.

    q, k (B,T,Hk,dk) and v (B,T,H,dv), float32 or bfloat16, dense in the last dimension only (views of one
    projection do); query/key head h // (H / Hk) serves head h.  g: log decays, float32, (B,T,H) or (H,).
    S0 (B,H,dv,dk) float32 or None (zeros).  lengths (B,) int32 or None: later steps are not read, leave the
    state as it is and give zeros."""
    import torch
    dims, per_head = _attn_inputs(q, k, v, g, S0, lengths)
    B, T, H, Hk, dk, dv = dims
    dev = v.device
    o = _out("o", o, (B, T, H, dv), v.dtype, dev)
    if ST is not None or want_state:
        ST = _out("ST", ST, (B, H, dv, dk), torch.float32, dev)
    d = LinattnDesc(*dims, _dtype(v.dtype), per_head, scale, q.stride()[:3], k.stride()[:3], v.stride()[:3], _NONE,
                    _NONE if per_head else g.stride())
    ws = _scratch(ws, lambda: mgs_linattn_workspace_size(*dims, dtype=v.dtype), dev)
    check(load().mgs_linattn_fwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(lengths),
                                 _ptr(o), _ptr(ST), _ptr(ws), ws.numel(), _stream(stream)), "mgs_linattn_fwd")
    return o, ST, ws


def mgs_linattn_bwd(q, k, v, g, do, S0=None, dST=None, lengths=None, scale=1.0, out=None, ws=None, stream=None):
    """(dq, dk, dv, dg, dS0) for L = sum(do * o) + sum(dST * S_T); dg and, with decays per head, its sum over
    sequences and steps are float32, and so is dS0 (B,H,dv,dk).  do (B,T,H,dv) may be strided as v may.
    out: the five outputs, dense (dS0 may be None there)."""
    import torch
    dims, per_head = _attn_inputs(q, k, v, g, S0, lengths)
    B, T, H, Hk, dk, dv = dims
    dev = v.device
    _tensor("do", do, (B, T, H, dv), v.dtype, dev, dense=LAST)
    if dST is not None:
        _tensor("dST", dST, (B, H, dv, dk), torch.float32, dev)
    dq, dk_, dv_, dg, dS0 = out if out is not None else (None,) * 5
    dq = _out("dq", dq, (B, T, Hk, dk), v.dtype, dev)
    dk_ = _out("dk", dk_, (B, T, Hk, dk), v.dtype, dev)
    dv_ = _out("dv", dv_, (B, T, H, dv), v.dtype, dev)
    dg = _out("dg", dg, tuple(g.shape), torch.float32, dev)
    if out is None or dS0 is not None:
        dS0 = _out("dS0", dS0, (B, H, dv, dk), torch.float32, dev)
    d = LinattnDesc(*dims, _dtype(v.dtype), per_head, scale, q.stride()[:3], k.stride()[:3], v.stride()[:3],
                    do.stride()[:3], _NONE if per_head else g.stride())
    ws = _scratch(ws, lambda: mgs_linattn_workspace_size(*dims, dtype=v.dtype, backward=True), dev)
    check(load().mgs_linattn_bwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(do), _ptr(S0), _ptr(dST),
                                 _ptr(lengths), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(dS0), _ptr(ws),
                                 ws.numel(), _stream(stream)), "mgs_linattn_bwd")
    return dq, dk_, dv_, dg, dS0


def mgs_linattn_step(q, k, v, g, S, slots=None, scale=1.0, o=None, stream=None):
    """o (B,H,dv) of one step for each of B sequences; S (n_slots,H,dv,dk) float32 is updated in place.

    q, k (B,Hk,dk), v (B,H,dv), g (B,H) or (H,).  slots (B,) int32: the state of sequence b is S[slots[b]]
    (None: S[b]); the slots of a call are distinct, and one outside S (-1) is idle: zeros out, no state touched."""
    import torch
    if v.dim() != 3 or q.dim() != 3:
        raise ValueError("q, k must be (B,Hk,dk) and v (B,H,dv)")
    (B, H, dv), (Hk, dk), dev = v.shape, q.shape[1:], v.device
    _tensor("v", v, (B, H, dv), v.dtype, dev, dense=LAST)
    _tensor("q", q, (B, Hk, dk), v.dtype, dev, dense=LAST)
    _tensor("k", k, (B, Hk, dk), v.dtype, dev, dense=LAST)
    per_head = g is not None and g.dim() == 1
    _tensor("g", g, (H,) if per_head else (B, H), torch.float32, dev, dense=DENSE if per_head else ANY)
    _tensor("S", S, (S.shape[0], H, dv, dk), torch.float32, dev)
    if slots is not None:
        _tensor("slots", slots, (B,), torch.int32, dev)
    o = _out("o", o, (B, H, dv), v.dtype, dev)
    d = LinattnDesc(B, 1, H, Hk, dk, dv, _dtype(v.dtype), per_head, scale, _step_strides(q), _step_strides(k),
                    _step_strides(v), _NONE, _NONE if per_head else _step_strides(g))
    check(load().mgs_linattn_step(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S), S.shape[0],
                                  _ptr(slots), _ptr(o), _stream(stream)), "mgs_linattn_step")
    return o


# ------------------------------------------------------------------- norm

def _rows(name, t, d, dtype, device):
    """A (..., d) tensor as a row stride: rows evenly spaced, dense within."""
    if t.dim() < 1 or t.shape[-1] != d:
        raise ValueError(f"{name} must end in {d}, got {tuple(t.shape)}")
    _tensor(name, t, t.shape, dtype, device, dense=LAST)
    if t.dim() == 2:
        return t.stride(0)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous or two-dimensional")
    return d


def _norm_inputs(x, w, residual):
    d, dev = x.shape[-1], x.device
    _dtype(x.dtype)
    xs = _rows("x", x, d, x.dtype, dev)
    _tensor("w", w, (d,), x.dtype, dev)
    rs = d
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
        rs = _rows("residual", residual, d, x.dtype, dev)
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    return rows, d, xs, rs


def mgs_rmsnorm_fwd(x, w, residual=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """(y, h, rstd) of h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w over the last dimension.

    x, residual (...,d), w (d,), float32 or bfloat16; rstd float32, one for each row.  Without a residual h is x
    itself, not a copy, unless a buffer is passed.  h may be the residual's (or x's) own dense tensor."""
    import torch
    rows, d, xs, rs = _norm_inputs(x, w, residual)
    dev = x.device
    y = _out("y", y, x.shape, x.dtype, dev)
    write_h = h is not None or residual is not None or not x.is_contiguous()
    h_out = _out("h", h, x.shape, x.dtype, dev) if write_h else None
    rstd = _out("rstd", rstd, x.shape[:-1], torch.float32, dev)
    check(load().mgs_rmsnorm_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(h_out), _ptr(rstd), rows, d, xs, rs,
                                 float(eps), _dtype(x.dtype), _stream(stream)), "mgs_rmsnorm_fwd")
    return y, (h_out if write_h else x), rstd


def mgs_rmsnorm_fwd_fp8(x, w, residual=None, eps=1e-6, group=0, y=None, scale=None, h=None, stream=None):
    """(y, scale, h): the norm with y in float8_e4m3fn and a float32 scale for each row (group = 0; scale (...,1)) or
    for each 128 columns (group = 128; scale (..., ceil(d / 128))); y * scale stands for the norm's output."""
    import torch
    rows, d, xs, rs = _norm_inputs(x, w, residual)
    dev = x.device
    y = _out("y", y, x.shape, torch.float8_e4m3fn, dev)
    n_scales = -(-d // group) if group else 1
    scale = _out("scale", scale, (*x.shape[:-1], n_scales), torch.float32, dev)
    write_h = h is not None or residual is not None or not x.is_contiguous()
    h_out = _out("h", h, x.shape, x.dtype, dev) if write_h else None
    check(load().mgs_rmsnorm_fwd_fp8(_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(scale), _ptr(h_out), rows, d, xs,
                                     rs, float(eps), int(group), _dtype(x.dtype), _stream(stream)),
          "mgs_rmsnorm_fwd_fp8")
    return y, scale, (h_out if write_h else x)


def mgs_rmsnorm_workspace_size(rows, d):
    out = ctypes.c_size_t(0)
    check(load().mgs_rmsnorm_workspace_size(int(rows), int(d), ctypes.byref(out)), "mgs_rmsnorm_workspace_size")
    return int(out.value)


def mgs_rmsnorm_bwd(dy, h, w, rstd, dh=None, dx=None, dw=None, ws=None, stream=None):
    """(dx, dw) for L = sum(dy * y) + sum(dh * h), from the forward's h and rstd; dx is the gradient of x and of the
    residual alike, dw (d,) float32.  dx may be dy's or dh's own tensor."""
    import torch
    d, dev = h.shape[-1], h.device
    _tensor("h", h, h.shape, h.dtype, dev)
    _tensor("dy", dy, h.shape, h.dtype, dev)
    _tensor("w", w, (d,), h.dtype, dev)
    _tensor("rstd", rstd, h.shape[:-1], torch.float32, dev)
    if dh is not None:
        _tensor("dh", dh, h.shape, h.dtype, dev)
    dx = _out("dx", dx, h.shape, h.dtype, dev)
    dw = _out("dw", dw, (d,), torch.float32, dev)
    rows = rstd.numel()   # one for each row of h
    ws = _scratch(ws, lambda: mgs_rmsnorm_workspace_size(rows, d), dev)
    check(load().mgs_rmsnorm_bwd(_ptr(dy), _ptr(h), _ptr(w), _ptr(rstd), _ptr(dh), _ptr(dx), _ptr(dw), rows, d,
                                 _dtype(h.dtype), _ptr(ws), ws.numel(), _stream(stream)), "mgs_rmsnorm_bwd")
    return dx, dw


# --------------------------------------------------------------- clipping

def _sizes(sizes):
    n = len(sizes)
    return n, (ctypes.c_int64 * max(n, 1))(*sizes)


def mgs_clip_norm_workspace_size(sizes):
    """sizes: element counts of the tensors."""
    n, arr = _sizes([int(s) for s in sizes])
    out = ctypes.c_size_t(0)
    check(load().mgs_clip_norm_workspace_size(n, arr, ctypes.byref(out)), "mgs_clip_norm_workspace_size")
    return int(out.value)


def mgs_clip_norm(tensors, max_norm=None, out=None, norm=None, ws=None, stream=None):
    """(norm (1,) float32 on the GPU, tensors scaled by min(1, max_norm / (norm + 1e-6))).

    tensors: contiguous, float32 or bfloat16 or both, any shapes.  out: tensors of the same shapes and types, or
    None to scale in place.  max_norm None: only the norm (second value None).  A norm that is not finite leaves
    the values as they are."""
    import torch
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    dev = tensors[0].device
    for i, t in enumerate(tensors):
        _dtype(t.dtype)
        _tensor(f"tensors[{i}]", t, t.shape, t.dtype, dev)
    outs = None
    if max_norm is not None:
        outs = tensors if out is None else list(out)
        if len(outs) != len(tensors):
            raise ValueError(f"out has {len(outs)} tensors, expected {len(tensors)}")
        if out is not None:
            for i, (o, t) in enumerate(zip(outs, tensors)):
                _tensor(f"out[{i}]", o, t.shape, t.dtype, dev)
    elif out is not None:
        raise ValueError("out needs max_norm")
    norm = _out("norm", norm, (1,), torch.float32, dev)
    counts = [t.numel() for t in tensors]
    n, sizes = _sizes(counts)
    ws = _scratch(ws, lambda: mgs_clip_norm_workspace_size(counts), dev)
    pointers = ctypes.c_void_p * n
    ins = pointers(*[t.data_ptr() for t in tensors])
    outp = pointers(*[t.data_ptr() for t in outs]) if outs is not None else None
    dtypes = (ctypes.c_int * n)(*[_dtype(t.dtype) for t in tensors])
    check(load().mgs_clip_norm(n, ins, outp, sizes, dtypes, 0.0 if max_norm is None else float(max_norm), _ptr(norm),
                               _ptr(ws), ws.numel(), _stream(stream)), "mgs_clip_norm")
    return norm, outs
