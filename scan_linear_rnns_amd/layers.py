"""Binding of the layer operators (include/mgs_layers.h): linear attention with a
decay per head, the root-mean-square norm with the residual's addition, and the
global gradient norm with clipping.

As in the package's other functions, each carries the name of the C entry point
that it calls and only marshals arguments; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import struct
from array import array

from ._lib import LinattnDesc, check, load

__all__ = [
    "mgs_linattn_workspace_size", "mgs_linattn_fwd", "mgs_linattn_bwd", "mgs_linattn_step",
    "mgs_rmsnorm_fwd", "mgs_rmsnorm_fwd_fp8", "mgs_rmsnorm_workspace_size", "mgs_rmsnorm_bwd",
    "mgs_clip_norm_workspace_size", "mgs_clip_norm",
]

# A single step is a few microseconds of GPU work, so what a call does on the host shows: the checks below are few
# while everything is in order, and say what is wrong only once something is.


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(torch, dev):
    """The current stream of GPU `dev`, the current one, as a pointer."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on GPU {dev}, the current one is {torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _on(stream, call, *args):
    """call(*args) with `stream` current, so that what it allocates belongs to that stream: the allocator hands memory
    that is freed to later work of the stream it came from, which has to be the one that the kernels run on."""
    import torch
    with torch.cuda.stream(stream):
        return call(*args)


def _dtype(torch, dtype):
    if dtype is torch.bfloat16:
        return 1
    if dtype is torch.float32:
        return 0
    raise TypeError(f"elements must be float32 or bfloat16, got {dtype}")


DENSE, LAST, ANY = 0, 1, 2   # what of a tensor has to be contiguous: all of it, its last dimension, nothing


def _device(name, t):
    """Index of the GPU that t is on."""
    if t is None:
        raise ValueError(f"{name} is required")
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a GPU tensor (no CPU path exists)")
    return dev


def _tensor(name, t, shape, dtype, dev, dense=DENSE):
    """Raises unless t is what it should be."""
    if (t is not None and t.dtype is dtype and t.get_device() == dev and t.shape == shape and
            (t.is_contiguous() if dense == DENSE else dense == ANY or t.stride(-1) == 1 or t.shape[-1] <= 1)):
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if _device(name, t) != dev:
        raise ValueError(f"{name} is on {t.device}, expected GPU {dev}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous" + ("" if dense == DENSE else " in its last dimension"))


def _out(torch, name, t, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _tensor(name, t, shape, dtype, dev)
    return t


def _like(name, t, x):
    """t, or a new tensor of x's shape and type."""
    if t is None:
        return x.new_empty(x.shape)
    _tensor(name, t, x.shape, x.dtype, x.get_device())
    return t


def _scratch(torch, ws, nbytes, dev):
    """ws, or a new workspace of nbytes() bytes (the operators here need no zero-fill)."""
    if ws is None:
        return torch.empty(max(nbytes(), 256), dtype=torch.uint8, device=dev)
    _tensor("ws", ws, ws.shape, torch.uint8, dev)
    return ws


# ------------------------------------------------------- linear attention

_NONE = (0, 0, 0)   # strides that are not read
_pack_desc = struct.Struct("6q2if4x15q").pack   # mgs_linattn_desc
assert struct.calcsize("6q2if4x15q") == ctypes.sizeof(LinattnDesc)


def mgs_linattn_workspace_size(B, T, H, Hk, dk, dv, dtype=None, backward=False):
    """Bytes, with backward=True enough for the forward and the backward; dtype (the inputs') defaults to float32."""
    import torch
    out = ctypes.c_size_t(0)
    d = _pack_desc(B, T, H, Hk, dk, dv, _dtype(torch, dtype or torch.float32), 0, 1.0, *_NONE * 5)
    check(load().mgs_linattn_workspace_size(d, int(bool(backward)), ctypes.byref(out)), "mgs_linattn_workspace_size")
    return int(out.value)


def _attn_inputs(torch, q, k, v, g, S0, lengths):
    """Checks the inputs of a whole-sequence call; (B, T, H, Hk, dk, dv), GPU, per-head decay?"""
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k must be (B,T,Hk,dk) and v (B,T,H,dv)")
    B, T, H, dv = v.shape
    Hk, dk = q.shape[2:]
    dev, dt = _device("v", v), v.dtype
    _tensor("v", v, (B, T, H, dv), dt, dev, LAST)
    _tensor("q", q, (B, T, Hk, dk), dt, dev, LAST)
    _tensor("k", k, (B, T, Hk, dk), dt, dev, LAST)
    per_head = g is not None and g.dim() == 1
    _tensor("g", g, (H,) if per_head else (B, T, H), torch.float32, dev, DENSE if per_head else ANY)
    if S0 is not None:
        _tensor("S0", S0, (B, H, dv, dk), torch.float32, dev)
    if lengths is not None:
        _tensor("lengths", lengths, (B,), torch.int32, dev)
    return (B, T, H, Hk, dk, dv), dev, per_head


def mgs_linattn_fwd(q, k, v, g, S0=None, lengths=None, scale=1.0, o=None, ST=None, ws=None, want_state=True,
                    stream=None):
    """(o (B,T,H,dv), S_T (B,H,dv,dk) or None, ws) of S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t
    per sequence and head.

    q, k (B,T,Hk,dk) and v (B,T,H,dv), float32 or bfloat16, dense in the last dimension only (views of one
    projection do); query/key head h // (H / Hk) serves head h.  g: log decays, float32, (B,T,H) or (H,).
    S0 (B,H,dv,dk) float32 or None (zeros).  lengths (B,) int32 or None: later steps are not read, leave the
    state as it is and give zeros."""
    if stream is not None:
        return _on(stream, mgs_linattn_fwd, q, k, v, g, S0, lengths, scale, o, ST, ws, want_state)
    import torch
    dims, dev, per_head = _attn_inputs(torch, q, k, v, g, S0, lengths)
    B, T, H, Hk, dk, dv = dims
    o = _like("o", o, v)
    if ST is not None or want_state:
        ST = _out(torch, "ST", ST, (B, H, dv, dk), torch.float32, dev)
    d = _pack_desc(*dims, _dtype(torch, v.dtype), per_head, scale, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3],
                   *_NONE, *(_NONE if per_head else g.stride()))
    ws = _scratch(torch, ws, lambda: mgs_linattn_workspace_size(*dims, dtype=v.dtype), dev)
    check(load().mgs_linattn_fwd(d, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(lengths), _ptr(o), _ptr(ST),
                                 _ptr(ws), ws.numel(), _raw_stream(torch, dev)), "mgs_linattn_fwd")
    return o, ST, ws


def mgs_linattn_bwd(q, k, v, g, do, S0=None, dST=None, lengths=None, scale=1.0, out=None, ws=None, stream=None):
    """(dq, dk, dv, dg, dS0) for L = sum(do * o) + sum(dST * S_T); dg and, with decays per head, its sum over
    sequences and steps are float32, and so is dS0 (B,H,dv,dk).  do (B,T,H,dv) may be strided as v may.
    out: the five outputs, dense (dS0 may be None there)."""
    if stream is not None:
        return _on(stream, mgs_linattn_bwd, q, k, v, g, do, S0, dST, lengths, scale, out, ws)
    import torch
    dims, dev, per_head = _attn_inputs(torch, q, k, v, g, S0, lengths)
    B, T, H, Hk, dk, dv = dims
    _tensor("do", do, (B, T, H, dv), v.dtype, dev, LAST)
    if dST is not None:
        _tensor("dST", dST, (B, H, dv, dk), torch.float32, dev)
    dq, dk_, dv_, dg, dS0 = out if out is not None else (None,) * 5
    dq = _out(torch, "dq", dq, (B, T, Hk, dk), v.dtype, dev)
    dk_ = _out(torch, "dk", dk_, (B, T, Hk, dk), v.dtype, dev)
    dv_ = _out(torch, "dv", dv_, (B, T, H, dv), v.dtype, dev)
    dg = _out(torch, "dg", dg, tuple(g.shape), torch.float32, dev)
    if out is None or dS0 is not None:
        dS0 = _out(torch, "dS0", dS0, (B, H, dv, dk), torch.float32, dev)
    d = _pack_desc(*dims, _dtype(torch, v.dtype), per_head, scale, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3],
                   *do.stride()[:3], *(_NONE if per_head else g.stride()))
    ws = _scratch(torch, ws, lambda: mgs_linattn_workspace_size(*dims, dtype=v.dtype, backward=True), dev)
    check(load().mgs_linattn_bwd(d, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(do), _ptr(S0), _ptr(dST), _ptr(lengths),
                                 _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(dS0), _ptr(ws), ws.numel(),
                                 _raw_stream(torch, dev)), "mgs_linattn_bwd")
    return dq, dk_, dv_, dg, dS0


def mgs_linattn_step(q, k, v, g, S, slots=None, scale=1.0, o=None, stream=None):
    """o (B,H,dv) of one step for each of B sequences; S (n_slots,H,dv,dk) float32 is updated in place.

    q, k (B,Hk,dk), v (B,H,dv), g (B,H) or (H,).  slots (B,) int32: the state of sequence b is S[slots[b]]
    (None: S[b]); the slots of a call are distinct, and one outside S (-1) is idle: zeros out, no state touched."""
    if stream is not None:
        return _on(stream, mgs_linattn_step, q, k, v, g, S, slots, scale, o)
    import torch
    if v.dim() != 3 or q.dim() != 3 or S.dim() != 4:
        raise ValueError("q, k must be (B,Hk,dk), v (B,H,dv) and S (n_slots,H,dv,dk)")
    B, H, dv = v.shape
    Hk, dk = q.shape[1:]
    dev, dt = _device("v", v), v.dtype
    _tensor("v", v, (B, H, dv), dt, dev, LAST)
    _tensor("q", q, (B, Hk, dk), dt, dev, LAST)
    _tensor("k", k, (B, Hk, dk), dt, dev, LAST)
    per_head = g is not None and g.dim() == 1
    _tensor("g", g, (H,) if per_head else (B, H), torch.float32, dev, DENSE if per_head else ANY)
    n_slots = S.shape[0]
    _tensor("S", S, (n_slots, H, dv, dk), torch.float32, dev)
    if slots is not None:
        _tensor("slots", slots, (B,), torch.int32, dev)
    o = _like("o", o, v)
    (qb, qh, _), (kb, kh, _), (vb, vh, _) = q.stride(), k.stride(), v.stride()
    gb, gh = (0, 0) if per_head else g.stride()
    d = _pack_desc(B, 1, H, Hk, dk, dv, _dtype(torch, dt), per_head, scale, qb, 0, qh, kb, 0, kh, vb, 0, vh, 0, 0, 0,
                   gb, 0, gh)
    check(load().mgs_linattn_step(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), S.data_ptr(), n_slots,
                                  _ptr(slots), o.data_ptr(), _raw_stream(torch, dev)), "mgs_linattn_step")
    return o


# ------------------------------------------------------------------- norm

def _rows(name, t, d, dtype, dev):
    """Row stride of a (...,d) tensor: rows evenly spaced, dense within."""
    if t.dim() < 1 or t.shape[-1] != d:
        raise ValueError(f"{name} must end in {d}, got {tuple(t.shape)}")
    if t.is_contiguous():
        _tensor(name, t, t.shape, dtype, dev, ANY)
        return d
    _tensor(name, t, t.shape, dtype, dev, LAST)
    if t.dim() != 2:
        raise ValueError(f"{name} must be contiguous or two-dimensional")
    return t.stride(0)


def _norm_inputs(torch, x, w, residual):
    shape, dev, dt = x.shape, _device("x", x), x.dtype
    if not shape:
        raise ValueError("x must have at least one dimension")
    d, code = shape[-1], _dtype(torch, dt)
    xs = rs = d
    if not x.is_contiguous():
        xs = _rows("x", x, d, dt, dev)
    _tensor("w", w, (d,), dt, dev)
    if residual is not None:
        _tensor("residual", residual, shape, dt, dev, ANY)
        if not residual.is_contiguous():
            rs = _rows("residual", residual, d, dt, dev)
    return x.numel() // d if d else 0, d, xs, rs, dev, code


def mgs_rmsnorm_fwd(x, w, residual=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """(y, h, rstd) of h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w over the last dimension.

    x, residual (...,d), w (d,), float32 or bfloat16; rstd float32, one for each row.  Without a residual h is x
    itself, not a copy, unless a buffer is passed.  h may be the residual's (or x's) own dense tensor."""
    if stream is not None:
        return _on(stream, mgs_rmsnorm_fwd, x, w, residual, eps, y, h, rstd)
    import torch
    rows, d, xs, rs, dev, code = _norm_inputs(torch, x, w, residual)
    y = _like("y", y, x)
    write_h = h is not None or residual is not None or not x.is_contiguous()
    h_out = _like("h", h, x) if write_h else None
    rstd = _out(torch, "rstd", rstd, x.shape[:-1], torch.float32, dev)
    check(load().mgs_rmsnorm_fwd(x.data_ptr(), _ptr(residual), w.data_ptr(), y.data_ptr(), _ptr(h_out), rstd.data_ptr(),
                                 rows, d, xs, rs, eps, code, _raw_stream(torch, dev)), "mgs_rmsnorm_fwd")
    return y, (h_out if write_h else x), rstd


def mgs_rmsnorm_fwd_fp8(x, w, residual=None, eps=1e-6, group=0, y=None, scale=None, h=None, stream=None):
    """(y, scale, h): the norm with y in float8_e4m3fn and a float32 scale for each row (group = 0; scale (...,1)) or
    for each 128 columns (group = 128; scale (..., ceil(d / 128))); y * scale stands for the norm's output."""
    if stream is not None:
        return _on(stream, mgs_rmsnorm_fwd_fp8, x, w, residual, eps, group, y, scale, h)
    import torch
    rows, d, xs, rs, dev, code = _norm_inputs(torch, x, w, residual)
    y = _out(torch, "y", y, x.shape, torch.float8_e4m3fn, dev)
    n_scales = -(-d // group) if group > 0 else 1
    scale = _out(torch, "scale", scale, (*x.shape[:-1], n_scales), torch.float32, dev)
    write_h = h is not None or residual is not None or not x.is_contiguous()
    h_out = _like("h", h, x) if write_h else None
    check(load().mgs_rmsnorm_fwd_fp8(x.data_ptr(), _ptr(residual), w.data_ptr(), y.data_ptr(), scale.data_ptr(),
                                     _ptr(h_out), rows, d, xs, rs, eps, group, code, _raw_stream(torch, dev)),
          "mgs_rmsnorm_fwd_fp8")
    return y, scale, (h_out if write_h else x)


def mgs_rmsnorm_workspace_size(rows, d):
    out = ctypes.c_size_t(0)
    check(load().mgs_rmsnorm_workspace_size(int(rows), int(d), ctypes.byref(out)), "mgs_rmsnorm_workspace_size")
    return int(out.value)


def mgs_rmsnorm_bwd(dy, h, w, rstd, dh=None, dx=None, dw=None, ws=None, stream=None):
    """(dx, dw) for L = sum(dy * y) + sum(dh * h), from the forward's h and rstd; dx is the gradient of x and of the
    residual alike, dw (d,) float32.  dx may be dy's or dh's own tensor."""
    if stream is not None:
        return _on(stream, mgs_rmsnorm_bwd, dy, h, w, rstd, dh, dx, dw, ws)
    import torch
    d, dev, dt = h.shape[-1], _device("h", h), h.dtype
    code = _dtype(torch, dt)
    _tensor("h", h, h.shape, dt, dev)
    _tensor("dy", dy, h.shape, dt, dev)
    _tensor("w", w, (d,), dt, dev)
    _tensor("rstd", rstd, h.shape[:-1], torch.float32, dev)
    if dh is not None:
        _tensor("dh", dh, h.shape, dt, dev)
    dx = _like("dx", dx, h)
    dw = _out(torch, "dw", dw, (d,), torch.float32, dev)
    rows = rstd.numel()   # one for each row of h
    ws = _scratch(torch, ws, lambda: mgs_rmsnorm_workspace_size(rows, d), dev)
    check(load().mgs_rmsnorm_bwd(dy.data_ptr(), h.data_ptr(), w.data_ptr(), rstd.data_ptr(), _ptr(dh), dx.data_ptr(),
                                 dw.data_ptr(), rows, d, code, ws.data_ptr(), ws.numel(),
                                 _raw_stream(torch, dev)), "mgs_rmsnorm_bwd")
    return dx, dw


# --------------------------------------------------------------- clipping

def mgs_clip_norm_workspace_size(sizes):
    """sizes: element counts of the tensors."""
    counts = array("q", sizes)
    out = ctypes.c_size_t(0)
    check(load().mgs_clip_norm_workspace_size(len(counts), counts.buffer_info()[0], ctypes.byref(out)),
          "mgs_clip_norm_workspace_size")
    return int(out.value)


def mgs_clip_norm(tensors, max_norm=None, out=None, norm=None, ws=None, stream=None):
    """(norm () float32 on the GPU, tensors scaled by min(1, max_norm / (norm + 1e-6))).

    tensors: contiguous, float32 or bfloat16 or both, any shapes.  out: tensors of the same shapes and types, or
    None to scale in place.  max_norm None: only the norm (second value None).  A norm that is not finite leaves
    the values as they are."""
    if stream is not None:
        return _on(stream, mgs_clip_norm, tensors, max_norm, out, norm, ws)
    import torch
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    dev = _device("tensors[0]", tensors[0])
    of = torch.Tensor

    def usable(ts):
        return set(map(of.get_device, ts)) == {dev} and all(map(of.is_contiguous, ts))

    kinds = [t.dtype for t in tensors]
    types = set(kinds)
    if not types <= {torch.float32, torch.bfloat16} or not usable(tensors):
        for i, t in enumerate(tensors):
            _dtype(torch, t.dtype)
            _tensor(f"tensors[{i}]", t, t.shape, t.dtype, dev)
    outs = None
    if max_norm is not None:
        outs = tensors if out is None else list(out)
        if len(outs) != len(tensors):
            raise ValueError(f"out has {len(outs)} tensors, expected {len(tensors)}")
        if out is not None and not ([o.dtype for o in outs] == kinds and usable(outs) and
                                    [o.shape for o in outs] == [t.shape for t in tensors]):
            for i, (o, t) in enumerate(zip(outs, tensors)):
                _tensor(f"out[{i}]", o, t.shape, t.dtype, dev)
    elif out is not None:
        raise ValueError("out needs max_norm")
    if len(types) == 1:
        dtypes = array("i", (_dtype(torch, kinds[0]),)) * len(kinds)
    else:
        dtypes = array("i", [k is torch.bfloat16 for k in kinds])
    norm = _out(torch, "norm", norm, (), torch.float32, dev)
    counts = array("q", map(of.numel, tensors))
    ws = _scratch(torch, ws, lambda: mgs_clip_norm_workspace_size(counts), dev)
    ins = array("Q", map(of.data_ptr, tensors))
    outp = array("Q", map(of.data_ptr, outs)) if outs is not None else None
    check(load().mgs_clip_norm(len(counts), ins.buffer_info()[0], outp.buffer_info()[0] if outp is not None else None,
                               counts.buffer_info()[0], dtypes.buffer_info()[0],
                               0.0 if max_norm is None else max_norm, norm.data_ptr(), ws.data_ptr(), ws.numel(),
                               _raw_stream(torch, dev)), "mgs_clip_norm")
    return norm, outs
