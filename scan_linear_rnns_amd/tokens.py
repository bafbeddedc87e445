"""Binding of the operators on the path from a token to the next one (include/mgs_tokens.h): the embedding lookup with
its gradient, the gated linear recurrence, and sampling.

As in layers.py, each function carries the name of the C entry point that it calls and only marshals arguments; there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import struct

from ._lib import GatedDesc, SampleDesc, check, load
from .layers import LAST, _device, _dtype, _on, _out, _ptr, _raw_stream, _rows, _scratch, _tensor

__all__ = [
    "mgs_embed_fwd", "mgs_embed_workspace_size", "mgs_embed_bwd",
    "mgs_gated_workspace_size", "mgs_gated_fwd", "mgs_gated_bwd", "mgs_gated_step",
    "mgs_sample_workspace_size", "mgs_sample",
]


# -------------------------------------------------------------- embedding

def _ids(torch, ids, dev):
    """Bits of an id."""
    if ids.dtype is not torch.int64 and ids.dtype is not torch.int32:
        raise TypeError(f"ids must be int64 or int32, got {ids.dtype}")
    _tensor("ids", ids, ids.shape, ids.dtype, dev)
    return 64 if ids.dtype is torch.int64 else 32


def mgs_embed_fwd(ids, W, scale=1.0, y=None, stream=None):
    """y (...,d) = scale W[ids]: ids (...) int64 or int32, W (vocab,d) float32 or bfloat16, rows evenly spaced.  An id
    outside the table (-1: padding) gives zeros."""
    if stream is not None:
        return _on(stream, mgs_embed_fwd, ids, W, scale, y)
    import torch
    dev = _device("W", W)
    if W.dim() != 2:
        raise ValueError(f"W must be (vocab,d), got {tuple(W.shape)}")
    vocab, d = W.shape
    code, bits, ws = _dtype(torch, W.dtype), _ids(torch, ids, dev), _rows("W", W, d, W.dtype, dev)
    if y is None:
        y = W.new_empty((*ids.shape, d))
    else:
        _tensor("y", y, (*ids.shape, d), W.dtype, dev)
    check(load().mgs_embed_fwd(ids.data_ptr(), bits, W.data_ptr(), y.data_ptr(), ids.numel(), vocab, d, ws, scale, code,
                               _raw_stream(torch, dev)), "mgs_embed_fwd")
    return y


def mgs_embed_workspace_size(n, vocab, d):
    """Bytes for mgs_embed_bwd of n ids."""
    out = ctypes.c_size_t(0)
    check(load().mgs_embed_workspace_size(int(n), int(vocab), int(d), ctypes.byref(out)), "mgs_embed_workspace_size")
    return int(out.value)


def mgs_embed_bwd(ids, dy, vocab, scale=1.0, dW=None, accumulate=False, dtype=None, ws=None, stream=None):
    """dW (vocab,d): for each id, scale times the sum of its rows of dy (...,d), zeros for ids that do not occur, in
    `dtype` (float32 by default; dW's own where it is given).  accumulate=True adds to dW and touches the rows that
    occur only.  Sums are float32 and run in an order that the ids fix.  ws: any memory, but not the recurrence's
    workspace, which this overwrites."""
    if stream is not None:
        return _on(stream, mgs_embed_bwd, ids, dy, vocab, scale, dW, accumulate, dtype, ws)
    import torch
    dev = _device("dy", dy)
    bits, code = _ids(torch, ids, dev), _dtype(torch, dy.dtype)
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(*ids.shape, 'd')}")
    n, d = ids.numel(), dy.shape[-1]
    gs = _rows("dy", dy, d, dy.dtype, dev)
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs dW")
        dW = torch.empty((vocab, d), dtype=dtype or torch.float32, device=dev)
    else:
        _tensor("dW", dW, (vocab, d), dtype or dW.dtype, dev)
    ws = _scratch(torch, ws, lambda: mgs_embed_workspace_size(n, vocab, d), dev)
    check(load().mgs_embed_bwd(ids.data_ptr(), bits, dy.data_ptr(), dW.data_ptr(), n, vocab, d, gs, scale,
                               int(bool(accumulate)), code, _dtype(torch, dW.dtype), ws.data_ptr(), ws.numel(),
                               _raw_stream(torch, dev)), "mgs_embed_bwd")
    return dW


# ------------------------------------------------- gated linear recurrence

_pack_gated = struct.Struct("3qif8q").pack   # mgs_gated_desc
assert struct.calcsize("3qif8q") == ctypes.sizeof(GatedDesc)
_NONE = (0, 0)   # strides that are not read


def mgs_gated_workspace_size(B, T, D, dtype=None, backward=False):
    """Bytes, with backward=True enough for the forward and the backward; dtype (the inputs') defaults to float32."""
    import torch
    out = ctypes.c_size_t(0)
    d = _pack_gated(B, T, D, _dtype(torch, dtype or torch.float32), 1.0, *_NONE * 4)
    check(load().mgs_gated_workspace_size(d, int(bool(backward)), ctypes.byref(out)), "mgs_gated_workspace_size")
    return int(out.value)


def _gated_scratch(torch, ws, B, T, D, dtype, backward, dev):
    """ws, or a new workspace: zeros, which it has to hold before its first use."""
    if ws is None:
        return torch.zeros(max(mgs_gated_workspace_size(B, T, D, dtype, backward), 256), dtype=torch.uint8, device=dev)
    _tensor("ws", ws, ws.shape, torch.uint8, dev)
    return ws


def _gated_inputs(torch, x, r, i, lam, lengths, reset):
    """Checks the inputs of a whole-sequence call; B, T, D, GPU."""
    if x.dim() != 3:
        raise ValueError("x, r, i must be (B,T,D)")
    dev, dt, shape = _device("x", x), x.dtype, x.shape
    _tensor("x", x, shape, dt, dev, LAST)
    _tensor("r", r, shape, dt, dev, LAST)
    _tensor("i", i, shape, dt, dev, LAST)
    B, T, D = shape
    _tensor("lam", lam, (D,), torch.float32, dev)
    if lengths is not None:
        _tensor("lengths", lengths, (B,), torch.int32, dev)
    if reset is not None:
        _tensor("reset", reset, (B, T), torch.uint8 if reset.dtype is torch.uint8 else torch.bool, dev)
    return B, T, D, dev


def mgs_gated_fwd(x, r, i, lam, h0=None, lengths=None, reset=None, rate=8.0, y=None, hT=None, states=None, ws=None,
                  want_state=True, want_states=False, stream=None):
    """(y (B,T,D), h_T (B,D) or None, states (B, ceil(T / 64), D) or None) of
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, log a_t = -rate softplus(lam) sigmoid(r_t), y = h.

    x, r, i (B,T,D), float32 or bfloat16, dense in the last dimension only (views of one projection do); lam (D,), h0
    (B,D) or None (zeros) float32.  lengths (B,) int32 or None: later steps are not read, leave the state as it is and
    give zeros.  reset (B,T) bool or uint8, or None: steps that start a document, which nothing before them reaches.
    states (want_states): what mgs_gated_bwd reads.  ws: a workspace (see `workspace`), zero-filled before its first
    use, and again after any other operator's call has had it."""
    if stream is not None:
        return _on(stream, mgs_gated_fwd, x, r, i, lam, h0, lengths, reset, rate, y, hT, states, ws, want_state,
                   want_states)
    import torch
    B, T, D, dev = _gated_inputs(torch, x, r, i, lam, lengths, reset)
    if h0 is not None:
        _tensor("h0", h0, (B, D), torch.float32, dev)
    if y is None:
        y = torch.empty((B, T, D), dtype=x.dtype, device=dev)
    else:
        _tensor("y", y, x.shape, x.dtype, dev)
    if hT is not None or want_state:
        hT = _out(torch, "hT", hT, (B, D), torch.float32, dev)
    if states is not None or want_states:
        states = _out(torch, "states", states, (B, -(-T // 64), D), torch.float32, dev)
    d = _pack_gated(B, T, D, _dtype(torch, x.dtype), rate, *x.stride()[:2], *r.stride()[:2], *i.stride()[:2], *_NONE)
    ws = _gated_scratch(torch, ws, B, T, D, x.dtype, False, dev)
    check(load().mgs_gated_fwd(d, _ptr(x), _ptr(r), _ptr(i), _ptr(lam), _ptr(h0), _ptr(lengths), _ptr(reset), _ptr(y),
                               _ptr(hT), _ptr(states), _ptr(ws), ws.numel(), _raw_stream(torch, dev)),
          "mgs_gated_fwd")
    return y, hT, states


def mgs_gated_bwd(x, r, i, lam, dy, states, dhT=None, lengths=None, reset=None, rate=8.0, out=None, ws=None,
                  want_dh0=True, stream=None):
    """(dx, dr, di, dlam, dh0) for L = sum(dy * y) + sum(dhT * h_T), from the forward's states; dlam (D,) and dh0 (B,D)
    (None without want_dh0) are float32.  dy (B,T,D) may be strided as x may.  out: the five outputs, dense (dh0 may be
    None there).  ws: as mgs_gated_fwd's."""
    if stream is not None:
        return _on(stream, mgs_gated_bwd, x, r, i, lam, dy, states, dhT, lengths, reset, rate, out, ws, want_dh0)
    import torch
    B, T, D, dev = _gated_inputs(torch, x, r, i, lam, lengths, reset)
    dt = x.dtype
    _tensor("dy", dy, (B, T, D), dt, dev, LAST)
    _tensor("states", states, (B, -(-T // 64), D), torch.float32, dev)
    if dhT is not None:
        _tensor("dhT", dhT, (B, D), torch.float32, dev)
    dx, dr, di, dlam, dh0 = out if out is not None else (None,) * 5
    dx = _out(torch, "dx", dx, (B, T, D), dt, dev)
    dr = _out(torch, "dr", dr, (B, T, D), dt, dev)
    di = _out(torch, "di", di, (B, T, D), dt, dev)
    dlam = _out(torch, "dlam", dlam, (D,), torch.float32, dev)
    if dh0 is not None or (out is None and want_dh0):
        dh0 = _out(torch, "dh0", dh0, (B, D), torch.float32, dev)
    d = _pack_gated(B, T, D, _dtype(torch, dt), rate, *x.stride()[:2], *r.stride()[:2], *i.stride()[:2],
                    *dy.stride()[:2])
    ws = _gated_scratch(torch, ws, B, T, D, dt, True, dev)
    check(load().mgs_gated_bwd(d, _ptr(x), _ptr(r), _ptr(i), _ptr(lam), _ptr(dy), _ptr(dhT), _ptr(states),
                               _ptr(lengths), _ptr(reset), _ptr(dx), _ptr(dr), _ptr(di), _ptr(dlam), _ptr(dh0),
                               _ptr(ws), ws.numel(), _raw_stream(torch, dev)), "mgs_gated_bwd")
    return dx, dr, di, dlam, dh0


def mgs_gated_step(x, r, i, lam, h, slots=None, rate=8.0, y=None, stream=None):
    """y (B,D) of one step for each of B sequences; h (n_slots,D) float32 is updated in place.

    x, r, i (B,D), dense in the last dimension.  slots (B,) int32: the state of sequence b is h[slots[b]] (None: h[b]);
    the slots of a call are distinct, and one outside h (-1) is idle: zeros out, no state touched."""
    if stream is not None:
        return _on(stream, mgs_gated_step, x, r, i, lam, h, slots, rate, y)
    import torch
    if x.dim() != 2 or h.dim() != 2:
        raise ValueError("x, r, i must be (B,D) and h (n_slots,D)")
    dev, dt, shape = _device("x", x), x.dtype, x.shape
    _tensor("x", x, shape, dt, dev, LAST)
    _tensor("r", r, shape, dt, dev, LAST)
    _tensor("i", i, shape, dt, dev, LAST)
    B, D = shape
    _tensor("lam", lam, (D,), torch.float32, dev)
    n_slots = h.shape[0]
    _tensor("h", h, (n_slots, D), torch.float32, dev)
    if slots is not None:
        _tensor("slots", slots, (B,), torch.int32, dev)
    if y is None:
        y = torch.empty(shape, dtype=dt, device=dev)
    else:
        _tensor("y", y, shape, dt, dev)
    d = _pack_gated(B, 1, D, _dtype(torch, dt), rate, x.stride(0), 0, r.stride(0), 0, i.stride(0), 0, 0, 0)
    check(load().mgs_gated_step(d, x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), h.data_ptr(), n_slots,
                                _ptr(slots), y.data_ptr(), _raw_stream(torch, dev)), "mgs_gated_step")
    return y


# --------------------------------------------------------------- sampling

_pack_sample = struct.Struct("3q2i3f4x").pack   # mgs_sample_desc
assert struct.calcsize("3q2i3f4x") == ctypes.sizeof(SampleDesc)


def mgs_sample_workspace_size(B, vocab, dtype=None):
    """Bytes; dtype (the logits') defaults to float32."""
    import torch
    out = ctypes.c_size_t(0)
    d = _pack_sample(B, vocab, vocab, _dtype(torch, dtype or torch.float32), 0, 1.0, 1.0, 0.0)
    check(load().mgs_sample_workspace_size(d, ctypes.byref(out)), "mgs_sample_workspace_size")
    return int(out.value)


def _setting(torch, name, value, dtype, B, dev, off):
    """A setting as the desc's number (the nearest that its type holds) and a pointer to one for each row, or None."""
    if isinstance(value, torch.Tensor):
        _tensor(name, value, (B,), dtype, dev)
        return off, value.data_ptr()
    return max(0, min(value, 2 ** 31 - 1)) if dtype is torch.int32 else value, None


def mgs_sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, logp=None, ws=None, stream=None):
    """(token (B,) int64, logp (B,) float32): the next token of each row of logits (B,vocab), float32 or bfloat16, rows
    evenly spaced, from uniform numbers u (B,) float32 in [0, 1).

    temperature, top_p, min_p and top_k are numbers, or (B,) tensors on the GPU (float32; top_k int32).  Of the tokens
    in order of their logits, the first top_k (0: all) stay, of these the fewest that hold top_p of their weight, of
    these the ones of at least min_p times the largest weight; the token is the first, by index, at which the kept
    weight exceeds u times its sum.  temperature 0 takes the largest.  logp: the log of the token's share of the kept
    weight.  A row with nothing but -inf, or with a NaN, gives -1 and -inf.  Numbers count as float32 holds them (0.8 is
    0.800000012).  ws: any memory, but not the recurrence's workspace, which this overwrites."""
    if stream is not None:
        return _on(stream, mgs_sample, logits, u, temperature, top_k, top_p, min_p, token, logp, ws)
    import torch
    if logits.dim() != 2:
        raise ValueError(f"logits must be (B,vocab), got {tuple(logits.shape)}")
    B, vocab = logits.shape
    dev, code = _device("logits", logits), _dtype(torch, logits.dtype)
    _tensor("logits", logits, logits.shape, logits.dtype, dev, LAST)
    _tensor("u", u, (B,), torch.float32, dev)
    f32 = torch.float32
    tau, taus = _setting(torch, "temperature", temperature, f32, B, dev, 1.0)
    k, ks = _setting(torch, "top_k", top_k, torch.int32, B, dev, 0)
    p, ps = _setting(torch, "top_p", top_p, f32, B, dev, 1.0)
    m, ms = _setting(torch, "min_p", min_p, f32, B, dev, 0.0)
    token = _out(torch, "token", token, (B,), torch.int64, dev)
    logp = _out(torch, "logp", logp, (B,), f32, dev)
    ws = _scratch(torch, ws, lambda: mgs_sample_workspace_size(B, vocab, logits.dtype), dev)
    d = _pack_sample(B, vocab, logits.stride(0), code, k, tau, p, m)
    check(load().mgs_sample(d, logits.data_ptr(), u.data_ptr(), taus, ks, ps, ms, token.data_ptr(), logp.data_ptr(),
                            ws.data_ptr(), ws.numel(), _raw_stream(torch, dev)), "mgs_sample")
    return token, logp
