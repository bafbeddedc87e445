"""Plain 64-bit implementations of the layer operators, for the tests: the definitions of include/mgs_layers.h
written as loops over steps and rows in numpy.  Test infrastructure; nothing here shares code with the library."""
import numpy as np


def expand(x, H):
    """(B,T,Hk,d) to (B,T,H,d): each query/key head for its group of heads."""
    return np.repeat(x, H // x.shape[2], axis=2)


def linattn(q, k, v, g, S0=None, lengths=None, scale=1.0, do=None, dST=None):
    """Outputs of the recurrence and, with do, its gradients, as a dict of float64 arrays."""
    B, T, H, dv = v.shape
    Hk, dk = q.shape[2:]
    per_head = g.ndim == 1
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    q, k, v = (np.asarray(x, np.float64) for x in (expand(q, H), expand(k, H), v))
    a = np.exp(np.broadcast_to(np.asarray(g, np.float64), (B, T, H)))
    S = np.zeros((B, H, dv, dk)) if S0 is None else np.array(S0, np.float64)
    o = np.zeros((B, T, H, dv))
    states = np.zeros((T + 1, B, H, dv, dk)) if do is not None else None
    if do is not None:
        states[0] = S
    for t in range(T):
        for b in range(B):
            if t < n[b]:
                S[b] = a[b, t][:, None, None] * S[b] + v[b, t][:, :, None] * k[b, t][:, None, :]
                o[b, t] = scale * np.einsum("hrc,hc->hr", S[b], q[b, t])
        if do is not None:
            states[t + 1] = S
    out = dict(o=o, ST=S.copy())
    if do is None:
        return out
    do = np.asarray(do, np.float64)
    D = np.zeros_like(S) if dST is None else np.array(dST, np.float64)
    dq, dkk, dvv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, T, H))
    for t in range(T - 1, -1, -1):
        for b in range(B):
            if t >= n[b]:
                continue
            dq[b, t] = scale * np.einsum("hrc,hr->hc", states[t + 1, b], do[b, t])
            D[b] += scale * do[b, t][:, :, None] * q[b, t][:, None, :]
            dkk[b, t] = np.einsum("hrc,hr->hc", D[b], v[b, t])
            dvv[b, t] = np.einsum("hrc,hc->hr", D[b], k[b, t])
            D[b] *= a[b, t][:, None, None]
            dg[b, t] = (D[b] * states[t, b]).sum((1, 2))
    group = lambda x: x.reshape(B, T, Hk, H // Hk, dk).sum(3)  # noqa: E731
    out.update(dq=group(dq), dk=group(dkk), dv=dvv, dg=dg.sum((0, 1)) if per_head else dg, dS0=D)
    return out


def linattn_abs(q, k, v, g, S0=None, lengths=None, scale=1.0, do=None, dST=None, **_):
    """The same sums over absolute values: what rounding errors are proportional to.  dg is computed by the library
    from sums of q . dq and k . dk along a segment, so its entry is the whole sum of their absolute values."""
    m = lambda x: None if x is None else np.abs(np.asarray(x, np.float64))  # noqa: E731
    r = linattn(m(q), m(k), m(v), g, m(S0), lengths, abs(scale), m(do), m(dST))
    if do is not None:
        H = v.shape[2]
        B, T = v.shape[:2]
        each = np.broadcast_to(np.asarray(g, np.float64), (B, T, H))
        per = linattn(m(expand(q, H)), m(expand(k, H)), m(v), each, m(S0), lengths, abs(scale), m(do), m(dST))
        x = (m(expand(q, H)) * per["dq"]).sum(-1) + (m(expand(k, H)) * per["dk"]).sum(-1)   # (B,T,H)
        seg = 512
        total = np.zeros_like(x)
        for t0 in range(0, T, seg):
            total[:, t0:t0 + seg] = x[:, t0:t0 + seg].sum(1, keepdims=True)
        full = total + per["dg"].max(1, keepdims=True) if T else total
        r["dg"] = full.sum((0, 1)) if g.ndim == 1 else full
    return r


def rmsnorm(x, w, residual=None, eps=1e-6):
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[..., None] * np.asarray(w, np.float64), h, rstd


def rmsnorm_bwd(dy, h, w, rstd, dh=None):
    dy, h, w, rstd = (np.asarray(t, np.float64) for t in (dy, h, w, rstd))
    e, r = dy * w, rstd[..., None]
    dx = r * (e - h * r * r * (e * h).mean(-1, keepdims=True)) + (0 if dh is None else np.asarray(dh, np.float64))
    return dx, (dy * h * r).reshape(-1, h.shape[-1]).sum(0)
