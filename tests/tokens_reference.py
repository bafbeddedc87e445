"""Plain 64-bit implementations of the token path's operators, for the tests: the definitions of include/mgs_tokens.h
in numpy.  Test infrastructure; nothing here shares code with the library."""
import numpy as np


def embed(ids, W, scale):
    ids, W = np.asarray(ids).reshape(-1), np.asarray(W, np.float64)
    y = np.zeros((len(ids), W.shape[1]))
    for n, v in enumerate(ids):
        if 0 <= v < W.shape[0]:
            y[n] = scale * W[v]
    return y


def embed_bwd(ids, dy, vocab, scale):
    """(dW, the same sum over absolute values, how many rows each id has)"""
    ids, dy = np.asarray(ids).reshape(-1), np.asarray(dy, np.float64)
    dy = dy.reshape(len(ids), -1)
    here = (ids >= 0) & (ids < vocab)
    dW, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(dW, ids[here], scale * dy[here])
    np.add.at(size, ids[here], np.abs(scale * dy[here]))
    return dW, size, np.bincount(ids[here].astype(np.int64), minlength=vocab)


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def gated(x, r, i, lam, h0=None, lengths=None, reset=None, rate=8.0, dy=None, dhT=None, eps=0.0, eps_step=0.0,
          tiny=0.0):
    """The recurrence and, with dy, its gradients as a dict of float64 arrays; under "err" the same names hold how far
    an evaluation may be off whose log a and sqrt(1 - a^2) are each within `eps` of themselves and that is off by
    eps_step of the state's absolute value for each step it goes through (running bounds, see the GPU test); `tiny` is
    how far sqrt(1 - a^2) may be off besides."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        return _gated(*(np.asarray(v, np.float64) for v in (x, r, i, lam)), h0, lengths, reset, rate, dy, dhT, eps,
                      eps_step, tiny)


def _gated(x, r, i, lam, h0, lengths, reset, rate, dy, dhT, eps, eps_step, tiny):
    B, T, D = x.shape
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    on = np.arange(T)[None, :, None] < n[:, None, None]
    fresh = np.zeros((B, T, 1), bool) if reset is None else np.asarray(reset, bool)[:, :, None]
    rho, iota = sigmoid(r), sigmoid(i)
    shut_r, shut_i = sigmoid(-r), sigmoid(-i)   # 1 - rho and 1 - iota, which cancel near one
    log_a = -rate * np.logaddexp(0.0, lam) * rho
    a, beta = np.exp(log_a), np.sqrt(-np.expm1(2 * log_a))
    la = np.where(fresh | (log_a == -np.inf), 0.0, np.abs(log_a))
    a, beta = np.where(fresh, 0.0, a), np.where(fresh, 1.0, beta)
    b = beta * iota * x
    h = np.zeros((B, T + 1, D))
    size, err = np.zeros((B, T + 1, D)), np.zeros((B, T + 1, D))   # of |h|'s recurrence, and of its errors
    if h0 is not None:
        h[:, 0] = h0
        size[:, 0] = np.abs(h0)
    ah = np.zeros((B, T, D))
    for t in range(T):
        f, live = fresh[:, t], on[:, t]
        ah[:, t] = np.where(f, 0.0, a[:, t] * h[:, t])
        old = np.where(f, 0.0, a[:, t] * size[:, t])
        old_err = np.where(f, 0.0, a[:, t] * err[:, t]) + old * (la[:, t] * eps + eps_step)
        h[:, t + 1] = np.where(live, ah[:, t] + b[:, t], h[:, t])
        size[:, t + 1] = np.where(live, old + np.abs(b[:, t]), size[:, t])
        err[:, t + 1] = np.where(live, old_err + 4 * eps * np.abs(b[:, t]) + tiny * np.abs(iota * x)[:, t],
                                 err[:, t] + eps_step * size[:, t])
    out = dict(y=np.where(on, h[:, 1:], 0.0), hT=h[:, -1].copy())
    errs = dict(y=np.where(on, err[:, 1:], 0.0), hT=err[:, -1])
    if dy is None:
        return dict(out, err=errs)
    G, Gs, Ge = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, T, D))
    K, Ks, Ke = (np.zeros((B, D)) for _ in range(3))   # what the step after hands back
    if dhT is not None:
        K, Ks = np.array(dhT, np.float64), np.abs(np.asarray(dhT, np.float64))
    for t in range(T - 1, -1, -1):
        live, f = on[:, t], fresh[:, t]
        G[:, t] = np.where(live, np.asarray(dy, np.float64)[:, t], 0.0) + K
        Gs[:, t] = np.where(live, np.abs(np.asarray(dy, np.float64)[:, t]), 0.0) + Ks
        Ge[:, t] = Ke + 2.0 ** -24 * Gs[:, t]
        K = np.where(live, np.where(f, 0.0, a[:, t] * G[:, t]), G[:, t])
        Ks = np.where(live, a[:, t] * Gs[:, t], Gs[:, t])
        Ke = np.where(live, a[:, t] * Ge[:, t] + Ks * (la[:, t] * eps + eps_step), Ge[:, t] + eps_step * Ks)
    out["dh0"], errs["dh0"] = K, Ke
    m = np.where(on, 1.0, 0.0)
    pull = np.where(fresh | (beta == 0), 0.0, iota * x * a * a / beta)
    dl = G * np.where(fresh, 0.0, ah - pull)
    held = np.where(fresh, 0.0, a * size[:, :-1])
    dl_err = Ge * (held + np.abs(pull)) + Gs * (
        np.where(fresh, 0.0, a * err[:, :-1]) + (held + np.abs(pull)) * (2 * la * eps + 2 * eps_step) +
        8 * eps * np.abs(pull))
    dx, di, dr, part = G * beta * iota, G * b * shut_i, dl * np.where(fresh, 0.0, log_a) * shut_r, dl * rho
    sl = -rate * sigmoid(lam)
    where = lambda v: np.where(on, v, 0.0)  # noqa: E731
    out.update(dx=where(dx), di=where(di), dr=where(dr), dlam=sl * where(part).sum((0, 1)))
    err_part = where(dl_err * rho + 4 * eps * np.abs(part))
    # (where 1 - a^2 counts as 0, pull does, and what it gives times log a, or times rate sigmoid(lam) rho, which
    # is no more, is beta / 2 and less)
    lost = where(tiny * Gs * iota * np.maximum(np.abs(x), 1))
    errs.update(dx=where((Ge + 6 * eps * Gs) * beta * iota) + lost,
                di=where((Ge + 8 * eps * Gs) * np.abs(b) * shut_i) + lost,
                dr=where((dl_err + 6 * eps * np.abs(dl)) * la * shut_r) + lost,
                dlam=np.abs(sl) * (err_part.sum((0, 1)) + 40 * 2.0 ** -24 * np.abs(where(part)).sum((0, 1))) +
                lost.sum((0, 1)))
    return dict(out, err=errs)


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, margin) of one row: margin is how far, as a share of the weight, the decisions are from the next
    other one (0 or more; small means that rounding might decide)."""
    x = np.asarray(logits, np.float64)
    if np.isnan(x).any() or (x == -np.inf).all():
        return -1, -np.inf, 1.0
    top = x.max()
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.where((x == -np.inf) | (top == np.inf), 0.0, np.exp((x - top) / temperature)))
    w = np.where(w < 2.0 ** -1000, 0.0, w)   # (as the operator is defined)
    order = np.argsort(-x, kind="stable")
    margin = 1.0
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        run = np.cumsum(w[order])
        want = top_p * run[-1]
        n = 1 + int((run < want).sum())
        margin = min(margin, np.abs(run - want)[:len(order) - 1].min(initial=1.0) / run[-1])
        order = order[:max(1, min(n, len(order)))]
    min_p = 0.0 if np.isnan(min_p) else min(max(min_p, 0.0), 1.0)
    near = w[order][w[order] < 1]
    if min_p > 0 and len(near):
        margin = min(margin, (np.abs(near - min_p) / np.maximum(near, min_p)).min())
    ids = np.sort(order[w[order] >= min_p])
    run = np.cumsum(w[ids])
    u = min(max(u, 0.0), float(np.float32(0.99999994))) if u == u else 0.0
    target = u * run[-1]
    at = int((run <= target).sum())
    if u > 0:
        margin = min(margin, np.abs(run - target).min() / run[-1])
    return int(ids[at]), float(np.log(w[ids[at]] / run[-1])), margin
