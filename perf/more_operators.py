"""Workloads of the operators of a recurrent language model's token path: the embedding lookup with its gradient, the
gated linear recurrence (forward, gradient, single step), and sampling of the next token.

Each case is one pass of one operator as a program calls it.  With `own` false, `run` computes it from elementary
torch operations (the plain form); with `own` true it calls scan_linear_rnns_amd.  `exact` computes the same outputs
in 64 bits straight from the definitions.

    lookup      y_n = scale W[id_n] (zeros for an id outside the table),   dW_v = scale sum over n with id_n = v of dy_n
    recurrence  log a_t = -c softplus(lam) sigmoid(r_t),   a_t = 0 where a document starts,
                h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t                    per sequence and channel
    sampling    w_i = exp((x_i - max x) / temperature); of the order by (w descending, index ascending): the first top_k,
                of these the fewest that hold top_p of their weight, of these the ones with w_i >= min_p;
                the token is the first, by index, at which the kept weight exceeds u times its total
"""
import math

import torch

own = False

RATE = 8.0   # c of the recurrence

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of one sequence through one layer: the latency of interactive generation
        dict(name="gated_step_one", op="gated", form="step", B=1, D=2048, slots=4, dtype="bf16"),
        # one token for each of a full batch of a server, states in a larger cache, in no order
        dict(name="gated_step_batch", op="gated", form="step", B=256, D=4096, slots=300, dtype="bf16"),
        # a batch of prompts of unlike lengths, inputs cut from one projection
        dict(name="gated_prompt_ragged", op="gated", form="fwd", B=8, T=1999, D=2560, dtype="bf16", ragged=True,
             packed=False, state=False, fused=True),
        # one long document: the parallel work lies along the steps
        dict(name="gated_prompt_long", op="gated", form="fwd", B=1, T=65536, D=1024, dtype="bf16", ragged=False,
             packed=False, state=True, fused=False),
        # training of a small layer, fp32, a width that fills no tile, states carried from the batch before
        dict(name="gated_train_f32", op="gated", form="train", B=16, T=1024, D=1000, dtype="f32", ragged=False,
             packed=False, state=True, fused=False),
        # training of a layer on packed documents
        dict(name="gated_train_bf16", op="gated", form="train", B=4, T=4096, D=4096, dtype="bf16", ragged=False,
             packed=True, state=False, fused=False),
        # the lookup while generating for a small batch
        dict(name="embed_step", op="embed", form="fwd", N=32, V=32000, D=2048, dtype="bf16"),
        # training of a small model, odd sizes, fp32: the lookup and the table's gradient
        dict(name="embed_train_f32", op="embed", form="train", N=4095, V=5003, D=1000, dtype="f32"),
        # training of a large one
        dict(name="embed_train_bf16", op="embed", form="train", N=32768, V=128000, D=2048, dtype="bf16"),
        # the next token of one sequence
        dict(name="sample_one", op="sample", B=1, V=32000, dtype="bf16", filters="all"),
        # the next tokens of a small batch, the whole distribution, a vocabulary that fills no tile
        dict(name="sample_plain", op="sample", B=37, V=50001, dtype="f32", filters="none"),
        # the next tokens of a full batch of a server, each request with its own settings
        dict(name="sample_batch", op="sample", B=256, V=128000, dtype="bf16", filters="mixed"),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated", "embed", "embed", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "sample":
        V = _span(rng, 100, 200000)
        return dict(op=op, B=_span(rng, 1, max(1, min(256, 32000000 // V))), V=V, dtype=dtype,
                    filters=rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]))
    width = _span(rng, 48, 8192)
    width = width - width % 8 if rng.random() < 0.6 else width
    if op == "embed":
        form = rng.choice(["fwd", "train", "train"])
        V = _span(rng, 300, min(200000, 200000000 // width))
        return dict(op=op, form=form, N=_span(rng, 1, min(65536, 60000000 // width)), V=V, D=width, dtype=dtype)
    form = rng.choice(["step", "fwd", "train", "train"])
    if form == "step":
        B = _span(rng, 1, 256)
        return dict(op=op, form=form, B=B, D=width, slots=B + rng.randint(0, 40), dtype=dtype)
    most = 60000000 if dtype == "bf16" else 30000000   # elements
    T = _span(rng, 1, min(65536, most // width))
    return dict(op=op, form=form, B=_span(rng, 1, max(1, min(64, most // (T * width)))), T=T, D=width, dtype=dtype,
                ragged=rng.random() < 0.3, packed=rng.random() < 0.3, state=rng.random() < 0.5,
                fused=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

def _settings(case, gen, dev):
    """Temperature, top_k, top_p, min_p: numbers, or one of each for every row."""
    kind, B = case["filters"], case["B"]
    if kind == "mixed":   # of requests that ask for different things; some leave a filter off
        def uniform(lo, hi):
            return lo + (hi - lo) * torch.rand(B, generator=gen, device=dev)

        def chosen(share):
            return torch.rand(B, generator=gen, device=dev) < share

        return dict(temperature=uniform(0.4, 1.3).where(chosen(0.95), 0.0),
                    top_k=uniform(1, 400).to(torch.int32).where(chosen(0.5), 0),
                    top_p=uniform(0.5, 1.0).where(chosen(0.7), 1.0), min_p=uniform(0.0, 0.2).where(chosen(0.4), 0.0))
    return dict(temperature=0.8, top_k=50 if kind in ("top_k", "all") else 0,
                top_p=0.95 if kind in ("top_p", "all") else 1.0, min_p=0.02 if kind in ("min_p", "all") else 0.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    st = dict(case=case)
    if own:
        import scan_linear_rnns_amd as mgs
        st["mgs"] = mgs

    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        # a few tokens well above a wide field; a part of the vocabulary is forbidden
        x = 2.0 * normal(B, V) + 6.0 * (normal(B, V) > 3.3)
        x = x.masked_fill(torch.rand(B, V, generator=gen, device=dev) < 0.02, -math.inf)
        st.update(logits=x.to(dt), u=torch.rand(B, generator=gen, device=dev), settings=_settings(case, gen, dev))
        if own:
            st["ws"] = mgs.workspace(mgs.mgs_sample_workspace_size(B, V), dev)
        return st

    if case["op"] == "embed":
        N, V, D = case["N"], case["V"], case["D"]
        # few tokens are most of a text; one in a hundred places is padding
        ids = torch.exp(math.log(V) * torch.rand(N, generator=gen, device=dev)).long().clamp_(1, V) - 1
        ids = ids.masked_fill(torch.rand(N, generator=gen, device=dev) < 0.01, -1)
        st.update(ids=ids, W=normal(V, D).to(dt), scale=D ** 0.5)
        if case["form"] == "train":
            st["dy"] = normal(N, D).to(dt)
            if own:
                st["ws"] = mgs.workspace(mgs.mgs_embed_workspace_size(N, V, D), dev)
        return st

    B, D = case["B"], case["D"]
    # decays between 0.9 and 0.999 with the gate open
    most = 0.9 + 0.099 * torch.rand(D, generator=gen, device=dev)
    st["lam"] = torch.log(torch.expm1(-torch.log(most) / RATE))
    if case["form"] == "step":
        st["slots"] = torch.randperm(case["slots"], generator=gen, device=dev)[:B].to(torch.int32)
        st["h"] = normal(case["slots"], D)
        st["x"], st["r"], st["i"] = (normal(B, D).to(dt) for _ in range(3))
        return st
    T = case["T"]
    if case["fused"]:   # views of one projection's output
        st["x"], st["r"], st["i"] = normal(B, T, 3 * D).to(dt).split(D, dim=2)
    else:
        st["x"], st["r"], st["i"] = (normal(B, T, D).to(dt) for _ in range(3))
    st["h0"] = normal(B, D) if case["state"] else None
    st["lengths"] = st["reset"] = None
    if case["ragged"]:
        st["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        st["lengths"][-1] = T
    if case["packed"]:   # documents of some 500 steps
        st["reset"] = torch.rand(B, T, generator=gen, device=dev) < 0.002
        st["reset"][:, 0] = True
    if case["form"] == "train":
        st["dy"] = normal(B, T, D).to(dt)
        st["dhT"] = normal(B, D) if case["state"] else None
    if own:
        st["ws"] = mgs.workspace(mgs.mgs_gated_workspace_size(B, T, D, dtype=dt, backward=case["form"] == "train"), dev)
    return st


# ------------------------------------------------------------- plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from zero: after each pass, sums over twice as many steps."""
    a, b = a.clone(), b.clone()
    s = 1
    while s < a.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _decay(lam, rho):
    """log a, a, sqrt(1 - a^2) of the gate's values."""
    log_a = -RATE * torch.nn.functional.softplus(lam) * rho
    return log_a, torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a))


def _plain_gated(st):
    case = st["case"]
    dt, T = st["x"].dtype, case["T"]
    x, rho, iota = st["x"].float(), torch.sigmoid(st["r"].float()), torch.sigmoid(st["i"].float())
    log_a, a, beta = _decay(st["lam"], rho)
    if st["reset"] is not None:
        new = st["reset"][:, :, None]
        a, beta = a.masked_fill(new, 0.0), beta.masked_fill(new, 1.0)
    b = beta * iota * x
    if st["lengths"] is not None:
        live = (torch.arange(T, device=x.device) < st["lengths"][:, None])[:, :, None]
        a, b = a.where(live, 1.0), b.where(live, 0.0)
    h0 = torch.zeros_like(b[:, :1]) if st["h0"] is None else st["h0"][:, None]
    h = _scan(a, torch.cat([b[:, :1] + a[:, :1] * h0, b[:, 1:]], 1))
    y = h if st["lengths"] is None else h.where(live, 0.0)
    out = {"y": y.to(dt)}
    if case["state"]:
        out["hT"] = h[:, -1]
    if case["form"] == "fwd":
        return out
    g = st["dy"].float()
    if st["lengths"] is not None:
        g = g.where(live, 0.0)
    if st["dhT"] is not None:
        g = torch.cat([g[:, :-1], g[:, -1:] + st["dhT"][:, None]], 1)
    # from the last step on: G_t = g_t + a_{t+1} G_{t+1}
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    G = _scan(after.flip(1), g.flip(1)).flip(1)
    if case["state"]:
        out["dh0"] = a[:, 0] * G[:, 0]
    if st["lengths"] is not None:
        G = G.where(live, 0.0)
    dl = G * (a * torch.cat([h0, h[:, :-1]], 1) - iota * x * a * a / beta)
    if st["reset"] is not None:
        dl = dl.masked_fill(new, 0.0)
    out["dx"] = (G * beta * iota).to(dt)
    out["dr"] = (dl * log_a * (1.0 - rho)).to(dt)
    out["di"] = (G * b * (1.0 - iota)).to(dt)
    out["dlam"] = (-RATE * torch.sigmoid(st["lam"]).double() * (dl * rho).sum((0, 1), dtype=torch.float64)).float()
    return out


def _plain_gated_step(st):
    x, rho, iota = st["x"].float(), torch.sigmoid(st["r"].float()), torch.sigmoid(st["i"].float())
    _, a, beta = _decay(st["lam"], rho)
    at = st["slots"].long()
    h = a * st["h"][at] + beta * iota * x
    st["h"][at] = h
    return {"y": h.to(st["x"].dtype), "h": st["h"]}


def _plain_embed(st):
    case = st["case"]
    ids, W = st["ids"], st["W"]
    here = ((ids >= 0) & (ids < case["V"]))[:, None]
    at = ids.clamp(0, case["V"] - 1)
    out = {"y": (st["scale"] * W[at].float()).where(here, 0.0).to(W.dtype)}
    if case["form"] == "train":
        dW = torch.zeros(W.shape, dtype=torch.float32, device=W.device)
        dW.index_add_(0, at, (st["scale"] * st["dy"].float()).where(here, 0.0))
        out["dW"] = dW.to(W.dtype)
    return out


def _column(value, B, dtype, dev):
    return value[:, None].to(dtype) if torch.is_tensor(value) else torch.full((B, 1), value, dtype=dtype, device=dev)


def _plain_sample(st):
    x = st["logits"].double()   # in 64 bits: sums of many small weights decide between neighbouring tokens
    B, V = x.shape
    tau, top_p, min_p = (_column(st["settings"][n], B, torch.float64, x.device)
                         for n in ("temperature", "top_p", "min_p"))
    top_k = _column(st["settings"]["top_k"], B, torch.int64, x.device)
    top, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((top - top[:, :1]) / tau.where(tau > 0, 1.0))
    rank = torch.arange(V, device=x.device)
    w = w.where((rank < top_k) | (top_k <= 0), 0.0)
    w = w.where((tau > 0) | (rank == 0), 0.0)
    before = torch.cumsum(w, 1) - w
    mass = w.sum(1, keepdim=True)
    w = w.where((before < top_p * mass) | (top_p >= 1) | (rank == 0), 0.0).where(w >= min_p, 0.0)
    kept = torch.zeros_like(w).scatter_(1, order, w)
    cdf = torch.cumsum(kept, 1)
    total = cdf[:, -1:]
    token = (cdf > st["u"].double()[:, None] * total).to(torch.uint8).argmax(1)
    return {"token": token, "logp": torch.log(kept.gather(1, token[:, None]) / total)[:, 0].float()}


# --------------------------------------------------------------------- run

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "sample":
            return _plain_sample(state)
        if op == "embed":
            return _plain_embed(state)
        return _plain_gated_step(state) if case["form"] == "step" else _plain_gated(state)

    mgs = state["mgs"]
    if op == "sample":
        token, logp = mgs.mgs_sample(state["logits"], state["u"], ws=state["ws"], **state["settings"])
        return {"token": token, "logp": logp}
    if op == "embed":
        out = {"y": mgs.mgs_embed_fwd(state["ids"], state["W"], scale=state["scale"])}
        if case["form"] == "train":
            out["dW"] = mgs.mgs_embed_bwd(state["ids"], state["dy"], case["V"], scale=state["scale"],
                                          dtype=state["W"].dtype, ws=state["ws"])
        return out
    inputs = (state["x"], state["r"], state["i"], state["lam"])
    if case["form"] == "step":
        y = mgs.mgs_gated_step(*inputs, state["h"], slots=state["slots"], rate=RATE)
        return {"y": y, "h": state["h"]}
    more = dict(h0=state["h0"], lengths=state["lengths"], reset=state["reset"], rate=RATE, ws=state["ws"])
    train = case["form"] == "train"
    y, hT, states = mgs.mgs_gated_fwd(*inputs, want_state=case["state"], want_states=train, **more)
    out = {"y": y}
    if case["state"]:
        out["hT"] = hT
    if train:
        del more["h0"]   # the first of the states
        dx, dr, di, dlam, dh0 = mgs.mgs_gated_bwd(*inputs, state["dy"], states, dhT=state["dhT"],
                                                  want_dh0=case["state"], **more)
        out.update(dx=dx, dr=dr, di=di, dlam=dlam)
        if case["state"]:
            out["dh0"] = dh0
    return out


# ------------------------------------------------------- 64-bit definitions

def _gates64(st):
    x, r, i = (st[n].double() for n in ("x", "r", "i"))
    rho, iota = 1.0 / (1.0 + torch.exp(-r)), 1.0 / (1.0 + torch.exp(-i))
    sp = torch.log1p(torch.exp(st["lam"].double()))
    a = torch.exp(-RATE * sp * rho)
    return x, rho, iota, sp, a, torch.sqrt((1.0 - a) * (1.0 + a))


def _exact_gated(st):
    """The recurrence step by step."""
    case = st["case"]
    B, T, D = case["B"], case["T"], case["D"]
    x, rho, iota, sp, a, beta = _gates64(st)
    on = torch.ones(B, T, 1, dtype=torch.bool, device=x.device)
    if st["lengths"] is not None:
        on = torch.arange(T, device=x.device)[None, :, None] < st["lengths"][:, None, None]
    fresh = torch.zeros_like(on) if st["reset"] is None else st["reset"][:, :, None]
    a, beta = torch.where(fresh, 0.0, a), torch.where(fresh, 1.0, beta)
    a_on = torch.where(on, a, 1.0).transpose(0, 1).contiguous()
    b_on = torch.where(on, beta * iota * x, 0.0).transpose(0, 1).contiguous()
    h = torch.zeros(T + 1, B, D, dtype=torch.float64, device=x.device)
    if st["h0"] is not None:
        h[0] = st["h0"].double()
    for t in range(T):
        torch.addcmul(b_on[t], a_on[t], h[t], out=h[t + 1])
    h = h.transpose(0, 1)
    out = {"y": torch.where(on, h[:, 1:], 0.0)}
    if case["state"]:
        out["hT"] = h[:, -1]
    if case["form"] == "fwd":
        return out
    del b_on
    G = torch.where(on, st["dy"].double(), 0.0).transpose(0, 1).contiguous()
    if st["dhT"] is not None:
        G[-1] += st["dhT"].double()
    for t in range(T - 2, -1, -1):
        G[t].addcmul_(a_on[t + 1], G[t + 1])
    if case["state"]:
        out["dh0"] = a_on[0] * G[0]
    G = torch.where(on, G.transpose(0, 1), 0.0)
    out["dx"] = G * beta * iota
    out["di"] = out["dx"] * x * (1.0 - iota)
    slope = torch.where(fresh, 0.0, a * h[:, :-1] - iota * x * a * a / beta)   # of h_t in log a_t
    pull = G * slope * rho * -RATE
    out["dr"] = pull * sp * (1.0 - rho)
    out["dlam"] = pull.sum((0, 1)) / (1.0 + torch.exp(-st["lam"].double()))
    return out


def _exact_sample(st):
    """Row by row."""
    case, s = st["case"], st["settings"]
    token, logp = [], []
    for n in range(case["B"]):
        tau, top_k, top_p, min_p = (float(s[name][n]) if torch.is_tensor(s[name]) else s[name]
                                    for name in ("temperature", "top_k", "top_p", "min_p"))
        x = st["logits"][n].double()
        if tau == 0:
            token.append(int((x == x.max()).nonzero()[0]))
            logp.append(0.0)
            continue
        w = torch.exp((x - x.max()) / tau)
        ids = torch.argsort(x, descending=True, stable=True)
        if top_k > 0:
            ids = ids[:int(top_k)]
        if top_p < 1:
            mass = torch.cumsum(w[ids], 0)
            ids = ids[:1 + int((mass < top_p * mass[-1]).sum())]
        ids = ids[w[ids] >= min_p].sort().values
        mass = torch.cumsum(w[ids], 0)
        at = int((mass <= float(st["u"][n]) * mass[-1]).sum())
        token.append(int(ids[at]))
        logp.append(math.log(float(w[ids[at]] / mass[-1])))
    dev = st["u"].device
    return {"token": torch.tensor(token, device=dev), "logp": torch.tensor(logp, dtype=torch.float64, device=dev)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(st)
    if case["op"] == "embed":
        ids, V = st["ids"], case["V"]
        here = (ids >= 0) & (ids < V)
        y = torch.zeros(case["N"], case["D"], dtype=torch.float64, device=ids.device)
        y[here] = st["W"][ids[here]].double() * st["scale"]
        if case["form"] == "fwd":
            return {"y": y}
        # sums of sorted rows, as differences of running sums
        order = torch.sort(ids[here], stable=True)
        running = torch.cumsum(st["dy"][here][order.indices].double() * st["scale"], 0)
        rows, counts = torch.unique_consecutive(order.values, return_counts=True)
        ends = running[counts.cumsum(0) - 1]
        dW = torch.zeros(V, case["D"], dtype=torch.float64, device=ids.device)
        dW[rows] = torch.diff(ends, dim=0, prepend=torch.zeros_like(ends[:1]))
        return {"y": y, "dW": dW}
    if case["form"] != "step":
        return _exact_gated(st)
    x, _, iota, _, a, beta = _gates64(st)
    h = st["h"].double()
    y = torch.empty_like(x)
    for n, slot in enumerate(st["slots"].tolist()):
        h[slot] = a[n] * h[slot] + beta[n] * iota[n] * x[n]
        y[n] = h[slot]
    return {"y": y, "h": h}


# -------------------------------------------------------------------- work

def work(case):
    """Bytes: every input once, every output once (of the table, the rows that are looked up; of the states, those in
    use).  Operations: those of the definitions, a function of one number (exp, a quotient, a root) as one."""
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        n = case["B"] * case["V"]
        return {"bytes": n * size + 32 * case["B"], "flops": 6 * n}
    if case["op"] == "embed":
        n, D = case["N"] * case["D"], case["D"]
        bytes_ = 8 * case["N"] + (min(case["N"], case["V"]) * D + n) * size
        if case["form"] == "fwd":
            return {"bytes": bytes_, "flops": n}
        return {"bytes": bytes_ + (n + case["V"] * D) * size, "flops": 3 * n}
    B, D = case["B"], case["D"]
    if case["form"] == "step":
        return {"bytes": B * D * (4 * size + 8) + 4 * (D + B), "flops": 16 * B * D}
    n = B * case["T"] * D
    more = 4 * D + (8 * B * D if case["state"] else 0) + (B * case["T"] if case["packed"] else 0)
    if case["form"] == "fwd":
        return {"bytes": 4 * size * n + more, "flops": 16 * n}
    return {"bytes": 8 * size * n + 2 * more, "flops": 50 * n}
