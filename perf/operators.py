"""Workloads of the layer operators: linear attention with a decay for each head, the root-mean-square norm with
the residual's addition, and the global gradient norm with clipping.

Each case is one pass of one operator as a program calls it.  With `own` false, `run` computes it from elementary
torch operations in 32 bits (the plain form); with `own` true it calls scan_linear_rnns_amd.  `exact` computes the
same outputs in 64 bits straight from the definitions.

    linear attention  S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t       per sequence and head
    norm              h = x + residual,   y = h / sqrt(mean(h^2) + eps) * w           per row; y also in 8 bits
    clipping          n = sqrt(sum over all tensors of g^2),   g <- g min(1, max_norm / (n + 1e-6))
"""
import math

import torch

own = False

EPS = 1e-6        # of the norm, under the root
CLIP_EPS = 1e-6   # of the clipping coefficient's denominator
E4M3_MAX = 448.0  # largest finite value of the 8-bit type
CHUNK = 64        # steps per chunk of the plain form

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of one sequence through one layer: the latency of interactive generation
        dict(name="attn_step_one", op="attn", form="step", B=1, H=16, Hk=16, dk=64, dv=64, slots=4, dtype="bf16"),
        # one token for each of a full batch of a server, states in a larger cache, in no order
        dict(name="attn_step_batch", op="attn", form="step", B=256, H=16, Hk=16, dk=128, dv=128, slots=300,
             dtype="bf16"),
        # a batch of prompts of unlike lengths, four value heads to a query/key head
        dict(name="attn_prompt_ragged", op="attn", form="fwd", B=8, T=1999, H=16, Hk=4, dk=64, dv=128, dtype="bf16",
             decay="step", ragged=True, state=True, fused=False),
        # one long document, few heads: all the parallel work lies along the steps
        dict(name="attn_prompt_long", op="attn", form="fwd", B=1, T=32768, H=8, Hk=8, dk=128, dv=128, dtype="bf16",
             decay="step", ragged=False, state=True, fused=False),
        # training at the long shape of the scans (16 sequences of 1024 steps, 64 wide), one decay per head, fp32
        dict(name="attn_train_f32", op="attn", form="train", B=16, T=1024, H=1, Hk=1, dk=64, dv=64, dtype="f32",
             decay="head", ragged=False, state=False, fused=False),
        # training of a layer, inputs cut from one fused projection
        dict(name="attn_train_bf16", op="attn", form="train", B=4, T=4096, H=16, Hk=16, dk=128, dv=128, dtype="bf16",
             decay="step", ragged=False, state=False, fused=True),
        # the norm ahead of an 8-bit projection while generating for a small batch
        dict(name="norm_step_8bit", op="norm", form="fp8", rows=32, d=2048, group=0, dtype="bf16"),
        # the same for a prompt, a scale for each 128 columns, a row count and width that fill no tile
        dict(name="norm_prompt_8bit", op="norm", form="fp8", rows=8191, d=5000, group=128, dtype="bf16"),
        # training: the norm and its gradient, fp32
        dict(name="norm_train_f32", op="norm", form="train", rows=4095, d=1000, group=0, dtype="f32"),
        # training: the norm and its gradient at a large layer's size
        dict(name="norm_train_bf16", op="norm", form="train", rows=16384, d=4096, group=0, dtype="bf16"),
        # the gradients of a small recurrent network: a few matrices and many vectors
        dict(name="clip_small", op="clip", tensors=40, most=65536, dtype="f32", spread=17),
        # the gradients of a large one, matrices in bf16 and vectors in fp32
        dict(name="clip_large", op="clip", tensors=150, most=12582912, dtype="bf16", spread=5),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "norm", "norm", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "attn":
        form = rng.choice(["step", "fwd", "train"])
        Hk = rng.choice([1, 2, 3, 4, 8])
        H = Hk * rng.choice([1, 1, 2, 4])
        dk, dv = rng.choice([32, 48, 64, 64, 96, 128, 128]), rng.choice([32, 40, 64, 64, 96, 128, 128])
        if form == "step":
            B = _span(rng, 1, 256)
            return dict(op=op, form=form, B=B, H=H, Hk=Hk, dk=dk, dv=dv, slots=B + rng.randint(0, 40), dtype=dtype)
        most = 262144 if form == "fwd" else 131072   # steps times heads
        T = _span(rng, 1, min(16384, most // H))
        B = _span(rng, 1, min(64, most // (T * H)))
        return dict(op=op, form=form, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype,
                    decay=rng.choice(["step", "step", "head"]), ragged=rng.random() < 0.4, state=rng.random() < 0.4,
                    fused=rng.random() < 0.3)
    if op == "norm":
        d = _span(rng, 64, 8192)
        d = d - d % 8 if rng.random() < 0.7 else d
        form = rng.choice(["fp8", "train"])
        return dict(op=op, form=form, rows=_span(rng, 1, min(32768, (16384 * 4096) // (2 * d))), d=d,
                    group=rng.choice([0, 128]) if form == "fp8" else 0, dtype=dtype)
    return dict(op=op, tensors=_span(rng, 3, 300), most=_span(rng, 1024, 2000000), dtype=dtype,
                spread=rng.randint(1, 1000))


# ------------------------------------------------------------------ inputs

def _clip_sizes(case):
    """Element counts of the tensors: a third matrices near `most`, the others vectors; odd ones among them."""
    n, most, s = case["tensors"], case["most"], case["spread"]
    sizes = []
    for i in range(n):
        f = ((i * 7919 + s * 104729) % 1000) / 1000.0
        sizes.append(max(1, int(most * (0.25 + 0.75 * f))) if i % 3 == 0 else max(1, int((most ** 0.5) * (0.5 + f))))
    return sizes


def _flat_like(tensors, dtype=None):
    """One zeroed flat buffer for each type, and a view in it for each tensor, 64 elements apart at the least."""
    size, at = {}, []
    for t in tensors:
        key = str(t.dtype)
        at.append((key, size.get(key, 0)))
        size[key] = at[-1][1] + -(-t.numel() // 64) * 64
    kind = {str(t.dtype): dtype or t.dtype for t in tensors}
    flat = {key: torch.zeros(size[key], dtype=kind[key], device=tensors[0].device) for key in sorted(size)}
    return flat, [flat[key][i:i + t.numel()] for (key, i), t in zip(at, tensors)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        # the residual stream has grown over the layers below; weights near one
        st = dict(case=case, x=normal(rows, d).to(dt), residual=(3.0 * normal(rows, d)).to(dt),
                  w=(1.0 + 0.1 * normal(d)).to(dt))
        if case["form"] == "train":
            st["dy"] = normal(rows, d).to(dt)
            st["dh"] = normal(rows, d).to(dt)   # what reaches the residual from above
        if own:
            import scan_linear_rnns_amd as mgs
            st["mgs"] = mgs
            if case["form"] == "train":
                st["ws"] = mgs.workspace(mgs.mgs_rmsnorm_workspace_size(rows, d), dev)
        return st

    if case["op"] == "clip":
        grads = []
        for i, n in enumerate(_clip_sizes(case)):
            t = 0.02 * (1 + i % 5) * normal(n)
            grads.append(t.to(dt) if i % 3 == 0 else t)
        # about a third of the usual norm, so that the gradients are scaled
        total = math.sqrt(sum(n * (0.02 * (1 + i % 5)) ** 2 for i, n in enumerate(_clip_sizes(case))))
        # the clipped gradients go to buffers of their own, so that a pass can be repeated: one flat buffer a type,
        # as an optimizer that walks flat memory keeps them
        flat, out = _flat_like(grads)
        st = dict(case=case, grads=grads, max_norm=total / 3, flat=flat, out=out)
        if own:
            import scan_linear_rnns_amd as mgs
            st["mgs"] = mgs
            st["ws"] = mgs.workspace(mgs.mgs_clip_norm_workspace_size([t.numel() for t in grads]), dev)
        return st

    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    rate = torch.exp(torch.linspace(math.log(0.002), math.log(0.7), H, device=dev))   # heads that forget slowly and fast

    def log_decay(*shape):   # -rate softplus(z): a decay for each step, as a projection and a learnt rate make it
        return -rate * torch.nn.functional.softplus(normal(*shape, H))

    if case["form"] == "step":
        slots = torch.randperm(case["slots"], generator=gen, device=dev)[:B].to(torch.int32)
        st = dict(case=case, q=normal(B, Hk, dk).to(dt), k=(normal(B, Hk, dk) * dk ** -0.5).to(dt),
                  v=normal(B, H, dv).to(dt), g=log_decay(B), S=normal(case["slots"], H, dv, dk), slots=slots)
        if own:
            import scan_linear_rnns_amd as mgs
            st["mgs"] = mgs
        return st
    T = case["T"]
    parts = [normal(B, T, Hk * dk), normal(B, T, Hk * dk) * dk ** -0.5, normal(B, T, H * dv)]
    if case["fused"]:   # views of one projection's output
        both = torch.cat(parts, dim=2).to(dt)
        q, k, v = torch.split(both, [Hk * dk, Hk * dk, H * dv], dim=2)
    else:
        q, k, v = (p.to(dt) for p in parts)
    st = dict(case=case, q=q.unflatten(2, (Hk, dk)), k=k.unflatten(2, (Hk, dk)), v=v.unflatten(2, (H, dv)),
              g=log_decay(B, T) if case["decay"] == "step" else -rate, S0=None, lengths=None)
    if case["ragged"]:
        lengths = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lengths[-1] = T
        st["lengths"] = lengths
    if case["state"]:
        st["S0"] = normal(B, H, dv, dk) * 0.5
    if case["form"] == "train":
        st["do"] = normal(B, T, H, dv).to(dt)
        st["dST"] = normal(B, H, dv, dk) * 0.1 if case["state"] else None
    if own:
        import scan_linear_rnns_amd as mgs
        st["mgs"] = mgs
        dims = (B, T, H, Hk, dk, dv)
        st["ws"] = mgs.workspace(mgs.mgs_linattn_workspace_size(*dims, dtype=dt, backward=case["form"] == "train"), dev)
    return st


# ------------------------------------------------------------- plain forms

def _chunks(st):
    """The inputs in 32 bits, heads expanded, steps past a sequence's length neutral, cut into chunks:
    q, k (B,H,N,C,dk), v (B,H,N,C,dv), log decays (B,H,N,C), the mask of live steps (B,T)."""
    q, k, v, g = st["q"].float(), st["k"].float(), st["v"].float(), st["g"].float()
    B, T, H, dv = v.shape
    rep = H // q.shape[2]
    q, k = q.repeat_interleave(rep, dim=2), k.repeat_interleave(rep, dim=2)
    g = g.expand(B, T, H)
    live = torch.ones(B, T, dtype=torch.bool, device=q.device)
    if st["lengths"] is not None:
        live = torch.arange(T, device=q.device) < st["lengths"][:, None]
    m = live[:, :, None, None]
    q, k, v = q.where(m, 0.0), k.where(m, 0.0), v.where(m, 0.0)
    g = g.where(live[:, :, None], 0.0)

    def cut(x):
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -T % CHUNK))
        return x.unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, 4).contiguous()

    return cut(q), cut(k), cut(v), cut(g[..., None])[..., 0], live


def _join(x, T):
    """(B,H,N,C,d) back to (B,T,H,d)."""
    return x.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :T]


def _decays(g):
    """Of log decays (B,H,N,C): cumulative sums in a chunk, the C x C decays, chunk totals, and the decays between
    chunks: (n, m) from the end of chunk m to the start of chunk n, m < n."""
    G = g.cumsum(-1)
    C, N = g.shape[-1], g.shape[-2]
    low = torch.ones(C, C, dtype=torch.bool, device=g.device).tril()
    L = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf))
    tot = G[..., -1]
    E = tot.cumsum(-1)
    before = torch.ones(N, N, dtype=torch.bool, device=g.device).tril(-1)
    M = torch.exp(((E - tot)[..., :, None] - E[..., None, :]).masked_fill(~before, -math.inf))
    return G, L, tot, E, M


def _plain_attention(st):
    case = st["case"]
    scale = case["dk"] ** -0.5
    T, dt = case["T"], st["q"].dtype
    q, k, v, g, live = _chunks(st)
    G, L, tot, E, M = _decays(g)
    U = (v * torch.exp(tot[..., None] - G)[..., None]).transpose(-1, -2) @ k         # (B,H,N,dv,dk)
    S = (M @ U.flatten(-2)).unflatten(-1, U.shape[-2:])                              # entering each chunk
    last = torch.exp(E[..., -1:] - E)
    ST = (last[..., None, None] * U).sum(2)
    if st["S0"] is not None:
        S = S + torch.exp(E - tot)[..., None, None] * st["S0"][:, :, None]
        ST = ST + torch.exp(E[..., -1])[..., None, None] * st["S0"]
    P = L * (q @ k.transpose(-1, -2))
    o = scale * (P @ v + torch.exp(G)[..., None] * (q @ S.transpose(-1, -2)))
    out = {"o": _join(o, T).to(dt)}
    if case["state"]:
        out["ST"] = ST
    if case["form"] == "fwd":
        return out
    do = st["do"].float().where(live[:, :, None, None], 0.0)
    do = torch.nn.functional.pad(do, (0, 0, 0, 0, 0, -T % CHUNK)).unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, 4)
    do = do.contiguous()
    F = scale * ((do * torch.exp(G)[..., None]).transpose(-1, -2) @ q)               # (B,H,N,dv,dk)
    Mt = M.transpose(-1, -2).contiguous()
    R = (Mt @ F.flatten(-2)).unflatten(-1, F.shape[-2:])                             # from the chunks after
    dS0 = (torch.exp(E - tot)[..., None, None] * F).sum(2)
    if st["dST"] is not None:
        R = R + last[..., None, None] * st["dST"][:, :, None]
        dS0 = dS0 + torch.exp(E[..., -1])[..., None, None] * st["dST"]
    W = scale * L * (do @ v.transpose(-1, -2))
    late = torch.exp(tot[..., None] - G)[..., None]
    dq = W @ k + scale * torch.exp(G)[..., None] * (do @ S)
    dk = W.transpose(-1, -2) @ q + late * (v @ R)
    dv = scale * (P.transpose(-1, -2) @ do) + late * (k @ R.transpose(-1, -2))
    Send = torch.exp(tot)[..., None, None] * S + U
    x = (q * dq).sum(-1) - (k * dk).sum(-1)
    dg = x.flip(-1).cumsum(-1).flip(-1) + (R * Send).sum((-1, -2))[..., None]
    dg = _join(dg[..., None], T)[..., 0].where(live[:, :, None], 0.0)
    out["dg"] = dg if st["g"].dim() == 3 else dg.sum((0, 1))
    groups = (case["Hk"], case["H"] // case["Hk"])
    out["dq"], out["dk"] = (_join(t, T).unflatten(2, groups).sum(3).to(dt) for t in (dq, dk))
    out["dv"] = _join(dv, T).to(dt)
    if case["state"]:
        out["dS0"] = dS0
    return out


def _plain_step(st):
    case = st["case"]
    rep = case["H"] // case["Hk"]
    q, k = (st[n].float().repeat_interleave(rep, dim=1) for n in ("q", "k"))
    v, at = st["v"].float(), st["slots"].long()
    S = torch.exp(st["g"])[..., None, None] * st["S"][at] + v[..., :, None] * k[..., None, :]
    st["S"][at] = S
    o = case["dk"] ** -0.5 * (S * q[..., None, :]).sum(-1)
    return {"o": o.to(st["q"].dtype), "S": st["S"]}


def _groups(y, group):
    """y (rows,d) as (rows, groups, width), the last group padded with zeros."""
    d = y.shape[1]
    width = group or d
    return torch.nn.functional.pad(y, (0, -d % width)).unflatten(1, (-1, width))


def _plain_norm(st):
    case = st["case"]
    dt = st["x"].dtype
    h = st["x"].float() + st["residual"].float()
    w = st["w"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = h * r * w
    if case["form"] == "fp8":
        y = _groups(y, case["group"])
        s = y.abs().amax(-1, keepdim=True).clamp_min(1e-30) / E4M3_MAX
        q = (y / s).flatten(1)[:, :case["d"]].to(torch.float8_e4m3fn)
        return {"y": q, "scale": s[..., 0], "h": h.to(dt)}
    hr = h.to(dt).float()   # the stored sum is what the gradient is taken at
    dy = st["dy"].float()
    e = dy * w
    dx = r * (e - hr * (r * r) * (e * hr).mean(-1, keepdim=True)) + st["dh"].float()
    dw = (dy * hr * r).sum(0)
    return {"y": y.to(dt), "h": h.to(dt), "dx": dx.to(dt), "dw": dw}


def _plain_clip(st):
    squares = torch.stack([t.float().square().sum() for t in st["grads"]])
    n = squares.sum().sqrt()
    c = (st["max_norm"] / (n + CLIP_EPS)).clamp_max(1.0)
    for t, out in zip(st["grads"], st["out"]):
        out.copy_(t.float() * c)
    return {"norm": n, "grads": st["flat"]}


# --------------------------------------------------------------------- run

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "attn":
            return _plain_step(state) if case["form"] == "step" else _plain_attention(state)
        return _plain_norm(state) if op == "norm" else _plain_clip(state)

    mgs = state["mgs"]
    if op == "clip":
        n, _ = mgs.mgs_clip_norm(state["grads"], state["max_norm"], out=state["out"], ws=state["ws"])
        return {"norm": n, "grads": state["flat"]}
    if op == "norm":
        if case["form"] == "fp8":
            y, scale, h = mgs.mgs_rmsnorm_fwd_fp8(state["x"], state["w"], state["residual"], eps=EPS,
                                                  group=case["group"])
            return {"y": y, "scale": scale, "h": h}
        y, h, rstd = mgs.mgs_rmsnorm_fwd(state["x"], state["w"], state["residual"], eps=EPS)
        dx, dw = mgs.mgs_rmsnorm_bwd(state["dy"], h, state["w"], rstd, dh=state["dh"], ws=state["ws"])
        return {"y": y, "h": h, "dx": dx, "dw": dw}
    scale = case["dk"] ** -0.5
    if case["form"] == "step":
        o = mgs.mgs_linattn_step(state["q"], state["k"], state["v"], state["g"], state["S"], slots=state["slots"],
                                 scale=scale)
        return {"o": o, "S": state["S"]}
    args = (state["q"], state["k"], state["v"], state["g"])
    more = dict(S0=state["S0"], lengths=state["lengths"], scale=scale, ws=state["ws"])
    o, ST, _ = mgs.mgs_linattn_fwd(*args, want_state=case["state"], **more)
    out = {"o": o}
    if case["state"]:
        out["ST"] = ST
    if case["form"] == "train":
        grads = mgs.mgs_linattn_bwd(*args, state["do"], dST=state["dST"], **more)
        out["dq"], out["dk"], out["dv"], out["dg"], dS0 = grads
        if case["state"]:
            out["dS0"] = dS0
    return out


# ------------------------------------------------------- 64-bit definitions

def _exact_attention(st):
    """The recurrences step by step; states are kept every 64 steps and stepped again for the gradient."""
    case = st["case"]
    B, T, H, Hk = (case[n] for n in ("B", "T", "H", "Hk"))
    scale = case["dk"] ** -0.5
    time_first = lambda x, rep: x.double().repeat_interleave(rep, dim=2).transpose(0, 1).contiguous()  # noqa: E731
    q, k, v = time_first(st["q"], H // Hk), time_first(st["k"], H // Hk), time_first(st["v"], 1)
    a = torch.exp(st["g"].double()).expand(B, T, H).transpose(0, 1)
    lengths = st["lengths"] if st["lengths"] is not None else torch.full((B,), T, device=q.device)
    on = torch.arange(T, device=q.device)[:, None] < lengths[None, :]            # (T,B)
    a = torch.where(on[:, :, None], a, 1.0)
    m = on[:, :, None, None].double()
    q, k, v = q * m, k * m, v * m
    S = torch.zeros(B, H, case["dv"], case["dk"], dtype=torch.float64, device=q.device)
    if st["S0"] is not None:
        S = st["S0"].double().clone()
    train = case["form"] == "train"
    kept, o = [], torch.empty_like(v)

    def step(S, t):
        return a[t][:, :, None, None] * S + v[t][..., :, None] * k[t][..., None, :]

    for t in range(T):
        if train and t % 64 == 0:
            kept.append(S)
        S = step(S, t)
        o[t] = scale * (S @ q[t][..., None])[..., 0]
    out = {"o": o.transpose(0, 1)}
    if case["state"]:
        out["ST"] = S
    if not train:
        return out
    do = st["do"].double().transpose(0, 1) * m
    D = torch.zeros_like(S) if st["dST"] is None else st["dST"].double().clone()
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a)
    for c in range(len(kept) - 1, -1, -1):
        t0, t1 = 64 * c, min(T, 64 * c + 64)
        states = [kept[c]]
        for t in range(t0, t1):
            states.append(step(states[-1], t))
        for t in range(t1 - 1, t0 - 1, -1):
            dq[t] = scale * (do[t][..., None, :] @ states[t - t0 + 1])[..., 0, :]
            D = D + scale * do[t][..., :, None] * q[t][..., None, :]
            dv[t] = (D @ k[t][..., None])[..., 0]
            dk[t] = (v[t][..., None, :] @ D)[..., 0, :]
            D = a[t][:, :, None, None] * D
            dg[t] = (D * states[t - t0]).sum((-1, -2)) * on[t][:, None]
    per_group = lambda x: (x * m).transpose(0, 1).unflatten(2, (Hk, H // Hk)).sum(3)  # noqa: E731
    dg = dg.transpose(0, 1)
    out.update(dq=per_group(dq), dk=per_group(dk), dv=(dv * m).transpose(0, 1),
               dg=dg if st["g"].dim() == 3 else dg.sum((0, 1)))
    if case["state"]:
        out["dS0"] = D
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float((t.double() ** 2).sum()) for t in st["grads"])
        n = math.sqrt(total)
        c = min(1.0, st["max_norm"] / (n + CLIP_EPS))
        flat, views = _flat_like(st["grads"], torch.float64)
        for t, view in zip(st["grads"], views):
            view.copy_(t.double() * c)
        return {"norm": torch.tensor(n, dtype=torch.float64), "grads": flat}
    if case["op"] == "norm":
        h = st["x"].double() + st["residual"].double()
        w = st["w"].double()
        root = torch.sqrt((h ** 2).sum(1, keepdim=True) / case["d"] + EPS)
        y = h / root * w
        if case["form"] == "fp8":
            width = case["group"] or case["d"]
            starts = range(0, case["d"], width)
            s = torch.stack([y[:, i:i + width].abs().max(1).values.clamp_min(1e-30) / E4M3_MAX for i in starts], 1)
            # the value that the 8 bits round
            ratio = torch.cat([y[:, i:i + width] / s[:, j:j + 1] for j, i in enumerate(starts)], 1)
            return {"y": ratio, "scale": s, "h": h}
        hs = h.to(st["x"].dtype).double()
        e = st["dy"].double() * w
        dot = (e * hs).sum(1, keepdim=True) / case["d"]
        return {"y": y, "h": h, "dx": (e - hs * dot / root ** 2) / root + st["dh"].double(),
                "dw": (st["dy"].double() * hs / root).sum(0)}
    if case["form"] != "step":
        return _exact_attention(st)
    rep = case["H"] // case["Hk"]
    S = st["S"].double()
    o = torch.empty(case["B"], case["H"], case["dv"], dtype=torch.float64, device=S.device)
    for b, slot in enumerate(st["slots"].tolist()):
        k, q = (st[n][b].double().repeat_interleave(rep, dim=0) for n in ("k", "q"))
        S[slot] = torch.exp(st["g"][b].double())[:, None, None] * S[slot] + st["v"][b].double()[:, :, None] * k[:, None, :]
        o[b] = case["dk"] ** -0.5 * (S[slot] @ q[:, :, None])[..., 0]
    return {"o": o, "S": S}


# -------------------------------------------------------------------- work

def work(case):
    """Bytes: every input once, every output once.  Operations: of the recurrence itself, a multiplication and an
    addition for each state element and product (state update, output; for gradients the two state passes and the
    three products)."""
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip":
        sizes = _clip_sizes(case)
        total = sum(n * (size if i % 3 == 0 else 4) for i, n in enumerate(sizes))
        return {"bytes": 2 * total, "flops": 3 * sum(sizes)}
    if case["op"] == "norm":
        n, d = case["rows"] * case["d"], case["d"]
        if case["form"] == "fp8":
            groups = -(-d // case["group"]) if case["group"] else 1
            return {"bytes": n * (3 * size + 1) + d * size + 4 * case["rows"] * groups, "flops": 7 * n}
        return {"bytes": n * 7 * size + d * (size + 4), "flops": 16 * n}
    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    if case["form"] == "step":
        return {"bytes": B * (8 * H * dk * dv + size * (2 * Hk * dk + 2 * H * dv) + 4 * H), "flops": 5 * B * H * dk * dv}
    steps = B * case["T"]
    decay = 4 * steps * H if case["decay"] == "step" else 4 * H
    states = 4 * B * H * dk * dv if case["state"] else 0
    inputs = steps * size * (2 * Hk * dk + H * dv) + decay
    if case["form"] == "fwd":
        return {"bytes": inputs + steps * size * H * dv + 2 * states, "flops": 4 * steps * H * dk * dv}
    # forward and backward: q, k, v, g, do in; o, dq, dk, dv, dg out
    return {"bytes": 2 * inputs + 2 * steps * size * H * dv + 4 * states, "flops": 14 * steps * H * dk * dv}
