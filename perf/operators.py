"""Timed cases of the gated delta rule and of the norms around its block.

Operators (state h [P, N] per batch row b and head h, group of head h: h // (H / G)):

    delta      h' = exp(g_t) h_{t-1},  u_t = beta_t (x_t - h' B_t),  h_t = h' + u_t B_t^T,  y_t = h_t C_t
               fwd  a whole sequence, step  one token from a saved state,
               bwd  the gradients of sum(dy y) + sum(dh_final h_final)
    add_norm   r = residual + scale x,  out = weight r / sqrt(mean(r^2) + eps)           (fwd and bwd)
    norm_gate  out = weight (y / sqrt(mean over the group of y^2 + eps)) silu(z)         (fwd and bwd)

`run` computes them from elementary torch operations in 32 bits (64 for the cumulated decays and
the sums that carry their gradient), or, with `own`, through the library's binding. `exact` walks the
definitions in 64 bits, the delta rule token by token.
"""
import math

import torch

own = False
EPS = 1e-5
CHUNK = 64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases --------------------------------------------------------------------------


def listed():
    return [
        # a short piece appended to a running sequence of a 130M-like layer: latency
        dict(name="delta_fwd_append", op="delta_fwd", dtype="bf16", B=1, L=37, H=24, P=64, G=1, N=128, h0=True),
        # prefill or training forward, 130M-like layer
        dict(name="delta_fwd_130m", op="delta_fwd", dtype="bf16", B=8, L=2048, H=24, P=64, G=1, N=128, h0=False),
        # the same, 2.7B-like layer
        dict(name="delta_fwd_2p7b", op="delta_fwd", dtype="bf16", B=4, L=8192, H=80, P=64, G=1, N=128, h0=False),
        # fp32 storage with odd sizes
        dict(name="delta_fwd_f32_odd", op="delta_fwd", dtype="f32", B=2, L=777, H=6, P=40, G=3, N=36, h0=True),
        # one generated token, one sequence: latency
        dict(name="delta_step_b1", op="delta_step", dtype="bf16", B=1, L=1, H=24, P=64, G=1, N=128, h0=True),
        # one generated token, a serving batch, heads that share keys and queries
        dict(name="delta_step_b64", op="delta_step", dtype="bf16", B=64, L=1, H=32, P=128, G=8, N=128, h0=True),
        # training backward, 130M-like layer
        dict(name="delta_bwd_130m", op="delta_bwd", dtype="bf16", B=4, L=2048, H=24, P=64, G=1, N=128, h0=False),
        # a ragged segment of a longer sequence: state and its cotangent carried over, shared keys
        dict(name="delta_bwd_segment", op="delta_bwd", dtype="bf16", B=1, L=1531, H=32, P=128, G=8, N=128, h0=True),
        # the norm before a block, with the residual stream in fp32
        dict(name="add_norm_fwd_2560", op="add_norm_fwd", dtype="bf16", rdtype="f32", rows=32768, dim=2560, scale=True),
        # its gradient, ragged rows, the residual stream in bf16
        dict(name="add_norm_bwd_2560", op="add_norm_bwd", dtype="bf16", rdtype="bf16", rows=8191, dim=2560, scale=True),
        # the norm after the layer: one group per head, z a column slice of the projection's rows
        dict(name="norm_gate_fwd_5120", op="norm_gate_fwd", dtype="bf16", rows=32768, dim=5120, groups=80),
        # its gradient
        dict(name="norm_gate_bwd_1536", op="norm_gate_bwd", dtype="bf16", rows=16384, dim=1536, groups=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _within(case, n, gbytes, gflops):
    """case with its length n ("L" or "rows") cut so that a pass stays within that work."""
    w = work(case)
    f = min(1.0, gbytes * 1e9 / w["bytes"], gflops * 1e9 / max(1, w["flops"]))
    return case if f == 1.0 else dict(case, **{n: max(1, int(f * case[n]))})


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_step", "delta_bwd", "delta_bwd", "add_norm_fwd", "add_norm_bwd",
                     "norm_gate_fwd", "norm_gate_bwd"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op.startswith("delta"):
        G = rng.choice([1, 1, 2, 4, 8])
        H = G * rng.randint(1, 80 // G)
        if rng.random() < 0.7:
            P, N = rng.choice([64, 128]), rng.choice([64, 128])
        else:
            P, N = rng.randint(1, 256), 4 * rng.randint(1, 64) if op == "delta_step" else rng.randint(1, 256)
        if op == "delta_step":
            return _within(dict(op=op, dtype=dtype, B=_log(rng, 1, 128), L=1, H=H, P=P, G=G, N=N, h0=True), "B", 0.5, 100)
        case = dict(op=op, dtype=dtype, B=rng.randint(1, 8), L=_log(rng, 1, 8192), H=H, P=P, G=G, N=N, h0=rng.random() < 0.5)
        return _within(case, "L", 0.5, 40 if dtype == "bf16" else 10)
    if op.startswith("add_norm"):
        dim = _log(rng, 64, 8192) if rng.random() < 0.5 else 64 * _log(rng, 1, 128)
        return _within(dict(op=op, dtype=dtype, rdtype=rng.choice(["f32", dtype]), rows=_log(rng, 1, 65536), dim=dim,
                            scale=rng.random() < 0.5), "rows", 0.7, 100)
    gs = rng.choice([64, 128, 256]) if rng.random() < 0.6 else 64 * rng.randint(1, 32)
    groups = rng.randint(1, max(1, 8192 // gs))
    return _within(dict(op=op, dtype=dtype, rows=_log(rng, 1, 65536), dim=gs * groups, groups=groups), "rows", 0.7, 100)


# ---- inputs -------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=gen, device="cuda")

    if case["op"].startswith("delta"):
        B, L, H, P, G, N = (case[k] for k in ("B", "L", "H", "P", "G", "N"))
        unit = lambda v: v / v.norm(dim=-1, keepdim=True)  # noqa: E731
        s["x"] = normal(B, L, H, P).to(dt)
        s["Bm"] = unit(normal(B, L, G, N)).to(dt)
        s["Cm"] = (unit(normal(B, L, G, N)) * N ** -0.5).to(dt)
        # a layer's step sizes (softplus of a projection plus a per-head bias) times its decay rates
        step = torch.nn.functional.softplus(normal(B, L, H) + uniform(-7.0, -2.3, H))
        s["g"] = (-step * torch.exp(uniform(0.0, math.log(16.0), H))).to(dt)
        s["beta"] = torch.sigmoid(normal(B, L, H)).to(dt)
        s["h0"] = 0.1 * normal(B, H, P, N) if case["h0"] else None
        if case["op"] == "delta_step":
            for k in ("x", "Bm", "Cm", "g", "beta"):
                s[k] = s[k][:, 0].contiguous()
        if case["op"] == "delta_bwd":
            s["dy"] = normal(B, L, H, P).to(dt)
            s["dh_final"] = normal(B, H, P, N) if case["h0"] else None
        return s
    rows, dim = case["rows"], case["dim"]
    s["weight"] = 1 + 0.1 * normal(dim)
    if case["op"].startswith("add_norm"):
        s["x"] = normal(rows, dim).to(dt)
        s["residual"] = (2 * normal(rows, dim)).to(DT[case["rdtype"]])
        s["scale"] = 1 + 0.1 * normal(dim) if case["scale"] else None
    else:
        s["y"] = normal(rows, dim).to(dt)
        s["z"] = normal(rows, 2 * dim).to(dt)[:, :dim]  # columns of the input projection's rows
    if case["op"].endswith("bwd"):
        s["dout"] = normal(rows, dim).to(dt)
        if case["op"] == "add_norm_bwd":
            s["dres"] = normal(rows, dim).to(DT[case["rdtype"]])
    return s


# ---- plain forms --------------------------------------------------------------------


def _chunks(s):
    """The chunked form's parts, [B, H, chunks, tokens, ...] in fp32 (cumulated decays in fp64), tokens
    padded with zeros."""
    B, L, H, P = s["x"].shape
    G, N = s["Bm"].shape[2:]
    C = 1 << (min(CHUNK, L) - 1).bit_length()
    n = -(-L // C)

    def cut(t, rep):
        t = torch.nn.functional.pad(t.float(), (0, 0) * (t.dim() - 2) + (0, n * C - L))
        t = t.reshape(B, n, C, *t.shape[2:]).transpose(2, 3).transpose(1, 2)
        return t.repeat_interleave(rep, dim=1) if rep > 1 else t

    x, k, q = cut(s["x"], 1), cut(s["Bm"], H // G), cut(s["Cm"], H // G)
    g, beta = cut(s["g"], 1), cut(s["beta"], 1).unsqueeze(-1)
    cum = g.double().cumsum(-1)
    i = torch.arange(C, device=x.device)
    low = i[:, None] >= i[None, :]
    E = (cum.unsqueeze(-1) - cum.unsqueeze(-2)).masked_fill(~low, -math.inf).exp().float()
    KK = (k @ k.mT) * E
    KK = KK.masked_fill(i[:, None] <= i[None, :], 0.0)
    # T = (I + beta KK)^-1, its diagonal blocks joined in pairs: the block below two of them is -T2 A21 T1
    A = beta * KK
    T, w = torch.ones(*A.shape[:3], C, 1, 1, device=x.device), 1
    while w < C:
        m = C // (2 * w)
        pair = A.reshape(*A.shape[:3], m, 2, w, m, 2, w)[..., 1, :, :, 0, :]
        A21 = pair.diagonal(dim1=3, dim2=5).movedim(-1, 3)
        T = T.reshape(*T.shape[:3], m, 2, w, w)
        T1, T2 = T[:, :, :, :, 0], T[:, :, :, :, 1]
        below = torch.cat([-T2 @ A21 @ T1, T2], -1)
        T = torch.cat([torch.nn.functional.pad(T1, (0, w)), below], -2)
        w *= 2
    T = T.reshape(A.shape)
    return dict(x=x, k=k, q=q, beta=beta, E=E, KK=KK, T=T, PQ=(q @ k.mT) * E, eg=cum.exp().float().unsqueeze(-1),
                ek=(cum[..., -1:] - cum).exp().float().unsqueeze(-1), gamma=cum[..., -1].exp().float()[..., None, None],
                n=n, L=L)


def _uncut(t, L):
    """[B, H, n, C, ...] -> [B, L, H, ...]"""
    t = t.transpose(1, 2).transpose(2, 3)
    return t.reshape(t.shape[0], -1, *t.shape[3:])[:, :L]


def _plain_states(s, c):
    """The state entering each chunk, u, and the final state."""
    B, L, H, P = s["x"].shape
    N = s["Bm"].shape[3]
    S = s["h0"].float() if s["h0"] is not None else torch.zeros(B, H, P, N, device=s["x"].device)
    U0 = c["T"] @ (c["beta"] * c["x"])
    W = c["T"] @ (c["beta"] * c["eg"] * c["k"])
    kd = c["ek"] * c["k"]
    S0, u = [], []
    for m in range(c["n"]):
        S0.append(S)
        u.append(U0[:, :, m] - W[:, :, m] @ S.mT)
        S = c["gamma"][:, :, m] * S + u[m].mT @ kd[:, :, m]
    return torch.stack(S0, 2), torch.stack(u, 2), S


def _plain_delta_fwd(s):
    c = _chunks(s)
    S0, u, S = _plain_states(s, c)
    y = (c["eg"] * c["q"]) @ S0.mT + c["PQ"] @ u
    return {"y": _uncut(y, c["L"]).to(s["x"].dtype), "h_final": S}


def _plain_delta_step(s):
    H, G = s["x"].shape[1], s["Bm"].shape[1]
    k, q = (s[n].float().repeat_interleave(H // G, dim=1) for n in ("Bm", "Cm"))
    S = s["g"].float().exp()[..., None, None] * s["h0"]
    u = s["beta"].float()[..., None] * (s["x"].float() - (S * k.unsqueeze(2)).sum(-1))
    S = S + u.unsqueeze(-1) * k.unsqueeze(2)
    return {"y": (S * q.unsqueeze(2)).sum(-1).to(s["x"].dtype), "state": S}


def _plain_delta_bwd(s):
    c = _chunks(s)
    S0, u, S1 = _plain_states(s, c)
    B, L, H, P = s["x"].shape
    G, N = s["Bm"].shape[2:]
    C = c["x"].shape[3]
    pad = (0, 0) * 2 + (0, c["n"] * C - L)
    dy = torch.nn.functional.pad(s["dy"].float(), pad).reshape(B, c["n"], C, H, P).transpose(2, 3).transpose(1, 2)
    k, q, eg, ek, beta, E = (c[n] for n in ("k", "q", "eg", "ek", "beta", "E"))
    dS = s["dh_final"] if s["dh_final"] is not None else torch.zeros_like(S1)
    W = c["T"].mT @ (c["PQ"].mT @ dy)
    Tk = c["T"].mT @ (ek * k)
    a, b = (eg * q).mT, eg * k
    own_S = a @ dy
    dS1, z = [None] * c["n"], [None] * c["n"]
    for m in reversed(range(c["n"])):
        dS1[m] = dS
        z[m] = W[:, :, m] + Tk[:, :, m] @ dS.mT
        dS = c["gamma"][:, :, m] * dS + own_S[:, :, m].mT - (beta[:, :, m] * z[m]).mT @ b[:, :, m]
    dS1, z = torch.stack(dS1, 2), torch.stack(z, 2)
    dr = beta * z
    rhat = c["x"] - eg * (k @ S0.mT) - c["KK"] @ u
    dP = (dy @ u.mT) * E
    dM = -((dr @ u.mT) * E).tril(-1)
    dyS, drS, udS = eg * (dy @ S0), eg * (dr @ S0), ek * (u @ dS1)
    dq = dyS + dP @ k
    dk = dP.mT @ q + dM @ k + dM.mT @ k + udS - drS
    pairs = (dP * (q @ k.mT)).double() + (dM * (k @ k.mT)).double()
    dot = lambda v, w: (v * w).sum(-1, dtype=torch.float64)  # noqa: E731
    U = dot(udS, k)
    dcum = pairs.sum(-1) - pairs.sum(-2) + dot(dyS, q) - dot(drS, k) - U
    dcum[..., -1] += U.sum(-1) + (c["gamma"] * dS1 * S0).sum((-1, -2), dtype=torch.float64)
    dg = dcum.flip(-1).cumsum(-1).flip(-1)

    def grouped(t):
        return _uncut(t.reshape(B, G, H // G, c["n"], C, N).sum(2), L).to(s["x"].dtype)

    out = {"dx": _uncut(dr, L), "dg": _uncut(dg, L), "dbeta": _uncut((z * rhat).sum(-1), L)}
    out = {n: t.to(s["x"].dtype) for n, t in out.items()}
    return out | {"dB": grouped(dk), "dC": grouped(dq)} | ({"dh0": dS} if s["h0"] is not None else {})


def _plain_add_norm_fwd(s):
    x = s["x"].float()
    r = s["residual"].float() + (x if s["scale"] is None else s["scale"] * x)
    out = s["weight"] * r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return {"res": r.to(s["residual"].dtype), "out": out.to(s["x"].dtype)}


def _plain_add_norm_bwd(s):
    r, do = s["residual"].float(), s["dout"].float()  # the saved sum
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n = r * rstd
    wdo = s["weight"] * do
    dr = s["dres"].float() + rstd * (wdo - n * (wdo * n).mean(-1, keepdim=True))
    out = {"dres": dr.to(s["residual"].dtype), "dw": (do * n).sum(0)}
    out["dx"] = (dr if s["scale"] is None else s["scale"] * dr).to(s["x"].dtype)
    if s["scale"] is not None:
        out["dscale"] = (dr * s["x"].float()).sum(0)
    return out


def _grouped_norm(s):
    shape = (s["y"].shape[0], s["case"]["groups"], -1)
    y, z, w = s["y"].float().reshape(shape), s["z"].float().reshape(shape), s["weight"].reshape(1, *shape[1:])
    rstd = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    sig = torch.sigmoid(z)
    return shape, y * rstd, rstd, z, sig, w


def _plain_norm_gate_fwd(s):
    shape, n, rstd, z, sig, w = _grouped_norm(s)
    return {"out": (w * n * z * sig).reshape(s["y"].shape).to(s["y"].dtype)}


def _plain_norm_gate_bwd(s):
    shape, n, rstd, z, sig, w = _grouped_norm(s)
    do = s["dout"].float().reshape(shape)
    gate = z * sig
    dn = w * do * gate
    dy = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    dz = w * n * do * sig * (1 + z * (1 - sig))
    to = lambda t: t.reshape(s["y"].shape).to(s["y"].dtype)  # noqa: E731
    return {"dy": to(dy), "dz": to(dz), "dw": (do * n * gate).sum(0).reshape(-1)}


# ---- the library's calls ------------------------------------------------------------


def _own(s):
    from state_space_sequence_chunked_b200 import _binding as ssd

    op = s["case"]["op"]
    if op == "delta_fwd":
        y, hf = ssd.ssd_delta_fwd(s["x"], s["g"], s["beta"], s["Bm"], s["Cm"], s["h0"])
        return {"y": y, "h_final": hf}
    if op == "delta_step":
        state = torch.empty_like(s["h0"])  # not in place, so that a pass can be repeated on the same state
        y = ssd.ssd_delta_decode_step(s["h0"], s["x"], s["g"], s["beta"], s["Bm"], s["Cm"], state_out=state)
        return {"y": y, "state": state}
    if op == "delta_bwd":
        o = ssd.ssd_delta_bwd(s["x"], s["g"], s["beta"], s["Bm"], s["Cm"], s["h0"], s["dy"], s["dh_final"],
                              want_dh0=s["h0"] is not None)
        return {n: o[n] for n in ("dx", "dg", "dbeta", "dB", "dC", "dh0") if o[n] is not None}
    if op == "add_norm_fwd":
        res, out = ssd.ssd_add_rmsnorm(s["x"], s["residual"], s["weight"], scale=s["scale"], eps=EPS)
        return {"res": res, "out": out}
    if op == "add_norm_bwd":
        o = ssd.ssd_add_rmsnorm_bwd(s["residual"], s["weight"], s["dout"], s["dres"], x=s["x"], scale=s["scale"], eps=EPS)
        return {n: o[n] for n in ("dres", "dx", "dw", "dscale") if o[n] is not None}
    if op == "norm_gate_fwd":
        return {"out": ssd.ssd_norm_gate(s["y"], s["z"], s["weight"], ngroups=s["case"]["groups"], eps=EPS)}
    o = ssd.ssd_norm_gate_bwd(s["y"], s["z"], s["weight"], s["dout"], ngroups=s["case"]["groups"], eps=EPS)
    return {n: o[n] for n in ("dy", "dz", "dw")}


PLAIN = {"delta_fwd": _plain_delta_fwd, "delta_step": _plain_delta_step, "delta_bwd": _plain_delta_bwd,
         "add_norm_fwd": _plain_add_norm_fwd, "add_norm_bwd": _plain_add_norm_bwd,
         "norm_gate_fwd": _plain_norm_gate_fwd, "norm_gate_bwd": _plain_norm_gate_bwd}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- the work that cannot be avoided ------------------------------------------------


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("delta"):
        B, L, H, P, G, N = (case[k] for k in ("B", "L", "H", "P", "G", "N"))
        tok, state = B * L, B * H * P * N
        inputs = es * tok * (H * P + 2 * H + 2 * G * N)
        if op == "delta_bwd":  # inputs, dy; gradients of all; h0, dh_final, dh0
            return {"bytes": 2 * inputs + es * tok * H * P + (12 * state if case["h0"] else 0), "flops": 16 * tok * H * P * N}
        states = 8 * state if case["h0"] else 4 * state
        return {"bytes": inputs + es * tok * H * P + states, "flops": 6 * tok * H * P * N}
    n = case["rows"] * case["dim"]
    if op.startswith("add_norm"):
        rs = 2 if case["rdtype"] == "bf16" else 4
        if op == "add_norm_fwd":
            return {"bytes": n * (2 * es + 2 * rs) + 8 * case["dim"], "flops": 6 * n}
        return {"bytes": n * (2 * es + 3 * rs + (es if case["scale"] else 0)) + 16 * case["dim"], "flops": 14 * n}
    if op == "norm_gate_fwd":
        return {"bytes": 3 * es * n + 4 * case["dim"], "flops": 9 * n}
    return {"bytes": 5 * es * n + 8 * case["dim"], "flops": 24 * n}


# ---- the definitions in 64 bits -----------------------------------------------------


def _tokens(s):
    """fp64 x, beta, k, q, decay with the token axis first and keys, queries per head."""
    H, G = s["x"].shape[2], s["Bm"].shape[2]
    first = lambda t: t.double().transpose(0, 1)  # noqa: E731
    heads = lambda t: first(t).repeat_interleave(H // G, dim=2)  # noqa: E731
    return first(s["x"]), first(s["beta"]), heads(s["Bm"]), heads(s["Cm"]), first(s["g"]).exp()


def _token(S, x, beta, k, a):
    """One token: the decayed state, the prediction error, and the state after it."""
    Sd = a[..., None, None] * S
    err = x - torch.einsum("bhpn,bhn->bhp", Sd, k)
    return Sd, err, Sd + torch.einsum("bhp,bhn->bhpn", beta[..., None] * err, k)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("delta"):
        if op == "delta_step":
            s = {n: v.unsqueeze(1) if n in ("x", "Bm", "Cm", "g", "beta") else v for n, v in s.items()}
        x, beta, k, q, a = _tokens(s)
        L, B, H, P = x.shape
        N = k.shape[3]
        S = s["h0"].double() if s["h0"] is not None else torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda")
        if op != "delta_bwd":
            y = torch.empty_like(x)
            for t in range(L):
                S = _token(S, x[t], beta[t], k[t], a[t])[2]
                y[t] = torch.einsum("bhpn,bhn->bhp", S, q[t])
            if op == "delta_step":
                return {"y": y[0], "state": S}
            return {"y": y.transpose(0, 1), "h_final": S}
        # reverse walk; the states of one segment at a time are formed again from its first
        seg = max(1, min(64, (1 << 27) // max(1, B * H * P * N)))
        starts = []
        for t in range(L):
            if t % seg == 0:
                starts.append(S)
            S = _token(S, x[t], beta[t], k[t], a[t])[2]
        dS = s["dh_final"].double() if s["dh_final"] is not None else torch.zeros_like(S)
        dy = s["dy"].double().transpose(0, 1)
        dx, dbeta, dg = torch.empty_like(x), torch.empty_like(beta), torch.empty_like(a)
        dk, dq = torch.empty_like(k), torch.empty_like(q)
        for m in reversed(range(len(starts))):
            S, kept = starts[m], []
            for t in range(m * seg, min(L, (m + 1) * seg)):
                Sd, err, S = _token(S, x[t], beta[t], k[t], a[t])
                kept.append((t, Sd, err, S))
            while kept:
                t, Sd, err, S = kept.pop()
                dq[t] = torch.einsum("bhp,bhpn->bhn", dy[t], S)
                dS = dS + torch.einsum("bhp,bhn->bhpn", dy[t], q[t])
                du = torch.einsum("bhpn,bhn->bhp", dS, k[t])
                dbeta[t] = (du * err).sum(-1)
                dx[t] = beta[t][..., None] * du
                dk[t] = torch.einsum("bhp,bhpn->bhn", beta[t][..., None] * err, dS) - torch.einsum("bhp,bhpn->bhn", dx[t], Sd)
                dS = dS - torch.einsum("bhp,bhn->bhpn", dx[t], k[t])
                dg[t] = (dS * Sd).sum((-1, -2))
                dS = a[t][..., None, None] * dS
        G = s["Bm"].shape[2]
        back = lambda t: t.transpose(0, 1)  # noqa: E731
        heads = lambda t: back(t).reshape(B, L, G, H // G, N).sum(3)  # noqa: E731
        out = {"dx": back(dx), "dg": back(dg), "dbeta": back(dbeta), "dB": heads(dk), "dC": heads(dq)}
        return out | ({"dh0": dS} if s["h0"] is not None else {})
    w = s["weight"].double()
    if op.startswith("add_norm"):
        scale = 1.0 if s["scale"] is None else s["scale"].double()
        r = s["residual"].double()
        if op == "add_norm_fwd":
            r = r + scale * s["x"].double()
            return {"res": r, "out": w * r / ((r ** 2).mean(1, keepdim=True) + EPS).sqrt()}
        root = ((r ** 2).mean(1, keepdim=True) + EPS).sqrt()
        do = s["dout"].double()
        # out_i = w_i r_i / root: d out_i / d r_j = w_i (1[i = j] / root - r_i r_j / (dim root^3))
        dr = s["dres"].double() + w * do / root - r * (w * do * r).sum(1, keepdim=True) / (case["dim"] * root ** 3)
        out = {"dres": dr, "dx": scale * dr, "dw": (do * r / root).sum(0)}
        return out | ({"dscale": (dr * s["x"].double()).sum(0)} if s["scale"] is not None else {})
    rows, groups = case["rows"], case["groups"]
    y, z = s["y"].double().view(rows, groups, -1), s["z"].double().reshape(rows, groups, -1)
    w = w.view(groups, -1)
    root = ((y ** 2).mean(2, keepdim=True) + EPS).sqrt()
    silu = z / (1 + (-z).exp())
    if op == "norm_gate_fwd":
        return {"out": (w * y / root * silu).reshape(rows, -1)}
    do = s["dout"].double().view(rows, groups, -1)
    v = w * do * silu
    dy = v / root - y * (v * y).sum(2, keepdim=True) / (y.shape[2] * root ** 3)
    dsilu = (1 + (-z).exp() * (1 + z)) / (1 + (-z).exp()) ** 2
    flat = lambda t: t.reshape(rows, -1)  # noqa: E731
    return {"dy": flat(dy), "dz": flat(w * y / root * do * dsilu), "dw": (do * y / root * silu).sum(0).reshape(-1)}
