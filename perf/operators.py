"""Cases of the delta-rule fast weight and of the norms around it.

Operators:
  fwd       gated delta rule over a sequence (chunked form), start state in, end state out
  bwd       its gradients
  step      its form for single tokens: one token of every row, states in a pool, by slot
  norm      row norm with weight, gate and scaled residual
  norm_bwd  its gradients

With a_t = exp(g_t) and a state S [dk, dv] per head:
  e_t = v_t - a_t S_{t-1}^T k_t,  S_t = a_t S_{t-1} + beta_t k_t e_t^T,  o_t = scale S_t^T q_t
  y = res + rscale * x * r(x) * w * act(z)
"""
import math

import torch

own = False

CHUNK = 64
F32, BF16 = torch.float32, torch.bfloat16
_TYPES = {"f32": F32, "bf16": BF16}


def listed():
    return [
        # the smallest float32 layer: latency of one call, every token's work in 32 bits
        dict(name="fwd_f32_n256", op="fwd", type="f32", B=1, H=2, N=256, dk=32, dv=32, decay=True),
        # a language layer's whole 32K context, 64 heads of 64 (training forward, prefill)
        dict(name="fwd_n32k_d64", op="fwd", type="bf16", B=4, H=16, N=32768, dk=64, dv=64, decay=True),
        # few heads of 128 over a long odd prompt: little to run side by side
        dict(name="fwd_n32749_d128", op="fwd", type="bf16", B=2, H=4, N=32749, dk=128, dv=128, decay=True),
        # unequal odd dims, no decay, fewer tokens than one tile
        dict(name="bwd_f32_n77", op="bwd", type="f32", B=2, H=3, N=77, dk=24, dv=40, decay=False),
        # a training step's backward, 32 heads of 64
        dict(name="bwd_n8k_d64", op="bwd", type="bf16", B=2, H=16, N=8192, dk=64, dv=64, decay=True),
        # the same for heads of 128, odd length
        dict(name="bwd_n4111_d128", op="bwd", type="bf16", B=2, H=4, N=4111, dk=128, dv=128, decay=True),
        # serving one sequence: latency
        dict(name="step_b1", op="step", type="bf16", B=1, H=16, dk=128, dv=128, slots=4, idle=0, decay=True),
        # serving a large batch, some rows idle, states scattered over a pool
        dict(name="step_b256", op="step", type="bf16", B=256, H=16, dk=128, dv=128, slots=320, idle=9, decay=True),
        # keys of a short call before the layer
        dict(name="norm_l2_f32", op="norm", type="f32", rows=515, D=40, kind="l2", weight=False, gate="none", res=False),
        # the layer's outputs: norm, gate, residual
        dict(name="norm_gate_res", op="norm", type="bf16", rows=262144, D=128, kind="rms", weight=True, gate="silu", res=True),
        # gradients of a short call
        dict(name="norm_bwd_l2_f32", op="norm_bwd", type="f32", rows=771, D=24, kind="l2", weight=False, gate="none", res=False),
        # gradients of a training step's outputs
        dict(name="norm_bwd_gate", op="norm_bwd", type="bf16", rows=262144, D=128, kind="rms", weight=True, gate="silu", res=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd"])
    if op in ("fwd", "bwd"):
        # half of the draws: the 16-bit type with heads of 64 or 128, over the whole range of lengths
        if rng.random() < 0.6:
            d, B, H = rng.choice([64, 128]), rng.randint(1, 4), rng.choice([1, 2, 3, 4, 6, 8, 16])
            most = (4 * 16 * 32768 * 64 if op == "fwd" else 2 * 16 * 8192 * 64) // (B * H * d)
            N = _log(rng, 1, min(most, 32768 if op == "fwd" else 8192))
            return dict(op=op, type="bf16", B=B, H=H, N=N, dk=d, dv=d, decay=rng.random() < 0.8)
        return dict(op=op, type=rng.choice(["f32", "bf16"]), B=rng.randint(1, 3), H=rng.randint(1, 5), N=_log(rng, 1, 2048),
                    dk=rng.randint(1, 16) * 8, dv=rng.randint(1, 16) * 8, decay=rng.random() < 0.8)
    if op == "step":
        B = _log(rng, 1, 256)
        d = rng.choice([(64, 64), (128, 128), (rng.randint(1, 16) * 8, rng.randint(1, 16) * 8)])
        return dict(op=op, type=rng.choice(["f32", "bf16", "bf16"]), B=B, H=rng.choice([1, 2, 4, 8, 16]), dk=d[0], dv=d[1],
                    slots=B + rng.randint(0, 64), idle=rng.randint(0, B // 8), decay=rng.random() < 0.8)
    D = 8 * _log(rng, 1, 256)
    return dict(op=op, type=rng.choice(["f32", "bf16", "bf16"]), rows=_log(rng, 1, min(262144, 262144 * 128 // D)), D=D,
                kind=rng.choice(["rms", "l2"]), weight=rng.random() < 0.7, gate=rng.choice(["none", "silu", "sigmoid"]), res=op == "norm" and rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["type"]]

    def normal(*shape, type=t, scale=1.0):
        x = torch.randn(shape, generator=gen, device="cuda")
        return (x if scale == 1.0 else x * scale).to(type)

    st = dict(case=dict(case))
    if case["op"] in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        st["x"] = normal(R, D)
        st["w"] = 1 + normal(D, type=F32, scale=0.1) if case["weight"] else None
        st["z"] = normal(R, D) if case["gate"] != "none" else None
        st["res"] = normal(R, D) if case["res"] else None
        if case["op"] == "norm_bwd":
            st["dout"] = normal(R, D)
        return st

    B, H, dk, dv = (case[n] for n in ("B", "H", "dk", "dv"))
    lead = (B, H) if case["op"] == "step" else (B, H, case["N"])
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    # queries and keys of unit length, as the norm before the layer leaves them
    st["q"] = unit(normal(*lead, dk, type=F32)).to(t)
    st["k"] = unit(normal(*lead, dk, type=F32)).to(t)
    st["v"] = normal(*lead, dv)
    st["beta"] = torch.sigmoid(normal(*lead, type=F32)).to(t)
    # decays between nearly none and about a half a token
    st["g"] = (-torch.nn.functional.softplus(1.5 * normal(*lead, type=F32) - 4)).to(t) if case["decay"] else None
    if case["op"] == "step":
        st["S"] = normal(case["slots"], H, dk, dv, type=F32, scale=0.1)
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        rows = torch.randperm(B, generator=gen, device="cuda")
        idle = rows[: case["idle"]]
        slots[idle] = -1
        st["slots"] = slots
        st["rows"] = rows[case["idle"]:].sort().values  # the rows that hold a sequence
        st["at"] = slots[st["rows"]].long()  # and their states
        st["out"] = torch.zeros(B, H, dv, dtype=t, device="cuda")
        return st
    st["S"] = normal(B, H, dk, dv, type=F32, scale=0.1)
    if case["op"] == "bwd":
        st["dout"] = normal(*lead, dv)
        st["dS"] = normal(B, H, dk, dv, type=F32, scale=0.1)
    return st


# ------------------------------------------------------------------ plain forms
def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., C, C], C a power of two, by blocks of 1, 2, 4, ... rows."""
    C = A.shape[-1]
    T = torch.eye(C, dtype=A.dtype, device=A.device).expand(A.shape)
    s = 1
    while s < C:
        n = C // (2 * s)
        at = lambda X: X.reshape(*X.shape[:-2], n, 2 * s, n, 2 * s).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)  # noqa: E731
        Ab, Tb = at(A), at(T)
        low = -(Tb[..., s:, s:] @ Ab[..., s:, :s] @ Tb[..., :s, :s])
        blocks = torch.cat([torch.cat([Tb[..., :s, :s], torch.zeros_like(low)], -1), torch.cat([low, Tb[..., s:, s:]], -1)], -2)
        T = torch.diag_embed(blocks.movedim(-3, -1), dim1=-4, dim2=-2).reshape(A.shape)
        s *= 2
    return T


def _delta(q, k, v, g, beta, S, scale):
    """Chunked form in 32 bits: q, k [M, N, dk], v [M, N, dv], g, beta [M, N], S [M, dk, dv] -> (o, end state)."""
    M, N, _ = q.shape
    C, n = CHUNK, -(-N // CHUNK)
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, n * C - N)).reshape(M, n, C, x.shape[-1])  # noqa: E731
    q, k, v, beta = cut(q), cut(k), cut(v), cut(beta.unsqueeze(-1))
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    strict = low.tril(-1)
    if g is None:
        G = torch.zeros(M, n, C, 1, dtype=torch.float64, device=q.device)
    else:
        G = cut(g.unsqueeze(-1)).double().cumsum(2)
    gam = torch.exp(G).float()
    dec = torch.exp((G - G.transpose(-1, -2)).masked_fill(~low, 0.0)).float()
    last = G[:, :, -1:]
    end, rest = torch.exp(last).float(), torch.exp(last - G).float()
    A = (beta * dec * (k @ k.transpose(-1, -2))).masked_fill(~strict, 0.0)
    T = _inverse(A)
    W, Ut = T @ (beta * gam * k), T @ (beta * v)
    Kt = (rest * k).transpose(-1, -2)
    starts, us = [], []
    for c in range(n):
        starts.append(S)
        us.append(Ut[:, c] - W[:, c] @ S)
        S = end[:, c] * S + Kt[:, c] @ us[-1]
    S0, U = torch.stack(starts, 1), torch.stack(us, 1)
    P = (dec * (q @ k.transpose(-1, -2))).masked_fill(~low, 0.0)
    o = scale * ((gam * q) @ S0 + P @ U)
    return o.reshape(M, n * C, -1)[:, :N], S


def _heads(st, names):
    """The tensors of those names as 32-bit values [heads, ...]; None stays."""
    return [None if st[n] is None else st[n].float().flatten(0, 1) for n in names]


def _act(z, gate):
    return torch.sigmoid(z) if gate == "sigmoid" else z * torch.sigmoid(z)


def _rstd(x, case):
    eps, sq = 1e-6, x.square().sum(-1, keepdim=True)
    return 1 / torch.sqrt(sq / case["D"] + eps) if case["kind"] == "rms" else 1 / torch.sqrt(sq).clamp_min(eps)


def _norm(st):
    c, x = st["case"], st["x"].float()
    y = x * _rstd(x, c)
    if st["w"] is not None:
        y = y * st["w"]
    if st["z"] is not None:
        y = y * _act(st["z"].float(), c["gate"])
    y = y * _RSCALE
    if st["res"] is not None:
        y = y + st["res"].float()
    return y.to(st["x"].dtype)


def _norm_bwd(st):
    c, x, dy = st["case"], st["x"].float(), st["dout"].float() * _RSCALE
    r = _rstd(x, c)
    xn, out = x * r, {}
    dn = dy
    if st["z"] is not None:
        z = st["z"].float()
        s = torch.sigmoid(z)
        a = s if c["gate"] == "sigmoid" else z * s
        da = s * (1 - s) if c["gate"] == "sigmoid" else s * (1 + z * (1 - s))
        yw = xn if st["w"] is None else xn * st["w"]
        out["dz"] = (dy * yw * da).to(st["x"].dtype)
        dn = dn * a
    if st["w"] is not None:
        out["dw"] = (dn * xn).sum(0)
        dn = dn * st["w"]
    n = c["D"] if c["kind"] == "rms" else 1
    out["dx"] = (r * (dn - xn * (dn * xn).sum(-1, keepdim=True) / n)).to(st["x"].dtype)
    return out


def _plain(st):
    c = st["case"]
    if c["op"] == "norm":
        return _norm(st)
    if c["op"] == "norm_bwd":
        return _norm_bwd(st)
    scale, t = c["dk"] ** -0.5, st["q"].dtype
    if c["op"] == "fwd":
        q, k, v, g, beta = _heads(st, ("q", "k", "v", "g", "beta"))
        o, S = _delta(q, k, v, g, beta, st["S"].flatten(0, 1), scale)
        st["S"].copy_(S.reshape(st["S"].shape))
        return {"out": o.reshape(st["v"].shape).to(t), "S": st["S"]}
    if c["op"] == "bwd":
        names = [n for n in ("q", "k", "v", "g", "beta") if st[n] is not None]
        leaf = {n: x.requires_grad_() for n, x in zip(names, _heads(st, names))}
        S0 = st["S"].flatten(0, 1).clone().requires_grad_()
        o, S = _delta(leaf["q"], leaf["k"], leaf["v"], leaf.get("g"), leaf["beta"], S0, scale)
        ins = [leaf[n] for n in names] + [S0]
        got = torch.autograd.grad([o, S], ins, [st["dout"].float().flatten(0, 1), st["dS"].flatten(0, 1)])
        out = {"d" + n: x.reshape(st[n].shape).to(t) for n, x in zip(names, got)}
        out["dS0"] = got[-1].reshape(st["S"].shape)
        return out
    # one token of every row that holds a sequence
    q, k, v, beta = (st[n][st["rows"]].float() for n in ("q", "k", "v", "beta"))
    S = st["S"][st["at"]]
    if st["g"] is not None:
        S = S * torch.exp(st["g"][st["rows"]].float())[..., None, None]
    e = v - (k.unsqueeze(-2) @ S).squeeze(-2)
    S = S + k.unsqueeze(-1) * (beta.unsqueeze(-1) * e).unsqueeze(-2)
    st["S"][st["at"]] = S
    st["out"][st["rows"]] = (scale * (q.unsqueeze(-2) @ S).squeeze(-2)).to(t)
    return {"out": st["out"], "S": st["S"]}


# ------------------------------------------------------------------ the framework's operators
_RSCALE = 0.5
_kept = {}


def _workspace(T, nbytes):
    """The one workspace of this program: it grows to the largest call."""
    if _kept.get("size", -1) < nbytes:
        _kept["ws"] = T.alloc_workspace(nbytes)
        _kept["size"] = nbytes
    return _kept["ws"]


def _own(st):
    import learned_linear_attention_b200 as T

    c, new = st["case"], torch.empty_like
    if c["op"] in ("norm", "norm_bwd"):
        d = T.make_norm_desc(c["rows"], c["D"], kind=c["kind"], gate=c["gate"], eps=1e-6, scale=_RSCALE, dtype=c["type"])
        if c["op"] == "norm":
            out = new(st["x"])
            T.ttt_norm_fwd(d, st["x"], st["w"], st["z"], st["res"], out)
            return out
        out = {"dx": new(st["x"])}
        if st["w"] is not None:
            out["dw"] = new(st["w"])
        if st["z"] is not None:
            out["dz"] = new(st["z"])
        ws = _workspace(T, T.ttt_norm_bwd_workspace_bytes(d))
        T.ttt_norm_bwd(d, st["x"], st["w"], st["z"], st["dout"], out["dx"], out.get("dw"), out.get("dz"), ws)
        return out
    N = 1 if c["op"] == "step" else c["N"]
    d = T.make_delta_desc(c["B"], c["H"], N, c["dk"], c["dv"], in_dtype=c["type"], out_dtype=c["type"])
    if c["op"] == "step":
        T.ttt_delta_step(d, st["q"], st["k"], st["v"], st["g"], st["beta"], st["slots"], c["slots"], st["S"], st["out"])
        return {"out": st["out"], "S": st["S"]}
    if c["op"] == "fwd":
        out = new(st["v"])
        ws = _workspace(T, T.ttt_delta_workspace_bytes(d))
        T.ttt_delta_fwd(d, st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], out, ws)
        return {"out": out, "S": st["S"]}
    out = {"d" + n: new(st[n]) for n in ("q", "k", "v", "g", "beta") if st[n] is not None}
    out["dS0"] = new(st["S"])
    ws = _workspace(T, T.ttt_delta_bwd_workspace_bytes(d))
    T.ttt_delta_bwd(d, st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], st["dout"], st["dS"],
                    out["dq"], out["dk"], out["dv"], out.get("dg"), out["dbeta"], out["dS0"], ws)
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] in ("norm", "norm_bwd"):
        n = case["rows"] * case["D"]
        gate, res, w = case["gate"] != "none", case["res"], case["weight"]
        if case["op"] == "norm":
            return {"bytes": n * size * (2 + gate + res) + 4 * case["D"] * w, "flops": n * (4 + 5 * gate + res + w)}
        return {"bytes": n * size * (3 + 2 * gate) + 8 * case["D"] * w, "flops": n * (9 + 9 * gate + 3 * w)}
    B, H, dk, dv = (case[n] for n in ("B", "H", "dk", "dv"))
    gates = 1 + case["decay"]
    if case["op"] == "step":
        rows = (B - case["idle"]) * H
        return {"bytes": rows * (8 * dk * dv + size * (2 * dk + 2 * dv + gates)) + 4 * B, "flops": rows * 7 * dk * dv}
    t = B * H * case["N"]
    if case["op"] == "fwd":
        return {"bytes": t * size * (2 * dk + 2 * dv + gates) + 8 * B * H * dk * dv, "flops": t * 6 * dk * dv}
    return {"bytes": t * size * (4 * dk + 3 * dv + 2 * gates) + 12 * B * H * dk * dv, "flops": t * 18 * dk * dv}


# ------------------------------------------------------------------ 64 bits, from the definition
def _exact_norm(st, c):
    d = lambda n: None if st[n] is None else st[n].double()  # noqa: E731
    x, w, z, res = d("x"), d("w"), d("z"), d("res")
    ins = {n: t.requires_grad_() for n, t in (("x", x), ("w", w), ("z", z)) if t is not None}
    length = (x * x).sum(1).sqrt()
    y = x / ((length ** 2 / c["D"] + 1e-6).sqrt() if c["kind"] == "rms" else length.clamp(min=1e-6)).unsqueeze(1)
    for f in (w, None if z is None else 1 / (1 + torch.exp(-z)) * (z if c["gate"] == "silu" else 1)):
        y = y if f is None else y * f
    y = _RSCALE * y if res is None else _RSCALE * y + res
    if c["op"] == "norm":
        return y.detach()
    got = torch.autograd.grad(y, list(ins.values()), d("dout"))
    return {"d" + n: g for n, g in zip(ins, got)}


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] in ("norm", "norm_bwd"):
        return _exact_norm(st, c)
    dk, s = c["dk"], 1 / math.sqrt(c["dk"])
    q, k, v, b, S = (st[n].double() for n in ("q", "k", "v", "beta", "S"))
    a = torch.ones_like(b) if st["g"] is None else st["g"].double().exp()
    outer = lambda x, y: torch.einsum("bhi,bhj->bhij", x, y)  # noqa: E731
    down = lambda X, x: torch.einsum("bhij,bhi->bhj", X, x)  # noqa: E731
    over = lambda X, x: torch.einsum("bhij,bhj->bhi", X, x)  # noqa: E731
    if c["op"] == "step":
        out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
        for row, slot in enumerate(st["slots"].tolist()):
            if slot >= 0:
                X = S[slot] * a[row][:, None, None]
                e = v[row] - (X * k[row][:, :, None]).sum(1)
                S[slot] = X + k[row][:, :, None] * (b[row][:, None] * e)[:, None, :]
                out[row] = s * (S[slot] * q[row][:, :, None]).sum(1)
        return {"out": out, "S": S}
    N, o, held = c["N"], torch.empty_like(v), [S]
    e = torch.empty_like(v)
    for t in range(N):
        S = S * a[:, :, t, None, None]
        e[:, :, t] = v[:, :, t] - down(S, k[:, :, t])
        S = S + outer(k[:, :, t], b[:, :, t, None] * e[:, :, t])
        o[:, :, t] = s * down(S, q[:, :, t])
        if c["op"] == "bwd":
            held.append(S)
    if c["op"] == "fwd":
        return {"out": o, "S": S}
    do, X = st["dout"].double(), st["dS"].double()
    dq, dk_, dv_, db, dg = (torch.empty_like(x) for x in (q, k, v, b, b))
    for t in range(N - 1, -1, -1):
        kt, at, bt, before = k[:, :, t], a[:, :, t, None], b[:, :, t, None], held[t]
        X = X + s * outer(q[:, :, t], do[:, :, t])
        dq[:, :, t] = s * over(held[t + 1], do[:, :, t])
        du = down(X, kt)
        dv_[:, :, t] = bt * du
        db[:, :, t] = (du * e[:, :, t]).sum(-1)
        dk_[:, :, t] = over(X, bt * e[:, :, t]) - at * bt * over(before, du)
        Y = X - outer(kt, bt * du)  # of the decayed state
        dg[:, :, t] = a[:, :, t] * (Y * before).sum((-1, -2))
        X = at.unsqueeze(-1) * Y
    out = {"dq": dq, "dk": dk_, "dv": dv_, "dbeta": db, "dS0": X}
    if st["g"] is not None:
        out["dg"] = dg
    return out
