"""What is measured of the gated delta rule and of the root-mean-square norm.

Each case names an operator: the gated delta rule over sequences (``gdr_fwd``), its decode step
on a pool of states (``gdr_step``), its gradients (``gdr_bwd``), the norm of a residual stream
with its addition, in the input's type or in 8 bits with scales (``rms_norm``), and the norm's
gradients (``rms_norm_bwd``).  ``run`` computes a case in elementary torch operations, or, where
``own`` is true, by the library's entry point.

The gated delta rule, per value head with state S [K, V] and for each token:
    S' = e^g S;  r = S'^T k;  S = S' + beta k (v - r)^T;  o = S^T q
The norm:  r = x + residual;  y = r / sqrt(mean(r^2) + eps) * weight.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-6
_CHUNK = 64  # tokens that the plain form of the recurrence takes at a time
_TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------------------------ the cases

def listed():
    def fwd(name, B, HK, H, T, K, V, dtype="bf16", packed=0):
        return {"name": name, "op": "gdr_fwd", "B": B, "HK": HK, "H": H, "T": T, "K": K, "V": V,
                "dtype": dtype, "packed": packed}

    def bwd(name, B, HK, H, T, K, V, dtype="bf16", packed=0):
        return dict(fwd(name, B, HK, H, T, K, V, dtype, packed), op="gdr_bwd")

    def step(name, B, HK, H, K, V, dtype="bf16", slots=0):
        return {"name": name, "op": "gdr_step", "B": B, "HK": HK, "H": H, "K": K, "V": V, "dtype": dtype,
                "slots": slots}

    def norm(name, rows, D, dtype, quant, group, residual):
        return {"name": name, "op": "rms_norm", "rows": rows, "D": D, "dtype": dtype, "quant": quant,
                "group": group, "residual": residual}

    def norm_bwd(name, rows, D, dtype, residual):
        return {"name": name, "op": "rms_norm_bwd", "rows": rows, "D": D, "dtype": dtype, "residual": residual}

    return [
        # a batch of prompts of one length: the sizes of the Gated DeltaNet-2 prefill workload
        fwd("prefill batch", 8, 16, 16, 2048, 128, 128),
        # one long prompt, two value heads to a key head: few chains, many chunks in each
        fwd("prefill long grouped", 1, 8, 16, 8192, 128, 128),
        # prompts of unlike lengths in one packed batch, some of them empty
        fwd("prefill packed ragged", 1, 4, 8, 6007, 64, 128, packed=13),
        # a short sequence in single precision, odd length
        fwd("short fp32", 2, 4, 4, 101, 64, 64, "fp32"),
        # decoding at full load: states in a pool, a few rows of the batch are padding
        step("decode pool", 256, 16, 16, 128, 128, slots=300),
        # one request alone: latency
        step("decode single", 1, 8, 16, 128, 128),
        # a training step's share of one GPU
        bwd("train batch", 4, 16, 16, 2048, 128, 128),
        # a small packed training batch with grouped heads
        bwd("train packed grouped", 1, 4, 8, 1000, 64, 128, packed=5),
        # the pre-norm of a prefill whose projections run in 8 bits (embedding width 4096)
        norm("norm prefill e4m3", 16384, 4096, "bf16", "e4m3", 0, True),
        # the same at a decode step, with a scale for every 128 channels
        norm("norm decode int8", 7, 4096, "bf16", "int8", 128, True),
        # training: the norm's gradients with the residual stream's own
        norm_bwd("norm gradient", 8192, 4096, "bf16", True),
        # a width that no vector access divides
        norm_bwd("norm gradient odd", 333, 1001, "fp32", False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_step", "gdr_bwd", "rms_norm", "rms_norm_bwd"])
    if op in ("gdr_fwd", "gdr_bwd"):
        most = 131072 if op == "gdr_bwd" else 262144  # tokens times value heads
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        if dtype == "fp32":
            most //= 8
        group = rng.choice([1, 1, 2, 4])
        HK = rng.choice([1, 2, 3, 4, 8, 16])
        H = HK * group
        K = rng.choice([16, 32, 40, 64, 64, 96, 128, 128])
        V = rng.choice([16, 32, 64, 64, 88, 128, 128, 256]) if H <= 16 else rng.choice([32, 64, 128])
        cap = min(8192, most // H * 128 // max(128, V))
        T = _log_int(rng, 1, cap)
        packed = rng.choice([0, 0, _log_int(rng, 2, 40)])
        B = 1 if packed else _log_int(rng, 1, max(1, min(16, cap // T)))
        return {"op": op, "B": B, "HK": HK, "H": H, "T": T, "K": K, "V": V, "dtype": dtype, "packed": packed}
    if op == "gdr_step":
        group = rng.choice([1, 1, 2, 4])
        HK = rng.choice([1, 2, 4, 8])
        K = rng.choice([16, 32, 64, 96, 128, 128, 256])
        V = rng.choice([16, 32, 64, 88, 128, 128, 256])
        most = 256 * 16 * 128 * 128 // (K * V * HK * group)
        B = _log_int(rng, 1, max(1, min(512, most)))
        return {"op": op, "B": B, "HK": HK, "H": HK * group, "K": K, "V": V,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "slots": rng.choice([0, B + rng.randrange(1, 40)])}
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    D = rng.choice([64, 128, 1000, 1001, 2048, 4096, 4096, 8192, _log_int(rng, 8, 12000)])
    rows = _log_int(rng, 1, (1 << 25) // D)
    if op == "rms_norm":
        quant = rng.choice(["", "e4m3", "int8"])
        return {"op": op, "rows": rows, "D": D, "dtype": dtype, "quant": quant,
                "group": rng.choice([0, 128]) if quant else 0, "residual": rng.random() < 0.7}
    return {"op": op, "rows": rows, "D": D, "dtype": dtype, "residual": rng.random() < 0.7}


# ----------------------------------------------------------------------------------- the inputs

def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)


def _lengths(case, seed):
    """Lengths of the packed sequences: uneven, now and then zero, and a few tokens behind the last
    one that belong to none."""
    import random
    r = random.Random(seed * 7919 + case["T"])
    n, T = case["packed"], case["T"]
    used = T - min(T // 10, r.randrange(0, 6))
    w = [0.0 if r.random() < 0.15 else r.expovariate(1.0) for _ in range(n)]
    w[r.randrange(n)] += 1.0
    total, lengths, at = sum(w), [], 0.0
    for x in w:
        lo, at = round(at / total * used), at + x
        lengths.append(round(at / total * used) - lo)
    return lengths


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2 + 1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op, dt = case["op"], _DT[case["dtype"]]
    st = {"case": dict(case)}
    if op in ("gdr_fwd", "gdr_bwd"):
        B, HK, H, T, K, V = (case[n] for n in ("B", "HK", "H", "T", "K", "V"))
        N = B
        st["offsets"] = None
        if case["packed"]:
            lengths = _lengths(case, int(seed))
            N, at = len(lengths), [0]
            for x in lengths:
                at.append(at[-1] + x)
            st["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
            st["longest"] = max(lengths)
        st["q"] = (normal(B, HK, T, K) / math.sqrt(K)).to(dt)
        st["k"] = _unit(normal(B, HK, T, K)).to(dt)
        st["v"] = normal(B, H, T, V).to(dt)
        # memories of some tokens to some hundreds of them, by head
        pace = torch.linspace(-6.5, -1.5, H, device="cuda").view(1, H, 1)
        st["g"] = -torch.exp(pace + 0.5 * normal(B, H, T))
        st["beta"] = torch.sigmoid(normal(B, H, T))
        st["S0"] = 0.1 * normal(N, H, K, V)
        if op == "gdr_bwd":
            st["do"] = normal(B, H, T, V).to(dt)
            st["dS"] = 0.1 * normal(N, H, K, V)
    elif op == "gdr_step":
        B, HK, H, K, V = (case[n] for n in ("B", "HK", "H", "K", "V"))
        st["q"] = (normal(B, HK, K) / math.sqrt(K)).to(dt)
        st["k"] = _unit(normal(B, HK, K)).to(dt)
        st["v"] = normal(B, H, V).to(dt)
        pace = torch.linspace(-6.5, -1.5, H, device="cuda").view(1, H)
        st["g"] = -torch.exp(pace + 0.5 * normal(B, H))
        st["beta"] = torch.sigmoid(normal(B, H))
        st["S"] = 0.1 * normal(case["slots"] or B, H, K, V)
        st["slots"] = None
        if case["slots"]:
            slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B]
            if B > 8:
                slots[B - B // 50 - 1:] = -1  # padding of the batch
            st["slots"] = slots.to(torch.int32)
    else:
        rows, D = case["rows"], case["D"]
        # a residual stream has a few channels much larger than the others
        loud = torch.exp(0.7 * normal(D))
        st["weight"] = 1.0 + 0.3 * normal(D)
        if op == "rms_norm":
            st["x"] = normal(rows, D).to(dt)
            st["residual"] = (normal(rows, D) * loud).to(dt) if case["residual"] else None
        else:
            st["r"] = (normal(rows, D) * loud).to(dt)
            st["dy"] = normal(rows, D).to(dt)
            st["dresidual"] = normal(rows, D).to(dt) if case["residual"] else None
    return st


# --------------------------------------------------------------------------------- the plain forms

def _padded(st, x, longest):
    """[1, H, T, ...] of a packed batch as [N, H, longest, ...], zeros behind each sequence."""
    off = st["offsets"].long()
    at = off[:-1, None] + torch.arange(longest, device=x.device)
    inside = at < off[1:, None]
    rows = x[0].transpose(0, 1)[torch.where(inside, at, 0)]  # [N, longest, H, ...]
    rows = rows * inside.view(*inside.shape, *([1] * (rows.dim() - 2)))
    return rows.transpose(1, 2)


def _unpadded(st, x, like):
    """The inverse of _padded; tokens behind the last sequence get zero."""
    off = st["offsets"].long()
    N, longest = x.shape[0], x.shape[2]
    at = off[:-1, None] + torch.arange(longest, device=x.device)
    inside = at < off[1:, None]
    out = torch.zeros(like.shape[2], x.shape[1], *x.shape[3:], device=x.device, dtype=x.dtype)
    out[at[inside]] = x.transpose(1, 2)[inside]
    return out.transpose(0, 1)[None]


def _chunks(x, L):
    """[N, H, T, ...] -> [N, H, chunks, L, ...], zeros behind the end."""
    T = x.shape[2]
    n = -(-T // L)
    if n * L != T:
        x = torch.cat([x, x.new_zeros(*x.shape[:2], n * L - T, *x.shape[3:])], 2)
    return x.reshape(*x.shape[:2], n, L, *x.shape[3:])


def _inside(q, k, g, beta, L):
    """The matrices of every chunk that do not depend on the state."""
    G = g.double().cumsum(-1)
    low = torch.ones(L, L, device=q.device).tril().bool()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    M = ((k @ k.transpose(-1, -2)) * D).tril(-1)  # beta_t M[t, s] is what token s leaves at t
    A = -beta[..., None] * M
    eye = torch.eye(L, device=q.device)
    T, power, reach = eye + A, A, 2
    while reach < L:  # (I - A)^-1 of a nilpotent A: the product of I + A^(2^i)
        power = power @ power
        T = T + T @ power
        reach *= 2
    P = (q @ k.transpose(-1, -2)) * D
    gam = torch.exp(G).float()
    w = torch.exp(G[..., -1:] - G).float()
    return D, M, T, P, gam, w


def _gdr_operands(st, names):
    case = st["case"]
    L = _CHUNK
    out = {}
    for n in names:
        x = st[n].float()
        if st["offsets"] is not None:
            x = _padded(st, x, st["longest"])
        if n in ("q", "k") and case["HK"] != case["H"]:
            x = x.repeat_interleave(case["H"] // case["HK"], 1)
        out[n] = x
    T = out["q"].shape[2]
    L = min(L, max(T, 1))
    return {n: _chunks(x, L) for n, x in out.items()}, L, T


def _walk(c, L, S):
    """The forward pass over the chunks: states at the chunks' starts, u, v - r, and the last state."""
    D, M, T, P, gam, w = _inside(c["q"], c["k"], c["g"], c["beta"], L)
    states, us, zs = [], [], []
    wk = (w[..., None] * c["k"]).transpose(-1, -2)
    for i in range(c["q"].shape[2]):
        states.append(S)
        z = c["v"][:, :, i] - gam[:, :, i, :, None] * (c["k"][:, :, i] @ S)
        u = T[:, :, i] @ (c["beta"][:, :, i, :, None] * z)
        S = gam[:, :, i, -1, None, None] * S + wk[:, :, i] @ u
        us.append(u)
        zs.append(z)
    return (D, M, T, P, gam, w), torch.stack(states, 2), torch.stack(us, 2), torch.stack(zs, 2), S


def _merge(x, T):
    return x.reshape(*x.shape[:2], -1, *x.shape[4:])[:, :, :T]


def _gdr_fwd(st):
    c, L, T = _gdr_operands(st, ("q", "k", "v", "g", "beta"))
    (_, _, _, P, gam, _), S, U, _, last = _walk(c, L, st["S0"])
    o = _merge(gam[..., None] * (c["q"] @ S) + P @ U, T)
    if st["offsets"] is not None:
        o = _unpadded(st, o, st["v"])
    return {"o": o.to(st["v"].dtype), "S": last}


def _gdr_bwd(st):
    case = st["case"]
    c, L, T = _gdr_operands(st, ("q", "k", "v", "g", "beta", "do"))
    (D, M, Ti, P, gam, w), S, U, Z, _ = _walk(c, L, st["S0"])
    q, k, v, beta, do = (c[n] for n in ("q", "k", "v", "beta", "do"))
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    dS, dSs, dYs = st["dS"], [], []
    Pdo, gq = tr(P) @ do, tr(gam[..., None] * q)
    for i in reversed(range(q.shape[2])):
        dSs.append(dS)
        dU = Pdo[:, :, i] + w[:, :, i, :, None] * (k[:, :, i] @ dS)
        dY = tr(Ti[:, :, i]) @ dU
        dX = -(beta * gam)[:, :, i, :, None] * dY
        dS = gam[:, :, i, -1, None, None] * dS + gq[:, :, i] @ do[:, :, i] + tr(k[:, :, i]) @ dX
        dYs.append(dY)
    dSs, dY = torch.stack(dSs[::-1], 2), torch.stack(dYs[::-1], 2)
    dX = -(beta * gam)[..., None] * dY
    dP = (do @ tr(U)).tril()
    dA = -(dY @ tr(U)).tril(-1)
    dPD, dAD = dP * D, dA * beta[..., None] * D
    inter = gam[..., None] * (do @ tr(S))
    dq = inter + dPD @ k
    wUdS = w[..., None] * (U @ tr(dSs))
    dk = dX @ tr(S) + tr(dPD) @ q + dAD @ k + tr(dAD) @ k + wUdS
    dv = beta[..., None] * dY
    dAM = dA * M
    dbeta = (dY * Z).sum(-1) + dAM.sum(-1)
    E = beta[..., None] * dAM + dP * P
    keep = (wUdS * k).sum(-1)
    dG = E.sum(-1) - E.sum(-2) + (inter * q).sum(-1) - (beta[..., None] * (v - Z) * dY).sum(-1) - keep
    dG[..., -1] += keep.sum(-1) + gam[..., -1] * (dSs * S).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
    for n, x in out.items():
        x = _merge(x, T)
        if n in ("dq", "dk") and case["HK"] != case["H"]:
            x = x.unflatten(1, (case["HK"], -1)).sum(2)
        if st["offsets"] is not None:
            x = _unpadded(st, x, st["v"])
        out[n] = x.to(st["v"].dtype) if n in ("dq", "dk", "dv") else x
    out["dS0"] = dS
    return out


def _gdr_step(st):
    case = st["case"]
    q, k, v = (st[n].float() for n in ("q", "k", "v"))
    if case["HK"] != case["H"]:
        q, k = (x.repeat_interleave(case["H"] // case["HK"], 1) for x in (q, k))
    S, g, beta, slots = st["S"], st["g"], st["beta"], st["slots"]
    o = torch.zeros_like(v)
    live = slice(None)
    if slots is not None:
        live = (slots >= 0).nonzero()[:, 0]
        old = S[slots[live].long()]
    else:
        old = S
    new = torch.exp(g[live])[..., None, None] * old
    r = (k[live].unsqueeze(-2) @ new).squeeze(-2)
    new = new + k[live].unsqueeze(-1) * (beta[live].unsqueeze(-1) * (v[live] - r)).unsqueeze(-2)
    o[live] = (q[live].unsqueeze(-2) @ new).squeeze(-2)
    if slots is not None:
        S[slots[live].long()] = new
    else:
        S.copy_(new)
    return {"o": o.to(st["v"].dtype), "S": S}


def _groups(y, group):
    """[rows, D] as [rows, groups, group], zeros behind the end; one group where `group` is 0."""
    D = y.shape[-1]
    size = group or D
    n = -(-D // size)
    if n * size != D:
        y = torch.cat([y, y.new_zeros(y.shape[0], n * size - D)], -1)
    return y.view(-1, n, size)


def _values(q, scales, D, group):
    """The values that 8-bit integers and their scales stand for, in bf16; 8-bit floating-point numbers
    as they are, in units of their scales."""
    if q.dtype != torch.int8:
        return q
    x = _groups(q.float(), group) * scales.view(q.shape[0], -1, 1)
    return x.reshape(q.shape[0], -1)[:, :D].to(torch.bfloat16)


def _rms_norm(st):
    case = st["case"]
    r = st["x"].float()
    if st["residual"] is not None:
        r = r + st["residual"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS) * st["weight"]
    out = {} if st["residual"] is None else {"residual": r.to(st["x"].dtype)}
    if not case["quant"]:
        return {"y": y.to(st["x"].dtype), **out}
    top = _TOP[case["quant"]]
    z = _groups(y, case["group"])
    amax = z.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    z = (z / scale).clamp(-top, top).reshape(y.shape[0], -1)[:, :case["D"]]
    z = z.to(torch.float8_e4m3fn) if case["quant"] == "e4m3" else torch.round(z).to(torch.int8)
    scale = scale[..., 0]
    return {"y": _values(z, scale, case["D"], case["group"]), "scales": scale, **out}


def _rms_norm_bwd(st):
    r, dy = st["r"].float(), st["dy"].float()
    s = torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS)
    n, wdy = r * s, dy * st["weight"]
    dx = s * (wdy - n * (wdy * n).mean(-1, keepdim=True))
    if st["dresidual"] is not None:
        dx = dx + st["dresidual"].float()
    return {"dx": dx.to(st["r"].dtype), "dweight": (dy * n).sum(0)}


_PLAIN = {"gdr_fwd": _gdr_fwd, "gdr_bwd": _gdr_bwd, "gdr_step": _gdr_step, "rms_norm": _rms_norm,
          "rms_norm_bwd": _rms_norm_bwd}


# ----------------------------------------------------------------------------- the library's calls

def _own(st):
    from linear_recurrent_token_b200 import mlstm
    case = st["case"]
    op = case["op"]
    if op == "gdr_fwd":
        o, S = mlstm.gdr_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"], seq_offsets=st["offsets"])
        return {"o": o, "S": S}
    if op == "gdr_bwd":
        d = mlstm.gdr_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"], st["S0"], st["dS"],
                          seq_offsets=st["offsets"])
        return {n: d[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dS0")}
    if op == "gdr_step":
        o = mlstm.gdr_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], slots=st["slots"])
        return {"o": o, "S": st["S"]}
    if op == "rms_norm":
        y, residual, scales = mlstm.rms_norm(st["x"], st["residual"], st["weight"], _EPS,
                                             quant=case["quant"] or None, group=case["group"])
        out = {} if residual is None else {"residual": residual}
        if not case["quant"]:
            return {"y": y, **out}
        return {"y": _values(y, scales, case["D"], case["group"]), "scales": scales, **out}
    dx, dweight = mlstm.rms_norm_bwd(st["dy"], st["r"], st["weight"], _EPS, st["dresidual"])
    return {"dx": dx, "dweight": dweight}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- the work

def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "gdr_step":
        B, HK, H, K, V = (case[n] for n in ("B", "HK", "H", "K", "V"))
        live = B - (B // 50 + 1 if case["slots"] and B > 8 else 0)
        return {"bytes": live * H * K * V * 8 + e * B * (2 * HK * K + 2 * H * V) + 8 * B * H,
                "flops": 7 * live * H * K * V}
    if op in ("gdr_fwd", "gdr_bwd"):
        B, HK, H, T, K, V = (case[n] for n in ("B", "HK", "H", "T", "K", "V"))
        N = case["packed"] or B
        state = 4 * N * H * K * V
        if op == "gdr_fwd":  # q, k, v, o, the gates, two states; decay, read, write, read-out
            return {"bytes": B * T * (2 * HK * K + 2 * H * V) * e + 8 * B * T * H + 2 * state,
                    "flops": 7 * B * T * H * K * V}
        # q, k and their gradients, v, do, dv, the gates and theirs, three states; the state again
        # (5 K V), then the gradients of the read-out, the write, the read and the decay
        return {"bytes": B * T * (4 * HK * K + 3 * H * V) * e + 16 * B * T * H + 3 * state,
                "flops": 20 * B * T * H * K * V}
    rows, D = case["rows"], case["D"]
    if op == "rms_norm":
        streams = e * (3 if case["residual"] else 1) + (1 if case["quant"] else e)
        scales = 4 * rows * (-(-D // case["group"]) if case["group"] else 1) if case["quant"] else 0
        return {"bytes": rows * D * streams + scales + 4 * D, "flops": 5 * rows * D}
    return {"bytes": rows * D * e * (4 if case["residual"] else 3) + 8 * D, "flops": 12 * rows * D}


# ------------------------------------------------------------------- the definition, in 64 bits

def _exact_sequences(st):
    """The sequences of a case, one after another: their rows and their place in the state."""
    case = st["case"]
    if st["offsets"] is None:
        return [(b, 0, case["T"], b) for b in range(case["B"])]
    off = st["offsets"].tolist()
    return [(0, off[n], off[n + 1], n) for n in range(len(off) - 1)]


def _exact_step(S, q, k, v, g, beta):
    """One token of the definition; [H, ...] operands.  Returns S', v - r, u, S, o."""
    Sp = torch.exp(g)[:, None, None] * S
    z = v - torch.einsum("hkv,hk->hv", Sp, k)
    u = beta[:, None] * z
    S = Sp + torch.einsum("hk,hv->hkv", k, u)
    return Sp, z, u, S, torch.einsum("hkv,hk->hv", S, q)


def _exact_gdr(st, gradients):
    case = st["case"]
    wide = {n: st[n].double() for n in ("q", "k", "v", "g", "beta", "S0", "do", "dS") if n in st}
    group = case["H"] // case["HK"]
    for n in ("q", "k"):
        wide[n] = wide[n].repeat_interleave(group, 1)
    out = {n: torch.zeros_like(wide[m]) for n, m in (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                                     ("dbeta", "beta"), ("S", "S0"), ("dS0", "S0"))}
    for b, lo, hi, n in _exact_sequences(st):
        at = lambda m, t: wide[m][b, :, t]  # noqa: E731
        S, kept = wide["S0"][n], []
        for t in range(lo, hi):
            Sp, z, u, S, o = _exact_step(S, *(at(m, t) for m in ("q", "k", "v", "g", "beta")))
            out["o"][b, :, t] = o
            if gradients:
                kept.append((Sp, z, u))
        out["S"][n] = S
        if not gradients:
            continue
        dS = wide["dS"][n]
        for t in reversed(range(lo, hi)):
            Sp, z, u = kept.pop()
            q, k, do, beta = (at(m, t) for m in ("q", "k", "do", "beta"))
            S = Sp + k[:, :, None] * u[:, None, :]
            dS = dS + q[:, :, None] * do[:, None, :]
            out["dq"][b, :, t] = (S * do[:, None, :]).sum(-1)
            du = (dS * k[:, :, None]).sum(-2)
            dr = -beta[:, None] * du
            out["dv"][b, :, t] = -dr
            out["dbeta"][b, :, t] = (du * z).sum(-1)
            out["dk"][b, :, t] = (dS * u[:, None, :]).sum(-1) + (Sp * dr[:, None, :]).sum(-1)
            dSp = dS + k[:, :, None] * dr[:, None, :]
            out["dg"][b, :, t] = (dSp * Sp).sum((-1, -2))
            dS = torch.exp(at("g", t))[:, None, None] * dSp
        out["dS0"][n] = dS
    if not gradients:
        return {"o": out["o"], "S": out["S"]}
    for n in ("dq", "dk"):
        out[n] = out[n].unflatten(1, (case["HK"], group)).sum(2)
    return {n: out[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dS0")}


def _exact_batch(st):
    """The forward definition for whole batches of one length, all sequences side by side."""
    case = st["case"]
    B, H, group = case["B"], case["H"], case["H"] // case["HK"]
    q, k = (st[n].double().repeat_interleave(group, 1).flatten(0, 1) for n in ("q", "k"))
    v, g, beta, S = (st[n].double().flatten(0, 1) for n in ("v", "g", "beta", "S0"))
    o = torch.zeros_like(v)
    for t in range(case["T"]):
        _, _, _, S, o[:, t] = _exact_step(S, q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t])
    return {"o": o.unflatten(0, (B, H)), "S": S.unflatten(0, (B, H))}


def _exact_quantised(y, kind, group):
    """Integers are rounded.  Of an 8-bit floating-point number this gives the value that is rounded to
    it: three bits are so few that which of two neighbours a value at their border takes would
    outweigh everything that the operator computes."""
    D = y.shape[-1]
    size = group or D
    scales = torch.ones(y.shape[0], -(-D // size), dtype=torch.float64, device=y.device)
    out = torch.zeros_like(y)
    for j in range(scales.shape[1]):
        part = y[:, j * size:(j + 1) * size]
        amax = part.abs().amax(-1)
        scales[:, j] = torch.where(amax > 0, amax / _TOP[kind], 1.0)
        z = part / scales[:, j, None]
        out[:, j * size:(j + 1) * size] = z if kind == "e4m3" else torch.round(z) * scales[:, j, None]
    return out, scales


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gdr_fwd":
        return _exact_batch(st) if st["offsets"] is None else _exact_gdr(st, False)
    if op == "gdr_bwd":
        if case["T"] * case["H"] * case["K"] * case["V"] * 8 > 40e9 or case["B"] * case["T"] > 20000:
            return None
        return _exact_gdr(st, True)
    if op == "gdr_step":
        group = case["H"] // case["HK"]
        S, o = st["S"].double(), torch.zeros(st["v"].shape, dtype=torch.float64, device=st["v"].device)
        slots = st["slots"].tolist() if st["slots"] is not None else range(case["B"])
        for b, s in enumerate(slots):
            if s >= 0:
                q, k = (st[n][b].double().repeat_interleave(group, 0) for n in ("q", "k"))
                _, _, _, S[s], o[b] = _exact_step(S[s], q, k, st["v"][b].double(), st["g"][b].double(),
                                                  st["beta"][b].double())
        return {"o": o, "S": S}
    if op == "rms_norm":
        r = st["x"].double()
        out = {}
        if st["residual"] is not None:
            r = r + st["residual"].double()
            out["residual"] = r
        y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + _EPS) * st["weight"].double()
        if not case["quant"]:
            return {"y": y, **out}
        y, scales = _exact_quantised(y, case["quant"], case["group"])
        return {"y": y, "scales": scales, **out}
    r, dy, w = st["r"].double(), st["dy"].double(), st["weight"].double()
    D = case["D"]
    ms = (r * r).mean(-1, keepdim=True) + _EPS
    dot = (dy * w * r).sum(-1, keepdim=True)
    dx = dy * w / ms.sqrt() - r * dot / (D * ms * ms.sqrt())
    if st["dresidual"] is not None:
        dx = dx + st["dresidual"].double()
    return {"dx": dx, "dweight": (dy * r / ms.sqrt()).sum(0)}
