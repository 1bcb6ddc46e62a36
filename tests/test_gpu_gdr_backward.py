"""Gradients of the gated delta rule (mlstm_gdr_bwd) against reverse-mode differentiation of its steps in
64 bits, and against differences.

Tolerances.  What is summed in fp32 accuracy (dS0, dbeta, dv) is held like the forward pass: 2^-14 of a
head's largest value (about eight roundings a token, at most 128 tokens of them count), plus half a step of
the storage type.  dg_t is a sum over the chunk of dO.O - dV.V and <dS, S> at its end, whose terms can be
larger than itself: 2^-18 of the sum of their magnitudes (|dO||O| + |dV||V| over the chunk, |dS||S|; each
product carries the forward pass's relative error, 64 of them are summed).  dq and dk in bf16 come from
products whose operands S, dS, U, dV, dP o D, dW o D have 11 bits (half a step 2^-11), at most three of them
in a term (dV, U and the product of both): 3.1 * 2^-11 of the sum of the terms' magnitudes, which
magnitudes() computes in 64 bits; in fp32 the operands have 22 bits: 2^-19 of it."""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_token_b200 import inputs, mlstm
from tests.helpers import TORCH_DTYPE, dev

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
COARSE = {"f32": 2.0 ** -19, "bf16": 3.1 * 2.0 ** -11}
NAMES = ("q", "k", "v", "g", "beta")


def make(shape, dtype, seed, states=True, seqs=None):
    inp = inputs.gdr_inputs(*shape, dtype, seed=seed, with_state=states)
    B, HK, H, T, K, V = shape
    rng = np.random.default_rng(seed + 1)
    N = seqs or B
    if states:
        inp["S0"] = (0.1 * rng.standard_normal((N, H, K, V))).astype(np.float32)
    inp["do"] = inputs.round_to(rng.standard_normal((B, H, T, V)), dtype)
    inp["dS"] = (0.1 * rng.standard_normal((N, H, K, V))).astype(np.float32) if states else None
    return inp


def magnitudes(inp):
    """Sums of the magnitudes of the terms of dq and dk [B,HK,T,K] and of dg [B,H,T], chunk by chunk."""
    q, k, v, g, beta, do = (np.asarray(inp[n], np.float64) for n in NAMES + ("do",))
    g = np.maximum(g, -1e4)
    B, H, T, V = v.shape
    HK, K = q.shape[1], q.shape[-1]
    q, k = (np.repeat(x, H // HK, axis=1) for x in (q, k))
    zero = np.zeros((B, H, K, V))
    S = zero if inp["S0"] is None else np.asarray(inp["S0"], np.float64)
    states, us, os = [S], [], []
    for t in range(T):
        Sd = np.exp(g[:, :, t])[..., None, None] * S
        u = beta[:, :, t, None] * (v[:, :, t] - np.einsum("bhkv,bhk->bhv", Sd, k[:, :, t]))
        S = Sd + np.einsum("bhk,bhv->bhkv", k[:, :, t], u)
        states.append(S), us.append(u), os.append(np.einsum("bhkv,bhk->bhv", S, q[:, :, t]))
    d = oracle.gdr_sequential_backward(inp["q"], inp["k"], v, g, beta, do, inp["S0"], inp["dS"])
    D = zero if inp["dS"] is None else np.asarray(inp["dS"], np.float64)
    grads = [D]  # gradient of the state behind each token, from the last one on
    for t in reversed(range(T)):
        D = D + np.einsum("bhk,bhv->bhkv", q[:, :, t], do[:, :, t])
        D = np.exp(g[:, :, t])[..., None, None] * (D - np.einsum("bhk,bhv->bhkv", k[:, :, t], d["dv"][:, :, t]))
        grads.append(D)
    grads = grads[::-1]
    Tq, Tk, Tg = np.zeros((B, H, T, K)), np.zeros((B, H, T, K)), np.zeros((B, H, T))
    for c in range(0, T, 64):
        e = min(c + 64, T)
        G = np.cumsum(g[:, :, c:e], -1)
        low = np.tril(np.ones((e - c, e - c)))
        Dm = np.exp(np.minimum(G[..., :, None] - G[..., None, :], 0)) * low
        gam, w = np.exp(G), np.exp(G[..., -1:] - G)
        aq, ak, ado, adv = (np.abs(x[:, :, c:e]) for x in (q, k, do, d["dv"]))
        au = np.abs(np.stack(us[c:e], 2))
        tr = lambda x: np.swapaxes(x, -1, -2)
        S0, D1 = np.abs(states[c]), np.abs(grads[e])
        P, W = (ado @ tr(au)) * Dm, (adv @ tr(au)) * Dm
        Tq[:, :, c:e] = gam[..., None] * (ado @ tr(S0)) + P @ ak
        Tk[:, :, c:e] = gam[..., None] * (adv @ tr(S0)) + w[..., None] * (au @ tr(D1)) + tr(P) @ aq + W @ ak + tr(W) @ ak
        norm = lambda x: np.sqrt((x * x).sum(-1))
        terms = norm(do[:, :, c:e]) * norm(np.stack(os[c:e], 2)) + norm(d["dv"][:, :, c:e]) * norm(v[:, :, c:e])
        end = np.sqrt((states[e] ** 2).sum((-1, -2)) * (grads[e] ** 2).sum((-1, -2)))
        Tg[:, :, c:e] = terms.sum(-1, keepdims=True) + end[..., None]
    shared = lambda x: x.reshape(B, HK, H // HK, T, K).sum(2)
    return {"dq": shared(Tq), "dk": shared(Tk), "dg": Tg}


def close(x, ref, half, extra, rel=2.0 ** -14):
    x = x.double().cpu().numpy()
    assert x.shape == ref.shape
    axes = (-1, -2) if ref.ndim == 4 else (-1,)
    big = np.abs(ref).max(axis=axes, keepdims=True)
    bad = ~(np.abs(x - ref) <= half * np.abs(ref) + rel * big + extra + 1e-30)
    assert not bad.any(), float((np.abs(x - ref) / (big + 1e-30)).max())


def check(out, inp, dtype, ref=None, mag=None):
    ref = oracle.gdr_sequential_backward(*(inp[n] for n in NAMES), inp["do"], inp["S0"], inp["dS"]) if ref is None else ref
    mag = magnitudes(inp) if mag is None else mag
    for n in ("dq", "dk"):
        close(out[n], ref[n], HALF[dtype], COARSE[dtype] * mag[n])
    close(out["dv"], ref["dv"], HALF[dtype], 0.0)
    close(out["dbeta"], ref["dbeta"], 0.0, 0.0)
    close(out["dg"], ref["dg"], 0.0, 2.0 ** -18 * mag["dg"], rel=0.0)
    close(out["dS0"], ref["dS0"], 0.0, 0.0)


def call(inp, dtype, **kw):
    td = TORCH_DTYPE[dtype]
    a = [dev(inp[n], td) for n in ("q", "k", "v")] + [dev(inp[n]) for n in ("g", "beta")] + [dev(inp["do"], td)]
    return mlstm.gdr_bwd(*a, dev(inp["S0"]), dev(inp["dS"]), **kw)


SHAPES = [  # B, HK, H, T, K, V
    (1, 1, 1, 1, 8, 8), (2, 1, 3, 2, 16, 24), (1, 2, 2, 17, 64, 40), (1, 1, 2, 63, 40, 88), (1, 2, 2, 64, 64, 64),
    (2, 1, 1, 65, 128, 128), (1, 2, 4, 129, 96, 48), (1, 1, 1, 300, 128, 256), (1, 1, 2, 200, 120, 16),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("states", [True, False])
def test_gradients(shape, dtype, states):
    inp = make(shape, dtype, sum(shape), states)
    out = call(inp, dtype)
    check(out, inp, dtype)
    again = call(inp, dtype)
    assert all(torch.equal(out[n], again[n]) for n in out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_heads_take_wider_blocks(dtype):
    """Enough heads for blocks of eight and of four tiles."""
    for shape in ((8, 16, 16, 70, 64, 72), (10, 5, 10, 66, 128, 64), (4, 4, 8, 130, 128, 128), (2, 8, 16, 65, 40, 136)):
        inp = make(shape, dtype, 5)
        check(call(inp, dtype), inp, dtype)


@pytest.mark.parametrize("dtype,shape", [  # one, two and four tiles of values a block
    ("bf16", (1, 16, 32, 140, 128, 128)), ("bf16", (1, 32, 32, 80, 72, 256)), ("bf16", (3, 16, 32, 140, 64, 64)),
    ("bf16", (2, 37, 37, 66, 32, 64)), ("f32", (2, 16, 16, 140, 128, 128)), ("f32", (3, 8, 16, 140, 64, 64)),
])
def test_tiles_a_block(dtype, shape):
    inp = make(shape, dtype, 7)
    check(call(inp, dtype), inp, dtype)


def test_many_heads_packed():
    lengths, T = (70, 0, 1, 64, 130, 5), 273
    inp = make((1, 4, 8, T, 64, 48), "bf16", 6, True, len(lengths))
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    out = call(inp, "bf16", seq_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    for n, x in enumerate(lengths):
        if x:
            lo = offsets[n]
            one = {m: inp[m][:, :, lo:lo + x] for m in NAMES + ("do",)} | {m: inp[m][n:n + 1] for m in ("S0", "dS")}
            check({m: out[m][:, :, lo:lo + x] for m in ("dq", "dk", "dv", "dg", "dbeta")} | {"dS0": out["dS0"][n:n + 1]},
                  one, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,T", [((5, 0, 70, 1, 64, 0), 147), ((0, 0), 3), ((63, 65), 128)])
def test_packed_sequences(lengths, T, dtype):
    inp = make((1, 2, 4, T, 64, 48), dtype, T, True, len(lengths))
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    out = call(inp, dtype, seq_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    for n, x in enumerate(lengths):
        lo = offsets[n]
        if x == 0:
            assert np.array_equal(out["dS0"][n].cpu().numpy(), inp["dS"][n])
            continue
        one = {m: inp[m][:, :, lo:lo + x] for m in NAMES + ("do",)} | {m: inp[m][n:n + 1] for m in ("S0", "dS")}
        check({m: out[m][:, :, lo:lo + x] for m in ("dq", "dk", "dv", "dg", "dbeta")} | {"dS0": out["dS0"][n:n + 1]},
              one, dtype)
    for m in ("dq", "dk", "dv", "dg", "dbeta"):
        assert bool((out[m][:, :, offsets[-1]:] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_extremes(dtype):
    """Full resets, strong and no decay, write strengths 0, 1 and 2."""
    inp = make((1, 2, 2, 150, 64, 32), dtype, 12)
    rng = np.random.default_rng(1)
    inp["g"][0, 0] = rng.choice([0.0, -np.inf, -90.0, -5.0, -1e-4, -1e30], 150)
    inp["beta"][:] = rng.choice([0.0, 1.0, 2.0], (1, 2, 150))
    check(call(inp, dtype), inp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_scales_of_the_inputs(dtype, scale):
    inp = make((1, 1, 2, 100, 64, 32), dtype, 13)
    for n, f in (("v", scale), ("S0", scale), ("q", 1 / scale), ("do", 1e3 / scale)):
        inp[n] = inputs.round_to(inp[n].astype(np.float64) * f, dtype if n != "S0" else "f32")
    inp["dS"] = (inp["dS"] / scale).astype(np.float32)
    check(call(inp, dtype), inp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_views_and_layout_of_the_gradients(dtype):
    B, HK, H, T, K, V = 2, 2, 4, 77, 32, 24
    inp = make((B, HK, H, T, K, V), dtype, 8)
    ref = call(inp, dtype)
    td = TORCH_DTYPE[dtype]
    flip = lambda n, d=td: dev(inp[n], d).transpose(1, 2).contiguous().transpose(1, 2)
    q, v, do = flip("q"), flip("v"), flip("do")
    fused = torch.zeros(B, T, HK * K + 8, dtype=td, device="cuda")
    k = fused[..., 8:].view(B, T, HK, K).transpose(1, 2)
    k.copy_(dev(inp["k"], td))
    out = mlstm.gdr_bwd(q, k, v, flip("g", torch.float32), flip("beta", torch.float32), do, dev(inp["S0"]), dev(inp["dS"]))
    assert out["dq"].stride() == q.stride() and out["dv"].stride() == v.stride()
    assert all(torch.equal(out[n], ref[n]) for n in ref)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "S0"])
def test_against_differences(name):
    """Central differences (64 bits, h = 1e-5, error ~ h^2) of <do, o> + <dS, S_T> along a random
    direction; fp32's share of the gradient's inner product with it, 2^-14 of the magnitudes."""
    inp = make((1, 2, 4, 70, 16, 24), "f32", 21)
    out = call(inp, "f32")
    grad = out["dS0" if name == "S0" else "d" + name].double().cpu().numpy()
    rng = np.random.default_rng(3)
    d, h = rng.standard_normal(inp[name].shape), 1e-5

    def loss(x):
        y = {n: np.asarray(inp[n], np.float64) for n in NAMES + ("S0",)}
        y[name] = x
        o, S = oracle.gdr_sequential(*(y[n] for n in NAMES), y["S0"])
        return (o * inp["do"]).sum() + (S * inp["dS"]).sum()

    base = np.asarray(inp[name], np.float64)
    num = (loss(base + h * d) - loss(base - h * d)) / (2 * h)
    assert abs(num - (grad * d).sum()) <= 2.0 ** -14 * np.abs(grad * d).sum()


def test_nothing_but_the_final_state_and_no_tokens():
    inp = make((1, 1, 2, 70, 32, 16), "bf16", 31)
    inp["do"][:] = 0
    inp["dS"][:] = 0
    out = call(inp, "bf16")
    assert all(bool((x == 0).all()) for x in out.values())
    e = torch.empty(2, 1, 0, 16, device="cuda")
    ev, eg = torch.empty(2, 2, 0, 8, device="cuda"), torch.empty(2, 2, 0, device="cuda")
    dS = torch.randn(2, 2, 16, 8, device="cuda")
    assert torch.equal(mlstm.gdr_bwd(e, e, ev, eg, eg, ev, None, dS)["dS0"], dS)
    assert bool((mlstm.gdr_bwd(e, e, ev, eg, eg, ev)["dS0"] == 0).all())


def test_offsets_out_of_order_stay_inside():
    inp = make((1, 1, 2, 90, 32, 16), "bf16", 2, True, 2)
    for bad in ([-5, 40, 1000], [80, 10, 90], [2**31 - 1, -2**31, 5], [91, 92, 93]):
        out = call(inp, "bf16", seq_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert out["dS0"].shape == (2, 2, 32, 16)


def test_captured_replayed_on_another_stream_and_beside_another_call():
    inp = make((2, 2, 4, 200, 64, 64), "bf16", 51)
    other = make((2, 2, 4, 200, 64, 64), "bf16", 52)
    td = torch.bfloat16
    args = lambda i: [dev(i[n], td) for n in ("q", "k", "v")] + [dev(i[n]) for n in ("g", "beta")] + [
        dev(i["do"], td), dev(i["S0"]), dev(i["dS"])]
    a, b = args(inp), args(other)
    ref, ref2 = mlstm.gdr_bwd(*a), mlstm.gdr_bwd(*b)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mlstm.gdr_bwd(*x))
        graphs.append(graph)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0][n], ref[n]) and torch.equal(outs[1][n], ref2[n]) for n in ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = mlstm.gdr_bwd(*a, stream=side)
    beside = mlstm.gdr_bwd(*b)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(on_side[n], ref[n]) and torch.equal(beside[n], ref2[n]) for n in ref)


def test_a_training_step_of_norm_and_recurrence():
    """Forward and backward through the norm, the gated delta rule on its output and the norm's own
    gradients, as a step runs them, against autograd in 64 bits through the same rounded tensors."""
    B, T, H, K = 2, 80, 2, 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, res, w = n(B, T, H * K), n(B, T, H * K), 1 + 0.1 * n(H * K)
    g, beta = -torch.exp(n(B, H, T) - 3), torch.sigmoid(n(B, H, T))
    kk = torch.nn.functional.normalize(n(B, H, T, K), dim=-1)
    y, r, _ = mlstm.rms_norm(x, res, w)
    v = y.view(B, T, H, K).transpose(1, 2)  # the norm's output as values and queries
    o, S = mlstm.gdr_fwd(v, kk, v, g, beta)
    do, dS = n(B, H, T, K), 0.1 * n(B, H, K, K)
    d = mlstm.gdr_bwd(v, kk, v, g, beta, do, None, dS)
    dy = (d["dq"] + d["dv"]).transpose(1, 2).reshape(B, T, H * K)
    dx, dw = mlstm.rms_norm_bwd(dy.contiguous(), r, w)
    x6, w6, g6, b6 = (t.double().requires_grad_() for t in (x, w, g, beta))
    r6 = x6 + res.double()
    v6 = (r6 / torch.sqrt((r6 * r6).mean(-1, keepdim=True) + 1e-6) * w6).view(B, T, H, K).transpose(1, 2)
    Sx, outs = torch.zeros(B, H, K, K, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        Sd = torch.exp(g6[:, :, t])[..., None, None] * Sx
        kt = kk[:, :, t].double()
        u = b6[:, :, t, None] * (v6[:, :, t] - torch.einsum("bhkv,bhk->bhv", Sd, kt))
        Sx = Sd + torch.einsum("bhk,bhv->bhkv", kt, u)
        outs.append(torch.einsum("bhkv,bhk->bhv", Sx, v6[:, :, t]))
    loss = (torch.stack(outs, 2) * do.double()).sum() + (Sx * dS.double()).sum()
    ref = torch.autograd.grad(loss, (x6, w6, g6, b6))
    for got, want in zip((dx, dw, d["dg"], d["dbeta"]), ref):
        assert float((got.double() - want).abs().max()) <= 2.0 ** -12 * float(want.abs().max())
