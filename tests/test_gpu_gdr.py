"""The gated delta rule (mlstm_gdr_fwd, mlstm_gdr_step) against its token-by-token oracle in 64 bits.

Tolerances.  fp32 arithmetic with about eight roundings a token and value (two products over K in partial
sums, the decay, the update); an error made at one token decays with the state, at most 128 tokens of it
count for the decays drawn here: 8 * 128 * 2^-24 < 2^-14 of the largest value of a head's state or
output.  Outputs in bf16 add half a step, 2^-8 of the value.

Chunk mode in bf16 reads out with 11-bit operands (fp16, half a step 2^-11): o_t = gam_t sum_i q_i S_i +
sum_s P_ts U_s over the chunk, where S (first sum), P and U (second sum) are each rounded once, q is exact.
So |error| <= 2^-11 sum|gam q_i S_i| + (2 * 2^-11 + 2^-22) sum|P_ts U_s| < 2^-9.9 * (the sums of
magnitudes), which readout_terms computes in 64 bits; states are not touched by it."""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_token_b200 import inputs, mlstm
from tests.helpers import TORCH_DTYPE, Guarded, dev, slice_relerr

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -14
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def to_dev(inp, dtype):
    td = TORCH_DTYPE[dtype]
    t = {n: dev(inp[n], td) for n in ("q", "k", "v")}
    return t | {n: dev(inp[n]) for n in ("g", "beta", "S0")}


def readout_terms(inp):
    """Sums of the magnitudes that chunk mode adds up for each output: [B,H,T,V]."""
    q, k, v, g, beta, S0 = (None if inp[n] is None else np.asarray(inp[n], np.float64)
                            for n in ("q", "k", "v", "g", "beta", "S0"))
    B, H, T, V = v.shape
    q, k = (np.repeat(x, H // x.shape[1], axis=1) for x in (q, k))
    S = np.zeros((B, H, q.shape[-1], V)) if S0 is None else S0
    out = np.zeros((B, H, T, V))
    for c in range(0, T, 64):
        start, us = S, []
        decay = np.ones((B, H, 0))
        for t in range(c, min(c + 64, T)):
            e = np.exp(g[:, :, t])
            Sd = e[..., None, None] * S
            u = beta[:, :, t, None] * (v[:, :, t] - np.einsum("bhkv,bhk->bhv", Sd, k[:, :, t]))
            S = Sd + np.einsum("bhk,bhv->bhkv", k[:, :, t], u)
            us.append(np.abs(u))
            decay = np.concatenate([decay * e[..., None], np.ones((B, H, 1))], -1)
            first = np.prod(np.exp(g[:, :, c:t + 1]), axis=-1)
            qk = np.abs(np.einsum("bhd,bhsd->bhs", q[:, :, t], k[:, :, c:t + 1])) * decay
            out[:, :, t] = first[..., None] * np.einsum("bhkv,bhk->bhv", np.abs(start), np.abs(q[:, :, t])) \
                + np.einsum("bhs,sbhv->bhv", qk, np.stack(us))
    return out


def coarse(inp, dtype, mode):
    return 2.0 ** -9.9 * readout_terms(inp) if dtype == "bf16" and mode != "recurrent" else 0.0


def close(x, ref, dtype, extra=0.0, rel=F32):
    """Elementwise: half a step of the value, rel of the head's largest, and extra."""
    x, ref = x.double().cpu().numpy(), np.asarray(ref)
    assert x.shape == ref.shape
    big = np.abs(ref).max(axis=(-1, -2), keepdims=True) if ref.size else ref
    bad = ~(np.abs(x - ref) <= HALF[dtype] * np.abs(ref) + rel * big + extra + 1e-30)
    assert not bad.any(), float((np.abs(x - ref) / (big + 1e-30)).max())


SHAPES = [  # B, HK, H, T, K, V
    (1, 1, 1, 1, 8, 8), (2, 1, 3, 2, 16, 24), (1, 2, 2, 17, 64, 40), (2, 2, 4, 31, 32, 32), (1, 1, 2, 63, 40, 88),
    (1, 2, 2, 64, 64, 64), (2, 1, 1, 65, 128, 128), (1, 2, 4, 129, 96, 48), (1, 1, 1, 300, 128, 256),
    (1, 1, 2, 200, 120, 16),
]


@pytest.mark.parametrize("mode", ["recurrent", "chunk", "auto"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("state", [True, False])
def test_forward(shape, dtype, mode, state):
    inp = inputs.gdr_inputs(*shape, dtype, seed=sum(shape), with_state=state)
    B, HK, H, T, K, V = shape
    t = to_dev(inp, dtype)
    o, S = Guarded((B, H, T, V), TORCH_DTYPE[dtype]), Guarded((B, H, K, V), torch.float32)
    mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode, o=o.t, S_out=S.t)
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o.t, o_ref, dtype, coarse(inp, dtype, mode))
    close(S.t, S_ref, "f32")
    assert o.intact() and S.intact()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_keys(dtype):
    inp = inputs.gdr_inputs(1, 1, 2, 70, 256, 72, dtype, seed=3)
    t = to_dev(inp, dtype)
    o, S = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"])
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, dtype)
    close(S, S_ref, "f32")


def packed(inp, lengths):
    """The oracle over each sequence of a packed batch; offsets."""
    at, o, S = 0, np.zeros_like(inp["v"], dtype=np.float64), []
    terms = np.zeros_like(o)
    offsets = [0]
    for n, x in enumerate(lengths):
        sl = {m: inp[m][:, :, at:at + x] for m in ("q", "k", "v", "g", "beta")}
        o[:, :, at:at + x], s = oracle.gdr_sequential(*(sl[m] for m in ("q", "k", "v", "g", "beta")),
                                                      inp["S0"][n:n + 1])
        terms[:, :, at:at + x] = readout_terms(sl | {"S0": inp["S0"][n:n + 1]})
        S.append(s[0])
        at += x
        offsets.append(at)
    return o, np.stack(S), torch.tensor(offsets, dtype=torch.int32, device="cuda"), 2.0 ** -9.9 * terms


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,T", [((5, 0, 70, 1, 64, 0), 147), ((0, 0), 3), ((63, 65), 128), ((130,), 130)])
def test_packed_sequences(lengths, T, dtype, mode):
    inp = inputs.gdr_inputs(1, 2, 4, T, 64, 48, dtype, seed=T)
    rng = np.random.default_rng(T)
    inp["S0"] = (0.1 * rng.standard_normal((len(lengths), 4, 64, 48))).astype(np.float32)
    o_ref, S_ref, off, terms = packed(inp, lengths)
    t = to_dev(inp, dtype)
    o = Guarded((1, 4, T, 48), TORCH_DTYPE[dtype])
    o.t.fill_(7.0)
    _, S = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], seq_offsets=off, mode=mode, o=o.t)
    used = sum(lengths)
    close(o.t[:, :, :used], o_ref[:, :, :used], dtype,
          terms[:, :, :used] if dtype == "bf16" and mode == "chunk" else 0.0)
    assert bool((o.t[:, :, used:] == 7.0).all()) and o.intact()
    close(S, S_ref, "f32")
    fresh, _ = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], seq_offsets=off, mode=mode)
    assert bool((fresh[:, :, used:] == 0).all()) and torch.equal(fresh[:, :, :used], o.t[:, :, :used])


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
def test_offsets_out_of_order_stay_inside(mode):
    """Offsets that leave the tokens or fall are bounded: finite results, guards intact."""
    inp = inputs.gdr_inputs(1, 1, 2, 90, 32, 16, "bf16", seed=2)
    t = to_dev(inp, "bf16")
    for bad in ([-5, 40, 1000], [80, 10, 90], [2**31 - 1, -2**31, 5], [91, 92, 93]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, S = Guarded((1, 2, 90, 16), torch.bfloat16), Guarded((2, 2, 32, 16), torch.float32)
        o.t.zero_()
        S0 = torch.zeros(2, 2, 32, 16, device="cuda")
        mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], S0, seq_offsets=off, mode=mode, o=o.t, S_out=S.t)
        assert o.intact() and S.intact() and bool(torch.isfinite(S.t).all())


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_views(dtype, mode):
    """Slices of one projection [B,T,width], gates [B,T,H], and one key row for all tokens (stride 0)."""
    B, HK, H, T, K, V = 2, 2, 4, 77, 32, 24
    inp = inputs.gdr_inputs(B, HK, H, T, K, V, dtype, seed=8)
    inp["k"][:] = inp["k"][:, :, :1]
    t = to_dev(inp, dtype)
    fused = torch.cat([t["q"].transpose(1, 2).reshape(B, T, -1), t["v"].transpose(1, 2).reshape(B, T, -1)], -1)
    q = fused[..., :HK * K].view(B, T, HK, K).transpose(1, 2)
    v = fused[..., HK * K:].view(B, T, H, V).transpose(1, 2)
    k = t["k"][:, :, :1].expand(B, HK, T, K)
    g, beta = (t[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("g", "beta"))
    o = torch.empty(B, T, H, V, dtype=q.dtype, device="cuda").transpose(1, 2)
    assert not q.is_contiguous() and k.stride(2) == 0
    _, S = mlstm.gdr_fwd(q, k, v, g, beta, t["S0"], mode=mode, o=o)
    o2, S2 = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, dtype, coarse(inp, dtype, mode))
    close(S, S_ref, "f32")


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_extremes(dtype, mode):
    """Full resets, decays down to e^-90, no decay at all, write strengths 0, 1 and 2."""
    inp = inputs.gdr_inputs(1, 2, 2, 150, 64, 32, dtype, seed=12)
    rng = np.random.default_rng(1)
    inp["g"][0, 0] = rng.choice([0.0, -np.inf, -90.0, -5.0, -1e-4, -1e30], 150)
    inp["beta"][:] = rng.choice([0.0, 1.0, 2.0], (1, 2, 150))
    t = to_dev(inp, dtype)
    o, S = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode)
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, dtype, coarse(inp, dtype, mode))
    close(S, S_ref, "f32")


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_scales_of_the_inputs(dtype, mode, scale):
    """Values and states far from one; k stays of unit length, q takes the other end."""
    inp = inputs.gdr_inputs(1, 1, 2, 100, 64, 32, "f64", seed=13)
    for n, f in (("v", scale), ("S0", scale), ("q", 1 / scale)):
        inp[n] = inp[n] * f
    for n in ("q", "k", "v"):
        inp[n] = inputs.round_to(inp[n], dtype)
    t = to_dev(inp, dtype)
    inp = {n: x.double().cpu().numpy() for n, x in t.items()}
    o, S = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode)
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, dtype, coarse(inp, dtype, mode))
    close(S, S_ref, "f32")


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
def test_values_that_are_not_finite_stay_in_their_head(mode):
    inp = inputs.gdr_inputs(2, 2, 2, 80, 64, 32, "bf16", seed=14)
    t = to_dev(inp, "bf16")
    o1, S1 = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode)
    t["v"][0, 1, 40, 3] = float("nan")
    t["g"][1, 0, 70] = float("nan")
    o2, S2 = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode)
    for a, b in ((o1, o2), (S1, S2)):
        assert torch.equal(a[0, 0], b[0, 0]) and torch.equal(a[1, 1], b[1, 1])
    assert bool(torch.isnan(o2[0, 1, 40:, 3]).all()) and bool(torch.isnan(S2[1, 0]).all())
    assert bool(torch.isfinite(o2[1, 0, :64].float()).all())


MANY = [  # enough heads for the tcgen05 pass: B, HK, H, T, K, V
    (20, 2, 4, 130, 128, 128), (10, 4, 8, 64, 64, 128), (5, 8, 16, 200, 96, 88), (10, 4, 8, 65, 40, 104), (5, 4, 8, 63, 128, 256),
    (3, 16, 16, 33, 16, 248), (81, 1, 1, 129, 128, 104),
]


@pytest.mark.parametrize("shape", MANY)
def test_many_heads(shape):
    inp = inputs.gdr_inputs(*shape, "bf16", seed=sum(shape))
    B, HK, H, T, K, V = shape
    t = to_dev(inp, "bf16")
    a = [t[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    o, S = Guarded((B, H, T, V), torch.bfloat16), Guarded((B, H, K, V), torch.float32)
    p = mlstm.gdr_params(*a[:5], o.t)
    ws = torch.empty(mlstm.gdr_fwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    mlstm.gdr_fwd(*a, o=o.t, S_out=S.t, workspace=ws)
    assert mlstm.gdr_status(p, ws) == 0 and mlstm.gdr_status(p, None) != 0  # (that pass, which has waits)
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o.t, o_ref, "bf16", coarse(inp, "bf16", "chunk"))
    close(S.t, S_ref, "f32")
    assert o.intact() and S.intact()
    o2, S2 = mlstm.gdr_fwd(*a)
    assert torch.equal(o.t, o2) and torch.equal(S.t, S2)


@pytest.mark.parametrize("dtype,shape", [  # B, HK, H, T, K, V: one, two and four tiles of values a block
    ("bf16", (1, 12, 24, 150, 128, 128)), ("bf16", (4, 12, 12, 150, 72, 128)), ("bf16", (2, 20, 40, 150, 64, 64)),
    ("f32", (2, 16, 16, 150, 128, 128)), ("f32", (3, 8, 16, 150, 64, 64)), ("f32", (1, 2, 2, 200, 128, 72)),
])
def test_tiles_a_block(dtype, shape):
    inp = inputs.gdr_inputs(*shape, dtype, seed=sum(shape))
    t = to_dev(inp, dtype)
    o, S = mlstm.gdr_fwd(*(t[n] for n in ("q", "k", "v", "g", "beta", "S0")), mode="chunk")
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, dtype, coarse(inp, dtype, "chunk"))
    close(S, S_ref, "f32")


def test_four_tiles_a_block_packed():
    lengths, T, H = (70, 0, 1, 64, 130, 5, 3, 128, 65, 12), 480, 14
    inp = inputs.gdr_inputs(1, 7, H, T, 72, 128, "bf16", seed=8)
    inp["S0"] = (0.1 * np.random.default_rng(8).standard_normal((10, H, 72, 128))).astype(np.float32)
    o_ref, S_ref, off, terms = packed(inp, lengths)
    t = to_dev(inp, "bf16")
    o, S = mlstm.gdr_fwd(*(t[n] for n in ("q", "k", "v", "g", "beta", "S0")), seq_offsets=off)
    used = sum(lengths)
    close(o[:, :, :used], o_ref[:, :, :used], "bf16", terms[:, :, :used])
    close(S, S_ref, "f32")
    assert bool((o[:, :, used:] == 0).all())


def test_many_heads_packed_strided_and_extreme():
    """Unlike lengths, token-major views, full resets and values that are not finite, on the tcgen05 pass."""
    lengths, T, H = (70, 0, 1, 64, 130, 5), 273, 32
    inp = inputs.gdr_inputs(1, 4, H, T, 64, 104, "bf16", seed=6)
    rng = np.random.default_rng(6)
    inp["S0"] = (0.1 * rng.standard_normal((6, H, 64, 104))).astype(np.float32)
    inp["g"][0, 0, ::7] = -np.inf
    inp["g"][0, 1] *= 300
    inp["beta"][0, 2] = 0.0
    o_ref, S_ref, off, terms = packed(inp, lengths)
    t = to_dev(inp, "bf16")
    flip = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)
    a = [flip(t[n]) for n in ("q", "k", "v", "g", "beta")]
    o = torch.full((1, T, H, 104), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    _, S = mlstm.gdr_fwd(*a, t["S0"], seq_offsets=off, mode="chunk", o=o)
    used = sum(lengths)
    close(o[:, :, :used], o_ref[:, :, :used], "bf16", terms[:, :, :used])
    close(S, S_ref, "f32")
    assert bool((o[:, :, used:] == 7.0).all())
    a[2][0, 3, 75] = float("nan")
    o2, S2 = mlstm.gdr_fwd(*a, t["S0"], seq_offsets=off, mode="chunk")
    clean = [h for h in range(H) if h != 3]
    assert torch.equal(o2[:, clean, :used], o[:, clean, :used]) and torch.equal(S2[:, clean], S[:, clean])
    assert bool(torch.isnan(o2[0, 3, 75:135]).all()) and bool(torch.isnan(S2[3, 3]).any()) and torch.equal(S2[4], S[4])


@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_many_heads_at_other_scales(scale):
    inp = inputs.gdr_inputs(10, 8, 8, 100, 64, 104, "f64", seed=13)
    for n, f in (("v", scale), ("S0", scale), ("q", 1 / scale)):
        inp[n] = inp[n] * f
    t = {n: dev(inp[n], torch.bfloat16) for n in ("q", "k", "v")} | {n: dev(inp[n]) for n in ("g", "beta", "S0")}
    inp = {n: x.double().cpu().numpy() for n, x in t.items()}
    o, S = mlstm.gdr_fwd(*(t[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, "bf16", coarse(inp, "bf16", "chunk"))
    close(S, S_ref, "f32")


def test_a_wait_that_runs_out_is_reported_and_the_workspace_stays_usable():
    """A limit shorter than any copy takes: the status says so, and an ordinary call on the same workspace is right."""
    inp = inputs.gdr_inputs(20, 4, 4, 130, 128, 128, "bf16", seed=9)
    t = to_dev(inp, "bf16")
    a = [t[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    short = mlstm.gdr_params(*a[:5], wait_limit_cycles=256)
    ws = torch.empty(mlstm.gdr_fwd_workspace_size(short), dtype=torch.uint8, device="cuda")
    mlstm.gdr_fwd(*a, workspace=ws, wait_limit_cycles=256)
    assert mlstm.gdr_status(short, ws) == 8
    o, S = mlstm.gdr_fwd(*a, workspace=ws)
    assert mlstm.gdr_status(mlstm.gdr_params(*a[:5]), ws) == 0
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o, o_ref, "bf16", coarse(inp, "bf16", "chunk"))
    close(S, S_ref, "f32")


def test_no_tokens_and_state_in_place():
    q = torch.empty(2, 1, 0, 16, device="cuda")
    v = torch.empty(2, 2, 0, 8, device="cuda")
    g = torch.empty(2, 2, 0, device="cuda")
    S0 = torch.randn(2, 2, 16, 8, device="cuda")
    _, S = mlstm.gdr_fwd(q, q, v, g, g, S0)
    assert torch.equal(S, S0)
    _, S = mlstm.gdr_fwd(q, q, v, g, g)
    assert bool((S == 0).all())
    for mode in ("recurrent", "chunk"):
        t = to_dev(inputs.gdr_inputs(2, 1, 2, 70, 16, 8, "bf16", seed=3), "bf16")
        o, S = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode)
        o2, S2 = mlstm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], mode=mode, S_out=t["S0"])
        assert S2 is t["S0"] and torch.equal(S, S2) and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,HK,H,K,V", [(1, 1, 1, 8, 8), (3, 2, 4, 64, 40), (2, 1, 3, 128, 128), (5, 2, 2, 256, 256),
                                        (2, 1, 1, 100 - 4, 24), (90, 2, 4, 128, 128), (300, 2, 2, 32, 64)])
def test_step(B, HK, H, K, V, dtype):
    inp = inputs.gdr_inputs(B, HK, H, 1, K, V, dtype, seed=K + V)
    t = to_dev(inp, dtype)
    one = {n: t[n][:, :, 0] for n in ("q", "k", "v", "g", "beta")}
    S = Guarded((B, H, K, V), torch.float32)
    S.fill(t["S0"])
    o = Guarded((B, H, V), TORCH_DTYPE[dtype])
    mlstm.gdr_step(*one.values(), S.t, o=o.t)
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    close(o.t[:, :, None], o_ref, dtype)
    close(S.t, S_ref, "f32")
    assert o.intact() and S.intact()


def test_step_with_slots_padding_and_a_slot_named_twice():
    B, HK, H, K, V, pool = 9, 1, 2, 64, 72, 12
    inp = inputs.gdr_inputs(B, HK, H, 1, K, V, "bf16", seed=31)
    t = to_dev(inp, "bf16")
    one = {n: t[n][:, :, 0] for n in ("q", "k", "v", "g", "beta")}
    slots = [3, -1, 11, 3, 0, 12, 3, 11, -2**31]
    S0 = torch.randn(pool, H, K, V, device="cuda") * 0.1
    S = S0.clone()
    o = mlstm.gdr_step(*one.values(), S, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    ref = S0.double().cpu().numpy()
    for b, s in enumerate(slots):
        if not 0 <= s < pool:
            assert bool((o[b] == 0).all())
            continue
        sl = slice(b, b + 1)
        o_ref, new = oracle.gdr_sequential(*(inp[n][sl] for n in ("q", "k", "v", "g", "beta")), ref[s:s + 1])
        ref[s] = new[0]
        close(o[sl][:, :, None], o_ref, "bf16")
    close(S, ref, "f32")
    untouched = [s for s in range(pool) if s not in slots]
    assert torch.equal(S[untouched], S0[untouched])


def test_steps_continue_a_prefill():
    """A prefill and single tokens after it give what one prefill over all of them gives."""
    inp = inputs.gdr_inputs(3, 2, 4, 75, 64, 32, "bf16", seed=41)
    t = to_dev(inp, "bf16")
    o_ref, S_ref = oracle.gdr_sequential(*(inp[n] for n in ("q", "k", "v", "g", "beta", "S0")))
    head = {n: t[n][:, :, :70] for n in ("q", "k", "v", "g", "beta")}
    _, S = mlstm.gdr_fwd(*head.values(), t["S0"])
    for i in range(70, 75):
        o = mlstm.gdr_step(*(t[n][:, :, i] for n in ("q", "k", "v", "g", "beta")), S)
        close(o[:, :, None], o_ref[:, :, i:i + 1], "bf16")
    close(S, S_ref, "f32")


def test_captured_replayed_and_on_another_stream():
    t = to_dev(inputs.gdr_inputs(2, 2, 2, 200, 64, 64, "bf16", seed=51), "bf16")
    a = [t[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    ref = {m: mlstm.gdr_fwd(*a, mode=m) for m in ("recurrent", "chunk")}
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):  # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append({m: mlstm.gdr_fwd(*a, mode=m) for m in ref})
        graphs.append(graph)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs.append({m: mlstm.gdr_fwd(*a, mode=m, stream=side) for m in ref})
    torch.cuda.current_stream().wait_stream(side)
    for out in outs:
        for m in ref:
            assert torch.equal(out[m][0], ref[m][0]) and torch.equal(out[m][1], ref[m][1])


def test_a_block_of_norm_projections_recurrence_and_norm():
    """The operators as a layer uses them: the pre-norm of the residual stream, projections (library
    products of the caller), the gated delta rule on strided slices of them, the output's norm per head.
    Against the same chain in 64 bits; each bf16 tensor between them is rounded there as well, the
    projections' rounding can differ by one step: 2^-7 of the largest value through the rest."""
    B, T, D, HK, H, K, V = 2, 90, 256, 2, 4, 32, 64
    gen = torch.Generator(device="cuda").manual_seed(7)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, res = n(B, T, D).bfloat16(), n(B, T, D).bfloat16()
    w, W = 1 + 0.1 * n(D), (n(D, 2 * HK * K + H * V) / 16).bfloat16()
    g, beta = -torch.exp(n(B, T, H) - 3), torch.sigmoid(n(B, T, H))
    y, r, _ = mlstm.rms_norm(x, res, w)
    p = y @ W
    cut = lambda lo, heads, d: p[..., lo:lo + heads * d].view(B, T, heads, d).transpose(1, 2)
    q, k, v = cut(0, HK, K), cut(HK * K, HK, K), cut(2 * HK * K, H, V)
    k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
    q = (q.float() / K ** 0.5).bfloat16()
    o = torch.empty(B, T, H, V, device="cuda", dtype=torch.bfloat16)
    mlstm.gdr_fwd(q, k, v, g.transpose(1, 2), beta.transpose(1, 2), o=o.transpose(1, 2))
    out, _, _ = mlstm.rms_norm(o)
    r64 = x.double() + res.double()
    y64 = r64 / torch.sqrt((r64 * r64).mean(-1, keepdim=True) + 1e-6) * w.double()
    close(y.flatten(0, 1)[None], y64.flatten(0, 1)[None].cpu(), "bf16", rel=2.0 ** -19)
    o_ref, _ = oracle.gdr_sequential(*(a.double().cpu().numpy() for a in (q, k, v, g.transpose(1, 2),
                                                                          beta.transpose(1, 2))))
    wide = dict(zip(("q", "k", "v", "g", "beta"), (a.double().cpu().numpy() for a in (q, k, v, g.transpose(1, 2),
                                                                                     beta.transpose(1, 2)))))
    close(o.transpose(1, 2), o_ref, "bf16", coarse(wide | {"S0": None}, "bf16", "auto"))
    o64 = o.double()
    out64 = o64 / torch.sqrt((o64 * o64).mean(-1, keepdim=True) + 1e-6)
    close(out.flatten(0, 2)[None], out64.flatten(0, 2)[None].cpu(), "bf16", rel=2.0 ** -19)
