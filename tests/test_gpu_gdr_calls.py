"""Calls of the gated delta rule that its documentation allows, one by one: sequences that begin behind the first
token, offsets that pass 32 bits, captured decode steps, calls without a state or without rows.  References and
tolerances of test_gpu_gdr.py and test_gpu_gdr_backward.py."""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_token_b200 import inputs, mlstm
from tests.helpers import TORCH_DTYPE
from tests.test_gpu_gdr import close, coarse, readout_terms, to_dev
from tests.test_gpu_gdr_backward import NAMES, call, check, make

pytestmark = pytest.mark.gpu

FAR = (1 << 32) + 64  # elements


@pytest.fixture
def give_back():
    """What a test of 10 to 20 GB held goes back to the device."""
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", [(7, 77, 77, 140), (70, 71, 150), (128, 192)])
def test_sequences_that_begin_behind_the_first_token(offsets, dtype, mode):
    T, H, N = 200, 4, len(offsets) - 1
    inp = inputs.gdr_inputs(1, 2, H, T, 64, 48, dtype, seed=T + N)
    inp["S0"] = (0.1 * np.random.default_rng(N).standard_normal((N, H, 64, 48))).astype(np.float32)
    t = to_dev(inp, dtype)
    o = torch.full((1, H, T, 48), 7.0, dtype=TORCH_DTYPE[dtype], device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    _, S = mlstm.gdr_fwd(*(t[n] for n in ("q", "k", "v", "g", "beta", "S0")), seq_offsets=off, mode=mode, o=o)
    for n in range(N):
        lo, hi = offsets[n], offsets[n + 1]
        one = {m: inp[m][:, :, lo:hi] for m in NAMES} | {"S0": inp["S0"][n:n + 1]}
        o_ref, S_ref = oracle.gdr_sequential(*(one[m] for m in NAMES), one["S0"])
        if hi > lo:
            close(o[:, :, lo:hi], o_ref, dtype, 2.0 ** -9.9 * readout_terms(one) if dtype == "bf16" else 0.0)
        close(S[n:n + 1], S_ref, "f32")
    assert bool((o[:, :, :offsets[0]] == 7.0).all()) and bool((o[:, :, offsets[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", [(7, 77, 77, 140), (128, 192)])
def test_gradients_of_sequences_that_begin_behind_the_first_token(offsets, dtype):
    T, H, N = 200, 4, len(offsets) - 1
    inp = make((1, 2, H, T, 64, 48), dtype, T + N, True, N)
    out = call(inp, dtype, seq_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    for n in range(N):
        lo, hi = offsets[n], offsets[n + 1]
        if hi > lo:
            one = {m: inp[m][:, :, lo:hi] for m in NAMES + ("do",)} | {m: inp[m][n:n + 1] for m in ("S0", "dS")}
            check({m: out[m][:, :, lo:hi] for m in ("dq", "dk", "dv", "dg", "dbeta")} | {"dS0": out["dS0"][n:n + 1]},
                  one, dtype)
        else:
            assert np.array_equal(out["dS0"][n].cpu().numpy(), inp["dS"][n])
    for m in ("dq", "dk", "dv", "dg", "dbeta"):
        assert bool((out[m][:, :, :offsets[0]] == 0).all()) and bool((out[m][:, :, offsets[-1]:] == 0).all())


def far(x, buffer, at):
    """x [1 or 2, heads, tokens, d] laid out in buffer from element `at`, FAR elements between tokens (or, of one token,
    between batch rows)."""
    B, H, T, D = x.shape
    view = buffer.as_strided((B, H, T, D), (FAR if T == 1 else 0, D, FAR, 1), at)
    view.copy_(x)
    return view


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
def test_strides_that_pass_32_bits(mode, give_back):
    inp = inputs.gdr_inputs(1, 1, 2, 2, 64, 64, "bf16", seed=5)
    t = to_dev(inp, "bf16")
    a = [t[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    ref, S_ref = mlstm.gdr_fwd(*a, mode=mode)
    wide, out = (torch.empty(FAR + 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (far(t[n], wide, at) for n, at in (("q", 0), ("k", 128), ("v", 256)))
    o = far(torch.zeros_like(t["v"]), out, 64)
    _, S = mlstm.gdr_fwd(q, k, v, *a[3:], mode=mode, o=o)
    assert torch.equal(o, ref) and torch.equal(S, S_ref)
    if mode == "chunk":
        do, dS = torch.randn_like(t["v"]), torch.randn_like(t["S0"])
        want = mlstm.gdr_bwd(*a[:5], do, a[5], dS)
        got = mlstm.gdr_bwd(q, k, v, *a[3:5], far(do, out, 64), a[5], dS)
        assert all(torch.equal(want[n], got[n]) for n in want)


def test_a_step_whose_rows_and_states_lie_far_apart(give_back):
    """Batch strides of more than 2^32 elements, and a pool of more than 2^31."""
    inp = inputs.gdr_inputs(2, 1, 2, 1, 64, 64, "bf16", seed=6)
    t = to_dev(inp, "bf16")
    S = t["S0"].clone()
    ref = mlstm.gdr_step(*(t[n][:, :, 0] for n in NAMES), S)
    wide, out = (torch.empty(FAR + 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (far(t[n], wide, at)[:, :, 0] for n, at in (("q", 0), ("k", 128), ("v", 256)))
    o = far(torch.zeros_like(t["v"]), out, 64)[:, :, 0]
    pool = (1 << 31) // (2 * 64 * 64) + 5
    states = torch.empty(pool, 2, 64, 64, device="cuda")
    slots = torch.tensor([pool - 1, 1], dtype=torch.int32, device="cuda")
    states[slots.long()] = t["S0"]
    mlstm.gdr_step(q, k, v, t["g"][:, :, 0], t["beta"][:, :, 0], states, slots=slots, o=o)
    assert torch.equal(o, ref) and torch.equal(states[slots.long()], S)


def test_captured_steps_follow_their_slots():
    """One captured step, replayed on other slots and inputs in the captured tensors, one slot named twice among them."""
    B, H, K, V, pool = 5, 2, 64, 72, 8
    inp = inputs.gdr_inputs(B, 1, H, 3, K, V, "bf16", seed=7)
    t = to_dev(inp, "bf16")
    now = [t[n][:, :, 0].clone() for n in NAMES]
    S0 = 0.1 * torch.randn(pool, H, K, V, device="cuda")
    S, slots = S0.clone(), torch.zeros(B, dtype=torch.int32, device="cuda")
    mlstm.gdr_step(*now, S, slots=slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = mlstm.gdr_step(*now, S, slots=slots)
    S.copy_(S0)
    ref = S0.clone()
    for i, names in enumerate(([3, 1, 0, 7, 2], [1, -1, 1, 9, 4], [5, 5, 5, 5, 5])):
        for x, n in zip(now, NAMES):
            x.copy_(t[n][:, :, i])
        slots.copy_(torch.tensor(names, dtype=torch.int32))
        graph.replay()
        want = mlstm.gdr_step(*(t[n][:, :, i] for n in NAMES), ref, slots=slots)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(S, ref)


@pytest.mark.parametrize("mode", ["recurrent", "chunk"])
def test_without_a_state(mode):
    inp = inputs.gdr_inputs(2, 1, 2, 70, 32, 24, "bf16", seed=8, with_state=False)
    t = to_dev(inp, "bf16")
    o, S = mlstm.gdr_fwd(*(t[n] for n in NAMES), mode=mode, return_state=False)
    assert S is None
    close(o, oracle.gdr_sequential(*(inp[n] for n in NAMES))[0], "bf16", coarse(inp, "bf16", mode))


def test_no_rows():
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
    q, v, g = e(0, 1, 5, 16), e(0, 2, 5, 8), e(0, 2, 5)
    o, S = mlstm.gdr_fwd(q, q, v, g, g)
    assert o.shape == v.shape and S.shape == (0, 2, 16, 8)
    d = mlstm.gdr_bwd(q, q, v, g, g, v)
    assert d["dq"].shape == q.shape and d["dS0"].shape == (0, 2, 16, 8)
    S = torch.randn(3, 2, 16, 8, device="cuda")
    before = S.clone()
    slots = e(0, dtype=torch.int32)
    assert mlstm.gdr_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], g[:, :, 0], S, slots=slots).shape == (0, 2, 8)
    torch.cuda.synchronize()
    assert torch.equal(S, before)


def test_more_rows_than_32_bits_of_elements(give_back):
    """The norm and its gradients over 2^31 elements and a few rows more: the last rows as alone."""
    D = 4096
    rows = (1 << 31) // D + 3
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, D, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    y, r, s = mlstm.rms_norm(x, x, w, quant="int8", group=128)
    y1, r1, s1 = mlstm.rms_norm(x[-5:].clone(), x[-5:].clone(), w, quant="int8", group=128)
    assert torch.equal(y[-5:], y1) and torch.equal(r[-5:], r1) and torch.equal(s[-5:], s1)
    dx, _ = mlstm.rms_norm_bwd(x, r, w)
    dx1, _ = mlstm.rms_norm_bwd(x[-5:].clone(), r1, w)
    assert torch.equal(dx[-5:], dx1)
