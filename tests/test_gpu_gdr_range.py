"""The gated delta rule where magnitudes differ within a call: gradients far below their neighbours', and
columns with an infinity beside others without."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_token_b200 import inputs, mlstm
from tests.helpers import TORCH_DTYPE, Guarded, dev
from tests.test_gpu_gdr import to_dev
from tests.test_gpu_gdr_backward import COARSE, HALF, NAMES, call, magnitudes, make

pytestmark = pytest.mark.gpu

SHAPES = [  # B, HK, H, T, K, V
    ("bf16", (1, 2, 2, 140, 64, 48)), ("bf16", (1, 1, 2, 140, 128, 72)), ("f32", (1, 2, 2, 140, 64, 48)),
    ("f32", (1, 1, 2, 140, 128, 72)),
]


def held_by_row(x, ref, mag, dtype):
    """Each gradient of q or k against the magnitudes of its own terms.  It is a sum of products of what the
    passes left (S, dS, U, dV: within 2^-14 of their largest, as everywhere) and dO or k, so beside the
    operands' bits the row's largest sum of magnitudes counts with 2^-14; no other row does."""
    x = x.double().cpu().numpy()
    bound = HALF[dtype] * np.abs(ref) + COARSE[dtype] * mag + 2.0 ** -14 * mag.max(axis=-1, keepdims=True)
    bad = ~(np.abs(x - ref) <= bound)
    assert not bad.any(), float((np.abs(x - ref) / (mag + 1e-300)).max())


def both(inp, dtype):
    ref = oracle.gdr_sequential_backward(*(inp[n] for n in NAMES), inp["do"], inp["S0"], inp["dS"])
    return call(inp, dtype), ref, magnitudes(inp)


@pytest.mark.parametrize("factor", [2.0 ** -12, 2.0 ** -30, 2.0 ** -60])
@pytest.mark.parametrize("dtype,shape", SHAPES)
def test_a_group_of_small_output_gradients_keeps_its_dq(dtype, shape, factor):
    inp = make(shape, dtype, 61)
    inp["do"][:, :, 80:96] *= factor  # a power of two: exact
    out, ref, mag = both(inp, dtype)
    held_by_row(out["dq"], ref["dq"], mag["dq"], dtype)
    assert bool((out["dq"][:, :, 80:96] != 0).any(-1).all())


@pytest.mark.parametrize("factor", [2.0 ** -12, 2.0 ** -30, 2.0 ** -60])
@pytest.mark.parametrize("dtype,shape", SHAPES)
def test_a_group_of_small_write_strengths_keeps_its_dk(dtype, shape, factor):
    inp = make(shape, dtype, 62)
    inp["beta"][:, :, 64:80] *= factor  # U, dV, and so every term of dk, are as small
    out, ref, mag = both(inp, dtype)
    held_by_row(out["dk"], ref["dk"], mag["dk"], dtype)
    assert bool((out["dk"][:, :, 64:80] != 0).any(-1).all())


@pytest.mark.parametrize("power", [10, 20, 30, 40])
@pytest.mark.parametrize("dtype,shape", SHAPES)
def test_large_output_gradients_beside_small_values_and_the_reverse(dtype, shape, power):
    """Columns 0 .. 15 have large dO and dS and small v and S0, the others the reverse: every product of the two
    counts alike in dq and dk."""
    inp = make(shape, dtype, 63)
    f = np.float32(2.0 ** (power / 2))
    for n in ("do", "dS"):
        inp[n][..., :16] *= f
        inp[n][..., 16:] /= f
    for n in ("v", "S0"):
        inp[n][..., :16] /= f
        inp[n][..., 16:] *= f
    out, ref, mag = both(inp, dtype)
    held_by_row(out["dq"], ref["dq"], mag["dq"], dtype)
    held_by_row(out["dk"], ref["dk"], mag["dk"], dtype)


@pytest.mark.parametrize("dtype,shape", SHAPES)
def test_small_rows_among_the_products_of_tokens(dtype, shape):
    """One token in each 16 with dO 2^-15 of the others', and beta 2^-15 at another: what reaches dq and dk by way
    of the other tokens of the chunk alone (S0 = dS = 0, one chunk)."""
    B, HK, H, _, K, V = shape
    inp = make((B, HK, H, 64, K, V), dtype, 64, states=False)
    inp["do"][:, :, 5::16] *= 2.0 ** -15
    inp["beta"][:, :, 9::16] *= 2.0 ** -15
    out, ref, mag = both(inp, dtype)
    held_by_row(out["dq"], ref["dq"], mag["dq"], dtype)
    held_by_row(out["dk"], ref["dk"], mag["dk"], dtype)


# One, two and four tiles of values a block in both types, and the tcgen05 pass: B, HK, H, T, K, V
FORWARD = [
    ("bf16", (1, 2, 4, 150, 64, 48)), ("bf16", (1, 1, 2, 150, 128, 72)), ("bf16", (1, 12, 24, 150, 128, 128)),
    ("bf16", (4, 12, 12, 150, 72, 128)), ("bf16", (2, 20, 40, 150, 64, 64)), ("bf16", (20, 2, 4, 130, 128, 128)),
    ("f32", (1, 2, 2, 150, 64, 48)), ("f32", (1, 2, 2, 200, 128, 72)), ("f32", (2, 16, 16, 150, 128, 128)),
    ("f32", (3, 8, 16, 150, 64, 64)),
]
BACKWARD = [
    ("bf16", (1, 2, 4, 140, 64, 48)), ("bf16", (1, 1, 2, 140, 128, 72)), ("bf16", (1, 16, 32, 140, 128, 128)),
    ("bf16", (1, 32, 32, 100, 72, 256)), ("bf16", (3, 16, 32, 140, 64, 64)), ("bf16", (2, 37, 37, 100, 32, 64)),
    ("f32", (1, 2, 2, 140, 64, 48)), ("f32", (2, 16, 16, 140, 128, 128)), ("f32", (3, 8, 16, 140, 64, 64)),
]
COLUMN, TOKEN, BEFORE = 3, 85, 80  # the infinity's, and the first token of its group of 16


def without_column(V):
    return [c for c in range(V) if c != COLUMN]


@pytest.mark.parametrize("name", ["v", "S0"])
@pytest.mark.parametrize("mode", ["chunk", "recurrent"])
@pytest.mark.parametrize("dtype,shape", FORWARD)
def test_an_infinity_stays_in_its_column(dtype, shape, mode, name):
    """Bitwise: the column is 2^-20 of the others, so no scale is its own with or without the infinity."""
    inp = inputs.gdr_inputs(*shape, dtype, seed=71)
    inp["v"][..., COLUMN] *= 2.0 ** -20
    inp["S0"][..., COLUMN] *= 2.0 ** -20
    t = to_dev(inp, dtype)
    run = lambda: mlstm.gdr_fwd(*(t[n] for n in ("q", "k", "v", "g", "beta", "S0")), mode=mode)
    o, S = run()
    if name == "v":
        t["v"][:, :, TOKEN, COLUMN] = float("inf")
    else:
        t["S0"][:, :, 5, COLUMN] = -float("inf")
    o2, S2 = run()
    rest = without_column(shape[-1])
    assert torch.equal(o[..., rest], o2[..., rest]) and torch.equal(S[..., rest], S2[..., rest])
    first = TOKEN if name == "v" else 0
    assert not bool(torch.isfinite(o2[:, :, first:, COLUMN]).any()) and not bool(torch.isfinite(S2[..., COLUMN]).any())
    if name == "v":  # nor does it reach the chunk before
        assert torch.equal(o[:, :, :64], o2[:, :, :64])


@pytest.mark.parametrize("name", ["v", "S0", "do", "dS"])
@pytest.mark.parametrize("dtype,shape", BACKWARD)
def test_an_infinity_stays_in_its_column_of_the_gradients(dtype, shape, name):
    inp = make(shape, dtype, 72)
    for n in ("v", "S0", "do", "dS"):
        inp[n][..., COLUMN] *= 2.0 ** -20
    a = call(inp, dtype)
    if name in ("v", "do"):
        inp[name][:, :, TOKEN, COLUMN] = np.inf
    else:
        inp[name][:, :, 5, COLUMN] = np.inf
    b = call(inp, dtype)
    rest = without_column(shape[-1])
    assert all(torch.equal(a[n][..., rest], b[n][..., rest]) for n in ("dv", "dS0"))
    if name in ("do", "dS"):  # (dv, dS0 are linear in these two; what v and S0 reach is dq, dk and the gates)
        assert not bool(torch.isfinite(b["dv"][:, :, :TOKEN, COLUMN]).any())
    if name == "v":  # a token's dq depends on tokens up to it
        assert torch.equal(a["dq"][:, :, :BEFORE], b["dq"][:, :, :BEFORE])
        assert not bool(torch.isfinite(b["dq"][:, :, TOKEN:]).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [[-5, 40, 1000], [80, 10, 90], [2**31 - 1, -2**31, 5], [91, 92, 93], [0, 90, 0]])
def test_gradients_with_offsets_out_of_order_stay_inside(dtype, bad):
    """The C entry between guards: outputs, workspace, and inputs that must not change."""
    B, HK, H, T, K, V = 1, 1, 2, 90, 32, 16
    inp = make((B, HK, H, T, K, V), dtype, 2, True, 2)
    td, f32 = TORCH_DTYPE[dtype], torch.float32
    ins = [dev(inp[n], td) for n in ("q", "k", "v")] + [dev(inp[n]) for n in ("g", "beta", "S0")]
    ins += [torch.tensor(bad, dtype=torch.int32, device="cuda"), dev(inp["do"], td), dev(inp["dS"])]
    kept = [x.clone() for x in ins]
    outs = [Guarded(s, d) for s, d in (((B, HK, T, K), td), ((B, HK, T, K), td), ((B, H, T, V), td), ((B, H, T), f32),
                                       ((B, H, T), f32), ((2, H, K, V), f32))]
    p = mlstm.gdr_params(*ins[:5], ins[7], seq_offsets=ins[6])
    ws = Guarded((mlstm.gdr_bwd_workspace_size(p),), torch.uint8)
    by = [mlstm.GdrStride(h * T * d, T * d, d) for h, d in ((HK, K), (HK, K), (H, V))]
    st = mlstm.lib().mlstm_gdr_bwd(ctypes.byref(p), *(x.data_ptr() for x in ins), *by, *(x.t.data_ptr() for x in outs),
                                   ws.t.data_ptr(), ws.t.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and ws.intact() and all(x.intact() for x in outs)
    assert all(torch.equal(x, y) for x, y in zip(ins, kept))
