"""The gated delta rule where magnitudes differ within a call: gradients far below their neighbours'."""
import numpy as np
import pytest

import oracle
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
