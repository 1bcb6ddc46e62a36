"""Root-mean-square norm (mlstm_rms_norm, mlstm_rms_norm_bwd) against its formulas in 64 bits.

Tolerances.  fp32 arithmetic: a row's mean of squares over D values is summed in at most 16 + 10
sequential steps (16 values a thread, then a tree), relative error <= 26 * 2^-24; the square root halves
it; the products, the division and the weight add 4 roundings: y within (13 + 4 + 2) * 2^-24 < 2^-19.7
relative.  Storage adds half a step.  The gradients' inner product mean(w dy r) has an absolute error of
26 * 2^-24 * mean|w dy r|, so dx is held to 2^-19 * (|w dy| + |r| s^2 mean|w dy r|) s + the rounding, and
dweight, a sum over rows in at most rows / 296 + 8 + 37 steps, to (rows + 40) * 2^-24 * sum|dy r s|."""
import numpy as np
import pytest
import torch

from linear_recurrent_token_b200 import mlstm
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TOP = {"e4m3": 448.0, "int8": 127.0}


def make(rows, D, dtype, seed, loud=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = n(rows, D).to(dtype)
    res = (n(rows, D) * (torch.exp(n(D)) if loud else 1.0)).to(dtype)
    return x, res, 1.0 + 0.3 * n(D), n(rows, D).to(dtype)


def norm64(x, res, w, eps):
    r = x.double() + (0 if res is None else res.double())
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, y if w is None else y * w.double()


def close(a, ref, half, rel=2.0 ** -19, extra=0.0):
    err = (a.double() - ref).abs()
    assert bool((err <= (half + rel) * ref.abs() + extra + 1e-30).all()), float((err / (ref.abs() + 1e-30)).max())


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 100), (9, 128), (300, 257), (7, 1000), (33, 1001), (4, 2048), (130, 4096),
          (3, 5000), (2, 8192), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("residual,weight", [(True, True), (False, False)])
def test_norm(rows, D, dtype, residual, weight):
    x, res, w, _ = make(rows, D, dtype, 3 + D)
    res, w = res if residual else None, w if weight else None
    y, r = Guarded((rows, D), dtype), Guarded((rows, D), dtype)
    mlstm.rms_norm(x, res, w, 1e-5, y=y.t, residual_out=r.t if residual else None)
    rr, yr = norm64(x, res, w, 1e-5)
    close(y.t, yr, HALF[dtype])
    if residual:
        close(r.t, rr, HALF[dtype], 2.0 ** -24)
    assert y.intact() and r.intact()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,D,group", [(1, 1, 0), (3, 7, 128), (2, 127, 128), (5, 128, 128), (9, 136, 128),
                                          (4, 129, 128), (33, 1001, 128), (33, 1001, 0), (7, 4096, 128), (130, 4096, 0),
                                          (3, 8192, 128), (2, 16383, 128), (2, 16384, 0), (300, 64, 0)])
def test_norm_in_8_bits(rows, D, group, dtype, quant):
    """Each value lies within half a step of the exact one: of 2^-4 relative (e4m3, 2^-10 of its unit under
    2^-6) or of the scale (int8), plus fp32's share; scales within fp32's share of the exact ones."""
    x, res, w, _ = make(rows, D, dtype, 5 + D)
    groups = -(-D // group) if group else 1
    q = Guarded((rows, D), torch.float8_e4m3fn if quant == "e4m3" else torch.int8)
    s = Guarded((rows, groups), torch.float32)
    _, r, _ = mlstm.rms_norm(x, res, w, 1e-5, quant=quant, group=group, y=q.t, scales=s.t)
    _, yr = norm64(x, res, w, 1e-5)
    size = group or D
    for j in range(groups):
        part = yr[:, j * size:(j + 1) * size]
        scale = part.abs().amax(-1) / TOP[quant]
        assert bool(((s.t[:, j].double() - scale).abs() <= 2.0 ** -19 * scale).all())
        got = q.t[:, j * size:(j + 1) * size].float().double()
        want = part / scale[:, None]
        step = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) if quant == "e4m3" else torch.full_like(want, 0.5)
        assert bool(((got - want).abs() <= step + 2.0 ** -18 * want.abs()).all())
        assert bool((got.abs().amax(-1) == TOP[quant]).all())  # the largest value takes the largest number
    assert q.intact() and s.intact()


@pytest.mark.parametrize("quant", [None, "e4m3", "int8"])
def test_rows_of_zeros_and_lone_nan_and_infinity(quant):
    for D in (256, 255):
        x = torch.zeros(4, D, device="cuda")
        x[1, 5], x[2, 7], x[3] = float("nan"), float("inf"), 1.0
        y, _, s = mlstm.rms_norm(x, eps=1e-6, quant=quant)
        y = y.float()
        assert bool((y[0] == 0).all()) and bool(torch.isfinite(y[3]).all())
        if quant is None:
            assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[2, 7]))
        else:
            assert float(s[0, 0]) == 1.0 and bool(torch.isnan(s[1, 0])) and bool(torch.isnan(s[2, 0]))
        if quant == "e4m3":
            assert bool(torch.isnan(y[1]).all())


def test_tiny_rows_keep_their_values():
    """Amplitudes near fp32's smallest: the scale's reciprocal would overflow."""
    x = torch.full((1, 128), 1e-36, device="cuda")
    w = torch.linspace(1e-4, 1.0, 128, device="cuda") * 1e-30
    y, _, s = mlstm.rms_norm(x, weight=w, eps=0.0, quant="e4m3")
    z = y.float().double() * s.double()
    ref = norm64(x, None, w, 0.0)[1]
    assert bool(((z - ref).abs() <= 2.0 ** -4 * ref.abs() + float(s) * 2.0 ** -10 + 1e-40).all())


@pytest.mark.parametrize("size", [1e-36, 1e-22, 1e18, 1e30])
def test_rows_whose_squares_leave_fp32(size):
    """Beside a row of ordinary size; values, and gradients in the range of fp32."""
    _, r, w, dy = make(9, 200, torch.float32, 23, loud=False)
    r[4] *= size
    y, _, _ = mlstm.rms_norm(r, weight=w, eps=0.0)
    close(y, norm64(r, None, w, 0.0)[1], HALF[torch.float32])
    dx, dw = mlstm.rms_norm_bwd(dy, r, w, 0.0)
    s = 1 / torch.sqrt((r.double() ** 2).mean(-1, keepdim=True))
    n, wd = r.double() * s, dy.double() * w.double()
    ref = s * (wd - n * (wd * n).mean(-1, keepdim=True))
    room = 2.0 ** -19 * s * (wd.abs() + n.abs() * (wd * n).abs().mean(-1, keepdim=True))
    close(dx, ref, HALF[torch.float32], 2.0 ** -24, room)
    assert bool(((dw.double() - (dy.double() * n).sum(0)).abs() <= 2.0 ** -18 * (dy.double() * n).abs().sum(0)).all())


@pytest.mark.parametrize("same", ["residual", "x"])
def test_sum_in_place(same):
    x, res, w, _ = make(37, 520, torch.bfloat16, 9)
    y0, r0, _ = mlstm.rms_norm(x, res, w)
    out = res if same == "residual" else x
    y1, r1, _ = mlstm.rms_norm(x, res, w, residual_out=out)
    assert r1 is out and torch.equal(r0, r1) and torch.equal(y0, y1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", SHAPES + [(1500, 72), (700, 2048)])
@pytest.mark.parametrize("extra,weight", [(True, True), (False, False)])
def test_gradients(rows, D, dtype, extra, weight):
    dr, r, w, dy = make(rows, D, dtype, 11 + D)
    dr, w = dr if extra else None, w if weight else None
    dx = Guarded((rows, D), dtype)
    _, dw = mlstm.rms_norm_bwd(dy, r, w, 1e-5, dr, dx=dx.t)
    r6, d6 = r.double(), dy.double()
    w6 = torch.ones(D, device="cuda", dtype=torch.float64) if w is None else w.double()
    s = 1 / torch.sqrt((r6 * r6).mean(-1, keepdim=True) + 1e-5)
    t = d6 * w6 * r6
    ref = s * (d6 * w6 - r6 * s * s * t.mean(-1, keepdim=True))
    room = 2.0 ** -19 * s * ((d6 * w6).abs() + r6.abs() * s * s * t.abs().mean(-1, keepdim=True))
    if extra:
        ref = ref + dr.double()
    close(dx.t, ref, HALF[dtype], 2.0 ** -24, room)
    terms = d6 * r6 * s
    err = (dw.double() - terms.sum(0)).abs()
    assert bool((err <= (2.0 ** -20 + (rows + 40) * 2.0 ** -24) * terms.abs().sum(0) + 1e-30).all())
    assert dx.intact()
    again, dw2 = mlstm.rms_norm_bwd(dy, r, w, 1e-5, dr)
    assert torch.equal(again, dx.t) and torch.equal(dw, dw2)


def test_gradients_against_differences():
    """Central differences of <dy, y> + <dr, r> in 64 bits along random directions, h = 1e-5: error ~ h^2."""
    dr, r, w, dy = make(4, 96, torch.float32, 21, loud=False)
    dx, dw = mlstm.rms_norm_bwd(dy, r, w, 1e-5, dr)
    loss = lambda a, b: float((norm64(a, None, b, 1e-5)[1] * dy.double()).sum() + (a * dr.double()).sum())
    gen = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(3):
        d = torch.randn(r.shape, generator=gen, device="cuda").double()
        e = torch.randn(w.shape, generator=gen, device="cuda").double()
        h = 1e-5
        num = (loss(r.double() + h * d, w.double() + h * e) - loss(r.double() - h * d, w.double() - h * e)) / (2 * h)
        got = float((dx.double() * d).sum() + (dw.double() * e).sum())
        assert abs(num - got) <= 1e-5 * (float((dx.double() * d).abs().sum()) + float((dw.double() * e).abs().sum()))


@pytest.mark.parametrize("same", ["dy", "dresidual"])
def test_gradient_in_place(same):
    dr, r, w, dy = make(50, 264, torch.bfloat16, 13)
    ref, dw = mlstm.rms_norm_bwd(dy, r, w, dresidual=dr)
    out = dy if same == "dy" else dr
    dx, dw2 = mlstm.rms_norm_bwd(dy, r, w, dresidual=dr, dx=out)
    assert dx is out and torch.equal(dx, ref) and torch.equal(dw, dw2)


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    y, r, s = mlstm.rms_norm(x, x.clone(), None, quant="e4m3")
    assert y.shape == (0, 64) and r.shape == (0, 64) and s.shape == (0, 1)
    dx, dw = mlstm.rms_norm_bwd(x, x.clone())
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_captured_and_replayed_on_another_stream():
    x, res, w, dy = make(65, 1024, torch.bfloat16, 17)
    y0, r0, _ = mlstm.rms_norm(x, res, w)
    dx0, dw0 = mlstm.rms_norm_bwd(dy, r0, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1, r1, _ = mlstm.rms_norm(x, res, w)
        dx1, dw1 = mlstm.rms_norm_bwd(dy, r1, w)
    for _ in range(2):
        y1.zero_(), dw1.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y0, y1) and torch.equal(r0, r1) and torch.equal(dx0, dx1) and torch.equal(dw0, dw1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, r2, _ = mlstm.rms_norm(x, res, w, stream=side)
    dx2, dw2 = mlstm.rms_norm_bwd(dy, r2, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y0, y2) and torch.equal(dx0, dx2) and torch.equal(dw0, dw2)
