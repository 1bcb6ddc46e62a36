"""The root-mean-square norm with more rows than its blocks take at once: at least six turns of a block's loop,
forward (444 blocks) and backward (296), one row a block and several.  References and tolerances of
test_gpu_rms_norm.py; the gradient of the weight sums more rows a block here: (rows + 40) * 2^-24 covers it."""
import pytest
import torch

from linear_recurrent_token_b200 import mlstm
from tests.helpers import Guarded
from tests.test_gpu_rms_norm import HALF, TOP, close, make, norm64

pytestmark = pytest.mark.gpu

# rows, D: one row a block with 256, 512 and 1024 threads, with and without 16-byte accesses (and the widest fp32 rows,
# which are read from memory as well); eight, four and two rows a block
SHAPES = [(3000, 4096), (3000, 1001), (2700, 5000), (2700, 5001), (2700, 10007), (2700, 16384), (25000, 72), (25000, 77),
          (13000, 1000), (13000, 513), (6000, 2048)]
DTYPES = [torch.float32, torch.bfloat16]


def held_in_8_bits(q, s, ref, quant, group):
    rows, D = ref.shape
    size = group or D
    for j in range(s.shape[-1]):
        part = ref[:, j * size:(j + 1) * size]
        scale = part.abs().amax(-1, keepdim=True) / TOP[quant]
        scale = torch.where(scale == 0, 1.0, scale)  # (one channel alone in a group now and then is x = -residual)
        assert bool(((s[:, j:j + 1].double() - scale).abs() <= 2.0 ** -19 * scale).all())
        got, want = q[:, j * size:(j + 1) * size].float().double(), part / scale
        step = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) if quant == "e4m3" else torch.full_like(want, 0.5)
        assert bool(((got - want).abs() <= step + 2.0 ** -18 * want.abs()).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("place", [None, "new", "residual", "x"])
def test_norm(rows, D, dtype, place):
    """place: no residual, a sum of its own, or the sum in the place of one of its terms."""
    x, res, w, _ = make(rows, D, dtype, 31 + D)
    rr, ref = norm64(x, res if place else None, w, 1e-5)
    kinds = [(None, 0), ("e4m3", 0), ("int8", 0), ("e4m3", 128), ("int8", 128)]
    for quant, group in kinds:
        a, b, r = (Guarded((rows, D), dtype) for _ in range(3))
        a.fill(x), b.fill(res)
        y = Guarded((rows, D), {None: dtype, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[quant])
        s = Guarded((rows, -(-D // group) if group else 1), torch.float32)
        out = {None: None, "new": r, "residual": b, "x": a}[place]
        mlstm.rms_norm(a.t, b.t if place else None, w, 1e-5, quant=quant, group=group, y=y.t,
                       residual_out=out.t if out else None, scales=s.t if quant else None)
        if quant:
            held_in_8_bits(y.t, s.t, ref, quant, group)
        else:
            close(y.t, ref, HALF[dtype])
        if out:
            close(out.t, rr, HALF[dtype], 2.0 ** -24)
        assert out is a or torch.equal(a.t, x)
        assert out is b or torch.equal(b.t, res)
        assert all(g.intact() for g in (a, b, r, y, s))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("place", [None, "new", "dy", "dresidual"])
def test_gradients(rows, D, dtype, place):
    """place: without the residual's gradient, or dx new or in the place of one of its terms."""
    dr, r, w, dy = make(rows, D, dtype, 37 + D)
    a, b, c, dx = (Guarded((rows, D), dtype) for _ in range(4))
    a.fill(dy), b.fill(dr), c.fill(r)
    out = {None: dx, "new": dx, "dy": a, "dresidual": b}[place]
    _, dw = mlstm.rms_norm_bwd(a.t, c.t, w, 1e-5, b.t if place else None, dx=out.t)
    r6, d6, w6 = r.double(), dy.double(), w.double()
    s = 1 / torch.sqrt((r6 * r6).mean(-1, keepdim=True) + 1e-5)
    t = d6 * w6 * r6
    ref = s * (d6 * w6 - r6 * s * s * t.mean(-1, keepdim=True))
    room = 2.0 ** -19 * s * ((d6 * w6).abs() + r6.abs() * s * s * t.abs().mean(-1, keepdim=True))
    close(out.t, ref + dr.double() if place else ref, HALF[dtype], 2.0 ** -24, room)
    terms = d6 * r6 * s
    err = (dw.double() - terms.sum(0)).abs()
    assert bool((err <= (2.0 ** -20 + (rows + 40) * 2.0 ** -24) * terms.abs().sum(0) + 1e-30).all())
    assert torch.equal(c.t, r) and (out is a or torch.equal(a.t, dy)) and (out is b or torch.equal(b.t, dr))
    assert all(g.intact() for g in (a, b, c, dx))
