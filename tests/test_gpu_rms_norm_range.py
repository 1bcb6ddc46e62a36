"""The root-mean-square norm at the ends of its range: outputs near fp32's largest."""
import pytest
import torch

from linear_recurrent_token_b200 import mlstm
from tests.test_gpu_rms_norm import TOP, norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("D,group", [(256, 0), (255, 0), (384, 128), (333, 128), (4096, 0)])
@pytest.mark.parametrize("power", [99.5, 100.5, 125.5, 126.5, 127.9])
def test_outputs_near_the_largest(dtype, quant, D, group, power):
    """Rows of +-1, whose norm is themselves, times weights up to 2^127.9.  Half a step of the format (e4m3: 2^-4 of
    the value, 2^-10 of its unit below 2^-6; int8: half the scale), and fp32's share as in every other test."""
    x = torch.where(torch.arange(D, device="cuda") % 3 == 0, -1.0, 1.0).to(dtype).repeat(3, 1)
    w = (torch.linspace(1e-3, 1.0, D, device="cuda").double() * 2.0 ** power).float()
    y, _, s = mlstm.rms_norm(x, weight=w, eps=0.0, quant=quant, group=group)
    ref = norm64(x, None, w, 0.0)[1]
    size = group or D
    for j in range(s.shape[-1]):
        part, got = ref[:, j * size:(j + 1) * size], y[:, j * size:(j + 1) * size].float().double()
        scale = part.abs().amax(-1, keepdim=True) / TOP[quant]
        assert bool(((s[:, j:j + 1].double() - scale).abs() <= 2.0 ** -19 * scale).all())
        want = part / scale
        step = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) if quant == "e4m3" else torch.full_like(want, 0.5)
        assert bool(((got - want).abs() <= step + 2.0 ** -18 * want.abs()).all())
        assert bool((got.abs().amax(-1) == TOP[quant]).all())
