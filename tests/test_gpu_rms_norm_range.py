"""The root-mean-square norm at the ends of its range: outputs near fp32's largest, calls of several threads at
once."""
import ctypes
import threading

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


def test_threads_with_rows_of_other_widths():
    """Four threads whose calls run the same kernel with other amounts of shared memory (widths 511 and 301 without
    whole 16-byte accesses, with the weight's gradient and without): none is refused, results as alone."""
    L, refused, wrong = mlstm.lib(), [], []

    def work(D, want_dw):
        stream = torch.cuda.Stream()
        gen = torch.Generator(device="cuda").manual_seed(D)
        r, dy = (torch.randn(8, D, generator=gen, device="cuda") for _ in range(2))
        ref, ref_dw = mlstm.rms_norm_bwd(dy, r)
        dx, dw = torch.empty_like(r), torch.empty(D, device="cuda")
        p = mlstm.RmsParams(8, D, 0, 0, 0, 1e-6)
        need = L.mlstm_rms_norm_bwd_workspace_size(ctypes.byref(p))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        args = (ctypes.byref(p), dy.data_ptr(), r.data_ptr(), None, None, dx.data_ptr(), dw.data_ptr() if want_dw else None,
                ws.data_ptr(), need, stream.cuda_stream)
        for _ in range(20000):
            if L.mlstm_rms_norm_bwd(*args) != 0:
                refused.append((D, want_dw))
        stream.synchronize()
        if not torch.equal(dx, ref) or (want_dw and not torch.equal(dw, ref_dw)):
            wrong.append((D, want_dw))

    threads = [threading.Thread(target=work, args=a) for a in ((511, True), (301, False), (511, True), (301, True))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not refused and not wrong
