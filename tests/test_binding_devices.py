"""Streams and devices in the binding of the gated delta rule and the norm, without a GPU: torch.cuda's switches are
replaced by ones that record."""
import contextlib
import types

import pytest
import torch

from linear_recurrent_token_b200 import mlstm

HERE, OTHER = torch.device("cuda", 0), torch.device("cuda", 1)


def test_a_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device=OTHER, cuda_stream=5)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        mlstm._on(HERE, stream, (), lambda cs: pytest.fail("launched"))


@pytest.mark.parametrize("given", [False, True])
def test_status_waits_on_the_workspace_s_device(monkeypatch, given):
    current, seen = [HERE], []

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()

    stream_of = lambda: types.SimpleNamespace(device=current[-1], cuda_stream=100 + current[-1].index)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", stream_of)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1].index, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    call = lambda p, ws, cs: seen.append((current[-1], ws, cs)) or 0
    monkeypatch.setattr(mlstm, "lib", lambda: types.SimpleNamespace(mlstm_gdr_status=call))
    ws = types.SimpleNamespace(device=OTHER, data_ptr=lambda: 4096)
    stream = types.SimpleNamespace(device=OTHER, cuda_stream=7) if given else None
    assert mlstm.gdr_status(mlstm.GdrParams(), ws, stream=stream) == 0
    assert seen == [(OTHER, 4096, 7 if given else 101)]
