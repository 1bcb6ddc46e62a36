"""Streams and devices in the binding of the gated delta rule and the norm, without a GPU."""
import types

import pytest
import torch

from linear_recurrent_token_b200 import mlstm

HERE, OTHER = torch.device("cuda", 0), torch.device("cuda", 1)


def test_a_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device=OTHER, cuda_stream=5)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        mlstm._on(HERE, stream, (), lambda cs: pytest.fail("launched"))
