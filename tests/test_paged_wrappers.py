"""Refusals of the paged and norm wrappers that need no GPU."""
import types

import pytest

torch = pytest.importorskip("torch")

import flash_attention_backward_gb300 as fb  # noqa: E402
from flash_attention_backward_gb300 import paged  # noqa: E402


def test_a_stream_of_another_device_is_refused():
    """Addresses of one device are not to be enqueued on another's stream."""
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)

    def enqueue(handle):
        raise AssertionError("enqueued")

    with pytest.raises(fb.FaBackError, match="cuda:1"):
        paged._call(enqueue, here, types.SimpleNamespace(device=there, cuda_stream=1))
