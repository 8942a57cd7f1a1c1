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


def paged_cache():
    k = torch.zeros(4, 16, 2, 136, dtype=torch.uint8)
    return fb.PagedCache(k, fb.FA_Q8_0, k.clone(), fb.FA_Q8_0, torch.zeros(2, 2, dtype=torch.int32), D=128, Dv=128)


@pytest.mark.parametrize("name", ["k", "v", "page_table", "B", "D", "k_type", "c"])
def test_a_cache_keeps_what_it_was_made_with(name):
    """Another tensor in a cache's place would leave the kernels the address of the old one, which may be freed."""
    c = paged_cache()
    was = getattr(c, name)
    with pytest.raises(fb.FaBackError, match=name):
        setattr(c, name, was.clone() if isinstance(was, torch.Tensor) else was)
    assert getattr(c, name) is was
    c.page_table.fill_(1)  # in place
    assert c.decode_workspace_size.__self__ is c


def test_single_values_in_the_place_of_tokens_are_refused():
    c, one = paged_cache(), torch.zeros((), dtype=torch.int32)
    for call in (lambda: fb.cache_read(c, one, one), lambda: fb.cache_append(one.float(), one.float(), c, one, one),
                 lambda: fb.paged_decode(one.float(), c, one, scale=1.0), lambda: fb.qk_norm_rope(one.float(), None, None),
                 lambda: fb.qk_norm_rope_backward(one.float(), None, one.float(), None, None)):
        with pytest.raises(fb.FaBackError):
            call()
