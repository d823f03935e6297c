"""CPU checks of the mixture-of-experts binding around its calls: where outputs are allocated, and what the
package does without the parts that are not everywhere."""
import contextlib

import pytest
import torch

from blockwise_scaled_fp8_act_amd import binding


class _Like:
    """Stands for a GPU tensor; notes the stream that is current when memory is asked for."""
    is_cuda = True
    device = "cuda:0"

    def __init__(self, current):
        self.current = current

    def new_empty(self, shape, dtype):
        return self.current[-1], shape, dtype


@pytest.mark.parametrize("handle,want", [(0, "default"), (7, "external 7")])
def test_outputs_belong_to_the_stream_whose_handle_is_given(monkeypatch, handle, want):
    """The handle 0 names the default stream and no new one: the memory of a call's outputs is handed on in
    the order of the work that uses it."""
    current = ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def external(handle, device=None):
        return f"external {handle}" if handle else "a new stream"
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    assert binding._empty(_Like(current), (2, 3), torch.int32, handle) == (want, (2, 3), torch.int32)
    assert binding._empty(_Like(current), 5, torch.uint8, None) == ("current", 5, torch.uint8)
