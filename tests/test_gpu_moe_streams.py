"""GPU tests of the mixture-of-experts calls' memory and streams: outputs belong to the stream that the call
names."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from tests._gpu import DEV

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _owner(t):
    """The stream whose pool holds a tensor's memory."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.parametrize("how", ["default handle", "default stream", "handle", "stream", "current"])
def test_outputs_belong_to_the_call_s_stream(how):
    ids = torch.randint(0, 8, (2000, 8), dtype=I32, device=DEV)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = {"default handle": 0, "default stream": torch.cuda.default_stream(), "handle": other.cuda_stream, "stream": other, "current": None}[how]
    want = other.cuda_stream if how in ("handle", "stream") else 0
    for t in bf.moe_plan(ids, 8, stream=stream):
        assert _owner(t) == want
    torch.cuda.synchronize()
