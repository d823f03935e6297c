"""A serving layer is the layer as it was when the serving one was made."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from test_gpu_ffn import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float32])
def test_later_steps_of_the_trained_layer_do_not_reach_it(weight):
    x, r, wn, w1, w2 = _case(5, 256, 136)
    params = [torch.nn.Parameter(t) for t in (wn.to(weight), w1, w2)]
    serve = bf.ServingInt8FeedForward(*params)
    want = serve(x, r)
    with torch.no_grad():
        for p in params:
            p.mul_(1.5)
    assert all(torch.equal(a, b) for a, b in zip(serve(x, r), want))
