"""SwiGLU's gradient where a partial product of dy, up and the gate's factor leaves fp32's ordinary range and the whole product
does not: through the bf16 form and both kernels of the form with both groupings, against 64 bits.

Errors as in test_gpu_swiglu.py (GRAD relative, near the gate's zero of dy u sig); below 2^-126 the fp32 result is off by at most
2^-150 and bf16's rounding by 2^-134 (half of its steps there): together below 2^-133."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from _ffn_ref import swiglu_grad64
from test_gpu_swiglu import BF16, DEV, GRAD, check_near_groups

pytestmark = pytest.mark.gpu
GATES = [-79.5, -79.0, -60.0, -30.0, -17.0, -5.0, -2.4, -1.28, -1.0, -1e-38, 0.0, 1e-38, 1.0, 2.4, 5.0, 30.0, 80.0, 80.5, 90.0, -80.0, -80.5, -90.0]
FACTORS = [0.0, 1e-38, 1e-30, -1e-11, 0.01, 1.0, -2.5, 1e11, 1e30, -1.6e38, 1.75e38, 3.2e38, -3.38e38]


def test_every_pair_of_factors():
    g, u, d = (t.reshape(-1) for t in torch.meshgrid(torch.tensor(GATES), torch.tensor(FACTORS), torch.tensor(FACTORS), indexing="ij"))
    gu, dy = torch.cat([g, u])[None].to(torch.bfloat16), d[None].to(torch.bfloat16)
    got, want = bf.swiglu_backward(dy.to(DEV), gu.to(DEV)).cpu().double(), swiglu_grad64(dy, gu)
    F = dy.shape[1]
    near = (dy.double() * gu[:, F:].double()).abs() * torch.sigmoid(gu[:, :F].double())
    near = torch.cat([near, torch.zeros_like(near)], 1)
    bound = want.abs() * (BF16 + GRAD) + near * GRAD + 2.0 ** -133
    fits = want.abs() < 3.38e38
    off = (got - want).abs() > bound
    assert not (off & fits).any(), [(float(gu[0, j % F]), float(gu[0, F + j % F]), float(dy[0, j % F]), float(got[0, j]), float(want[0, j]))
                                    for j in (off & fits)[0].nonzero().flatten().tolist()[:8]]
    over = want.abs() > 3.42e38
    assert got[over].isinf().all() and (got[over].sign() == want[over].sign()).all()


@pytest.mark.parametrize("F", [128, 384, 136, 101])
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz"])
def test_both_groupings(F, fmt):
    """A row for each pair of factors (no gradient of them leaves fp32), gates and signs in turn along it."""
    pairs = [(3.2e38, 0.01), (0.01, 3e36), (1e-11, 1e30), (1e30, 1e-11), (1e-30, 3e36), (3e36, 1e-30), (3.38e38, 0.5), (2e38, 1e-38), (1.0, 1.0)]
    gates = torch.tensor(GATES)[torch.arange(F) % len(GATES)]
    sign = 1.0 - 2.0 * (torch.arange(F) % 3 == 0)
    gu = torch.stack([torch.cat([gates, u * sign]) for u, _ in pairs]).to(torch.bfloat16)
    dy = torch.stack([d * sign.flip(0) for _, d in pairs]).to(torch.bfloat16)
    q, a_s, qT, s = (t.cpu() for t in bf.swiglu_backward_quantize(dy.to(DEV), gu.to(DEV), fmt=fmt))
    v = swiglu_grad64(dy, gu)
    assert v.abs().max() < 3.4e38
    near = (dy.double() * gu[:, F:].double()).abs() * torch.sigmoid(gu[:, :F].double())
    v_abs = v.abs() + torch.cat([near, torch.zeros_like(near)], 1)
    check_near_groups(q, a_s, v, v_abs, fmt)
    check_near_groups(qT, s, v.t(), v_abs.t(), fmt)


def test_ordinary_values_beside_far_ones():
    """The eight columns that share the test for far values keep their own bits."""
    g = torch.Generator().manual_seed(3)
    gu, dy = torch.randn(4, 512, generator=g).to(torch.bfloat16), torch.randn(4, 256, generator=g).to(torch.bfloat16)
    clean = bf.swiglu_backward(dy.to(DEV), gu.to(DEV)).cpu()
    gu[0, ::8], gu[1, 256::8], dy[2, ::8] = -90.0, 3.2e38, 3.2e38
    got = bf.swiglu_backward(dy.to(DEV), gu.to(DEV)).cpu()
    rest = torch.arange(512) % 8 != 0
    assert torch.equal(got[:, rest], clean[:, rest])
