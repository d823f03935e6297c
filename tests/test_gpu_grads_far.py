"""Clipping by factors below fp32's ordinary range: the products need not be there. Tolerances as in test_gpu_grads.py."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from test_gpu_grads import DEV, TYPES, check_clip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("out", [None, "f32", "bf16"])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-30])
@pytest.mark.parametrize("shift", [0, 1])
def test_factor_below_fp32(kind, out, max_norm, shift):
    g = torch.Generator().manual_seed(4)
    flat = ((1.0 + torch.rand(90000 + shift, generator=g)) * 1.6e38).to(TYPES[kind]).to(DEV)
    grads = [flat[shift:70000 + shift], flat[70000 + shift:]]
    check_clip(grads, max_norm, None if out is None else [torch.empty(t.shape, dtype=TYPES[out], device=DEV) for t in grads])


def test_ordinary_beside_large():
    """One value makes the norm; the others are products below what fp32 holds, or in its last steps."""
    grads = [torch.tensor([3e38, 1e30, 1.0, 0.0, -1e-38, -2e35], device=DEV)]
    check_clip(grads, 1e-5)
