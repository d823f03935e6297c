"""GPU tests of sigmoid routing where the scores leave fp32's ordinary range: logits from -80 on, whose scores
and their sums reach the smallest normal number (2^-126, the floor of a renormalized sum) and below.
References and bounds as in test_gpu_moe_ops.py: weights 32 * 2^-24 relative and one subnormal step; gradients
64 * 2^-24 of the magnitudes that enter an element, half a step of its type and one bf16 subnormal step."""
import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from tests import _moe_ref as ref
from tests._gpu import DEV

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
# experts and choices: 16 lanes a token, 64 lanes, a wave (more than 16 choices)
SHAPES = [(8, 1), (8, 8), (60, 6), (64, 16), (256, 8), (384, 8), (1000, 16), (64, 17), (300, 24)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _far_logits(seed, E, dtype):
    """Rows of logits around -81 to -104, equal ones, ones of both sides of each border, far ones beside
    ordinary ones, ordinary rows between, and rows past everything; on the device and as float64."""
    g = np.random.Generator(np.random.PCG64(seed))
    rows = []
    for at in (-80.0, -81.0, -85.0, -87.3, -88.5, -88.8, -89.0, -95.0, -100.0, -103.0, -104.0, -1e4):
        rows += [np.full(E, at), at + 0.25 * g.standard_normal(E), 1.5 * g.standard_normal(E)]
    mixed = 1.5 * g.standard_normal(E)
    mixed[1:] -= 90.0
    rows += [mixed, np.where(np.arange(E) % 2, -np.inf, -89.0), np.where(np.arange(E) == 0, -89.0, -np.inf)]
    z = torch.from_numpy(np.array(rows).astype(np.float32)).to(DEV).to(dtype)
    return z, _np(z)


@pytest.mark.parametrize("E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_sigmoid_weights_of_far_logits(E, k, dtype):
    z, zh = _far_logits(E + k, E, dtype)
    g = np.random.Generator(np.random.PCG64(k))
    for bias in (None, np.zeros(E, np.float32), (0.05 * g.standard_normal(E)).astype(np.float32)):
        for renorm in (True, False):
            for groups, top in ((1, 1), (4, 3)):
                if E % groups or k > top * (E // groups):
                    continue
                w, ids = bf.moe_route(z, k, score="sigmoid", bias=None if bias is None else torch.from_numpy(bias).to(DEV), groups=groups,
                                      top_groups=top, renormalize=renorm, scale=2.5)
                with np.errstate(over="ignore"):
                    want, want_ids = ref.route(zh, k, "sigmoid", bias, groups, top, renormalize=renorm, scale=2.5)
                assert np.array_equal(ids.cpu().numpy(), want_ids), (bias is None, renorm, groups)
                assert np.all(np.abs(_np(w) - want) <= 32 * E24 * np.abs(want) + 2.0 ** -149), (bias is None, renorm, groups)


def _check_gradient(z, zh, ids, dw, renorm, what):
    dz = bf.moe_route_backward(z, torch.from_numpy(ids).to(DEV), torch.from_numpy(dw).to(DEV), score="sigmoid", renormalize=renorm, scale=2.5)
    with np.errstate(over="ignore"):
        want, size = ref.route_backward(zh, ids, dw, "sigmoid", renorm, 2.5)
    half = 2.0 ** -8 if z.dtype == BF else E24
    assert np.all(np.abs(_np(dz) - want) <= 64 * E24 * size + half * np.abs(want) + 2.0 ** -133), what


def _gradients(seed, T, k):
    """Weights' gradients of ordinary size, of a loss scaled by 65536, and of 1e30."""
    g = np.random.Generator(np.random.PCG64(seed))
    dw = g.standard_normal((T, k))
    return [(s * dw).astype(np.float32) for s in (1.0, 65536.0, 1e30)] + [np.full((T, k), 2.0, np.float32)]


BACK = [(8, 1), (8, 8), (16, 4), (64, 16), (256, 8), (384, 8), (64, 17), (300, 24)]


@pytest.mark.parametrize("E,k", BACK)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_sigmoid_gradient_stays_finite_where_scores_are_small(E, k, dtype):
    """Scores that sum to 1e-37 (above the floor) or to nothing (below): the gradient is of the weights'
    gradient's size, however small the sum is that divides."""
    T = 12
    g = np.random.Generator(np.random.PCG64(E))
    zh = np.repeat(np.array([-70.0, -80.0, -85.0, -1e4, -3e38, -60.0])[:, None], 2, 0) + 0.5 * g.standard_normal((T, E))
    z = torch.from_numpy(zh.astype(np.float32)).to(DEV).to(dtype)
    ids = ref.choose(g, T, k, E, dropped=0.1)
    for i, dw in enumerate(_gradients(k, T, k)):
        for renorm in (True, False):
            _check_gradient(z, _np(z), ids, dw, renorm, (i, renorm))


@pytest.mark.parametrize("E,k", BACK)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_sigmoid_gradient_of_far_logits(E, k, dtype):
    z, zh = _far_logits(E + k, E, dtype)
    T = z.shape[0]
    ids = ref.choose(np.random.Generator(np.random.PCG64(E)), T, k, E, dropped=0.1)
    ids = np.where(np.isneginf(np.take_along_axis(zh, ids.clip(0, E - 1).astype(np.int64), 1)), -1, ids).astype(np.int32)
    for i, dw in enumerate(_gradients(k, T, k)):
        for renorm in (True, False):
            _check_gradient(z, zh, ids, dw, renorm, (i, renorm))
