"""Rows of odd lengths and alignments through every form of the norm, the gated activation and the int8 row quantizer: pieces
at any address, pieces cut off by a row's end, 128x1 groups cut off by the last token, the gradient's eight columns that lie
in both halves, several rows for each wave and workgroup of the norm's gradient. Inputs and outputs lie between guard
bytes; values and tolerances are those of the modules whose checks these are."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
import test_gpu_i8 as i8
import test_gpu_norm as norm
import test_gpu_swiglu as swiglu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(9, 9), (5, 511), (6, 1023), (3, 1025), (2, 2047), (3, 4097), (2, 6143), (2, 8191), (2, 12289), (1, 16383), (1, 16385)])
@pytest.mark.parametrize("residual,weight,fmt", [("none", "f32", "int8"), ("bf16", "bf16", "e4m3fn"), ("f32", "f32", "e4m3fnuz"), ("f32", "bf16", None)])
@pytest.mark.parametrize("ld,shift", [(0, 0), (7, 3)])
def test_norm(T, H, residual, weight, fmt, ld, shift):
    norm.check_forward(T, H, residual, weight, fmt, ld=ld, shift=shift)


@pytest.mark.parametrize("residual", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1001, 4097])
def test_norm_in_place(residual, H):
    norm.check_forward(7, H, residual, "bf16", "e4m3fn", ld=3, alias=True)


@pytest.mark.parametrize("T,H", [(127, 256), (129, 128), (255, 131), (17, 384), (2, 1000), (143, 9)])
@pytest.mark.parametrize("h_type,weight,fmt", [("bf16", "f32", "e4m3fn"), ("f32", "bf16", "e4m3fnuz")])
def test_norm_rhs(T, H, h_type, weight, fmt):
    for ld, shift in ((0, 0), (1, 7)):
        norm.test_rhs(T, H, h_type, weight, fmt, ld, shift)


@pytest.mark.parametrize("T,H", [(6200, 40), (4100, 600), (4099, 1001), (2000, 1100), (1031, 2047), (1100, 2600), (700, 4097), (5, 6143), (3, 8191),
                                 (3, 16383)])
@pytest.mark.parametrize("h_type,weight,with_dh", [("bf16", "f32", True), ("f32", "bf16", False), ("f32", "f32", True)])
def test_norm_backward(T, H, h_type, weight, with_dh):
    norm.check_backward(T, H, h_type, weight, with_dh)


@pytest.mark.parametrize("h_type,H", [("bf16", 600), ("f32", 600), ("bf16", 1001), ("f32", 2048)])
def test_norm_backward_into_dh(h_type, H):
    """In place over many rows, whose successors are read ahead."""
    norm.check_backward(4500, H, h_type, "bf16", True, ld=8, alias=True)


@pytest.mark.parametrize("T,F", [(9, 9), (5, 511), (6, 1023), (2, 2047), (3, 4097), (2, 6143), (2, 12289), (1, 16383), (1, 16385)])
@pytest.mark.parametrize("fmt", ["e4m3fn", "int8", None])
def test_swiglu_rows(T, F, fmt):
    swiglu.check_rows(T, F, fmt)
    swiglu.check_rows(T, F, fmt, ld=5, shift=1)


TILES = [(1, 3), (2, 5), (17, 9), (127, 256), (129, 128), (255, 131), (143, 127), (15, 260), (131, 252), (1, 1000)]


@pytest.mark.parametrize("T,F", TILES)
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz"])
@pytest.mark.parametrize("ld,shift", [(0, 0), (1, 7)])
def test_swiglu_both_groupings(T, F, fmt, ld, shift):
    swiglu.test_both_groupings(T, F, fmt, ld, shift)
    swiglu.test_gradient_in_both_groupings(T, F, fmt, ld, shift)


@pytest.mark.parametrize("T,F", [(9, 9), (5, 511), (3, 513), (2, 4097)])
@pytest.mark.parametrize("ld,shift", [(0, 0), (5, 1)])
def test_swiglu_gradient(T, F, ld, shift):
    swiglu.test_gradient(T, F, ld, shift)


@pytest.mark.parametrize("M,K", [(9, 9), (5, 511), (6, 1023), (3, 4097), (2, 6143), (2, 12289), (1, 16383), (1, 16385)])
def test_int8_rows(M, K):
    i8.test_rows(M, K, 0, 0)
    i8.test_rows(M, K, 3, 1)


def test_halves_of_the_gradient_meet_in_a_group():
    """The gradient in both groupings of a width whose halves meet inside a group, and inside eight columns, holds the values
    of the plain gradient: the codes times their scales are those within half a step."""
    T, F = 140, 131
    g = torch.Generator(device="cuda:0").manual_seed(5)
    gu = torch.randn(T, 2 * F, device="cuda:0", generator=g).to(torch.bfloat16)
    dy = torch.randn(T, F, device="cuda:0", generator=g).to(torch.bfloat16)
    q, a_s, qT, s = bf.swiglu_backward_quantize(dy, gu)
    plain = bf.swiglu_backward(dy, gu).double()
    rows = q.view(torch.float8_e4m3fn).double() * a_s.t().double().repeat_interleave(128, 1)[:, :2 * F]
    cols = qT.view(torch.float8_e4m3fn).double().t() * s.double().repeat_interleave(128, 0)[:T]
    least = 2.0 ** -10      # of a scale: half of the smallest code
    # a code is off by half a step, 2^-4, plus what the bf16 value it is compared with is off, 2^-8
    for got, scale in ((rows, a_s.t().double().repeat_interleave(128, 1)[:, :2 * F]), (cols, s.double().repeat_interleave(128, 0)[:T])):
        assert ((got - plain).abs() <= plain.abs() * (2.0 ** -4 + 2.0 ** -7) + scale * least * 1.01).all()
