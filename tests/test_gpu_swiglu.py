"""SwiGLU with 8-bit codes, and its gradient, against 64-bit formulas.

The value in fp32 is within VALUE of the 64-bit one: two for the exponential (its argument's split, the
instruction) and half a step for its correction, one and a half for the reciprocal, and a product each with
the gate, the sigmoid's share and up -- at most ten half steps; the gradient has three products and sums more."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from _ffn_ref import HALF, U, Guarded, codes_hold, swiglu64, swiglu_grad64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
VALUE, GRAD = 10 * U, 16 * U
TOP = {"e4m3fn": 448.0, "e4m3fnuz": 240.0}
LEAST = {"e4m3fn": 2.0 ** -10, "e4m3fnuz": 2.0 ** -11}      # half the smallest step
FLOAT8 = {"e4m3fn": torch.float8_e4m3fn, "e4m3fnuz": torch.float8_e4m3fnuz}
BF16 = HALF[torch.bfloat16]


def make(T, F, seed=0, scale=2.0):
    return (scale * torch.randn(T, 2 * F, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def amax_groups(v):
    T, H = v.shape
    return torch.nn.functional.pad(v, (0, -H % 128)).view(T, -1, 128).abs().amax(2).clamp_min(1e-12)


def spread(s, H):
    """(groups, rows) scales over the elements [rows, H]."""
    return s.t().repeat_interleave(128, 1)[:, :H]


def check_groups(q, s, v, fmt, slack):
    """Codes [R, C] and scales (Cb, R) of the 64-bit values v."""
    want = (amax_groups(v) / TOP[fmt]).t()
    assert ((s.double() - want).abs() <= want * (slack + 2 * U)).all()
    # the multiplier top / amax is rounded once, the product once
    codes_hold(q.view(FLOAT8[fmt]).float(), s, v, lambda x: spread(x, v.shape[1]), TOP[fmt], 2.0 ** -4, LEAST[fmt], slack + 4 * U)


def check_value(y, v, slack, tiny=1e-38):
    assert ((y.double() - v).abs() <= v.abs() * (BF16 + slack) + tiny).all()


SIZES = [(1, 1), (3, 7), (2, 8), (5, 120), (1, 128), (3, 129), (2, 512), (9, 520), (4, 1000), (3, 1001), (2, 1032), (3, 2048), (2, 4104), (1, 5120),
         (2, 8192), (2, 14336), (1, 16384), (2, 16392), (300, 136)]


@pytest.mark.parametrize("T,F", SIZES)
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz", "int8", None])
def test_rows(T, F, fmt):
    check_rows(T, F, fmt)


@pytest.mark.parametrize("fmt", ["e4m3fn", "int8"])
@pytest.mark.parametrize("ld,shift", [(8, 0), (3, 0), (16, 1), (16, 8), (0, 3)])
def test_row_strides(ld, shift, fmt):
    check_rows(5, 1280, fmt, ld, shift)


def check_rows(T, F, fmt, ld=0, shift=0):
    gu = make(T, F)
    gg = Guarded(T, 2 * F, gu.dtype, DEV, 2 * F + ld, shift, gu)
    gq = None if fmt is None else Guarded(T, F, torch.int8 if fmt == "int8" else torch.uint8, DEV, F + ld, shift)
    gy = Guarded(T, F, torch.bfloat16, DEV, F + ld, shift)
    q, s, y = bf.swiglu_quantize(gg.view, fmt=fmt, q=None if gq is None else gq.view, y=gy.view)
    v = swiglu64(gu)
    check_value(gy.host(), v, VALUE)
    if fmt == "int8":
        want = v.abs().amax(1).clamp_min(1e-12) / 127
        assert ((s.cpu().double() - want).abs() <= want * (VALUE + 2 * U)).all()
        codes_hold(gq.host().float(), s.cpu(), v, lambda x: x[:, None].expand(T, F), 127.0, 0.0, 0.5, VALUE + 5 * U)
    elif fmt is not None:
        check_groups(gq.host(), s.cpu(), v, fmt, VALUE)


DUAL = [(1, 1), (16, 128), (5, 8), (130, 1280), (128, 136), (127, 1001), (256, 384), (300, 520), (48, 1032), (144, 2048)]


@pytest.mark.parametrize("T,F", DUAL)
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz"])
@pytest.mark.parametrize("ld,shift", [(0, 0), (16, 16), (5, 1)])
def test_both_groupings(T, F, fmt, ld, shift):
    gu = make(T, F, 1)
    gg = Guarded(T, 2 * F, gu.dtype, DEV, 2 * F + ld, shift, gu)
    gq, gt = Guarded(T, F, torch.uint8, DEV, F + ld, shift), Guarded(F, T, torch.uint8, DEV, T + ld, shift)
    _, a_s, _, s = bf.swiglu_quantize_lhs_and_rhs(gg.view, q=gq.view, qT=gt.view, fmt=fmt)
    v = swiglu64(gu)
    check_groups(gq.host(), a_s.cpu(), v, fmt, VALUE)
    check_groups(gt.host(), s.cpu(), v.t(), fmt, VALUE)
    # the row form's codes, bit for bit
    q1, s1, _ = bf.swiglu_quantize(gu.to(DEV), fmt=fmt)
    assert torch.equal(gq.host(), q1.cpu()) and torch.equal(a_s, s1)


@pytest.mark.parametrize("T,F", DUAL)
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz"])
@pytest.mark.parametrize("ld,shift", [(0, 0), (16, 16), (5, 1)])
def test_gradient_in_both_groupings(T, F, fmt, ld, shift):
    gu, dy = make(T, F, 2), make(T, F, 3)[:, :F].contiguous()
    gg, gd = Guarded(T, 2 * F, gu.dtype, DEV, 2 * F + ld, shift, gu), Guarded(T, F, dy.dtype, DEV, F + ld, shift, dy)
    gq, gt = Guarded(T, 2 * F, torch.uint8, DEV, 2 * F + ld, shift), Guarded(2 * F, T, torch.uint8, DEV, T + ld, shift)
    _, a_s, _, s = bf.swiglu_backward_quantize(gd.view, gg.view, q=gq.view, qT=gt.view, fmt=fmt)
    v = swiglu_grad64(dy, gu)
    # near gate = -1.278 the gate's factor 1 + g (1 - sig) passes zero: its rounding there is absolute
    v_abs = v.abs() + torch.cat([(dy.double() * gu[:, F:].double()).abs(), torch.zeros(T, F, dtype=torch.float64)], 1)
    check_near_groups(gq.host(), a_s.cpu(), v, v_abs, fmt)
    check_near_groups(gt.host(), s.cpu(), v.t(), v_abs.t(), fmt)


def check_near_groups(q, s, v, v_abs, fmt):
    """As check_groups, for values that are off by GRAD of v_abs."""
    want, room = amax_groups(v), amax_groups(v_abs) * GRAD
    assert ((s.double() * TOP[fmt] - want.t()).abs() <= (room + want * 2 * U).t()).all()
    sc = spread(s.double(), v.shape[1])
    p = v / sc
    off = (q.view(FLOAT8[fmt]).double() - p.clamp(-TOP[fmt], TOP[fmt])).abs()
    near = v_abs / sc * GRAD + p.abs() * (4 * U + spread((room / want).t(), v.shape[1]))
    assert (off <= torch.maximum(p.abs() * 2.0 ** -4, torch.full_like(p, LEAST[fmt])) + 2 * near + 1e-30).all()


@pytest.mark.parametrize("T,F", [(1, 1), (3, 7), (5, 8), (2, 512), (3, 520), (2, 1001), (9, 4096)])
@pytest.mark.parametrize("ld,shift", [(0, 0), (8, 8), (3, 1)])
def test_gradient(T, F, ld, shift):
    gu, dy = make(T, F, 4), make(T, F, 5)[:, :F].contiguous()
    gg, gd = Guarded(T, 2 * F, gu.dtype, DEV, 2 * F + ld, shift, gu), Guarded(T, F, dy.dtype, DEV, F + ld, shift, dy)
    go = Guarded(T, 2 * F, torch.bfloat16, DEV, 2 * F + ld, shift)
    bf.swiglu_backward(gd.view, gg.view, dgu=go.view)
    v = swiglu_grad64(dy, gu)
    near = torch.cat([(dy.double() * gu[:, F:].double()).abs(), torch.zeros(T, F, dtype=torch.float64)], 1)
    assert ((go.host().double() - v).abs() <= v.abs() * (BF16 + GRAD) + near * GRAD + 1e-38).all()


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(8)
    gu, dy = torch.randn(1, 16, generator=g).to(torch.bfloat16), torch.randn(1, 8, generator=g).to(torch.bfloat16)
    dgu = bf.swiglu_backward(dy.to(DEV), gu.to(DEV)).cpu().double()

    def value(t):
        return (dy.double() * torch.nn.functional.silu(t[:, :8]) * t[:, 8:]).sum()
    for j in range(16):
        e = torch.zeros(1, 16, dtype=torch.float64)
        e[0, j] = 1e-5
        diff = float((value(gu.double() + e) - value(gu.double() - e)) / 2e-5)
        assert abs(float(dgu[0, j]) - diff) <= abs(diff) * 1.01 * BF16 + 1e-6


GATES = [-0.0, 0.0, 1e-38, -1e-38, -1.0, -1.28, 5.0, -17.0, 17.0, 60.0, -79.5, -80.0, -80.5, -87.0, -88.0, -89.0, -95.0, -104.0, -130.0, -160.0, 88.0, 89.0, 104.0,
         300.0, -300.0, 1e4, -1e4, 1e30, -1e30, 3e38, -3e38]
UPS = [0.0, 1.0, -2.5, 1e-30, 1e10, 1e30, 3e38]


def test_far_gates():
    """Gates whose sigmoid leaves fp32's ordinary range, with ups that bring the product back."""
    g = torch.tensor(GATES).repeat_interleave(len(UPS)).to(torch.bfloat16)
    u = torch.tensor(UPS).repeat(len(GATES)).to(torch.bfloat16)
    gu = torch.cat([g, u])[None]
    _, _, y = bf.swiglu_quantize(gu.to(DEV), fmt=None)
    v = swiglu64(gu)
    y, fits = y.cpu().double(), v.abs() < 3.38e38
    assert ((y - v).abs() <= v.abs() * (BF16 + VALUE) + 2e-38)[fits].all()
    assert y[~fits].isinf().all()
    dy = torch.full((1, g.numel()), 0.75, dtype=torch.bfloat16)
    d, want = bf.swiglu_backward(dy.to(DEV), gu.to(DEV)).cpu().double(), swiglu_grad64(dy, gu)
    fits = want.abs() < 3.38e38
    near = torch.cat([(dy.double() * u.double() * torch.sigmoid(g.double())).abs(), torch.zeros(1, g.numel(), dtype=torch.float64)], 1)
    assert ((d - want).abs() <= want.abs() * (BF16 + GRAD) + near * GRAD + 2e-38)[fits].all()


@pytest.mark.parametrize("F", [1280, 1281])
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz", "int8"])
def test_values_that_are_not_finite(F, fmt):
    gu = make(5, F)
    clean = bf.swiglu_quantize(gu.to(DEV), fmt=fmt)
    gu[1, 3], gu[3, F + 130] = float("nan"), float("inf")
    q, s, _ = bf.swiglu_quantize(gu.to(DEV), fmt=fmt)
    s, was, ok = (t[None].cpu() if fmt == "int8" else t.cpu() for t in (s, clean[1], s))
    assert not s[0, 1].isfinite() and not s[1 % s.shape[0], 3].isfinite()
    rows = [0, 2, 4]
    assert torch.equal(q.cpu()[rows], clean[0].cpu()[rows]) and torch.equal(s[:, rows], was[:, rows])


def test_empty():
    gu = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    q, s, y = bf.swiglu_quantize(gu, want_y=True)
    assert q.shape == (0, 32) and s.shape == (1, 0) and y.shape == (0, 32)
    assert [t.shape for t in bf.swiglu_quantize_lhs_and_rhs(gu)] == [(0, 32), (1, 0), (32, 0), (0, 32)]
    assert bf.swiglu_backward(torch.empty(0, 32, dtype=torch.bfloat16, device=DEV), gu).shape == (0, 64)
