"""RMS norm with the residual's addition and 8-bit codes, and its gradient, against plain formulas.

Given the rstd that the kernel wrote, v = fl(fl(h rstd) weight) is the same in any IEEE arithmetic, so codes,
scales and bf16 rows are compared bit for bit; rstd itself with the 64-bit value. The gradient's tolerance
counts the roundings of its fp32 sums."""
import math

import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from _ffn_ref import HALF, U, Guarded, i8_codes, lhs_codes, normed, rhs_codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(T, H, residual, weight, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * (0.1 + 3 * torch.rand(T, 1, generator=g))).to(torch.bfloat16)
    r = None if residual == "none" else (2 * torch.randn(T, H, generator=g)).to(TYPES[residual])
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(TYPES[weight])
    return x, r, w


def rstd64(h, eps):
    return (h.double().square().mean(1) + torch.tensor(eps, dtype=torch.float32).double()).rsqrt()


def check_forward(T, H, residual, weight, fmt, ld=0, shift=0, eps=1e-6, data=None, alias=False):
    x, r, w = data or make(T, H, residual, weight)
    pad = lambda t: Guarded(T, H, t.dtype, DEV, H + ld, shift, t)  # noqa: E731
    gx, gr = pad(x), None if r is None else pad(r)
    kind = torch.int8 if fmt == "int8" else torch.uint8
    gq = None if fmt is None else Guarded(T, H, kind, DEV, H + ld, shift)
    gh = None if r is None else gr if alias else Guarded(T, H, r.dtype, DEV, H + ld, shift)
    gy = Guarded(T, H, torch.bfloat16, DEV, H + ld, shift)
    wd = torch.empty(H + shift, dtype=w.dtype, device=DEV)[shift:].copy_(w)
    q, s, h, y, rstd = bf.rms_norm_quantize(gx.view, wd, residual=None if gr is None else gr.view, eps=eps, fmt=fmt,
                                            q=None if gq is None else gq.view, h=None if gh is None else gh.view, y=gy.view, want_rstd=True)
    kept = x if r is None else (x.float() + r.float()).to(r.dtype)
    if r is not None:
        assert torch.equal(gh.host(), kept)
    else:
        assert h is None
    rs = rstd.cpu()
    want = rstd64(kept, eps)
    assert ((rs.double() - want).abs() <= want * 1.01 * U).all()       # one rounding of the 64-bit value
    v = normed(kept, rs, w)
    assert torch.equal(gy.host(), v.to(torch.bfloat16))
    if fmt is None:
        assert q is None and s is None
    elif fmt == "int8":
        wq, ws = i8_codes(v)
        assert torch.equal(gq.host(), wq) and torch.equal(s.cpu(), ws)
    else:
        wq, ws = lhs_codes(v, fmt)
        assert torch.equal(s.cpu(), ws)
        assert torch.equal(gq.host(), wq)


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 8), (5, 120), (1, 128), (3, 129), (2, 512), (9, 520), (4, 1000), (3, 1001), (6, 1024),
                                 (2, 1032), (3, 2048), (2, 2056), (1, 4096), (2, 5120), (2, 8192), (2, 12288), (1, 16384), (2, 16392), (1, 20001)])
@pytest.mark.parametrize("residual,weight,fmt", [("none", "bf16", "e4m3fn"), ("bf16", "f32", "int8"), ("f32", "bf16", "e4m3fnuz"), ("bf16", "bf16", None)])
def test_forward(T, H, residual, weight, fmt):
    check_forward(T, H, residual, weight, fmt)


@pytest.mark.parametrize("fmt", ["e4m3fn", "int8"])
@pytest.mark.parametrize("ld,shift", [(8, 0), (3, 0), (16, 1), (0, 3), (16, 8), (16, 4)])
@pytest.mark.parametrize("residual", ["none", "bf16", "f32"])
def test_strides_and_alignment(residual, ld, shift, fmt):
    check_forward(5, 1280, residual, "f32", fmt, ld=ld, shift=shift)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 31, 64, 65, 1000, 4099])
def test_row_counts(T):
    check_forward(T, 256, "bf16", "bf16", "e4m3fn")
    check_forward(T, 1288, "f32", "bf16", "int8")


@pytest.mark.parametrize("residual", ["bf16", "f32"])
@pytest.mark.parametrize("H", [640, 2048, 1001, 20000])
def test_residual_in_place(residual, H):
    check_forward(7, H, residual, "bf16", "e4m3fn", alias=True)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e17, 3e19, 1e37])
def test_far_magnitudes(scale):
    """Squares that leave fp32 (from 1.8e19 up, and below 1e-23), eps far below and far above them."""
    x, _, w = make(4, 1280, "none", "bf16")
    x = (x.float() * scale / 8).to(torch.bfloat16)
    for eps in (1e-6, 1e-37):
        check_forward(4, 1280, "none", "bf16", "e4m3fn", eps=eps, data=(x, None, w))
        check_forward(4, 1280, "none", "bf16", "int8", eps=eps, data=(x, None, w))


def test_zero_rows():
    x = torch.zeros(3, 1280, dtype=torch.bfloat16)
    _, _, w = make(3, 1280, "none", "bf16")
    for fmt in ("e4m3fn", "int8"):
        check_forward(3, 1280, "none", "bf16", fmt, data=(x, None, w))


@pytest.mark.parametrize("H", [1280, 1281])
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz", "int8"])
def test_rows_that_are_not_finite(H, fmt):
    """A NaN makes its whole row NaN, an infinity its group (the rest of the row is then 0): their scales are
    not finite. The other rows are what they are without them."""
    x, r, w = make(6, H, "bf16", "bf16")
    clean = bf.rms_norm_quantize(x.to(DEV), w.to(DEV), residual=r.to(DEV), fmt=fmt)
    x[1, 5], x[3, H - 1], r[4, 200] = math.nan, math.inf, -math.inf
    q, s, h, y, rstd = bf.rms_norm_quantize(x.to(DEV), w.to(DEV), residual=r.to(DEV), fmt=fmt, want_y=True)
    s, ok = (s[None] if fmt == "int8" else s).cpu(), [0, 2, 5]
    assert not s[:, 1].isfinite().any() and not s[-1, 3].isfinite() and not s[1 % s.shape[0], 4].isfinite()
    assert y.cpu()[1].isnan().all()
    assert torch.equal(q.cpu()[ok], clean[0].cpu()[ok])
    assert torch.equal(s[:, ok], (clean[1][None] if fmt == "int8" else clean[1]).cpu()[:, ok])


@pytest.mark.parametrize("T,H", [(1, 8), (16, 128), (130, 1280), (127, 1001), (128, 136), (300, 520), (5, 4096)])
@pytest.mark.parametrize("h_type,weight,fmt", [("bf16", "bf16", "e4m3fn"), ("f32", "f32", "e4m3fn"), ("bf16", "f32", "e4m3fnuz")])
@pytest.mark.parametrize("ld,shift", [(0, 0), (16, 16), (5, 1)])
def test_rhs(T, H, h_type, weight, fmt, ld, shift):
    _, _, w = make(T, H, "none", weight)
    h = (3 * torch.randn(T, H, generator=torch.Generator().manual_seed(3))).to(TYPES[h_type])
    rstd = rstd64(h, 1e-6).float()
    gh, gq = Guarded(T, H, h.dtype, DEV, H + ld, shift, h), Guarded(H, T, torch.uint8, DEV, T + ld, shift)
    qT, s = bf.rms_norm_quantize_rhs(gh.view, w.to(DEV), rstd.to(DEV), qT=gq.view, fmt=fmt)
    wq, ws = rhs_codes(normed(h, rstd, w), fmt)
    assert torch.equal(s.cpu(), ws) and torch.equal(gq.host(), wq)


def backward64(dy, h, w, rstd, dh):
    d, n, w = dy.double(), h.double() * rstd.double()[:, None], w.double()
    g = d * w
    dx = rstd.double()[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    return dx if dh is None else dx + dh.double(), (d * n).sum(0)


def check_backward(T, H, h_type, weight, with_dh, ld=0, shift=0, alias=False):
    g = torch.Generator().manual_seed(T * 31 + H)
    _, _, w = make(T, H, "none", weight)
    h = (3 * torch.randn(T, H, generator=g)).to(TYPES[h_type])
    dy = torch.randn(T, H, generator=g).to(torch.bfloat16)
    dh = torch.randn(T, H, generator=g).to(h.dtype) if with_dh else None
    rstd = rstd64(h, 1e-6).float()
    pad = lambda t: Guarded(T, H, t.dtype, DEV, H + ld, shift, t)  # noqa: E731
    ghd = None if dh is None else pad(dh)
    gdx = ghd if alias else Guarded(T, H, h.dtype, DEV, H + ld, shift)
    dx, dw = bf.rms_norm_backward(pad(dy).view, pad(h).view, w.to(DEV), rstd.to(DEV), dh=None if ghd is None else ghd.view, dx=gdx.view)
    want_dx, want_dw = backward64(dy, h, w, rstd, dh)
    d, n = dy.double(), h.double() * rstd.double()[:, None]
    gn = d * w.double() * n
    # sum of g n: three roundings a term, at most H / 256 + 24 additions one behind the other (a thread's
    # columns, the lanes, the waves); then the mean, two products, a difference, r, dh
    chain = H / 256 + 24 + 12
    r = rstd.double()[:, None]
    bound = U * (r * (6 * (d * w.double()).abs() + n.abs() * gn.abs().mean(1, keepdim=True) * chain) + 2 * want_dx.abs()
                 + (0 if dh is None else 2 * dh.double().abs())) + HALF[h.dtype] * want_dx.abs()
    assert ((gdx.host().double() - want_dx).abs() <= bound).all()
    # a term: two roundings; additions one behind the other: a workgroup's rows, a run's parts, the runs
    chain = math.ceil(T / 512) + 16 + 32 + 3
    assert dw.dtype == w.dtype
    assert ((dw.cpu().double() - want_dw).abs() <= U * chain * (d * n).abs().sum(0) + HALF[w.dtype] * want_dw.abs() + 1e-30).all()


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 8), (5, 128), (600, 136), (513, 1001), (2, 2048), (70, 2056), (1030, 4096), (3, 5120), (2, 8192),
                                 (2, 9000), (3, 16384), (2, 16392)])
@pytest.mark.parametrize("h_type,weight,with_dh", [("bf16", "bf16", False), ("bf16", "f32", True), ("f32", "bf16", True), ("f32", "f32", False)])
def test_backward(T, H, h_type, weight, with_dh):
    check_backward(T, H, h_type, weight, with_dh)


@pytest.mark.parametrize("h_type", ["bf16", "f32"])
@pytest.mark.parametrize("ld,shift", [(8, 0), (3, 0), (16, 1), (16, 8), (0, 5)])
def test_backward_strides(h_type, ld, shift):
    check_backward(37, 1280, h_type, "bf16", True, ld, shift)


@pytest.mark.parametrize("h_type,H", [("bf16", 1280), ("f32", 4096), ("bf16", 1001)])
def test_backward_into_dh(h_type, H):
    check_backward(9, H, h_type, "bf16", True, alias=True)


def test_backward_against_differences():
    """Central differences of sum(dy * v) in 64 bits."""
    g = torch.Generator().manual_seed(5)
    h, dy, w = torch.randn(2, 24, generator=g), torch.randn(2, 24, generator=g).to(torch.bfloat16), torch.randn(24, generator=g)

    def value(h64, w64):
        return (dy.double() * h64 * (h64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w64).sum()
    rstd = rstd64(h, 1e-6).float()
    dx, dw = bf.rms_norm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV))
    step = 1e-5
    for i in range(2):
        for j in range(0, 24, 5):
            e = torch.zeros(2, 24, dtype=torch.float64)
            e[i, j] = step
            diff = (value(h.double() + e, w.double()) - value(h.double() - e, w.double())) / (2 * step)
            assert abs(float(dx[i, j]) - float(diff)) < 1e-5
    e = torch.zeros(24, dtype=torch.float64)
    e[3] = step
    diff = (value(h.double(), w.double() + e) - value(h.double(), w.double() - e)) / (2 * step)
    assert abs(float(dw[3]) - float(diff)) < 1e-5


def test_backward_without_rows():
    w = torch.ones(40, dtype=torch.bfloat16, device=DEV)
    empty = torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    dweight = torch.full_like(w, 3)
    dx, dw = bf.rms_norm_backward(empty, empty, w, torch.empty(0, device=DEV), dweight=dweight)
    assert dx.shape == (0, 40) and (dw == 0).all()


def test_empty():
    w = torch.ones(40, device=DEV)
    q, s, h, y, rstd = bf.rms_norm_quantize(torch.empty(0, 40, dtype=torch.bfloat16, device=DEV), w, want_y=True)
    assert q.shape == (0, 40) and s.shape == (1, 0) and y.shape == (0, 40)


def test_same_result_on_every_call():
    x, r, w = (t.to(DEV) for t in make(700, 1288, "bf16", "f32"))
    dy = torch.randn(700, 1288, device=DEV).to(torch.bfloat16)
    q, s, h, _, rstd = bf.rms_norm_quantize(x, w, residual=r, want_rstd=True)
    dx, dw = bf.rms_norm_backward(dy, h, w, rstd)
    for _ in range(3):
        q2, s2, _, _, _ = bf.rms_norm_quantize(x, w, residual=r)
        dx2, dw2 = bf.rms_norm_backward(dy, h, w, rstd)
        assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


