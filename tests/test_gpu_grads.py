"""Global gradient norm and clipping against sums in 64 bits. The norm is the 64-bit one rounded to fp32; its
sums differ in order alone, which 64 bits hide: within one step. The factor is rounded to fp32 from 64 bits
and each product once more, then to the output's type."""
import math

import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from _ffn_ref import HALF, U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(sizes, kinds, seed=0, scale=0.1):
    g = torch.Generator().manual_seed(seed)
    return [(scale * (1 + i % 4) * torch.randn(*(s if isinstance(s, tuple) else (s,)), generator=g)).to(TYPES[kinds[i % len(kinds)]]).to(DEV)
            for i, s in enumerate(sizes)]


def norm64(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def f32(v):
    return float(torch.tensor(v, dtype=torch.float64).float())


def factor64(grads, max_norm, eps):
    n = norm64(grads)       # max_norm and eps are taken as fp32
    return min(1.0, f32(max_norm) / (n + f32(eps))) if math.isfinite(n) else 1.0


def check_norm(norm, want):
    """The norm in fp32: infinite where the 64-bit one rounds to that; below 2^-126 fp32 has steps of 2^-149,
    and half of one is the rounding's."""
    got = float(norm)
    assert math.isinf(got) if math.isinf(f32(want)) else abs(got - want) <= want * 2 * U + 2.0 ** -150


def check_clip(grads, max_norm, outs=None, eps=1e-6):
    want_norm, c = norm64(grads), factor64(grads, max_norm, eps)
    want = [t.double() * c for t in grads]
    norm = bf.clip_grads(grads, max_norm, out=outs, eps=eps)
    assert norm.shape == (1,)
    check_norm(norm, want_norm)
    for got, w in zip(grads if outs is None else outs, want):
        # the factor, the product, and the output's type; below 2^-126 the product is rounded to steps of
        # 2^-149 (a half of one off) and bf16 has steps of 2^-133: half of one off, and fp32's rounding
        # before it can move that to the next by as much again as it was off
        tiny = 2.0 ** -150 if got.dtype == torch.float32 else 2.0 ** -134 + 2.0 ** -150
        assert ((got.double() - w).abs() <= w.abs() * (3 * U + HALF[got.dtype]) + tiny).all()


SIZES = [1, 7, 8, 100, 8191, 8192, 8193, (33, 257), (128, 512), 70001, 0, 5, (3, 0, 4)]


@pytest.mark.parametrize("kinds", [["bf16"], ["f32"], ["bf16", "f32", "f32"]])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e6])
def test_in_place(kinds, max_norm):
    check_clip(make(SIZES, kinds), max_norm)


@pytest.mark.parametrize("kinds,out", [(["bf16"], "f32"), (["f32"], "bf16"), (["bf16", "f32"], "bf16"), (["f32", "bf16"], "f32")])
@pytest.mark.parametrize("max_norm", [1.0, 1e6])
def test_into_others(kinds, out, max_norm):
    grads = make(SIZES, kinds)
    before = [t.clone() for t in grads]
    check_clip(grads, max_norm, [torch.full(t.shape, 9.0, dtype=TYPES[out], device=DEV) for t in grads])
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("n", [1, 95, 96, 97, 192, 300])
def test_many_tensors(n):
    grads = make([(37 * i) % 9001 for i in range(1, n + 1)], ["bf16", "f32"])
    assert abs(float(bf.grad_norm(grads)) - norm64(grads)) <= norm64(grads) * 2 * U
    check_clip(grads, 0.5)


def test_large_tensor():
    """More units than workgroups: each takes a run of them, across the tensors' borders."""
    grads = make([6_000_001, 3, 2_500_000], ["f32", "bf16"])
    check_clip(grads, 1.0, [torch.empty_like(t) for t in grads])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_views_of_odd_alignment(kind):
    """Gradients that begin anywhere in a buffer; what lies between them stays."""
    flat = torch.full((60000,), 5.0, dtype=TYPES[kind], device=DEV)
    at = [(1, 9000), (9003, 17), (9021, 8192), (20000, 30001)]
    grads = [flat[a:a + n] for a, n in at]
    for i, t in enumerate(grads):
        t.copy_(make([t.numel()], [kind], i)[0])
    gap = torch.ones(60000, dtype=torch.bool, device=DEV)
    for a, n in at:
        gap[a:a + n] = False
    check_clip(grads, 1.0)
    assert (flat[gap] == 5.0).all()


def test_transposed_and_permuted():
    a, b = make([(40, 56), (6, 10, 14)], ["bf16", "f32"])
    check_clip([a.t(), b.permute(2, 0, 1)], 0.5)


@pytest.mark.parametrize("scale", [1e-40, 1e-30, 1e20, 1e37])
def test_far_magnitudes(scale):
    """Squares outside fp32's range."""
    grads = [(torch.rand(5000, device=DEV) + 0.5) * scale, ((torch.rand(4000, device=DEV) + 0.5) * scale).to(torch.bfloat16)]
    want = norm64(grads)
    check_norm(bf.grad_norm(grads), want)
    check_clip(grads, want / 4, eps=0.0)


def test_norm_beyond_fp32_still_clips():
    grads = [torch.full((5000,), 3e38, device=DEV)]
    c = 1.0 / (norm64(grads) + 1e-6)
    norm = bf.clip_grads(grads, 1.0)
    assert math.isinf(float(norm))
    want = 3e38 * c
    assert abs(float(grads[0][17]) - want) <= want * 3e-7 + 2e-45 * 3e38


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("into", [False, True])
def test_norm_that_is_not_finite_leaves_the_gradients(bad, into):
    grads = make([5000, 300], ["bf16", "f32"])
    grads[1][7] = bad
    before = [t.clone() for t in grads]
    outs = [torch.zeros_like(t) for t in grads] if into else None
    norm = bf.clip_grads(grads, 1.0, out=outs)
    assert not math.isfinite(float(norm))
    for a, b in zip(outs or grads, before):
        assert torch.equal(torch.nan_to_num(a, 1.5), torch.nan_to_num(b, 1.5))


def test_nothing_and_zeros():
    norm = torch.full((1,), 5.0, device=DEV)
    assert bf.grad_norm([], norm=norm) is norm and float(norm) == 0
    norm.fill_(5.0)
    assert float(bf.clip_grads([], 1.0, norm=norm)) == 0
    empty = torch.empty(0, device=DEV)
    assert float(bf.clip_grads([empty], 1.0)) == 0
    zeros = [torch.zeros(100, device=DEV)]
    assert float(bf.clip_grads(zeros, 0.0, eps=0.0)) == 0 and (zeros[0] == 0).all()


def test_same_bits_on_every_call():
    grads = make([100003, 77, (512, 1001)], ["bf16", "f32"])
    first = bf.grad_norm(grads)
    need = bf.grad_workspace(grads)
    workspace = torch.empty(need, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(bf.grad_norm(grads, workspace=workspace), first)
    outs = [torch.empty_like(t) for t in grads]
    assert torch.equal(bf.clip_grads(grads, 1.0, out=outs, workspace=workspace), first)


def test_overlaps_are_refused():
    flat = torch.ones(1000, device=DEV)
    with pytest.raises(bf.Bsfp8Error, match="invalid"):
        bf.clip_grads([flat[:600], flat[500:]], 1.0)
    with pytest.raises(bf.Bsfp8Error, match="invalid"):
        bf.clip_grads([flat, flat], 1.0)
    with pytest.raises(bf.Bsfp8Error, match="invalid"):
        bf.clip_grads([flat[:500], flat[500:]], 1.0, out=[flat[500:], flat[:500]])
    with pytest.raises(bf.Bsfp8Error, match="invalid"):
        bf.clip_grads([flat[:500]], 1.0, out=[flat[1:501]])
    with pytest.raises(bf.Bsfp8Error, match="invalid"):
        bf.clip_grads([flat[:400], flat[400:800]], 1.0, out=[flat[:400], flat[401:801]])
    assert (flat == 1).all()
    assert float(bf.grad_norm([flat, flat])) == pytest.approx(math.sqrt(2000))
