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


@pytest.mark.parametrize("shape", [(50,), (2, 5, 5)])
def test_layer_with_one_output_used(shape):
    """Gradients where only y, or only h, goes on; those of x and of the residual are two tensors."""
    H, F = 136, 72
    g = torch.Generator(device="cuda:0").manual_seed(1)
    x, r = (torch.randn(*shape, H, device="cuda:0", generator=g).to(torch.bfloat16).requires_grad_() for _ in range(2))
    layer = bf.BlockwiseFp8FeedForward(H, F, device="cuda:0")
    dy = torch.randn(*shape, H, device="cuda:0", generator=g).to(torch.bfloat16)
    y, h = layer(x, r)
    assert y.shape == x.shape and h.shape == x.shape
    torch.autograd.backward([y, h], [dy, torch.zeros_like(h)])
    both = [t.grad.clone() for t in (x, r, *layer.parameters())]
    assert x.grad.data_ptr() != r.grad.data_ptr()
    x.grad = r.grad = None
    layer.zero_grad()
    layer(x, r)[0].backward(dy)
    assert all(torch.equal(a, t.grad) for a, t in zip(both, (x, r, *layer.parameters())))
    x.grad = r.grad = None
    layer.zero_grad()
    layer(x, r)[1].backward(dy)
    assert torch.equal(x.grad, dy) and torch.equal(r.grad, dy) and all(p.grad is None for p in layer.parameters())
    assert len({t.data_ptr() for t in (x.grad, r.grad, dy)}) == 3
    y, h = layer(x, r)
    first, = torch.autograd.grad(y, x, dy.clone().requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.sum().backward()


def test_layers_without_tokens():
    H, F = 136, 72
    layer = bf.BlockwiseFp8FeedForward(H, F, device="cuda:0")
    x = torch.empty(0, H, dtype=torch.bfloat16, device="cuda:0", requires_grad=True)
    y, h = layer(x, torch.empty(0, H, device="cuda:0"))
    assert y.shape == (0, H) and h.shape == (0, H) and h.dtype == torch.float32
    (y.float().sum() + h.sum()).backward()
    assert x.grad.shape == (0, H) and all((p.grad == 0).all() for p in layer.parameters())
    serve = bf.ServingInt8FeedForward(layer.weight_norm, layer.w_gate_up, layer.w_down)
    y, h = serve(x.detach(), None)
    assert y.shape == (0, H) and h.shape == (0, H)


def test_clipping_one_parameter():
    p = torch.nn.Parameter(torch.ones(1001, device="cuda:0"))
    p.grad = torch.full_like(p, 2.0)
    norm = bf.clip_grad_norm_(p, 1.0, eps=0.0)
    assert abs(float(norm) - 2 * 1001 ** 0.5) < 1e-5
    # c = 1 / norm and the product are rounded once each
    assert (p.grad.double() * 1001 ** 0.5 - 1).abs().max() <= 2.0 ** -22


def test_captured_training_step():
    """Forward, backward, clipping and the update in one graph, replayed with eager work between; every replay is the eager
    step's bits. The warm-up's autograd graph is gone before the capture."""
    torch.manual_seed(3)
    T, H, F = 77, 256, 200
    layer, twin = (bf.BlockwiseFp8FeedForward(H, F, device="cuda:0") for _ in range(2))
    start = [p.detach().clone() for p in layer.parameters()]
    x, dy = (torch.randn(T, H, device="cuda:0").to(torch.bfloat16) for _ in range(2))
    r, dh = (torch.randn(T, H, device="cuda:0") for _ in range(2))

    def step(m):
        for p in m.parameters():
            p.grad = None
        torch.autograd.backward(list(m(x, r)), [dy, dh])
        norm = bf.clip_grad_norm_(m.parameters(), 0.5)
        with torch.no_grad():
            for p in m.parameters():
                p.sub_(p.grad)
        return norm

    def reset(m):
        with torch.no_grad():
            for p, s in zip(m.parameters(), start):
                p.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    reset(layer)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step(layer)
    reset(layer)
    reset(twin)
    for i in range(4):
        want = step(twin)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(norm).all() and torch.equal(norm, want), i
        assert all(torch.equal(a, b) for a, b in zip(layer.parameters(), twin.parameters())), i
