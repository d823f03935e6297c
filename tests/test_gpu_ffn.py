"""The gated feed-forward layer: the operators run together, training against the layer in float64 and serving in
int8, a captured training step and decode step, the same calls by the long way, other streams.

Tolerances: as for the mixture-of-experts layer, one product of two quantized operands is off by 3.7e-2 of its
norm (SQNR 28.6 dB); the activation passes on the errors of both its factors (a gain of at most 1.5) before the
second product adds its own: below 0.1 for y; a gradient passes one product more: 0.15. int8 rows of normal
values have steps of amax / 127, about 4.5 sigma / 127 = 0.035 sigma, off by 0.035 / sqrt(12) = 1.0e-2 a factor: 1.4e-2
a product, and by the same chain below 0.04."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from blockwise_scaled_fp8_act_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _case(T, H, F, residual="bf16", seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, device=DEV, generator=g).to(BF)
    r = None if residual is None else (2 * torch.randn(T, H, device=DEV, generator=g)).to(BF if residual == "bf16" else torch.float32)
    wn = (1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(BF)
    w1 = (torch.randn(2 * F, H, device=DEV, generator=g) * H ** -0.5).to(BF)
    w2 = (torch.randn(H, F, device=DEV, generator=g) * F ** -0.5).to(BF)
    return x, r, wn, w1, w2


def _reference(x, r, wn, w1, w2, eps=1e-6):
    h = x if r is None else x + r
    n = h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * wn
    gu = n @ w1.t()
    F = w2.shape[1]
    return (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ w2.t(), h


def _off(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T,H,F,residual,fmt", [(300, 256, 384, "bf16", "e4m3fn"), (128, 512, 256, "f32", "e4m3fn"), (65, 200, 136, None, "e4m3fn"),
                                                (1, 128, 256, "bf16", "e4m3fn"), (257, 384, 128, "f32", "e4m3fnuz"), (40, 130, 101, "bf16", "e4m3fn")])
def test_training_and_gradients(T, H, F, residual, fmt):
    args = _case(T, H, F, residual)
    live = [None if a is None else a.clone().requires_grad_() for a in args]
    wide = [None if a is None else a.double().requires_grad_() for a in args]
    y, h = bf.blockwise_fp8_feed_forward(live[0], *live[2:], residual=live[1], fmt=fmt)
    want_y, want_h = _reference(*wide)
    assert y.dtype == BF and h.dtype == (BF if args[1] is None else args[1].dtype)
    assert _off(y, want_y) < 0.1 and _off(h, want_h) < 2.0 ** -8
    dy, dh = torch.randn_like(y), torch.randn_like(h)
    torch.autograd.backward([y, h], [dy, dh])
    torch.autograd.backward([want_y, want_h], [dy.double(), dh.double()])
    for a, b, name in zip(live, wide, ("x", "residual", "weight_norm", "w_gate_up", "w_down")):
        if a is not None:
            assert a.grad.dtype == a.dtype and _off(a.grad, b.grad) < 0.15, name


def test_only_some_gradients():
    x, r, wn, w1, w2 = _case(64, 256, 128)
    full = [t.clone().requires_grad_() for t in (x, r, wn, w1, w2)]
    y, h = bf.blockwise_fp8_feed_forward(full[0], *full[2:], residual=full[1])
    dy = torch.randn_like(y)
    y.backward(dy)                  # nothing reaches h by another way
    for only in range(5):
        some = [t.clone().requires_grad_(i == only) for i, t in enumerate((x, r, wn, w1, w2))]
        bf.blockwise_fp8_feed_forward(some[0], *some[2:], residual=some[1])[0].backward(dy)
        for i, t in enumerate(some):
            assert (t.grad is None) == (i != only)
        assert torch.equal(some[only].grad, full[only].grad)


@pytest.mark.parametrize("T,H,F,residual", [(1, 256, 384, "bf16"), (7, 1000, 520, "f32"), (64, 512, 1024, "bf16"), (300, 136, 130, None)])
def test_serving_int8(T, H, F, residual):
    x, r, wn, w1, w2 = _case(T, H, F, residual)
    y, h = bf.ServingInt8FeedForward(wn, w1, w2)(x, r)
    want_y, want_h = _reference(*(None if a is None else a.double() for a in (x, r, wn, w1, w2)))
    assert _off(y, want_y) < 0.04 and _off(h, want_h) < 2.0 ** -8


def test_module_steps_with_clipped_gradients():
    """A training step runs: forward, backward, clipping of all gradients, an optimizer's step; two layers share
    the residual stream."""
    torch.manual_seed(0)
    layers = torch.nn.ModuleList([bf.BlockwiseFp8FeedForward(256, 384, device=DEV) for _ in range(2)])
    x = torch.randn(4, 50, 256, device=DEV).to(BF)
    opt = torch.optim.SGD(layers.parameters(), lr=0.1)
    for _ in range(2):
        opt.zero_grad()
        y, h = layers[0](x)
        y, h = layers[1](y, h)
        ((y + h).float() ** 2).mean().backward()
        grads = [p.grad for p in layers.parameters()]
        want = torch.stack([g.double().norm() for g in grads]).norm()
        before = [g.clone() for g in grads]
        norm = bf.clip_grad_norm_(layers.parameters(), float(want) / 2)
        assert abs(float(norm) - float(want)) <= float(want) * 2.0 ** -23
        for g, b in zip(grads, before):
            assert torch.isfinite(g).all() and ((g.double() - b.double() / 2).abs() <= b.double().abs() * 2.0 ** -8).all()
        opt.step()
    with pytest.raises(ValueError, match="no parameter"):
        opt.zero_grad()
        bf.clip_grad_norm_(layers.parameters(), 1.0)


def _capture(run):
    """Runs `run` on a side stream first (memory, kernels), then into a graph."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    return graph, out


def _all_operators(T, H, F):
    """Every operator once, as a training step and a decode step call them; their outputs."""
    x, r, wn, w1, w2 = _case(T, H, F, "f32")
    dy = torch.randn(T, F, device=DEV).to(BF)
    dn = torch.randn(T, H, device=DEV).to(BF)
    grads = [torch.randn(H, F, device=DEV).to(BF), torch.randn(H, device=DEV)]
    outs = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    b, bs = bf.quantize_rows_i8(w1, q=torch.empty(2 * F, (H + 15) // 16 * 16, dtype=torch.int8, device=DEV)[:, :H])

    def run():
        q, s, h, y, rstd = bf.rms_norm_quantize(x, wn, residual=r, want_y=True, want_rstd=True)
        qT, sT = bf.rms_norm_quantize_rhs(h, wn, rstd)
        dx, dwn = bf.rms_norm_backward(dn, h, wn, rstd, dh=h)
        i8 = torch.empty(T, (H + 15) // 16 * 16, dtype=torch.int8, device=DEV)[:, :H]
        _, i8_s, _, _, _ = bf.rms_norm_quantize(x, wn, residual=r, fmt="int8", q=i8)
        gu = bf.gemm_i8(i8, i8_s, b, bs)
        rows = bf.swiglu_quantize(gu, "int8", want_y=True)
        both = bf.swiglu_quantize_lhs_and_rhs(gu)
        back = bf.swiglu_backward_quantize(dy, gu)
        plain = bf.swiglu_backward(dy, gu)
        xq, xs = bf.quantize_rows_i8(x)
        norm = bf.clip_grads(grads, 1.0, out=outs)
        alone = bf.grad_norm(grads)
        return [q, s, h, y, rstd, qT, sT, dx, dwn, i8, i8_s, gu, *rows, *both, *back, plain, xq, xs, norm, alone, *outs]
    return run


@pytest.mark.parametrize("T,H,F", [(1, 1280, 640), (130, 1000, 520), (1000, 2048, 1408)])
def test_captured_and_replayed(T, H, F):
    run = _all_operators(T, H, F)
    want = [t.clone() for t in run()]
    graph, out = _capture(run)
    junk = torch.randn(1 << 22, device=DEV)
    for i in range(4):
        for t in out:
            t.view(torch.uint8).zero_() if t.dtype == torch.int8 else t.zero_()
        junk.mul_(1.0001)
        eager = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b, c) in enumerate(zip(out, want, eager)):
            assert torch.equal(a, b) and torch.equal(c, b), (i, k)


def test_two_graphs_one_workspace():
    """Two captured norm gradients and clippings that a program gives the same workspace, replayed in turn."""
    x, r, wn, _, _ = _case(700, 1280, 8)
    dy = torch.randn(700, 1280, device=DEV).to(BF)
    rstd = (r.double().square().mean(1) + 1e-6).rsqrt().float()
    ws = torch.empty(bf.rms_norm_backward_workspace(700, 1280), dtype=torch.uint8, device=DEV)
    grads = [torch.randn(100000, device=DEV), torch.randn(33333, device=DEV).to(BF)]
    runs = [lambda: bf.rms_norm_backward(dy, r, wn, rstd, workspace=ws), lambda: bf.rms_norm_backward(dy, x, wn, rstd, workspace=ws),
            lambda: (bf.grad_norm(grads, workspace=ws),), lambda: (bf.grad_norm(grads[:1], workspace=ws),)]
    want = [[t.clone() for t in f()] for f in runs]
    graphs = [_capture(f) for f in runs]
    for _ in range(3):
        for (graph, out), w in zip(graphs, want):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_the_long_way_gives_the_same(monkeypatch):
    """Without the binding's C part, and on a named stream, the same bits come back."""
    for sizes in ((1, 1280, 640), (130, 1000, 520)):
        run = _all_operators(*sizes)
        want = run()
        with monkeypatch.context() as m:
            m.setattr(binding, "_calls", None)
            got = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_named_streams():
    """Calls on a stream that is not the current one: their outputs are ordered there, and belong to it."""
    x, r, wn, w1, _ = _case(2000, 2048, 256)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    want = bf.rms_norm_quantize(x, wn, residual=r, fmt="int8", want_rstd=True)
    b, bs = bf.quantize_rows_i8(w1)
    wc = bf.gemm_i8(want[0], want[1], b, bs)
    wn_grads = bf.rms_norm_backward(x, want[2], wn, want[4])
    norm = bf.grad_norm([x, r])
    torch.cuda.synchronize()
    q, s, h, _, rstd = bf.rms_norm_quantize(x, wn, residual=r, fmt="int8", want_rstd=True, stream=other)
    c = bf.gemm_i8(q, s, b, bs, stream=other)
    rows = bf.swiglu_quantize(c, stream=other)
    grads = bf.rms_norm_backward(x, h, wn, rstd, stream=other.cuda_stream)
    n2 = bf.grad_norm([x, r], stream=other)
    other.synchronize()
    for a, w in zip((q, s, h, rstd, c, *grads, n2), (want[0], want[1], want[2], want[4], wc, *wn_grads, norm)):
        assert torch.equal(a, w)
    assert torch.equal(rows[0], bf.swiglu_quantize(wc)[0])


def test_offsets_past_4_gib():
    """Rows that lie past 2^32 bytes of a tensor: the last ones are what they are in a small tensor."""
    T, H = 300, 1280
    ld = 8_000_000                  # 300 rows of 16 MB: 4.8 GB
    big = torch.empty(T * ld, dtype=BF, device=DEV)
    view = big.as_strided((T, 2 * H), (ld, 1))
    gu = torch.randn(T, 2 * H, device=DEV).to(BF)
    view.copy_(gu)
    wn = torch.ones(H, dtype=BF, device=DEV)
    assert torch.equal(bf.swiglu_quantize(view)[0], bf.swiglu_quantize(gu)[0])
    for a, b in zip(bf.swiglu_quantize_lhs_and_rhs(view), bf.swiglu_quantize_lhs_and_rhs(gu)):
        assert torch.equal(a, b)
    half = view[:, :H]
    for fmt in ("e4m3fn", "int8"):
        for a, b in zip(bf.rms_norm_quantize(half, wn, fmt=fmt, want_rstd=True), bf.rms_norm_quantize(gu[:, :H].contiguous(), wn, fmt=fmt, want_rstd=True)):
            assert (a is None and b is None) or torch.equal(a, b)
    rstd = torch.rand(T, device=DEV)
    dx = big.as_strided((T, H), (ld, 1), 4 * H)
    dw = bf.rms_norm_backward(half, half, wn, rstd, dx=dx)[1]
    want = bf.rms_norm_backward(gu[:, :H], gu[:, :H], wn, rstd)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    c = big.as_strided((T, 640), (ld, 1), 8 * H)
    q, s = bf.quantize_rows_i8(half)
    b, bs = bf.quantize_rows_i8(torch.randn(640, H, device=DEV).to(BF))
    assert torch.equal(bf.gemm_i8(q, s, b, bs, c=c), bf.gemm_i8(q, s, b, bs))
    del big, view, half, dx, c
    many = torch.zeros(2 ** 31 + 100_001, dtype=BF, device=DEV)         # more than 2^31 values, 4.3 GB
    many[-3:] = 2.0
    many[5] = 1.0
    assert float(bf.grad_norm([many])) == 13 ** 0.5 or abs(float(bf.grad_norm([many])) - 13 ** 0.5) < 4e-7
    bf.clip_grads([many], 13 ** 0.5 / 2, eps=0.0)
    assert float(many[-1]) == 1.0 and float(many[5]) == 0.5
