"""GPU tests of the mixture-of-experts layer: the training function and its gradients against the layer
in float64 with the same choices, the serving path against the same, empty experts, dropped choices,
a captured decode step.

Tolerances: one product of two quantized operands has a relative error of 3.7e-2 (SQNR 28.6 dB, pinned in
the oracle's tests). silu(G) U adds the errors of its two factors (a gain of at most about 1.5 in the
norm) before the second product adds its own: sqrt(2 * (1.5 * 3.7e-2)^2 ... ) < 0.1 for the output; a
gradient passes at most one product more: 0.15. The gradient of a choice's weight is one dot product
<dy, e> of vectors that may be nearly orthogonal: its error is bounded by the error of e, 0.1 |dy| |e|,
and not by its own size. The choices and plans are exact."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from tests._gpu import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _case(seed, T, E, k, F, H, experts=None):
    """Tokens, weights, router weights and ids (distinct, of the experts named) on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, device=DEV, generator=g).to(BF)
    w1 = (0.05 * torch.randn(E, 2 * F, H, device=DEV, generator=g)).to(BF)
    w2 = (0.05 * torch.randn(E, H, F, device=DEV, generator=g)).to(BF)
    z = torch.randn(T, E, device=DEV, generator=g)
    if experts is not None:
        mask = torch.ones(E, dtype=torch.bool, device=DEV)
        mask[experts] = False
        z = z.masked_fill(mask, float("-inf"))
    weights, ids = bf.moe_route(z, k)
    return x, weights, ids, w1, w2


def _reference(x, weights, ids, w1, w2, sizes=None):
    """The layer in float64, differentiable; ids outside the experts contribute nothing. sizes [T, k], if
    given, receives the norms of the experts' rows."""
    E, F = w1.shape[0], w2.shape[2]
    y = torch.zeros_like(x)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gu = x[t] @ w1[e].t()
            h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
            out = h @ w2[e].t()
            if sizes is not None:
                sizes[t, j] = out.detach().norm(dim=1)
            y = y.index_add(0, t, weights[t, j][:, None] * out)
    return y


def _off(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T,E,k,F,H,experts", [(300, 8, 2, 256, 384, None), (65, 4, 3, 128, 128, None), (40, 16, 2, 128, 256, [1, 5, 6]), (1, 8, 2, 128, 256, None),
                                               (1500, 8, 2, 128, 128, None)])
def test_training_layer_and_gradients(T, E, k, F, H, experts):
    args = _case(T, T, E, k, F, H, experts)
    live = [a.clone().requires_grad_(a.dtype != torch.int32) for a in args]
    wide = [a.double().requires_grad_() if a.dtype != torch.int32 else a for a in args]
    dy = torch.randn(T, H, device=DEV).to(BF)
    sizes = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    y, want = bf.blockwise_fp8_moe(*live), _reference(*wide, sizes)
    assert _off(y, want) < 0.1
    y.backward(dy)
    want.backward(dy.double())
    assert torch.all((live[1].grad.double() - wide[1].grad).abs() <= 0.1 * dy.double().norm(dim=1, keepdim=True) * sizes)
    for i, name in ((0, "x"), (3, "w_gate_up"), (4, "w_down")):
        assert live[i].grad.shape == args[i].shape and live[i].grad.dtype == args[i].dtype
        assert _off(live[i].grad, wide[i].grad) < 0.15, name
    if experts is not None:                                # experts without a token: zero gradient, not garbage
        idle = [e for e in range(E) if e not in experts]
        assert torch.all(live[3].grad[idle] == 0) and torch.all(live[4].grad[idle] == 0)


def test_dropped_choices_contribute_nothing():
    x, weights, ids, w1, w2 = _case(3, 200, 8, 2, 128, 256)
    ids = ids.clone()
    ids[::3, 1], ids[5], ids[7, 0] = -1, 8, 1000
    live = [a.clone().requires_grad_() for a in (x, weights, w1, w2)]
    wide = [a.double().requires_grad_() for a in (x, weights, w1, w2)]
    y = bf.blockwise_fp8_moe(live[0], live[1], ids, live[2], live[3])
    sizes = torch.zeros(200, 2, dtype=torch.float64, device=DEV)
    want = _reference(wide[0], wide[1], ids, wide[2], wide[3], sizes)
    dy = torch.randn_like(y)
    y.backward(dy)
    want.backward(dy.double())
    assert _off(y, want) < 0.1 and torch.all(y[5] == 0)
    for i in (0, 2, 3):
        assert torch.isfinite(live[i].grad).all() and _off(live[i].grad, wide[i].grad) < 0.15
    assert torch.all((live[1].grad.double() - wide[1].grad).abs() <= 0.1 * dy.double().norm(dim=1, keepdim=True) * sizes)
    assert torch.all(live[1].grad[5] == 0)
    assert _off(bf.ServingMoE(w1, w2)(x, weights, ids), want.detach()) < 0.1


@pytest.mark.parametrize("T", [1, 7, 64, 500])
def test_serving_layer(T):
    x, weights, ids, w1, w2 = _case(T, T, 16, 4, 256, 512)
    y = bf.ServingMoE(w1, w2)(x, weights, ids)
    assert _off(y, _reference(*(a.double() if a.dtype != torch.int32 else a for a in (x, weights, ids, w1, w2)))) < 0.1


def test_module_trains_and_serves():
    """A few steps of the module on one batch bring its loss down; the serving form of the trained weights
    agrees with its forward pass (they differ in the rounding of the gate and up products: 5e-2)."""
    torch.manual_seed(0)
    m = bf.BlockwiseFp8MoE(256, 128, experts=8, k=2, score="sigmoid", balance_bias=True, device=DEV)
    x = torch.randn(4, 64, 256, device=DEV).to(BF)
    goal = torch.randn(4, 64, 256, device=DEV).to(BF) * 0.1
    opt = torch.optim.Adam(m.parameters(), lr=1e-2)
    losses = []
    for _ in range(12):
        opt.zero_grad()
        loss = ((m(x) - goal).float() ** 2).mean()
        loss.backward()
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in m.parameters())
        opt.step()
        losses.append(loss.item())
    assert losses[-1] < 0.9 * losses[0], losses
    with torch.no_grad():
        flat = x.reshape(-1, 256)
        y = bf.ServingMoE(m.w_gate_up, m.w_down)(flat, *m.route(flat))
        assert _off(y, m(x).reshape(-1, 256).double()) < 5e-2


def test_route_gradient_reaches_the_logits():
    z = torch.randn(50, 16, device=DEV, dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        a, b = z.float().requires_grad_(), z.clone().requires_grad_()
        weights, ids = bf.route_experts(a, 4, score=score, scale=2.5)
        p = torch.softmax(b, 1) if score == "softmax" else torch.sigmoid(b)
        q = p.gather(1, ids.long())
        c = torch.randn(50, 4, device=DEV)
        (weights * c).sum().backward()
        (2.5 * q / q.sum(1, keepdim=True) * c).sum().backward()
        assert _off(a.grad, b.grad) < 1e-5
        assert not ids.requires_grad


def test_serving_step_replays_from_a_graph():
    x, _, _, w1, w2 = _case(9, 32, 16, 4, 128, 256)
    layer, z = bf.ServingMoE(w1, w2), torch.randn(32, 16, device=DEV)

    def step():
        return layer(x, *bf.moe_route(z, 4))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        z.copy_(torch.randn(32, 16, device=DEV))
        x.copy_(torch.randn(32, 256, device=DEV))
        want = step().clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_training_step_replays_from_a_graph():
    """Forward and backward of route and experts in one graph, on leaves of its own; every replay, with eager
    work on other leaves between, equals that eager step bit for bit."""
    T, E, k, F, H = 70, 8, 2, 128, 256
    x, _, _, w1, w2 = _case(11, T, E, k, F, H)
    z, dy = torch.randn(T, E, device=DEV), torch.randn(T, H, device=DEV).to(BF)

    def step(leaves, dy):
        x, z, w1, w2 = leaves
        y = bf.blockwise_fp8_moe(x, *bf.route_experts(z, k, score="sigmoid", scale=2.5), w1, w2)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))

    leaves = [t.clone().requires_grad_() for t in (x, z, w1, w2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(leaves, dy)
    for _ in range(4):
        with torch.no_grad():
            leaves[0].copy_(torch.randn(T, H, device=DEV))
            leaves[1].copy_(torch.randn(T, E, device=DEV))
            leaves[2].mul_(0.9)
        dy.copy_(torch.randn(T, H, device=DEV))
        want = step([t.detach().clone().requires_grad_() for t in leaves], dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, name in zip(got, want, ("y", "dx", "dlogits", "dw_gate_up", "dw_down")):
            assert torch.equal(a, b), name


def test_layer_rejects_malformed_weights():
    x, weights, ids, w1, w2 = _case(1, 4, 4, 2, 128, 128)
    with pytest.raises(TypeError, match="bf16"):
        bf.ServingMoE(w1.float(), w2)
    with pytest.raises(ValueError, match="w_gate_up has shape"):
        bf.ServingMoE(w1[:, :128], w2)
    with pytest.raises(ValueError, match="multiples of 128"):
        bf.ServingMoE(w1[:, :128, :], w2[:, :, :64])
    with pytest.raises(ValueError, match="bf16 tokens"):
        bf.blockwise_fp8_moe(x.float(), weights, ids, w1, w2)


def test_no_tokens():
    """A batch without tokens (an idle rank): empty results, zero weight gradients."""
    _, _, _, w1, w2 = _case(1, 4, 4, 2, 128, 128)
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    weights, ids = bf.moe_route(torch.empty(0, 4, device=DEV), 2)
    assert weights.shape == (0, 2) and ids.shape == (0, 2)
    live = [a.clone().requires_grad_() for a in (x, weights, w1, w2)]
    y = bf.blockwise_fp8_moe(live[0], live[1], ids, live[2], live[3])
    assert y.shape == (0, 128)
    y.sum().backward()
    assert live[0].grad.shape == (0, 128) and torch.all(live[2].grad == 0) and torch.all(live[3].grad == 0)
    assert bf.ServingMoE(w1, w2)(x, weights, ids).shape == (0, 128)
    assert bf.moe_route_backward(torch.empty(0, 4, device=DEV), ids, weights).shape == (0, 4)
