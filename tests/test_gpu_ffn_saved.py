"""The feed-forward layer keeps for the backward pass, and writes for it, what a gradient that was asked for reads; outputs and
gradients are the same bits whatever is asked."""
import itertools

import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from blockwise_scaled_fp8_act_amd import ffn
from test_gpu_ffn import _case

pytestmark = pytest.mark.gpu
T, H, F = 48, 256, 136


def run(live, fmt="e4m3fn"):
    x, r, wn, w1, w2 = live
    return bf.blockwise_fp8_feed_forward(x, wn, w1, w2, residual=r, fmt=fmt)


@pytest.fixture
def asked(monkeypatch):
    """The code buffers [rows, columns] that the layer asks for."""
    shapes, make = [], ffn._codes

    def codes(rows, cols, device):
        shapes.append((rows, cols))
        return make(rows, cols, device)
    monkeypatch.setattr(ffn, "_codes", codes)
    return shapes


TRANSPOSED = {(H, 2 * F), (F, H), (F, T)}       # codes of w_gate_up, of w_down and of the activation, for gradients alone


@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3fn", "e4m3fnuz"])
def test_without_gradients(residual, fmt, asked):
    args = _case(T, H, F, residual)
    live = [None if a is None else a.clone().requires_grad_() for a in args]
    want = run(live, fmt)
    assert TRANSPOSED <= set(asked)
    for mode in (torch.no_grad, torch.inference_mode):
        del asked[:]
        with mode():
            got = run(live, fmt)
        assert not TRANSPOSED & set(asked) and not got[0].requires_grad
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del asked[:]
    got = run(args, fmt)
    assert not TRANSPOSED & set(asked) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_every_choice_of_gradients(asked):
    args = _case(T, H, F, "f32")
    dy, dh = torch.randn(T, H, device="cuda:0").to(torch.bfloat16), torch.randn(T, H, device="cuda:0")
    full = [a.clone().requires_grad_() for a in args]
    torch.autograd.backward(list(run(full)), [dy, dh])
    for need in itertools.product([False, True], repeat=5):
        if not any(need):
            continue
        some = [a.clone().requires_grad_(n) for a, n in zip(args, need)]
        del asked[:]
        y, h = run(some)
        x, r, wn, w1, w2 = need
        want = {(H, 2 * F)} if x or r or wn else set()
        want |= ({(F, H)} if x or r or wn or w1 else set()) | ({(F, T)} if w2 else set())
        assert TRANSPOSED & set(asked) == want, need
        torch.autograd.backward([y, h], [dy, dh]) if h.requires_grad else y.backward(dy)
        for a, b, n in zip(some, full, need):
            assert torch.equal(a.grad, b.grad) if n else a.grad is None, need


def test_frozen_weights_hold_no_memory():
    """With w_down frozen the activation's transposed codes are not there, with gradients of w_down alone nothing but them is."""
    T, H, F = 4096, 1024, 4096
    args = _case(T, H, F, "bf16")

    def held(need):
        some = [a.clone().requires_grad_(n) for a, n in zip(args, need)]
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = run(some)
        return torch.cuda.memory_allocated() - before - sum(t.numel() * t.element_size() for t in out)
    everything, frozen, alone = held([True] * 5), held([True] * 4 + [False]), held([False] * 4 + [True])
    assert everything - frozen >= T * F and alone < 2 * T * F < frozen
