"""Gated mixture-of-experts layer in blockwise FP8, composed from the C-ABI kernels.

Every token goes to the k experts its router chooses; expert e computes
W_down[e] (silu(G) * U) with G, U the halves of W_gate_up[e] x, and a token's experts are added with the
router's weights:

    route     weights, ids = moe_route(router logits)                 (choice, weights; gradient)
    plan      offsets, slots, rows = moe_plan(ids)                    (pairs sorted by expert)
    dispatch  tokens in expert order, quantized                       moe_dispatch
    products  gate and up, then down, per expert                      the grouped FP8 GEMMs
    return    weighted sum of a token's rows                          moe_combine

Training (``blockwise_fp8_moe``) runs the grouped GEMMs of the dense layer's recipe: activations in
1x128 groups, weights in 128x128 blocks, the weight gradients over 128x1 groups that restart at every
expert's first token. Serving (``ServingMoE``) keeps the quantized weights and runs the routed
products, which read the tokens through the plan and join the gate and up halves, so a decode step
moves the chosen experts' weights and little else. silu(G) * U of the training path is elementwise
torch code; every other step runs in the library's kernels. Training holds G and U in bf16, the grouped
GEMM's output, since the backward takes them; serving joins them in fp32 before the one rounding, so the
two forms of one layer differ by those roundings (at most 2^-8 of G and of U). All activations and weights are bf16 on
the GPU, H and F multiples of 128.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as _b


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, top_groups, renormalize, scale):
        weights, ids = _b.moe_route(logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                                    renormalize=renormalize, scale=scale)
        ctx.save_for_backward(logits, ids)
        ctx.rule = (score, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _):
        logits, ids = ctx.saved_tensors
        score, renormalize, scale = ctx.rule
        dlogits = _b.moe_route_backward(logits, ids, dweights.contiguous(), score=score, renormalize=renormalize, scale=scale)
        return dlogits, None, None, None, None, None, None, None


def route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """moe_route with a gradient: (weights [T, k] fp32, ids [T, k] int32) of logits [T, E]. The bias takes
    part in the choice only and has no gradient."""
    return _RouteFn.apply(logits, k, score, bias, groups, top_groups, renormalize, scale)


def _expert_weights(w_gate_up, w_down):
    """Checks W_gate_up [E, 2 F, H] and W_down [E, H, F]; returns (E, F, H)."""
    if w_gate_up.dtype != torch.bfloat16 or w_down.dtype != torch.bfloat16:
        raise TypeError("blockwise FP8 experts expect bf16 weights")
    if w_gate_up.dim() != 3 or w_down.dim() != 3:
        raise ValueError(f"expected w_gate_up [E, 2 F, H] and w_down [E, H, F], got {tuple(w_gate_up.shape)}, {tuple(w_down.shape)}")
    E, H, F = w_down.shape
    if tuple(w_gate_up.shape) != (E, 2 * F, H):
        raise ValueError(f"w_gate_up has shape {tuple(w_gate_up.shape)}, expected {(E, 2 * F, H)} for w_down {(E, H, F)}")
    if H % _b.BLOCK or F % _b.BLOCK or H == 0 or F == 0:
        raise ValueError(f"H = {H} and F = {F} must be positive multiples of {_b.BLOCK}")
    return E, F, H


def _tokens(x, H):
    if x.dim() != 2 or x.shape[1] != H or x.dtype != torch.bfloat16:
        raise ValueError(f"expected bf16 tokens [T, {H}], got {x.dtype} {tuple(x.shape)}")
    return x.contiguous()


def _forward(q, a_s, w, s, offsets, E):
    """Grouped product with the experts' weights stacked in w [E N, K], scales s [E N / 128, K / 128]."""
    N, K = w.shape[0] // E, w.shape[1]
    return _b.gemm_1x128_128x128_grouped(q, a_s, w, s, offsets, E, b_stride=N * K, bs_stride=s.numel() // E,
                                         bs_stride_nb=s.shape[1], bs_stride_kb=1, N=N)


def _dgrad(q, a_s, wT, s, offsets, E):
    """The same product with the transposed weights: wT [K, E N] holds expert e in columns N e on, and the
    scales are those of the weights, read transposed."""
    K, N = wT.shape[0], wT.shape[1] // E
    return _b.gemm_1x128_128x128_grouped(q, a_s, wT, s, offsets, E, b_stride=N, bs_stride=s.numel() // E, bs_stride_nb=1,
                                         bs_stride_kb=s.shape[1], ldb=E * N, N=K)


def _wgrad(dy, x, offsets, E):
    """dW[e] = dy_e^T x_e over each expert's rows."""
    qy, sy, padded = _b.quantize_rhs_grouped(dy, offsets, E)
    qx, sx, _ = _b.quantize_rhs_grouped(x, offsets, E)
    return _b.gemm_1x128_128x1_grouped(qy, sy, qx, sx, padded, E)


class _MoEFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weights, ids, w_gate_up, w_down):
        E, F, H = _expert_weights(w_gate_up, w_down)
        x, weights = _tokens(x, H), weights.contiguous()
        offsets, slots, _ = _b.moe_plan(ids, E)
        q, a_s, xr = _b.moe_dispatch(x, slots, want_copy=True)
        q1, q1T, s1 = _b.quantize_weight_128x128(w_gate_up.reshape(E * 2 * F, H))
        q2, q2T, s2 = _b.quantize_weight_128x128(w_down.reshape(E * H, F))
        gu = _forward(q, a_s, q1, s1, offsets, E)
        g, u = gu[:, :F].float(), gu[:, F:].float()
        h = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
        e = _forward(*_b.quantize_lhs(h), q2, s2, offsets, E)
        y = _b.moe_combine(e, slots, weights)
        ctx.save_for_backward(weights, offsets, slots, xr, gu, h, e, q1T, s1, q2T, s2)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weights, offsets, slots, xr, gu, h, e, q1T, s1, q2T, s2 = ctx.saved_tensors
        E, F = offsets.numel() - 1, h.shape[1]
        de, dweights = _b.moe_combine_backward(dy.to(torch.bfloat16).contiguous(), e, slots, weights)
        dh = _dgrad(*_b.quantize_lhs(de), q2T, s2, offsets, E).float()
        g, u = gu[:, :F].float(), gu[:, F:].float()
        sg = torch.sigmoid(g)
        dgu = torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], dim=1).to(torch.bfloat16)
        dx = dw1 = dw2 = None
        if ctx.needs_input_grad[0]:
            dx = _b.moe_combine(_dgrad(*_b.quantize_lhs(dgu), q1T, s1, offsets, E), slots)
        if ctx.needs_input_grad[3]:
            dw1 = _wgrad(dgu, xr, offsets, E)
        if ctx.needs_input_grad[4]:
            dw2 = _wgrad(de, h, offsets, E)
        return dx, dweights if ctx.needs_input_grad[1] else None, None, dw1, dw2


def blockwise_fp8_moe(x, weights, ids, w_gate_up, w_down):
    """The experts of a gated layer for training: x [T, H] bf16, weights [T, k] fp32 and ids [T, k] int32 as
    route_experts gives them (ids outside [0, E) contribute nothing), w_gate_up [E, 2 F, H] (gate rows,
    then up rows), w_down [E, H, F]. Returns y [T, H] bf16; gradients of x, weights and both weights."""
    return _MoEFn.apply(x, weights, ids, w_gate_up, w_down)


class BlockwiseFp8MoE(torch.nn.Module):
    """Router and gated experts with bf16 parameters; the experts' products run in blockwise FP8. ``bias``
    (a buffer, fp32) is added to the scores for the choice only, where ``balance_bias`` is set."""

    def __init__(self, features: int, hidden: int, experts: int, k: int, score: str = "softmax", groups: int = 1,
                 top_groups: int = 1, renormalize: bool = True, scale: float = 1.0, balance_bias: bool = False, device=None):
        super().__init__()
        self.k, self.rule = k, dict(score=score, groups=groups, top_groups=top_groups, renormalize=renormalize, scale=scale)

        def parameter(*shape):
            return torch.nn.Parameter(torch.empty(shape, dtype=torch.bfloat16, device=device).normal_(std=0.02))
        self.router = parameter(experts, features)
        self.w_gate_up = parameter(experts, 2 * hidden, features)
        self.w_down = parameter(experts, features, hidden)
        self.register_buffer("bias", torch.zeros(experts, dtype=torch.float32, device=device) if balance_bias else None)

    def route(self, x: torch.Tensor):
        # the product's sums are in fp32, its logits rounded to bf16, the parameters' type; a router whose
        # choice or gradient needs more bits gives fp32 logits of its own to route_experts
        logits = torch.nn.functional.linear(x, self.router)
        return route_experts(logits, self.k, bias=self.bias, **self.rule)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        flat = x.reshape(-1, x.shape[-1])
        weights, ids = self.route(flat)
        return blockwise_fp8_moe(flat, weights, ids, self.w_gate_up, self.w_down).reshape(x.shape)


class ServingMoE:
    """The layer for inference: the experts' weights quantized once, products for few rows an expert. Any
    number of tokens is computed; from about 256 rows an expert the grouped GEMM is as fast."""

    def __init__(self, w_gate_up: torch.Tensor, w_down: torch.Tensor):
        self.E, self.F, self.H = _expert_weights(w_gate_up, w_down)
        with torch.no_grad():
            self.q1, _, self.s1 = _b.quantize_weight_128x128(w_gate_up.reshape(-1, self.H), want_qT=False)
            self.q2, _, self.s2 = _b.quantize_weight_128x128(w_down.reshape(-1, self.F), want_qT=False)

    @torch.no_grad()
    def __call__(self, x: torch.Tensor, weights: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
        """y [T, H] for tokens x [T, H], weights and ids as moe_route gives them."""
        E, F, H = self.E, self.F, self.H
        offsets, slots, rows = _b.moe_plan(ids, E)
        q, a_s = _b.quantize_lhs(_tokens(x, H))
        h = _b.gemm_1x128_128x128_routed(q, a_s, self.q1, self.s1, offsets, E, b_stride=2 * F * H, bs_stride=self.s1.numel() // E,
                                         bs_stride_nb=self.s1.shape[1], bs_stride_kb=1, rows=rows, k=ids.shape[1], swiglu=True)
        e = _b.gemm_1x128_128x128_routed(*_b.quantize_lhs(h), self.q2, self.s2, offsets, E, b_stride=H * F,
                                         bs_stride=self.s2.numel() // E, bs_stride_nb=self.s2.shape[1], bs_stride_kb=1)
        return _b.moe_combine(e, slots, weights)
