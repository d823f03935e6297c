"""Gated feed-forward layer with its norm, in 8 bits, composed from the C-ABI kernels: with the residual stream
h = x + residual,

    n = rms_norm(h) * weight_norm;   G, U = the halves of W_gate_up n;   y = W_down (silu(G) * U)

and h goes on to the next layer beside y (which is its x, as h is its residual).

Training (``blockwise_fp8_feed_forward``) follows the dense layer's FP8 recipe: activations in 1x128 groups,
weights in 128x128 blocks, the weight gradients over 128x1 groups of tokens. Neither the normed rows nor the
activation nor the gradient of G and U is ever held in bf16: the norm and the activation write the codes that the
products take, and the norm's 128x1 codes are formed again from h in the backward pass.

    forward   codes of n            rms_norm_quantize            G, U     gemm_1x128_128x128
              codes of silu(G) U    swiglu_quantize_lhs_and_rhs  y        gemm_1x128_128x128
    backward  codes of dy           quantize_lhs_and_rhs         dW_down  gemm_1x128_128x1, d(silu(G) U) gemm_1x128_128x128
              codes of dG, dU       swiglu_backward_quantize     dn       gemm_1x128_128x128
              codes of n (128x1)    rms_norm_quantize_rhs        dW_gate_up  gemm_1x128_128x1
              dh, dweight_norm      rms_norm_backward

Operands of the backward pass alone (the weights' transposed codes, the activation's 128x1 codes) are written and kept for
the gradients that are asked for, and not at all without gradients (swiglu_quantize then forms the activation's codes).

Serving (``ServingInt8FeedForward``) keeps the weights in int8 with a scale an output channel; the norm and the
activation write int8 rows with a scale a token, and both products are gemm_i8.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as _b
from .linear import _codes


def _layer(weight_norm, w_gate_up, w_down):
    """Checks weight_norm [H], w_gate_up [2 F, H] and w_down [H, F]; returns (F, H)."""
    if w_gate_up.dtype != torch.bfloat16 or w_down.dtype != torch.bfloat16:
        raise TypeError("the feed-forward layer expects bf16 weights")
    if w_gate_up.dim() != 2 or w_down.dim() != 2:
        raise ValueError(f"expected w_gate_up [2 F, H] and w_down [H, F], got {tuple(w_gate_up.shape)}, {tuple(w_down.shape)}")
    H, F = w_down.shape
    if tuple(w_gate_up.shape) != (2 * F, H) or H == 0 or F == 0:
        raise ValueError(f"w_gate_up has shape {tuple(w_gate_up.shape)}, expected {(2 * F, H)} for w_down {(H, F)}")
    if tuple(weight_norm.shape) != (H,):
        raise ValueError(f"weight_norm has shape {tuple(weight_norm.shape)}, expected {(H,)}")
    return F, H


def _rows(name, t, H, dtypes):
    if t.dim() != 2 or t.shape[1] != H or t.dtype not in dtypes:
        raise ValueError(f"expected {name} [T, {H}] of {[str(d) for d in dtypes]}, got {t.dtype} {tuple(t.shape)}")
    return _dense(t, t.dtype, *t.shape)


def _dense(t, dtype, T, H):
    """t as [T, H] of the type, its strides too (a gradient may be expanded, which sizes of 0 and 1 hide)."""
    t = t.to(dtype).reshape(T, H)
    return t if t.stride() == (H, 1) else torch.empty((T, H), dtype=dtype, device=t.device).copy_(t)


def _weight(w, fmt, transposed):
    """Codes, transposed codes (None unless the gradient goes through them) and scales."""
    N, K = w.shape
    return _b.quantize_weight_128x128(w, q=_codes(N, K, w.device), qT=_codes(K, N, w.device) if transposed else None, want_qT=transposed, fmt=fmt)


def _reads(needs):
    """Of the gradients asked for (x, residual, weight_norm, w_gate_up, w_down): whether one goes back through w_gate_up,
    through w_down, and whether w_down's own is among them."""
    through_1 = any(needs[:3])
    return through_1, through_1 or needs[3], needs[4]


class _FeedForwardFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight_norm, w_gate_up, w_down, eps, fmt, live):
        F, H = _layer(weight_norm, w_gate_up, w_down)
        through_1, through_2, own_2 = _reads(ctx.needs_input_grad) if live else (False, False, False)
        given, ctx.shape = x, x.shape
        if residual is not None:
            if residual.shape != x.shape:
                raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
            residual = _rows("residual", residual.reshape(-1, residual.shape[-1]), H, (torch.bfloat16, torch.float32))
        x = _rows("x", x.reshape(-1, x.shape[-1]), H, (torch.bfloat16,))
        T, dev = x.shape[0], x.device
        w_gate_up, w_down, weight_norm = w_gate_up.contiguous(), w_down.contiguous(), weight_norm.contiguous()
        q, s, h, _, rstd = _b.rms_norm_quantize(x, weight_norm, residual=residual, eps=eps, fmt=fmt, q=_codes(T, H, dev), want_rstd=through_2)
        h = x if h is None else h
        q1, q1T, s1 = _weight(w_gate_up, fmt, through_1)
        q2, q2T, s2 = _weight(w_down, fmt, through_2)
        gu = _b.gemm_1x128_128x128(q, s, q1, s1, fmt=fmt)
        qaT = saT = None
        if own_2:
            qa, sa, qaT, saT = _b.swiglu_quantize_lhs_and_rhs(gu, q=_codes(T, F, dev), qT=_codes(F, T, dev), fmt=fmt)
        else:
            qa, sa, _ = _b.swiglu_quantize(gu, fmt, q=_codes(T, F, dev))
        y = _b.gemm_1x128_128x128(qa, sa, q2, s2, fmt=fmt)
        # what a gradient that was asked for reads, and no more
        ctx.save_for_backward(*((h, weight_norm, rstd, gu, q2T, s2) if through_2 else (None,) * 6), q1T, s1 if through_1 else None, qaT, saT)
        ctx.fmt, ctx.x_dtype, ctx.h_dtype, ctx.sizes = fmt, x.dtype, h.dtype, (T, H, F)
        ctx.set_materialize_grads(False)        # an output that nothing was made of has no gradient to read
        return y.view(ctx.shape), given.view_as(given) if residual is None else h.view(ctx.shape)

    @staticmethod
    def backward(ctx, dy, dh):
        # With create_graph the kernels' results must not pass for constants. Else x and the residual get one tensor as
        # their gradient, and autograd sees that it is one: a leaf copies it instead of keeping memory that another keeps.
        return _gradients_once(ctx, dy, dh) if torch.is_grad_enabled() else _gradients(ctx, dy, dh)


def _gradients(ctx, dy, dh):
    h, weight_norm, rstd, gu, q2T, s2, q1T, s1, qaT, saT = ctx.saved_tensors
    fmt, T, H, F = ctx.fmt, *ctx.sizes
    need_x, need_r, need_n, need_1, need_2 = ctx.needs_input_grad[:5]
    dx = dw1 = dw2 = dwn = None
    if dy is None:                              # h alone was used
        dx = None if dh is None else dh.to(ctx.h_dtype)
    else:
        dy, dev = _dense(dy, torch.bfloat16, T, H), dy.device
        qd, sd, qdT, sdT = _b.quantize_lhs_and_rhs(dy, q=_codes(T, H, dev), qT=_codes(H, T, dev), fmt=fmt)
        if need_2:
            dw2 = _b.gemm_1x128_128x1(qdT, sdT, qaT, saT, fmt=fmt)
        if need_x or need_r or need_n or need_1:
            da = _b.gemm_1x128_128x128(qd, sd, q2T, s2, 1, s2.shape[1], fmt=fmt)
            qg, sg, qgT, sgT = _b.swiglu_backward_quantize(da, gu, q=_codes(T, 2 * F, dev), qT=_codes(2 * F, T, dev), fmt=fmt)
            h = h.reshape(T, H)
            if need_1:
                qn, sn = _b.rms_norm_quantize_rhs(h, weight_norm, rstd, qT=_codes(H, T, dev), fmt=fmt)
                dw1 = _b.gemm_1x128_128x1(qgT, sgT, qn, sn, fmt=fmt)
            if need_x or need_r or need_n:
                dn = _b.gemm_1x128_128x128(qg, sg, q1T, s1, 1, s1.shape[1], fmt=fmt)
                dh = None if dh is None else _dense(dh, ctx.h_dtype, T, H)
                dx, dwn = _b.rms_norm_backward(dn, h, weight_norm, rstd, dh=dh)
                dx = dx.view(ctx.shape)
    gx = dx if dx is None or dx.dtype == ctx.x_dtype else dx.to(ctx.x_dtype)
    return gx if need_x else None, dx if need_r else None, dwn if need_n else None, dw1, dw2, None, None, None


_gradients_once = once_differentiable(_gradients)


def blockwise_fp8_feed_forward(x, weight_norm, w_gate_up, w_down, residual=None, eps=1e-6, fmt="e4m3fn"):
    """The layer for training: x [..., H] bf16, residual of x's shape, bf16 or fp32 (None: x is the residual stream),
    weight_norm [H] bf16 or fp32, w_gate_up [2 F, H] (gate rows, then up rows) and w_down [H, F] bf16. Returns
    (y bf16, h of the residual's type), both of x's shape; gradients of x, residual and all weights. ``fmt``: the FP8 element
    format ("e4m3fn", "e4m3fnuz" or the torch float8 dtype)."""
    return _FeedForwardFn.apply(x, residual, weight_norm, w_gate_up, w_down, eps, _b.fp8_format(fmt), torch.is_grad_enabled())


class BlockwiseFp8FeedForward(torch.nn.Module):
    """Norm and gated feed-forward layer with bf16 parameters whose products run in blockwise FP8."""

    def __init__(self, features: int, hidden: int, eps: float = 1e-6, device=None, fmt="e4m3fn"):
        super().__init__()
        self.eps, self.fmt = eps, _b.fp8_format(fmt)

        def parameter(*shape):
            return torch.nn.Parameter(torch.empty(shape, dtype=torch.bfloat16, device=device).normal_(std=0.02))
        self.weight_norm = torch.nn.Parameter(torch.ones(features, dtype=torch.bfloat16, device=device))
        self.w_gate_up = parameter(2 * hidden, features)
        self.w_down = parameter(features, hidden)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(y, h): y of x's shape, h = x + residual."""
        return blockwise_fp8_feed_forward(x, self.weight_norm, self.w_gate_up, self.w_down, residual=residual, eps=self.eps, fmt=self.fmt)


def _int8_rows(rows, cols, device):
    """An int8 buffer whose row stride is the products' 16 bytes."""
    return torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.int8, device=device)[:, :cols]


class ServingInt8FeedForward:
    """The layer for inference: weights quantized to int8 once, a scale an output channel, and the norm's weight copied with them;
    any number of tokens."""

    def __init__(self, weight_norm: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, eps: float = 1e-6):
        self.F, self.H = _layer(weight_norm, w_gate_up, w_down)
        self.eps, self.weight_norm = eps, weight_norm.detach().clone(memory_format=torch.contiguous_format)     # as the codes: of now
        with torch.no_grad():
            self.q1, self.s1 = _b.quantize_rows_i8(w_gate_up.contiguous(), q=_int8_rows(2 * self.F, self.H, w_gate_up.device))
            self.q2, self.s2 = _b.quantize_rows_i8(w_down.contiguous(), q=_int8_rows(self.H, self.F, w_down.device))

    @torch.no_grad()
    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(y [T, H], h [T, H]) for tokens x [T, H] and their residual stream."""
        x = _rows("x", x, self.H, (torch.bfloat16,))
        T, dev = x.shape[0], x.device
        q, s, h, _, _ = _b.rms_norm_quantize(x, self.weight_norm, residual=residual, eps=self.eps, fmt="int8", q=_int8_rows(T, self.H, dev))
        gu = _b.gemm_i8(q, s, self.q1, self.s1)
        qa, sa, _ = _b.swiglu_quantize(gu, "int8", q=_int8_rows(T, self.F, dev))
        return _b.gemm_i8(qa, sa, self.q2, self.s2), x if h is None else h


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """clip_grads of the parameters' gradients, in place; parameters without one are passed over. Returns the norm
    before the clipping, (1,) fp32 on the device, without waiting for it. Unlike torch.nn.utils.clip_grad_norm_: no gradient
    at all is an error, the norm has one dimension, and gradients that hold an infinity or a NaN are left as they are."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        raise ValueError("no parameter has a gradient")
    return _b.clip_grads(grads, float(max_norm), eps=eps)
