"""Refusals of the operators between the 8-bit products, the int8 product and the gradient norm: the C entry
points before any HIP call, the binding's checks before the library. No GPU is touched."""
import ctypes
import math

import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from blockwise_scaled_fp8_act_amd import binding

P = ctypes.c_void_p(16 * 1024)      # 16-byte aligned, never dereferenced on these paths
ODD = ctypes.c_void_p(16 * 1024 + 2)
INVALID, ALIGN = 1, 2


@pytest.fixture(scope="module")
def L():
    return binding.lib()


def test_norm_entry(L):
    #                  x  T  H    ldx  res rt ldr w  wt eps   h  ldh  rstd codes q ldq s y    ldy stream
    def call(**over):
        a = dict(x=P, T=4, H=256, ldx=256, res=P, rt=0, ldr=256, w=P, wt=0, eps=1e-6, h=P, ldh=256, rstd=P, codes=1, q=P, ldq=256, s=P, y=None,
                 ldy=0, stream=None)
        assert not set(over) - set(a)
        a.update(over)
        return L.rms_norm_quantize(*a.values())
    for bad in (dict(T=-1), dict(H=-1), dict(T=2 ** 24), dict(H=2 ** 31), dict(ldx=255), dict(ldr=255), dict(ldh=255), dict(ldq=255), dict(x=None),
                dict(w=None), dict(h=None), dict(res=None), dict(q=None), dict(s=None), dict(codes=0), dict(codes=4), dict(codes=-1), dict(rt=2),
                dict(wt=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y=P, ldy=255),
                dict(codes=0, q=None, s=None)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, q=None, s=None) == 0
    assert call(H=0, ldx=0) == 0


def test_norm_rhs_and_backward_entries(L):
    def rhs(h=P, ht=0, T=4, H=256, ldh=256, w=P, wt=0, rstd=P, codes=1, qT=P, ldqT=4, s=P):
        return L.rms_norm_quantize_rhs(h, ht, T, H, ldh, w, wt, rstd, codes, qT, ldqT, s, None)
    for bad in (dict(T=-1), dict(H=-1), dict(ldh=255), dict(ldqT=3), dict(codes=0), dict(codes=3), dict(ht=2), dict(wt=2), dict(h=None), dict(w=None),
                dict(rstd=None), dict(qT=None), dict(s=None), dict(T=128 * 65535 + 1, ldqT=2 ** 24)):
        assert rhs(**bad) == INVALID, bad
    assert rhs(T=0) == 0 and rhs(H=0) == 0

    def back(dy=P, lddy=256, h=P, ht=0, ldh=256, w=P, wt=0, rstd=P, dh=P, lddh=256, T=4, H=256, dx=P, lddx=256, dw=P, ws=P, wsb=4096):
        return L.rms_norm_backward(dy, lddy, h, ht, ldh, w, wt, rstd, dh, lddh, T, H, dx, lddx, dw, ws, wsb, None)
    assert L.rms_norm_backward_workspace(4, 256) == 4096
    for bad in (dict(T=-1), dict(H=-1), dict(T=2 ** 24), dict(lddy=255), dict(ldh=255), dict(lddh=255), dict(lddx=255), dict(dy=None), dict(h=None),
                dict(w=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(wsb=4095), dict(ws=ODD), dict(ht=5), dict(wt=5)):
        assert back(**bad) == INVALID, bad
    assert back(H=0) == 0
    assert L.rms_norm_backward_workspace(-1, 4) == -1 and L.rms_norm_backward_workspace(4, -1) == -1


def test_more_columns_than_a_launch_holds(L):
    wide = 2 ** 30 - 127
    assert L.rms_norm_quantize_rhs(P, 0, 4, wide, wide, P, 0, P, 1, P, 4, P, None) == INVALID
    assert L.swiglu_quantize_lhs_and_rhs(P, 4, wide, 2 * wide, 1, P, wide, P, P, 4, P, None) == INVALID
    assert L.swiglu_backward_quantize(P, wide, P, 2 * wide, 4, 2 ** 29 - 63, 1, P, 2 * wide, P, P, 4, P, None) == INVALID
    assert L.rms_norm_backward_workspace(4, 2 ** 26 - 15) == -1 and L.rms_norm_backward_workspace(4, 2 ** 26 - 16) == 4 * 4 * (2 ** 26 - 16)
    deep = 2 ** 26
    assert L.rms_norm_backward(P, deep, P, 0, deep, P, 0, P, None, 0, 4, deep, P, deep, P, P, 2 ** 40, None) == INVALID


def test_swiglu_entries(L):
    def rows(gu=P, T=4, F=256, ldgu=512, codes=1, q=P, ldq=256, s=P, y=None, ldy=0):
        return L.swiglu_quantize(gu, T, F, ldgu, codes, q, ldq, s, y, ldy, None)
    for bad in (dict(T=-1), dict(F=-1), dict(T=2 ** 24), dict(ldgu=511), dict(ldq=255), dict(codes=0), dict(codes=7), dict(gu=None), dict(q=None),
                dict(s=None), dict(y=P, ldy=255)):
        assert rows(**bad) == INVALID, bad
    assert rows(T=0) == 0 and rows(F=0) == 0

    def both(gu=P, T=4, F=256, ldgu=512, codes=1, q=P, ldq=256, a_s=P, qT=P, ldqT=4, s=P):
        return L.swiglu_quantize_lhs_and_rhs(gu, T, F, ldgu, codes, q, ldq, a_s, qT, ldqT, s, None)

    def grad(dy=P, lddy=256, gu=P, ldgu=512, T=4, F=256, codes=1, q=P, ldq=512, a_s=P, qT=P, ldqT=4, s=P):
        return L.swiglu_backward_quantize(dy, lddy, gu, ldgu, T, F, codes, q, ldq, a_s, qT, ldqT, s, None)
    for f, q in ((both, 255), (grad, 511)):
        for bad in (dict(T=-1), dict(F=-1), dict(ldgu=511), dict(ldq=q), dict(ldqT=3), dict(codes=0), dict(codes=3), dict(gu=None), dict(q=None),
                    dict(a_s=None), dict(qT=None), dict(s=None), dict(T=128 * 65535 + 1, ldqT=2 ** 24)):
            assert f(**bad) == INVALID, (f, bad)
        assert f(T=0) == 0 and f(F=0) == 0
    assert grad(lddy=255) == INVALID and grad(dy=None) == INVALID
    assert L.swiglu_backward(P, 255, P, 512, 4, 256, P, 512, None) == INVALID
    assert L.swiglu_backward(P, 256, P, 511, 4, 256, P, 512, None) == INVALID
    assert L.swiglu_backward(P, 256, P, 512, 4, 256, P, 511, None) == INVALID
    assert L.swiglu_backward(P, 2 ** 30, P, 2 ** 31, 2 ** 24, 2 ** 29, P, 2 ** 31, None) == INVALID      # 2^32 lanes and more
    assert L.swiglu_backward(None, 0, None, 0, 0, 0, None, 0, None) == 0


def test_i8_entries(L):
    assert L.quantize_rows_i8(P, 4, 256, 255, P, 256, P, None) == INVALID
    assert L.quantize_rows_i8(P, 4, 256, 256, P, 255, P, None) == INVALID
    assert L.quantize_rows_i8(P, 4, 256, 256, None, 256, P, None) == INVALID
    assert L.quantize_rows_i8(P, 2 ** 24, 256, 256, P, 256, P, None) == INVALID
    assert L.quantize_rows_i8(P, 0, 256, 256, P, 256, P, None) == 0

    def gemm(a=P, lda=256, a_s=P, b=P, ldb=256, b_s=P, c=P, ldc=64, M=4, N=64, K=256):
        return L.gemm_i8(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K, None)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=131072, lda=131072, ldb=131072), dict(ldc=63), dict(lda=240), dict(ldb=240), dict(c=None), dict(a=None),
                dict(b=None), dict(a_s=None), dict(b_s=None), dict(lda=2 ** 23 + 16), dict(ldb=2 ** 23 + 16), dict(M=2 ** 20, N=2 ** 20, ldc=2 ** 20)):
        assert gemm(**bad) == INVALID, bad
    assert gemm(lda=257) == ALIGN and gemm(ldb=264) == ALIGN and gemm(a=ODD) == ALIGN and gemm(b=ODD) == ALIGN
    assert gemm(M=0) == 0 and gemm(N=0) == 0


def grads(addresses, sizes, types):
    n = len(sizes)
    return (ctypes.c_void_p * n)(*addresses), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types)


def test_gradient_entries(L):
    a, n, t = grads([4096, 8192], [100, 20000], [0, 1])
    assert L.grad_workspace(n, 2) == 8 * 4
    assert L.grad_workspace(None, 2) == -1 and L.grad_workspace(n, -1) == -1 and L.grad_workspace(None, 0) == 0
    assert L.grad_workspace((ctypes.c_int64 * 1)(-1), 1) == -1
    assert L.grad_workspace((ctypes.c_int64 * 200)(*[10 ** 9] * 200), 200) == 8 * 512 * 3
    norm = lambda a=a, n=n, t=t, c=2, o=P, w=P, wb=32: L.grad_norm(a, n, t, c, o, w, wb, None)  # noqa: E731
    assert norm(a=None) == INVALID and norm(n=None) == INVALID and norm(t=None) == INVALID and norm(c=-1) == INVALID
    assert norm(o=None) == INVALID and norm(w=None) == INVALID and norm(wb=31) == INVALID and norm(w=ctypes.c_void_p(4100)) == INVALID
    for addresses, sizes, types in (([0, 8192], [100, 20000], [0, 1]), ([4097, 8192], [100, 20000], [0, 1]), ([4096, 8194], [100, 20000], [0, 1]),
                                    ([4096, 8192], [100, -1], [0, 1]), ([4096, 8192], [100, 20000], [0, 2])):
        x, y, z = grads(addresses, sizes, types)
        assert norm(x, y, z) == INVALID, (addresses, sizes, types)

    def clip(outs, max_norm=1.0, eps=1e-6, out_types=t):
        o = None if outs is None else (ctypes.c_void_p * 2)(*outs)
        return L.clip_grads(a, o, n, t, out_types, 2, max_norm, eps, P, P, 32, None)
    far = 1 << 30
    assert clip([far, 2 * far], max_norm=-1.0) == INVALID and clip([far, 2 * far], max_norm=math.nan) == INVALID
    assert clip([far, 2 * far], eps=-1.0) == INVALID and clip([far, 2 * far], eps=math.inf) == INVALID and clip([far, 2 * far], eps=math.nan) == INVALID
    assert clip(None) == INVALID and clip([0, far]) == INVALID and clip([far + 1, 2 * far]) == INVALID and clip([far, 2 * far], out_types=None) == INVALID
    assert clip([far, 2 * far], out_types=(ctypes.c_int * 2)(0, 3)) == INVALID
    # an output over a gradient, over part of its own, over another output
    assert clip([8192, far]) == INVALID and clip([4098, far]) == INVALID and clip([far, far + 198]) == INVALID and clip([far, far]) == INVALID
    assert clip([4096, far], out_types=(ctypes.c_int * 2)(1, 1)) == INVALID        # its own place, in another type
    assert clip([8192 + 80000 - 2, far]) == INVALID


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def raises(kind, words, f, *args, **kw):
    with pytest.raises(kind, match=words):
        f(*args, **kw)


def test_norm_binding():
    x, w = bf16(4, 256), bf16(256)
    f = bf.rms_norm_quantize
    raises(TypeError, "x has dtype", f, x.float(), w)
    raises(ValueError, "x must be 2-D", f, bf16(256), w)
    raises(ValueError, "contiguous rows", f, bf16(256, 4).t(), w)
    raises(TypeError, "weight must be", f, x, w.half())
    raises(ValueError, "weight has shape", f, x, bf16(255))
    raises(ValueError, "eps must be positive", f, x, w, eps=0.0)
    raises(ValueError, "eps must be positive", f, x, w, eps=1e-60)
    raises(ValueError, "eps must be positive", f, x, w, eps=math.nan)
    raises(ValueError, "unsupported FP8 format", f, x, w, fmt="e5m2")
    raises(TypeError, "residual has dtype", f, x, w, residual=x.half())
    raises(ValueError, "residual has shape", f, x, w, residual=bf16(4, 255))
    raises(TypeError, "h has dtype", f, x, w, residual=x, h=x.float())
    raises(ValueError, "h is not written", f, x, w, h=x)
    raises(ValueError, "q and s are not written", f, x, w, fmt=None, q=torch.zeros(4, 256, dtype=torch.uint8))
    raises(TypeError, "q has dtype", f, x, w, fmt="int8", q=torch.zeros(4, 256, dtype=torch.uint8))
    raises(TypeError, "q has dtype", f, x, w, q=torch.zeros(4, 256, dtype=torch.int8))
    raises(ValueError, "s has shape", f, x, w, fmt="int8", s=torch.zeros(4, 2))
    raises(ValueError, "s has shape", f, x, w, s=torch.zeros(4, 2))
    raises(ValueError, "rstd has shape", f, x, w, rstd=torch.zeros(5))
    raises(ValueError, "must be a GPU tensor", f, x, w)
    f = bf.rms_norm_quantize_rhs
    raises(ValueError, "rstd has shape", f, x, w, torch.zeros(3))
    raises(ValueError, "qT has shape", f, x, w, torch.zeros(4), qT=torch.zeros(4, 256, dtype=torch.uint8))
    raises(ValueError, "unsupported FP8 format", f, x, w, torch.zeros(4), fmt="int8")
    raises(ValueError, "must be a GPU tensor", f, x, w, torch.zeros(4))
    f = bf.rms_norm_backward
    raises(TypeError, "dy has dtype", f, x.float(), x, w, torch.zeros(4))
    raises(ValueError, "h has shape", f, x, bf16(3, 256), w, torch.zeros(4))
    raises(TypeError, "dh has dtype", f, x, x, w, torch.zeros(4), dh=x.float())
    raises(TypeError, "dx has dtype", f, x, x.float(), w, torch.zeros(4), dx=x)
    raises(TypeError, "dweight has dtype", f, x, x, w, torch.zeros(4), dweight=torch.zeros(256))
    raises(TypeError, "workspace must be", f, x, x, w, torch.zeros(4), workspace=torch.zeros(4096))
    raises(ValueError, "workspace holds", f, x, x, w, torch.zeros(4), workspace=torch.zeros(4095, dtype=torch.uint8))
    raises(ValueError, "must be a GPU tensor", f, x, x, w, torch.zeros(4))
    raises(ValueError, "no norm of", bf.rms_norm_backward_workspace, -1, 3)


def test_swiglu_binding():
    gu, dy = bf16(4, 512), bf16(4, 256)
    raises(ValueError, "gate and up", bf.swiglu_quantize, bf16(4, 511))
    raises(TypeError, "gu has dtype", bf.swiglu_quantize, gu.float())
    raises(ValueError, "q has shape", bf.swiglu_quantize, gu, q=torch.zeros(4, 512, dtype=torch.uint8))
    raises(ValueError, "y has shape", bf.swiglu_quantize, gu, y=gu)
    raises(ValueError, "unsupported FP8 format", bf.swiglu_quantize_lhs_and_rhs, gu, fmt="int8")
    raises(ValueError, "a_s has shape", bf.swiglu_quantize_lhs_and_rhs, gu, a_s=torch.zeros(4, 2))
    raises(ValueError, "dy has shape", bf.swiglu_backward, gu, gu)
    raises(ValueError, "dgu has shape", bf.swiglu_backward, dy, gu, dgu=dy)
    raises(ValueError, "qT has shape", bf.swiglu_backward_quantize, dy, gu, qT=torch.zeros(256, 4, dtype=torch.uint8))
    for f, args in ((bf.swiglu_quantize, (gu,)), (bf.swiglu_quantize_lhs_and_rhs, (gu,)), (bf.swiglu_backward, (dy, gu)),
                    (bf.swiglu_backward_quantize, (dy, gu))):
        raises(ValueError, "must be a GPU tensor", f, *args)


def test_i8_binding():
    a, b, s = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(64, 256, dtype=torch.int8), torch.zeros
    raises(TypeError, "x has dtype", bf.quantize_rows_i8, a)
    raises(ValueError, "must be a GPU tensor", bf.quantize_rows_i8, bf16(4, 256))
    raises(TypeError, "a has dtype", bf.gemm_i8, a.view(torch.uint8), s(4), b, s(64))
    raises(ValueError, "a_s has shape", bf.gemm_i8, a, s(5), b, s(64))
    raises(ValueError, "b_s has shape", bf.gemm_i8, a, s(4), b, s(4))
    raises(ValueError, "c has shape", bf.gemm_i8, a, s(4), b, s(64), c=bf16(64, 4))
    raises(ValueError, "K = 257", bf.gemm_i8, a, s(4), b, s(64), K=257)
    long = torch.zeros(1, 131072, dtype=torch.int8)
    raises(ValueError, "may pass int32", bf.gemm_i8, long, s(1), long, s(1))
    raises(ValueError, "must be a GPU tensor", bf.gemm_i8, a, s(4), b, s(64))


def test_gradient_binding():
    g = [torch.zeros(3), bf16(5)]
    raises(ValueError, "no gradients", bf.grad_norm, [])
    raises(TypeError, r"grads\[1\] must be", bf.grad_norm, [g[0], None])
    raises(TypeError, r"grads\[0\] has dtype", bf.grad_norm, [torch.zeros(3, dtype=torch.float64)])
    raises(ValueError, r"grads\[0\] must be dense", bf.grad_norm, [torch.zeros(4, 4)[:, :3]])
    raises(ValueError, r"grads\[0\] must be dense", bf.grad_norm, [torch.zeros(4, 1).expand(4, 3)])
    raises(ValueError, "must be a GPU tensor", bf.grad_norm, g)
    raises(ValueError, "max_norm", bf.clip_grads, g, -1.0)
    raises(ValueError, "max_norm", bf.clip_grads, g, math.nan)
    raises(ValueError, "eps", bf.clip_grads, g, 1.0, eps=-1.0)
    raises(ValueError, "out holds 1", bf.clip_grads, g, 1.0, out=g[:1])
    raises(ValueError, r"out\[0\] has shape", bf.clip_grads, g, 1.0, out=[torch.zeros(4), bf16(5)])
    raises(ValueError, r"out\[0\] has shape", bf.clip_grads, [torch.zeros(3, 4)], 1.0, out=[torch.zeros(4, 3).t()])
