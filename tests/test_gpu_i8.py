"""int8 rows and products. Both are exact: codes and scales follow from IEEE arithmetic, the sum is whole, and
its two factors and the rounding to bf16 are single fp32 operations, so everything is compared bit for bit."""
import math

import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from _ffn_ref import Guarded, i8_codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 8), (5, 120), (4, 1000), (3, 1001), (2, 1032), (3, 2048), (2, 5120), (2, 14336), (1, 16384), (2, 16392),
                                 (1030, 256)])
@pytest.mark.parametrize("ld,shift", [(0, 0), (8, 8), (3, 1)])
def test_rows(M, K, ld, shift):
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(M + K)) * 3).to(torch.bfloat16)
    x[0, 0] = -0.0
    gx, gq = Guarded(M, K, x.dtype, DEV, K + ld, shift, x), Guarded(M, K, torch.int8, DEV, K + ld, shift)
    _, s = bf.quantize_rows_i8(gx.view, q=gq.view)
    q, want = i8_codes(x.float())
    assert torch.equal(gq.host(), q) and torch.equal(s.cpu(), want)


def test_rows_of_zeros_and_halves():
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    x[1] = torch.arange(256) - 127.5        # halves of a step: 127.5 -> 127
    x[2, :128] = 2.0 ** -120                # below the floor of the scale
    q, s = bf.quantize_rows_i8(x.to(DEV))
    wq, ws = i8_codes(x.float())
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), ws)


def reference(a, a_s, b, b_s):
    acc = torch.empty(a.shape[0], b.shape[0], dtype=torch.int64)
    bt = b.double().t().contiguous()
    for i in range(0, a.shape[0], 512):     # whole below 2^53
        acc[i:i + 512] = (a[i:i + 512].double() @ bt).long()
    return ((acc.to(torch.int32).float() * a_s[:, None]) * b_s).to(torch.bfloat16)


def codes(rows, K, seed, ld=0, edge=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int8) if not edge else torch.full((rows, K), -128, dtype=torch.int8)
    stride = (K + ld + 15) // 16 * 16
    buf = torch.randint(-128, 128, (rows, stride), generator=g, dtype=torch.int8).to(DEV)      # what lies behind K is not zero
    buf[:, :K] = v.to(DEV)
    return v, buf[:, :K], torch.rand(rows, generator=g) + 0.01


def check_product(M, N, K, ldc=0, shift=0, ld=0, edge=False):
    a, ad, a_s = codes(M, K, 1, ld, edge)
    b, bd, b_s = codes(N, K, 2, ld, edge)
    gc = Guarded(M, N, torch.bfloat16, DEV, N + ldc, shift)
    bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV), c=gc.view)
    assert torch.equal(gc.host(), reference(a, a_s, b, b_s)), (M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 16), (2, 3, 5), (1, 1000, 1000), (1, 4096, 128), (3, 1280, 640), (5, 130, 129), (7, 2048, 1111), (8, 640, 5120),
                                   (15, 500, 400), (16, 1024, 2048), (17, 96, 130), (31, 513, 257), (32, 512, 8192), (33, 64, 128), (64, 1280, 1280), (65, 130, 260),
                                   (100, 1000, 1000), (127, 256, 127), (128, 4096, 512), (129, 385, 1408), (250, 640, 384), (256, 256, 256), (300, 1001, 333),
                                   (512, 5120, 640), (1000, 1000, 1288), (1024, 2048, 512), (2049, 4100, 260), (4096, 4097, 384), (5000, 300, 144)])
def test_product(M, N, K):
    check_product(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 640, 512), (20, 333, 200), (70, 1280, 300), (600, 515, 384), (2100, 4100, 128)])
@pytest.mark.parametrize("ldc,shift,ld", [(4, 0, 32), (1, 0, 0), (8, 1, 48), (0, 3, 16), (8, 4, 64)])
def test_product_strides(M, N, K, ldc, shift, ld):
    check_product(M, N, K, ldc, shift, ld)


@pytest.mark.parametrize("M,N", [(1, 33), (16, 40), (70, 70), (300, 300)])
def test_longest_sum(M, N):
    """K = 131071 products of 16384 stay within int32; the last block is partial."""
    check_product(M, N, 131071, edge=True)


def test_inner_dimension_of_zero_and_of_a_part():
    a, ad, a_s = codes(40, 96, 3)
    b, bd, b_s = codes(50, 128, 4)
    c = torch.full((40, 50), 7.0, dtype=torch.bfloat16, device=DEV)
    bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV), c=c, K=0)
    assert (c == 0).all()
    got = bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV), K=70)
    assert torch.equal(got.cpu(), reference(a[:, :70], a_s, b[:, :70], b_s))
    assert bf.gemm_i8(ad[:0], a_s[:0].to(DEV), bd, b_s.to(DEV), K=96).shape == (0, 50)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_scales_that_are_not_finite(M):
    """A row whose scale is not finite (its codes are 0) comes out as NaN, the others as without it."""
    a, ad, a_s = codes(M, 640, 5)
    _, bd, b_s = codes(520, 640, 6)
    clean = bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV))
    ad = ad.clone()
    ad[1], a_s[1], ad[2], a_s[2] = 0, math.inf, 0, math.nan
    c = bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV))
    assert c[1].isnan().all() and c[2].isnan().all()
    c[1:3] = clean[1:3]
    assert torch.equal(c, clean)


def test_same_result_on_every_call():
    for M in (1, 64, 700):
        _, ad, a_s = codes(M, 2000, 7)
        _, bd, b_s = codes(1100, 2000, 8)
        first = bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV))
        for _ in range(3):
            assert torch.equal(bf.gemm_i8(ad, a_s.to(DEV), bd, b_s.to(DEV)), first)
