"""Every kernel of the int8 product, bit for bit against whole sums, with rows behind K and around C that are not
zero; scales of a row, shared operands, the same call twice at once."""
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from _ffn_ref import Guarded
from _i8_cases import CASES

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _codes(rows, K, seed):
    """Codes of the whole range in rows padded with others."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.randint(-128, 128, (rows, (K + 15) // 16 * 16 + 16), generator=g, device=DEV, dtype=torch.int8)
    return buf[:, :K], torch.rand(rows, generator=g, device=DEV) + 0.01


def _want(a, a_s, b, b_s):
    acc = a.double() @ b.double().t()           # whole numbers below 2^31
    return ((acc.float() * a_s[:, None]) * b_s).to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [s for _, _, shapes in CASES for s in shapes])
def test_kernel(M, N, K):
    (a, a_s), (b, b_s) = _codes(M, K, 1), _codes(N, K, 2)
    want = _want(a, a_s, b, b_s)
    for ldc, shift in ((0, 0), (3, 1)):
        c = Guarded(M, N, torch.bfloat16, DEV, N + ldc, shift)
        bf.gemm_i8(a, a_s, b, b_s, c=c.view)
        assert torch.equal(c.host(), want.cpu())


def test_two_calls_at_once():
    """Two products on two streams, over the same weight."""
    (a, a_s), (b, b_s) = _codes(1000, 1280, 3), _codes(2050, 1280, 4)
    (d, d_s) = _codes(16, 1280, 5)
    wants = [_want(a, a_s, b, b_s), _want(d, d_s, b, b_s)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [bf.gemm_i8(x, s, b, b_s, stream=st) for (x, s), st in zip(((a, a_s), (d, d_s)), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, wants))


def test_symmetric_product():
    """A and B the same tensor."""
    a, a_s = _codes(520, 520, 6)
    assert torch.equal(bf.gemm_i8(a, a_s, a, a_s), _want(a, a_s, a, a_s))
