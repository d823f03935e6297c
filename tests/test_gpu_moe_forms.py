"""GPU test of every kernel of the routed product (tests/_moe_cases.py; tests/test_moe_forms.py shows that each
case runs the one it names). Bounds as in test_gpu_moe_ops.py: 2^-10 of the magnitudes (with the gate through the
derivative of silu(g) u) and half a bf16 step."""
import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from tests import _moe_cases as cases
from tests import _moe_ref as ref
from tests._gpu import DEV, to_dev
from tests.test_gpu_moe_ops import _check_product, _codes, _g, _np, _product_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", cases.PRODUCT_FORMS, ids=[f"{c['kernel']}{'-gated' * c['swiglu']}-{i}" for i, c in enumerate(cases.PRODUCT_FORMS)])
def test_routed_product_of_every_kernel(case):
    """Codes over the whole range and scales of their own in every block: a row, a column, a chunk of K or a
    scale taken from elsewhere shows. Rows of C outside the experts stay as they are."""
    N, K, E, M, swiglu = case["N"], case["K"], cases.experts(case), cases.rows(case), case["swiglu"]
    g = _g(N + K + E)
    N2 = 2 * N if swiglu else N
    if "T" in case:
        k = case["k"]
        offsets, _, index = ref.plan(ref.choose(g, case["T"], k, E, case.get("dropped", 0.0)), E)
        source = np.where(index >= 0, index // k, 0)
        lhs = dict(rows=torch.from_numpy(index).to(DEV), k=k)
    else:
        offsets = 2 + np.concatenate([[0], np.cumsum(case["counts"])]).astype(np.int64)
        source, lhs = np.arange(M), {}
    A = int(source.max()) + 1 if "T" not in case else case["T"]
    _, b, b_s = _product_case(g, [0] * E, N2, K)
    if swiglu:
        b_s *= np.float32(2.0 ** -9)                  # gates of ordinary size
    a, a_s = _codes(g, (A, K)), (0.5 + g.random((K // 128, A))).astype(np.float32) * np.float32(2.0 ** -5)
    out = torch.full((M + 2, N + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    bf.gemm_1x128_128x128_routed(to_dev(a), to_dev(a_s), to_dev(b.reshape(E * N2, K)), to_dev(b_s.reshape(-1)), torch.from_numpy(offsets).to(DEV), E,
                                 b_stride=N2 * K, bs_stride=b_s[0].size, bs_stride_nb=K // 128, bs_stride_kb=1, N=N, swiglu=swiglu, c=out[1:M + 1, :N], **lhs)
    got = _np(out[1:M + 1, :N])
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        if r.size:
            _check_product(got[r], a[source[r]], a_s[:, source[r]], b[e], b_s[e], swiglu, f"expert {e}")
    assert np.all(got[:offsets[0]] == 7.0) and np.all(got[offsets[-1]:] == 7.0)
    assert torch.all(out[0] == 7.0) and torch.all(out[M + 1] == 7.0) and torch.all(out[:, N:] == 7.0)
