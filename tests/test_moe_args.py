"""Checks of the mixture-of-experts operators that need no GPU: the C ABI and the binding reject bad
arguments before any HIP call, the schedule's bounds hold, and the gradient formulas the GPU tests
compare with agree with differences of the forward definition."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from blockwise_scaled_fp8_act_amd import binding
from tests import _moe_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_scaled_fp8_act_amd", "csrc")
P = ctypes.c_void_p(16 * 1024)      # a fake, aligned address: never dereferenced on these paths
ODD = ctypes.c_void_p(16 * 1024 + 8)
F32, I32, I64, U8, BF = torch.float32, torch.int32, torch.int64, torch.uint8, torch.bfloat16


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from blockwise_scaled_fp8_act_amd import build
        build.build()
    return binding.lib()


def _passed(rc):
    return rc not in (1, 2)         # past the argument checks: no device here


def test_route_entry_rejects_bad_arguments(L):
    def f(logits=P, dtype=1, T=4, E=64, ld=64, bias=None, score=0, k=8, groups=1, top=1, renorm=1, scale=1.0, w=P, ids=P):
        return L.moe_route(logits, dtype, T, E, ld, bias, score, k, groups, top, renorm, scale, w, ids, None)
    assert _passed(f())
    assert f(T=0) == 0
    for bad in (dict(logits=None), dict(w=None), dict(ids=None), dict(dtype=2), dict(dtype=-1), dict(score=2), dict(T=-1),
                dict(E=0), dict(E=1025, ld=1025), dict(ld=63), dict(k=0), dict(k=65), dict(k=9, E=8), dict(groups=0), dict(groups=5),
                dict(groups=8, top=0), dict(groups=8, top=9), dict(groups=16, top=1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(T=2 ** 31 // 8)):
        assert f(**bad) == 1, bad
    assert _passed(f(E=1024, ld=1024, k=64))
    assert _passed(f(groups=8, top=1))                  # 8 experts hold k = 8


def test_route_backward_entry_rejects_bad_arguments(L):
    def f(logits=P, dtype=0, T=4, E=64, ld=64, score=1, k=8, scale=1.0, ids=P, dw=P, dl=P, lddl=64):
        return L.moe_route_backward(logits, dtype, T, E, ld, score, k, 1, scale, ids, dw, dl, lddl, None)
    assert _passed(f())
    assert f(T=0) == 0
    for bad in (dict(logits=None), dict(ids=None), dict(dw=None), dict(dl=None), dict(lddl=63), dict(ld=10), dict(k=65), dict(E=0),
                dict(score=3), dict(dtype=9), dict(scale=float("nan"))):
        assert f(**bad) == 1, bad


def test_plan_entry_rejects_bad_arguments(L):
    def f(ids=P, T=4, k=2, E=8, off=P, slots=P, rows=P, ws=None, n=0):
        return L.moe_plan(ids, T, k, E, off, slots, rows, ws, n, None)
    assert _passed(f())
    for bad in (dict(ids=None), dict(off=None), dict(slots=None), dict(rows=None), dict(E=0), dict(E=1025), dict(k=0), dict(k=65),
                dict(T=-1), dict(T=2 ** 30, k=2)):
        assert f(**bad) == 1, bad
    need = L.moe_plan_workspace(8192, 8, 64)
    assert need == 32 * 65 * 4
    assert f(T=8192, k=8, E=64) == 1 and f(T=8192, k=8, E=64, ws=P, n=need - 1) == 1
    assert f(T=8192, k=8, E=64, ws=ctypes.c_void_p(16385), n=need) == 1       # not 4-byte aligned
    assert _passed(f(T=8192, k=8, E=64, ws=P, n=need))
    assert L.moe_plan_workspace(512, 8, 1024) == 0
    assert L.moe_plan_workspace(1, 65, 8) == -1 and L.moe_plan_workspace(-1, 1, 8) == -1


def test_dispatch_and_combine_entries_reject_bad_arguments(L):
    def d(x=P, T=4, H=256, ldx=256, slots=P, k=2, q=P, ldq=256, a_s=P, copy=None, ldcopy=0):
        return L.moe_dispatch(x, T, H, ldx, slots, k, q, ldq, a_s, copy, ldcopy, None)
    assert _passed(d())
    assert d(T=0) == 0 and d(H=0) == 0
    for bad in (dict(x=None), dict(slots=None), dict(q=None), dict(a_s=None), dict(ldx=255), dict(ldq=255), dict(copy=P, ldcopy=255),
                dict(k=0), dict(k=65), dict(T=-1), dict(H=-1)):
        assert d(**bad) == 1, bad

    def c(rows=P, R=8, ldr=256, slots=P, w=P, T=4, k=2, H=256, y=P, ldy=256):
        return L.moe_combine(rows, R, ldr, slots, w, T, k, H, y, ldy, None)
    assert _passed(c()) and _passed(c(w=None)) and _passed(c(rows=None, R=0))
    assert c(T=0) == 0 and c(H=0) == 0
    for bad in (dict(rows=None), dict(slots=None), dict(y=None), dict(ldr=255), dict(ldy=255), dict(R=-1), dict(k=0)):
        assert c(**bad) == 1, bad

    def b(dy=P, lddy=256, rows=P, ldr=256, slots=P, w=P, T=4, k=2, H=256, dr=P, lddr=256, dw=P):
        return L.moe_combine_backward(dy, lddy, rows, ldr, slots, w, T, k, H, dr, lddr, dw, None)
    assert _passed(b())
    assert b(T=0) == 0
    for bad in (dict(dy=None), dict(rows=None), dict(slots=None), dict(w=None), dict(dr=None), dict(dw=None), dict(lddy=1),
                dict(ldr=1), dict(lddr=1), dict(k=65)):
        assert b(**bad) == 1, bad


def test_routed_product_entry_rejects_bad_arguments(L):
    def f(a=P, lda=256, a_s=P, a_rows=4, rows=None, k=1, b=P, ldb=256, bst=128 * 256, b_s=P, bss=2, nb=2, kb=1, off=P, E=8, c=P,
          ldc=128, M=4, N=128, K=256, sw=0):
        return L.gemm_1x128_128x128_routed(a, lda, a_s, a_rows, rows, k, b, ldb, bst, b_s, bss, nb, kb, off, E, c, ldc, M, N, K, sw,
                                           None)
    assert _passed(f()) and _passed(f(rows=P, k=2, a_rows=1)) and _passed(f(sw=1))
    assert f(E=0) == 0 and f(M=0) == 0 and f(N=0) == 0
    for bad in (dict(a=None), dict(a_s=None), dict(b=None), dict(b_s=None), dict(off=None), dict(c=None), dict(K=0), dict(K=200),
                dict(sw=1, N=64), dict(lda=128), dict(ldb=128), dict(ldc=127), dict(a_rows=3), dict(rows=P, a_rows=0), dict(k=0),
                dict(k=65), dict(E=1025), dict(E=-1), dict(M=-1), dict(M=2 ** 31, a_rows=2 ** 31), dict(bst=-16), dict(bss=-1),
                dict(nb=-1), dict(kb=-1)):
        assert f(**bad) == 1, bad
    for bad in (dict(a=ODD), dict(b=ODD), dict(lda=264), dict(ldb=264), dict(bst=8)):
        assert f(**bad) == 2, bad


def test_entries_reject_launches_of_2_32_lanes(L):
    """A launch's lanes are counted in 32 bits: a wave a token (or for so many of its columns), four for the
    gradient of the return, a workgroup a tile of the routed product."""
    most = 2 ** 26 - 64

    def route(T):
        return L.moe_route(P, 1, T, 8, 8, None, 0, 2, 1, 1, 1, 1.0, P, P, None)

    def route_backward(T):
        return L.moe_route_backward(P, 1, T, 8, 8, 0, 2, 1, 1.0, P, P, P, 8, None)
    for f in (route, route_backward):
        assert _passed(f(most)) and f(most + 1) == 1

    def dispatch(T, H):
        return L.moe_dispatch(P, T, H, H, P, 2, P, H, P, None, 0, None)
    assert _passed(dispatch(most, 1024)) and _passed(dispatch(most // 2, 1025))
    assert dispatch(most + 1, 1024) == 1 and dispatch(most, 1025) == 1

    def combine(T, H):
        return L.moe_combine(P, 8, H, P, P, T, 2, H, P, H, None)
    assert _passed(combine(most, 512)) and combine(most + 1, 512) == 1 and combine(most, 513) == 1

    def combine_backward(T):
        return L.moe_combine_backward(P, 8, P, 8, P, P, T, 2, 8, P, 8, P, None)
    assert _passed(combine_backward(most // 4)) and combine_backward(most // 4 + 1) == 1

    def product(M, N, E=2, sw=0):
        return L.gemm_1x128_128x128_routed(P, 128, P, M, P, 1, P, 128, 128, P, 1, 1, 1, P, E, P, N, M, N, 128, sw, None)
    rows = 64 * (2 ** 23 - 3) + 65                        # E = 2: (M - 2) / 64 + 2 tiles, at most 2^23 - 1
    assert _passed(product(rows, 1)) and product(rows + 1, 1) == 1 and product(rows, 129) == 1
    assert _passed(product(2, 128 * (2 ** 22 - 1))) and product(2, 128 * 2 ** 22) == 1
    assert _passed(product(2, 64 * (2 ** 22 - 2), sw=1)) and product(2, 64 * 2 ** 22, sw=1) == 1


def test_binding_rejects_malformed_tensors():
    z = torch.zeros(4, 16)
    for bad, kind in ((dict(logits=z.half()), TypeError), (dict(logits=z[0]), ValueError), (dict(logits=z.t()), ValueError),
                      (dict(k=0), ValueError), (dict(k=17), ValueError), (dict(score="relu"), ValueError), (dict(groups=3), ValueError),
                      (dict(groups=4, top_groups=5), ValueError), (dict(groups=8, top_groups=1, k=3), ValueError),
                      (dict(bias=torch.zeros(15)), ValueError), (dict(bias=torch.zeros(16, dtype=BF)), TypeError),
                      (dict(scale=float("nan")), ValueError), (dict(weights=torch.zeros(4, 3)), ValueError),
                      (dict(ids=torch.zeros(4, 2)), TypeError), (dict(logits=torch.zeros(4, 1025)), ValueError), ({}, ValueError)):
        with pytest.raises(kind):                       # the last: well formed, but in host memory
            bf.moe_route(**{"logits": z, "k": 2, **bad})
    ids = torch.zeros(4, 2, dtype=I32)
    dw = torch.zeros(4, 2)
    for bad, kind in ((dict(ids=ids.long()), TypeError), (dict(ids=ids[:3]), ValueError), (dict(ids=ids.t()), ValueError),
                      (dict(dweights=dw[:3]), ValueError), (dict(dlogits=torch.zeros(4, 16, dtype=BF)), TypeError), ({}, ValueError)):
        with pytest.raises(kind):
            bf.moe_route_backward(**{"logits": z, "ids": ids, "dweights": dw, **bad})
    for bad, kind in ((dict(ids=ids.long()), TypeError), (dict(E=0), ValueError), (dict(E=1025), ValueError),
                      (dict(offsets=torch.zeros(9, dtype=I32)), TypeError), (dict(offsets=torch.zeros(8, dtype=I64)), ValueError),
                      (dict(slots=torch.zeros(8, dtype=I32)), ValueError), (dict(workspace=torch.zeros(8)), TypeError),
                      (dict(ids=torch.zeros(4, 65, dtype=I32)), ValueError), ({}, ValueError)):
        with pytest.raises(kind):
            bf.moe_plan(**{"ids": ids, "E": 8, **bad})
    with pytest.raises(ValueError, match="the plan needs"):
        bf.moe_plan(torch.zeros(8192, 8, dtype=I32), 64, workspace=torch.zeros(16, dtype=U8))
    x = torch.zeros(4, 256, dtype=BF)
    for bad, kind in ((dict(x=x.float()), TypeError), (dict(x=x[:3]), ValueError), (dict(q=torch.zeros(8, 255, dtype=U8)), ValueError),
                      (dict(a_s=torch.zeros(8, 2)), ValueError), (dict(copy=torch.zeros(8, 256)), TypeError),
                      (dict(slots=ids.long()), TypeError), ({}, ValueError)):
        with pytest.raises(kind):
            bf.moe_dispatch(**{"x": x, "slots": ids, **bad})
    r = torch.zeros(8, 256, dtype=BF)
    for bad, kind in ((dict(rows=r.float()), TypeError), (dict(weights=dw.double()), TypeError), (dict(weights=dw[:3]), ValueError),
                      (dict(y=torch.zeros(4, 255, dtype=BF)), ValueError), ({}, ValueError)):
        with pytest.raises(kind):
            bf.moe_combine(**{"rows": r, "slots": ids, **bad})
    for bad, kind in ((dict(rows=r[:7]), ValueError), (dict(dy=x.float()), TypeError), (dict(weights=None), TypeError),
                      (dict(drows=torch.zeros(8, 128, dtype=BF)), ValueError), ({}, ValueError)):
        with pytest.raises(kind):
            bf.moe_combine_backward(**{"dy": x, "rows": r, "slots": ids, "weights": dw, **bad})


def test_routed_product_binding_checks():
    E, N, K, M = 4, 256, 256, 6
    good = dict(a=torch.zeros(M, K, dtype=U8), a_s=torch.ones(2, M), b=torch.zeros(E * N, K, dtype=U8), b_s=torch.ones(E * 2, 2),
                offsets=torch.zeros(E + 1, dtype=I64), E=E, b_stride=N * K, bs_stride=4, bs_stride_nb=2, bs_stride_kb=1)
    for bad, kind, text in (
            (dict(a=torch.zeros(M, K)), TypeError, "a has dtype"), (dict(a_s=torch.ones(M, 2)), ValueError, "a_s has shape"),
            (dict(a=torch.zeros(M, 200, dtype=U8)), ValueError, "multiple of 128"), (dict(rows=torch.zeros(M)), TypeError, "rows"),
            (dict(rows=torch.zeros(M, 1, dtype=I32)), ValueError, "1-D"), (dict(rows=torch.zeros(M, dtype=I32), k=0), ValueError, "k = 0"),
            (dict(offsets=torch.zeros(E, dtype=I64)), ValueError, "E \\+ 1"), (dict(offsets=torch.zeros(E + 1, dtype=I32)), TypeError, "int64"),
            (dict(b=torch.zeros(E * N - 1, K, dtype=U8), N=N), ValueError, "b holds"), (dict(b_stride=N * K + 16), ValueError, "b holds"),
            (dict(bs_stride=5), ValueError, "b_s holds"), (dict(bs_stride_nb=-1), ValueError, ">= 0"), (dict(swiglu=True, N=64), ValueError, "with swiglu"),
            (dict(swiglu=True, N=256), ValueError, "b holds"), (dict(c=torch.zeros(M, 128, dtype=BF)), ValueError, "c has shape"),
            (dict(E=1025), ValueError, "E = 1025"), ({}, ValueError, "GPU tensor"), (dict(swiglu=True), ValueError, "GPU tensor")):
        with pytest.raises(kind, match=text):
            bf.gemm_1x128_128x128_routed(**{**good, **bad})


def test_schedule_bounds(tmp_path):
    """The plan's workgroups cover every pair in whole 64-pair steps of eight waves, at most 512 of
    them; the routed product's row tiles are enough for the worst boundaries, found by brute force."""
    src = tmp_path / "check.cpp"
    src.write_text(r'''
#include <algorithm>
#include <cstdio>
#include "schedule.hpp"
using namespace bsfp8::sched;
int64_t worst(int64_t M, int64_t E, int64_t tm) {   // most tiles E experts with M rows in all can have
    if (E == 1) return M == 0 ? 0 : (M + tm - 1) / tm;
    int64_t best = 0;
    for (int64_t r = 0; r <= M; ++r) best = std::max(best, (r + tm - 1) / tm + worst(M - r, E - 1, tm));
    return best;
}
int main() {
    for (int64_t P : {0LL, 1LL, 511LL, 512LL, 513LL, 2048LL, 2049LL, 4096LL, 4097LL, 8192LL, 8193LL, 65536LL, 131072LL, 1048575LL, 1048577LL, 99999999LL, 2147483647LL}) {
        const int64_t s = plan_segment(P), b = plan_blocks(P);
        if (s % 512 != 0 || b < 1 || b > 512 || b * s < P || (P > 0 && (b - 1) * s >= P)) return std::printf("plan %lld\n", (long long)P), 1;
        if ((P <= 8192) != (b == 1)) return std::printf("blocks %lld\n", (long long)P), 1;
        if (b == 1 && plan_round(plan_waves(P), plan_steps(P)) < P) return std::printf("round %lld\n", (long long)P), 1;
        if (b > 1 && s % plan_round(plan_waves(P), plan_steps(P)) != 0) return std::printf("rounds %lld\n", (long long)P), 1;
    }
    for (int64_t tm : {1, 2, 4})
        for (int64_t M = 1; M <= 14; ++M)
            for (int64_t E = 1; E <= 5; ++E)
                if (routed_row_tiles(M, E, tm) != worst(M, E, tm)) return std::printf("tiles %d %d %d\n", (int)M, (int)E, (int)tm), 1;
    return 0;
}
''')
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_formula_against_differences(score, renormalize):
    """Central differences of the forward definition, with the choice held: step h = 1e-5 in 64 bits
    leaves an error of about h^2 + 1e-16 / h < 1e-9 of the weights' size."""
    g = np.random.Generator(np.random.PCG64(5))
    T, E, k, scale, h = 3, 12, 4, 1.7, 1e-5
    z, dw = g.standard_normal((T, E)), g.standard_normal((T, k))
    _, ids = ref.route(z, k, score, renormalize=renormalize, scale=scale)

    def weights(z):
        p = ref.scores(z, score)
        q = np.take_along_axis(p, ids.astype(np.int64), 1)
        return scale * q / (q.sum(axis=1, keepdims=True) if renormalize else 1.0)

    got, _ = ref.route_backward(z, ids, dw, score, renormalize, scale)
    for e in range(E):
        up, down = z.copy(), z.copy()
        up[:, e] += h
        down[:, e] -= h
        slope = ((weights(up) - weights(down)) * dw).sum(axis=1) / (2 * h)
        assert np.abs(slope - got[:, e]).max() < 1e-8


def test_route_reference_by_hand():
    """Rows small enough to work out: ties, a mask that leaves less than k, none, NaN, groups."""
    inf, nan = np.inf, np.nan
    z = np.array([[1.0, 1.0, 0.0, 1.0], [-inf, 2.0, -inf, -inf], [-inf] * 4, [0.0, nan, 0.0, 0.0]])
    w, ids = ref.route(z, 2)
    assert ids.tolist() == [[0, 1], [1, -1], [-1, -1], [-1, -1]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0] and np.isnan(w[3]).all()
    # groups of two: without a bias the group of the largest logit wins, with one the larger pair sum
    z = np.array([[2.0, -9.0, 1.5, 1.5]])
    assert ref.route(z, 2, "sigmoid", groups=2)[1].tolist() == [[0, 1]]
    assert ref.route(z, 2, "sigmoid", bias=np.zeros(4), groups=2)[1].tolist() == [[2, 3]]


def test_one_step_calls_leave_the_unusual_alone():
    """The C part of the binding answers None, without an exception and without keeping a reference, to whatever is no
    plain GPU tensor or out of range: the checks of the Python functions then say what is wrong."""
    from blockwise_scaled_fp8_act_amd import binding
    binding.lib()
    calls = binding._calls
    assert calls is not None
    z, f, i = torch.randn(4, 64), torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    good = {"moe_route": (z, 2, "softmax", None, 1, 1, True, 1.0, f, i), "moe_route_backward": (z, i, f, "softmax", True, 1.0, None),
            "moe_plan": (i, 8, None, None, None, None), "moe_dispatch": (x, i, None, None, None, False), "moe_combine": (x, i, f, None),
            "moe_combine_backward": (x, x, i, f, None, None),
            "gemm_1x128_128x128_routed": (x, f, x, f, f, 2, 128, 1, 1, 1, None, i, 2, False, None, None)}
    odd = (None, 3, "x", 2.5, float("nan"), 2 ** 70, -1, [1], torch.nn.Parameter(z), z.t(), z[0], z[:0], z.double(), torch.zeros(2, 2, 2))
    count = [sys.getrefcount(o) for o in odd + (z, f, i, x)]
    for name, args in good.items():
        call = getattr(calls, name)
        assert call(*args) is None                               # tensors of the CPU
        assert call() is None and call(*args[:-1]) is None and call(*args, 1) is None
        for at in range(len(args)):
            for o in odd:
                assert call(*args[:at], o, *args[at + 1:]) is None
    o = args = None
    good.clear()
    now = [sys.getrefcount(o) for o in odd + (z, f, i, x)]
    assert all(abs(a - b) <= 16 for a, b in zip(count, now)), (count, now)
