"""GPU tests of the mixture-of-experts operators against plain 64-bit references (tests/_moe_ref.py)
and, for codes and products, the CPU oracle.

Tolerances, all relative to a sum of magnitudes so that cancellation is counted:
  route weights   fp32 chain of at most 32 roundings of half a step: 32 * 2^-24 relative;
  dlogits         64 * 2^-24 of the magnitudes that enter an element, plus half a step of its type
                  (fp32 2^-24, bf16 2^-8) and one bf16 subnormal step;
  combine         (k + 2) * 2^-24 of the magnitudes, plus half a bf16 step (2^-8) of the result;
  drows           one fp32 product and one bf16 rounding: 2^-8 (1 + 2^-10) relative;
  dweights        a dot product in fp32 partial sums of at most H / 64 + 16 terms each:
                  (H / 64 + 32) * 2^-24 of the magnitudes;
  products        2^-10 of the magnitudes of the products (the matrix core's K-block sum is not an exactly
                  rounded one) plus half a bf16 step; with the gate: through the derivative of
                  silu(g) u, |silu'| <= 1.1.
Chosen experts, plans and codes have to be equal."""
import gc

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
import oracle
from blockwise_scaled_fp8_act_amd import inputs
from tests import _moe_ref as ref
from tests._gpu import DEV, to_dev

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _g(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _np(t):
    return t.detach().double().cpu().numpy()


def _logits(g, T, E, dtype, pad=0):
    """[T, E] logits on the device with `pad` extra columns between rows, and as float64."""
    z = torch.from_numpy((1.5 * g.standard_normal((T, E + pad))).astype(np.float32)).to(DEV).to(dtype)[:, :E]
    return z, _np(z)


def _check_weights(w, want):
    w = _np(w)
    assert np.array_equal(np.isnan(w), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(w - want)[ok] <= 32 * E24 * np.abs(want[ok]) + 2.0 ** -149)


ROUTES = [(1, 1, 1), (3, 2, 2), (5, 7, 3), (33, 8, 2), (1, 64, 8), (7, 65, 8), (129, 128, 6), (66, 256, 8), (9, 384, 8), (5, 1000, 64),
          (4, 1024, 10), (65, 60, 4), (2, 64, 64)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_route(T, E, k, dtype):
    for i, (score, bias, renorm) in enumerate([(s, b, r) for s in ("softmax", "sigmoid") for b in (0, 1) for r in (0, 1)]):
        print(f"route T={T} E={E} k={k} {dtype} {score} bias={bias} renorm={renorm}", flush=True)
        g = _g(100 + i)
        z, zh = _logits(g, T, E, dtype, pad=i % 3)
        b = torch.from_numpy((0.05 * g.standard_normal(E)).astype(np.float32)).to(DEV) if bias else None
        w, ids = bf.moe_route(z, k, score=score, bias=b, renormalize=bool(renorm), scale=2.5)
        want_w, want_ids = ref.route(zh, k, score, None if b is None else _np(b), renormalize=bool(renorm), scale=2.5)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        _check_weights(w, want_w)


@pytest.mark.parametrize("T,E,k", [(3, 1000, 8), (3, 513, 16), (2, 300, 16), (5, 250, 13), (9, 17, 16), (3, 255, 17)])
def test_route_odd_expert_counts(T, E, k):
    """Counts that leave lanes without experts in both team sizes, and the most choices a team ranks."""
    for score, bias in (("softmax", 0), ("sigmoid", 1), ("softmax", 1)):
        g = _g(E + k)
        z, zh = _logits(g, T, E, F32, pad=1)
        b = torch.from_numpy((0.05 * g.standard_normal(E)).astype(np.float32)).to(DEV) if bias else None
        w, ids = bf.moe_route(z, k, score=score, bias=b, renormalize=False)
        want_w, want_ids = ref.route(zh, k, score, None if b is None else _np(b), renormalize=False)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        _check_weights(w, want_w)


@pytest.mark.parametrize("E", [16, 256, 1024])
def test_route_of_quantized_logits_with_many_ties(E):
    """Logits of a few distinct values (the top ones tie by the dozen) in both types and signs, -0 beside
    0: ties go to the lower index."""
    g = _g(E)
    zh = np.round(g.standard_normal((40, E)) * 2) / 2
    zh[::2] *= -1.0                                     # leaves -0.0 among the zeros
    zh[5] = np.where(np.arange(E) % 2, 0.0, -0.0)
    for dtype in (F32, BF):
        z = torch.from_numpy(zh.astype(np.float32)).to(DEV).to(dtype)
        for bias in (None, np.zeros(E, np.float32), np.round(g.standard_normal(E) * 4).astype(np.float32) / 64):
            b = None if bias is None else torch.from_numpy(bias).to(DEV)
            _, ids = bf.moe_route(z, 8, score="sigmoid", bias=b)
            assert np.array_equal(ids.cpu().numpy(), ref.route(zh + 0.0, 8, "sigmoid", bias)[1])


@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (64, 8, 2, 6), (64, 4, 3, 8), (160, 8, 3, 6), (96, 8, 1, 8), (128, 16, 4, 8), (12, 3, 2, 8),
                                            (64, 64, 9, 9), (1024, 32, 5, 8), (200, 100, 30, 16), (256, 2, 1, 8), (384, 8, 4, 8)])
def test_route_groups(E, groups, top, k):
    for i, (score, bias) in enumerate([("softmax", 0), ("sigmoid", 1), ("softmax", 1), ("sigmoid", 0)]):
        print(f"groups E={E} groups={groups} top={top} k={k} {score} bias={bias}", flush=True)
        g = _g(200 + i)
        z, zh = _logits(g, 37, E, F32 if i % 2 else BF)
        b = torch.from_numpy((0.05 * g.standard_normal(E)).astype(np.float32)).to(DEV) if bias else None
        w, ids = bf.moe_route(z, k, score=score, bias=b, groups=groups, top_groups=top)
        want_w, want_ids = ref.route(zh, k, score, None if b is None else _np(b), groups, top)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        _check_weights(w, want_w)


@pytest.mark.parametrize("E,groups,top", [(8, 1, 1), (64, 1, 1), (256, 1, 1), (256, 8, 4), (384, 1, 1)])
def test_route_chooses_between_keys_closer_than_fp32(E, groups, top):
    """Biases that bring every key to 0.7 within fp32's resolution (about 3e-8): the order is the one of
    the 64-bit keys; and all-equal logits, where the lowest indexes win."""
    g = _g(7)
    for score in ("sigmoid", "softmax"):
        z, zh = _logits(g, 48, E, F32)
        z = z[:1].expand(48, E).contiguous() + torch.from_numpy((g.integers(0, 2, (48, E)) * 2.0 ** -22).astype(np.float32)).to(DEV)
        zh = _np(z)
        b = torch.from_numpy((0.7 - ref.scores(zh[:1], score)[0]).astype(np.float32)).to(DEV)
        _, ids = bf.moe_route(z, 8 if E > 8 else 4, score=score, bias=b, groups=groups, top_groups=top)
        _, want = ref.route(zh, 8 if E > 8 else 4, score, _np(b), groups, top)
        assert np.array_equal(ids.cpu().numpy(), want)
        same = torch.full((5, E), 0.3, device=DEV)
        for bias in (None, torch.zeros(E, device=DEV)):
            _, ids = bf.moe_route(same, 4, score=score, bias=bias, groups=groups, top_groups=top)
            assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 5


@pytest.mark.parametrize("E,groups,top", [(16, 4, 2), (64, 8, 3), (100, 5, 2), (256, 8, 4), (256, 1, 1), (512, 8, 4), (1000, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_of_rows_that_tie_beside_rows_that_do_not(E, groups, top, score):
    """Rows of a few distinct logits, of plain ones, with NaN, with nothing left and of equal logits in one wave, in
    every order: what a row needs to be told apart leaves its neighbours as they are."""
    g, k, T = _g(E + top), 4, 61
    few = np.round(g.standard_normal((T, E)) * 2) / 4
    kind = g.integers(0, 5, T)[:, None]
    zh = np.where(kind == 0, few, 1.5 * g.standard_normal((T, E))).astype(np.float32)
    zh = np.where((kind == 2) & (np.arange(E) == 3), np.nan, np.where(kind == 3, -np.inf, np.where(kind == 4, 0.25, zh)))
    z = torch.from_numpy(zh.astype(np.float32)).to(DEV)
    for bias in (np.zeros(E, np.float32), np.round(g.standard_normal(E) * 2).astype(np.float32) / 64):
        w, ids = bf.moe_route(z, k, score=score, bias=torch.from_numpy(bias).to(DEV), groups=groups, top_groups=top)
        want_w, want_ids = ref.route(_np(z), k, score, bias, groups, top)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        _check_weights(w, want_w)


@pytest.mark.parametrize("E", [8, 64, 100, 256, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_infinities_and_nan(E, score):
    """Masked experts (-inf) that leave less than k or nothing, NaN and +inf logits, far logits, biases of
    -inf and NaN: as the reference defines them, the other rows untouched."""
    g, k = _g(9), 4
    zh = 1.5 * g.standard_normal((12, E))
    zh[1] = -np.inf
    zh[2, 1:] = -np.inf
    zh[3, 2:] = -np.inf
    zh[4, E // 2] = np.nan
    zh[5] = np.nan
    zh[6, 3] = np.inf
    zh[7] = 1e4 * g.standard_normal(E)
    zh[8] = -200.0 + 0.1 * g.standard_normal(E)
    zh[9, ::2] = -np.inf
    zh[10] = np.finfo(np.float32).min
    zh[11, 0] = -3e38
    z = torch.from_numpy(zh.astype(np.float32)).to(DEV)
    zh = _np(z)
    bias = 0.05 * g.standard_normal(E)
    odd = bias.copy()
    odd[0], odd[1] = -np.inf, np.nan
    for b in (None, bias.astype(np.float32), odd.astype(np.float32)):
        for renorm in (True, False):
            for groups, top in ((1, 1), (4, 2)):
                w, ids = bf.moe_route(z, k, score=score, bias=None if b is None else torch.from_numpy(b).to(DEV), renormalize=renorm,
                                      groups=groups, top_groups=top)
                with np.errstate(all="ignore"):
                    want_w, want_ids = ref.route(zh, k, score, b, groups, top, renormalize=renorm)
                assert np.array_equal(ids.cpu().numpy(), want_ids), (b is None, renorm, groups)
                _check_weights(w, want_w)


@pytest.mark.parametrize("E,groups,top", [(64, 8, 2), (256, 8, 4), (96, 8, 3), (512, 16, 3), (64, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_with_biases_of_any_size(E, groups, top, score):
    """Biases that force experts in (+inf, 1e9), push them back (-1e9) or swamp the scores (+-100 and sums
    of such that cancel): the order is the one of the 64-bit keys."""
    g = _g(E + top)
    z, zh = _logits(g, 24, E, F32)
    for case in range(5):
        b = 0.01 * g.standard_normal(E)
        at = g.permutation(E)
        if case == 0:
            b[at[:5]] = np.inf
        elif case == 1:
            b[at[:E // 2]] = -1e9
            b[at[:2]] = 1e9
        elif case == 2:
            b += 100.0
        elif case == 3:
            b = np.where(g.integers(0, 2, E) == 1, 1e6, -1e6) + b
        else:
            b = np.round(g.standard_normal(E) * 2) * 1e4
        b = b.astype(np.float32)
        w, ids = bf.moe_route(z, 4, score=score, bias=torch.from_numpy(b).to(DEV), groups=groups, top_groups=top)
        want_w, want_ids = ref.route(zh, 4, score, b, groups, top)
        assert np.array_equal(ids.cpu().numpy(), want_ids), case
        _check_weights(w, want_w)


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_route_backward(T, E, k, dtype):
    for i, (score, renorm) in enumerate([(s, r) for s in ("softmax", "sigmoid") for r in (0, 1)]):
        g = _g(300 + i)
        z, zh = _logits(g, T, E, dtype, pad=i)
        ids = ref.choose(g, T, k, E, dropped=0.1 if i % 2 else 0.0)
        dw = g.standard_normal((T, k)).astype(np.float32)
        out = torch.full((T, E + 3), 7.0, dtype=dtype, device=DEV)
        dz = bf.moe_route_backward(z, torch.from_numpy(ids).to(DEV), torch.from_numpy(dw).to(DEV), score=score, renormalize=bool(renorm),
                                   scale=1.7, dlogits=out[:, :E])
        want, size = ref.route_backward(zh, ids, dw, score, bool(renorm), 1.7)
        half = 2.0 ** -8 if dtype == BF else E24
        assert np.all(np.abs(_np(dz) - want) <= 64 * E24 * size + half * np.abs(want) + 2.0 ** -133)
        assert torch.all(out[:, E:] == 7.0)


def test_route_backward_rows_without_a_choice():
    z = torch.randn(3, 64, device=DEV)
    z[1] = float("nan")
    ids = torch.full((3, 4), -1, dtype=I32, device=DEV)
    ids[2] = torch.tensor([5, -1, 64, 9], dtype=I32)
    dz = bf.moe_route_backward(z, ids, torch.ones(3, 4, device=DEV), score="softmax", renormalize=False)
    assert torch.all(dz[:2] == 0) and torch.any(dz[2] != 0)


PLANS = [(1, 1, 1), (1, 8, 64), (63, 1, 2), (64, 1, 63), (13, 5, 64), (511, 8, 65), (512, 8, 256), (513, 8, 8), (700, 6, 1024), (4096, 8, 64),
         (256, 8, 64), (2049, 1, 31), (1024, 4, 64), (4097, 1, 1024), (1365, 6, 100), (8192, 1, 1024), (8193, 1, 7), (33333, 3, 255), (131072, 8, 128)]


@pytest.mark.parametrize("T,k,E", PLANS)
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_plan(T, k, E, dropped):
    g = _g(T + E)
    ids = g.integers(0, E, (T, k)).astype(np.int32)
    bad = np.array([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=np.int64).astype(np.int32)
    ids = np.where(g.random((T, k)) < dropped, bad[g.integers(0, 4, (T, k))], ids).astype(np.int32)
    got = bf.moe_plan(torch.from_numpy(ids).to(DEV), E)
    for a, b, name in zip(got, ref.plan(ids, E), ("offsets", "slots", "rows")):
        assert np.array_equal(a.cpu().numpy(), b), name


def test_plan_of_no_tokens_and_of_one_expert():
    offsets, slots, rows = bf.moe_plan(torch.empty(0, 4, dtype=I32, device=DEV), 16, offsets=torch.full((17,), 9, device=DEV))
    assert torch.all(offsets == 0) and slots.shape == (0, 4) and rows.numel() == 0
    ids = torch.full((3000, 2), 5, dtype=I32, device=DEV)
    offsets, slots, rows = bf.moe_plan(ids, 16)
    assert offsets.tolist() == [0] * 6 + [6000] * 11 and torch.equal(slots.flatten().cpu(), torch.arange(6000, dtype=I32))


@pytest.mark.parametrize("T,H,k,pad,shift", [(1, 128, 1, 0, 0), (5, 1, 2, 0, 0), (7, 127, 3, 0, 0), (9, 129, 2, 3, 0), (33, 1000, 4, 0, 0), (17, 1040, 8, 16, 0),
                                             (40, 1280, 6, 0, 8), (64, 2056, 2, 0, 0), (130, 4096, 8, 0, 0), (3, 5120, 64, 32, 0), (21, 272, 4, 16, 1)])
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_dispatch(T, H, k, pad, shift, dropped):
    """Row r holds what quantize_lhs writes for its token, padding rows hold zeros; strides, odd lengths
    and bases that are not 16-byte aligned; nothing outside the rows is written."""
    g = _g(T + H)
    E, R = 64, T * k
    x = inputs.normal_bf16(g, (T, H))
    x[0] = 0
    if H > 200:
        x[T // 2, 130] = 0x7F00                       # a large finite value in one group
    slots = ref.plan(ref.choose(g, T, k, E, dropped), E)[1]
    buf = torch.zeros(T * (H + pad) + 16, dtype=torch.int16, device=DEV)
    xd = buf[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H]
    xd.copy_(torch.from_numpy(x.view(np.int16)))
    q = torch.full((R + 2, H + pad), 0xA5, dtype=torch.uint8, device=DEV)
    copy = torch.full((R + 2, H + pad), -1, dtype=torch.int16, device=DEV)
    _, a_s, _ = bf.moe_dispatch(xd, torch.from_numpy(slots).to(DEV), q=q[1:R + 1, :H], copy=copy[1:R + 1, :H])
    oq, os_ = oracle.quantize_lhs(x)
    want_q, want_s, want_c = np.zeros((R, H), np.uint8), np.zeros(((H + 127) // 128, R), np.float32), np.zeros((R, H), np.uint16)
    t, j = np.nonzero(slots >= 0)
    r = slots[t, j]
    want_q[r], want_s[:, r], want_c[r] = oq[t], os_[:, t], x[t]
    assert np.array_equal(q[1:R + 1, :H].cpu().numpy(), want_q)
    assert np.array_equal(a_s.cpu().numpy(), want_s)
    assert np.array_equal(copy[1:R + 1, :H].cpu().numpy().view(np.uint16), want_c)
    for b, v in ((q, 0xA5), (copy, -1)):
        assert torch.all(b[0] == v) and torch.all(b[R + 1] == v) and torch.all(b[:, H:] == v)


def test_dispatch_and_combine_skip_slots_out_of_range():
    x = torch.randn(2, 256, device=DEV).to(BF)
    slots = torch.tensor([[0, 4], [-6, 2 ** 31 - 1]], dtype=I32, device=DEV)     # rows 4, 5 and 2^31 - 1 of 4
    q = torch.full((4, 256), 0xA5, dtype=torch.uint8, device=DEV)
    bf.moe_dispatch(x, slots, q=q)
    assert torch.all(q[1:] == 0xA5) and torch.any(q[0] != 0xA5)
    rows = torch.randn(4, 256, device=DEV).to(BF)
    y = bf.moe_combine(rows, slots, torch.ones(2, 2, device=DEV))
    assert torch.equal(y[0], rows[0]) and torch.all(y[1] == 0)
    drows = torch.full((4, 256), 7.0, dtype=BF, device=DEV)
    _, dw = bf.moe_combine_backward(x, rows, slots, torch.ones(2, 2, device=DEV), drows=drows)
    assert torch.all(drows[1:] == 7.0) and torch.equal(drows[0], x[0])
    assert dw[0, 1] == 0 and torch.all(dw[1] == 0) and dw[0, 0] != 0


SIZES = [(1, 8, 1), (5, 1, 2), (7, 127, 3), (33, 1000, 4), (17, 1040, 8), (64, 2056, 2), (65, 4096, 8), (3, 5120, 64), (9, 512, 6)]


@pytest.mark.parametrize("T,H,k", SIZES)
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_combine(T, H, k, dropped):
    for pad, shift in ((0, 0), (8, 0), (3, 1)):
        g = _g(T + H + pad)
        E, R = 64, T * k
        slots = ref.plan(ref.choose(g, T, k, E, dropped), E)[1]
        buf = torch.from_numpy(g.standard_normal(R * (H + pad) + 16).astype(np.float32)).to(DEV).to(BF)
        rows = buf[shift:shift + R * (H + pad)].view(R, H + pad)[:, :H]
        w = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)).to(DEV)
        out = torch.full((T + 2, H + pad), 7.0, dtype=BF, device=DEV)
        for weights in (w, None):
            y = bf.moe_combine(rows, torch.from_numpy(slots).to(DEV), weights, y=out[1:T + 1, :H])
            want, size = ref.combine(_np(rows), slots, None if weights is None else _np(w))
            assert np.all(np.abs(_np(y) - want) <= (k + 2) * E24 * size + 2.0 ** -8 * np.abs(want) + 2.0 ** -133)
        assert torch.all(out[0] == 7.0) and torch.all(out[T + 1] == 7.0) and torch.all(out[:, H:] == 7.0)


@pytest.mark.parametrize("T,H,k", SIZES)
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_combine_backward(T, H, k, dropped):
    for pad, shift in ((0, 0), (8, 0), (3, 1)):
        g = _g(T + H + pad)
        E, R = 64, T * k
        slots = ref.plan(ref.choose(g, T, k, E, dropped), E)[1]
        buf = torch.from_numpy(g.standard_normal(R * (H + pad) + 16).astype(np.float32)).to(DEV).to(BF)
        rows = buf[shift:shift + R * (H + pad)].view(R, H + pad)[:, :H]
        dy = torch.from_numpy(g.standard_normal((T, H + pad)).astype(np.float32)).to(DEV).to(BF)[:, :H]
        w = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)).to(DEV)
        out = torch.full((R + 2, H + pad), 7.0, dtype=BF, device=DEV)
        drows, dw = bf.moe_combine_backward(dy, rows, torch.from_numpy(slots).to(DEV), w, drows=out[1:R + 1, :H])
        t, j = np.nonzero(slots >= 0)
        want, want_dw, size = np.zeros((R, H)), np.zeros((T, k)), np.zeros((T, k))
        want[slots[t, j]] = _np(w)[t, j][:, None] * _np(dy)[t]
        want_dw[t, j] = (_np(dy)[t] * _np(rows)[slots[t, j]]).sum(axis=1)
        size[t, j] = np.abs(_np(dy)[t] * _np(rows)[slots[t, j]]).sum(axis=1)
        assert np.all(np.abs(_np(drows) - want) <= 2.0 ** -8 * (1 + 2.0 ** -10) * np.abs(want) + 2.0 ** -133)
        assert np.all(np.abs(_np(dw) - want_dw) <= (H / 64 + 32) * E24 * size)
        assert torch.all(out[0] == 7.0) and torch.all(out[R + 1] == 7.0) and torch.all(out[:, H:] == 7.0)


def test_a_row_that_could_not_be_routed_shows_in_its_output():
    z = torch.randn(3, 16, device=DEV)
    z[1, 4] = float("nan")
    w, ids = bf.moe_route(z, 2)
    offsets, slots, rows = bf.moe_plan(ids, 16)
    assert offsets[-1].item() == 4 and rows.tolist()[4:] == [-1, -1]
    y = bf.moe_combine(torch.ones(6, 64, dtype=BF, device=DEV), slots, w)
    assert torch.all(torch.isnan(y[1])) and torch.all(y[0] == 1) and torch.all(y[2] == 1)


def _codes(g, shape):
    """Random finite e4m3 codes over the whole range."""
    c = g.integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 0x7F) == 0x7F, c & 0x80, c).astype(np.uint8)


def _product_case(g, counts, N2, K, lead=0):
    """Codes and scales of an expert product; counts: rows of each expert, `lead` rows before the first."""
    E, Kb, Nb = len(counts), K // 128, (N2 + 127) // 128
    offsets = lead + np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    b, b_s = _codes(g, (E, N2, K)), (0.5 + g.random((E, Nb, Kb))).astype(np.float32) * np.float32(2.0 ** -6)
    return offsets, b, b_s


def _product_reference(a, a_s, b, b_s):
    """The product and the sum of its magnitudes, 64-bit."""
    Kb = b_s.shape[1]
    return oracle.gemm_1x128_128x128(a, a_s, b, b_s, Kb, 1), oracle.gemm_1x128_128x128(a & 0x7F, a_s, b & 0x7F, b_s, Kb, 1)


def _silu(x):
    return x / (1 + np.exp(-x))


def _check_product(got, a, a_s, b, b_s, swiglu, what):
    v, size = _product_reference(a, np.ascontiguousarray(a_s), b, b_s)
    err = 2.0 ** -10 * size
    if swiglu:
        F = b.shape[0] // 2
        g, u, dg, du = v[:, :F], v[:, F:], err[:, :F], err[:, F:]
        v, err = _silu(g) * u, 1.1 * dg * (np.abs(u) + du) + np.abs(_silu(g)) * du
    assert np.all(np.abs(got - v) <= err + 2.0 ** -8 * np.abs(v) * (1 + 2.0 ** -10)), what


PRODUCTS = [([1], 16, 128), ([1], 100, 256), ([0, 3, 0, 1], 17, 384), ([5, 0, 16, 17, 33, 1], 128, 1280), ([64, 65, 1, 0], 1000, 128),
            ([2, 200, 7], 256, 512), ([130], 48, 640), ([0] * 60 + [3] * 10 + [0, 9], 33, 256), ([40, 30, 21], 144, 2176)]


@pytest.mark.parametrize("counts,N,K", PRODUCTS, ids=[f"case{i}" for i in range(len(PRODUCTS))])
def test_routed_product(counts, N, K):
    """Rows in expert order (A row r for C row r), odd columns, lead and tail rows outside every expert."""
    g = _g(N + K)
    lead, E = 2, len(counts)
    M = lead + sum(counts) + 3
    offsets, b, b_s = _product_case(g, counts, N, K, lead)
    a, a_s = _codes(g, (M, K)), (0.5 + g.random((K // 128, M))).astype(np.float32) * np.float32(2.0 ** -5)
    out = torch.full((M + 2, N + 5), 7.0, dtype=BF, device=DEV)
    c = bf.gemm_1x128_128x128_routed(to_dev(a), to_dev(a_s), to_dev(b.reshape(E * N, K)), to_dev(b_s.reshape(-1)), torch.from_numpy(offsets).to(DEV), E,
                                     b_stride=N * K, bs_stride=b_s[0].size, bs_stride_nb=K // 128, bs_stride_kb=1, N=N, c=out[1:M + 1, :N])
    got = _np(c)
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        if r.size:
            _check_product(got[r], a[r], a_s[:, r], b[e], b_s[e], False, f"expert {e}")
    assert np.all(got[:lead] == 7.0) and np.all(got[offsets[-1]:] == 7.0)
    assert torch.all(out[0] == 7.0) and torch.all(out[M + 1] == 7.0) and torch.all(out[:, N:] == 7.0)


@pytest.mark.parametrize("T,k,E,F,K,dropped", [(1, 8, 64, 128, 256, 0.0), (1, 2, 8, 256, 1280, 0.0), (3, 1, 4, 128, 128, 0.0), (20, 4, 8, 384, 512, 0.3), (64, 8, 16, 128, 256, 0.1),
                                               (130, 2, 3, 128, 384, 0.0), (9, 6, 100, 128, 128, 0.5), (5, 2, 8, 128, 128, 1.0)])
@pytest.mark.parametrize("swiglu", [True, False])
def test_routed_product_through_the_plan(T, k, E, F, K, dropped, swiglu):
    """A in token order, read through the plan's rows; gate and up halves joined."""
    g = _g(T + E)
    ids = ref.choose(g, T, k, E, dropped)
    offsets, slots, rows = ref.plan(ids, E)
    N2 = 2 * F if swiglu else F
    _, b, b_s = _product_case(g, [0] * E, N2, K)
    if swiglu:
        b_s *= np.float32(2.0 ** -9)                  # gates of ordinary size
    a, a_s = _codes(g, (T, K)), (0.5 + g.random((K // 128, T))).astype(np.float32) * np.float32(2.0 ** -5)
    c = torch.full((T * k, F), 7.0, dtype=BF, device=DEV)
    plan = [t.to(DEV) for t in map(torch.from_numpy, (offsets, rows))]
    bf.gemm_1x128_128x128_routed(to_dev(a), to_dev(a_s), to_dev(b.reshape(E * N2, K)), to_dev(b_s.reshape(-1)), plan[0], E, b_stride=N2 * K,
                                 bs_stride=b_s[0].size, bs_stride_nb=K // 128, bs_stride_kb=1, rows=plan[1], k=k, swiglu=swiglu, c=c)
    got = _np(c)
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        if r.size:
            t = rows[r] // k
            _check_product(got[r], a[t], a_s[:, t], b[e], b_s[e], swiglu, f"expert {e}")
    assert np.all(got[offsets[-1]:] == 7.0)


@pytest.mark.parametrize("offsets", [[3, 60, 40, 90, 104], [-5, 10, 2000, 30, 104], [104, 0, 0, 0, 0], [0, 0, 0, 0, 0]],
                         ids=["decreasing", "outside", "past the end", "empty"])
def test_routed_product_clamps_boundaries_and_rows(offsets):
    """Boundaries that decrease or leave [0, M] are clamped as the grouped GEMM clamps them; a row whose
    map entry names no token is zero."""
    g = _g(3)
    E, N, K, M, T, k = 4, 96, 256, 104, 26, 4
    _, b, b_s = _product_case(g, [0] * E, N, K)
    a, a_s = _codes(g, (T, K)), (0.5 + g.random((K // 128, T))).astype(np.float32)
    rows = g.permutation(M).astype(np.int32)
    lost = {5: -1, 50: 104, 70: 2 ** 31 - 1, 99: -2 ** 31}
    for r, v in lost.items():
        rows[r] = v
    c = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    bf.gemm_1x128_128x128_routed(to_dev(a), to_dev(a_s), to_dev(b.reshape(E * N, K)), to_dev(b_s.reshape(-1)), torch.tensor(offsets, device=DEV), E,
                                 b_stride=N * K, bs_stride=b_s[0].size, bs_stride_nb=K // 128, bs_stride_kb=1, rows=torch.from_numpy(rows).to(DEV), k=k, c=c)
    got, covered, prev = _np(c), np.zeros(M, bool), 0
    for e in range(E):
        lo = min(max(offsets[e], prev, 0), M)
        hi = min(max(offsets[e + 1], lo), M)
        prev = hi
        covered[lo:hi] = True
        r = np.array([i for i in range(lo, hi) if i not in lost], dtype=np.int64)
        if r.size:
            _check_product(got[r], a[rows[r] // k], a_s[:, rows[r] // k], b[e], b_s[e], False, f"expert {e}")
    for r in lost:
        if covered[r]:
            assert np.all(got[r] == 0), r
    assert np.all(got[~covered] == 7.0)


def test_routed_product_with_padded_weights_and_transposed_scales():
    """Rows of B with a longer stride, experts apart, scales read transposed, K = 0-free ends: against the
    grouped GEMM on the same operands, whose sums differ in order only."""
    g = _g(12)
    E, N, K, M = 3, 256, 384, 70
    ldb, gap = K + 48, 1024
    buf = torch.zeros(E * (N * ldb + gap), dtype=torch.uint8, device=DEV)
    b = _codes(g, (E, N, K))
    for e in range(E):
        buf[e * (N * ldb + gap):][:N * ldb].view(N, ldb)[:, :K].copy_(torch.from_numpy(b[e]))
    b_s = (0.5 + g.random((E, K // 128, N // 128))).astype(np.float32)       # [kb][nb]
    a, a_s = _codes(g, (M, K)), (0.5 + g.random((K // 128, M))).astype(np.float32)
    off = torch.tensor([0, 20, 20, 70], device=DEV)
    c = bf.gemm_1x128_128x128_routed(to_dev(a), to_dev(a_s), buf[:N * ldb].view(N, ldb)[:, :K], to_dev(b_s.reshape(-1)), off, E, b_stride=N * ldb + gap,
                                     bs_stride=b_s[0].size, bs_stride_nb=1, bs_stride_kb=N // 128, N=N)
    got = _np(c)
    for e, (lo, hi) in enumerate(((0, 20), (20, 20), (20, 70))):
        if hi > lo:
            _check_product(got[lo:hi], a[lo:hi], a_s[:, lo:hi], b[e], np.ascontiguousarray(b_s[e].T), False, e)


def _layer(z, x, w1, s1, w2, s2, E, k, F, H, stream=None):
    """A decode step of a gated expert layer, operator by operator."""
    weights, ids = bf.moe_route(z, k, score="sigmoid", stream=stream)
    offsets, slots, rows = bf.moe_plan(ids, E, stream=stream)
    q, a_s = bf.quantize_lhs(x, stream=stream)
    h = bf.gemm_1x128_128x128_routed(q, a_s, w1, s1, offsets, E, 2 * F * H, s1.numel() // E, H // 128, 1, rows=rows, k=k, swiglu=True, stream=stream)
    qh, sh = bf.quantize_lhs(h, stream=stream)
    e = bf.gemm_1x128_128x128_routed(qh, sh, w2, s2, offsets, E, H * F, s2.numel() // E, F // 128, 1, stream=stream)
    qd, sd, _ = bf.moe_dispatch(x, slots, stream=stream)
    return weights, ids, e, bf.moe_combine(e, slots, weights, stream=stream), qd, sd


def _layer_inputs(seed, T, E, k, F, H):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z, x = torch.randn(T, E, device=DEV, generator=g), torch.randn(T, H, device=DEV, generator=g).to(BF)
    w1 = (0.05 * torch.randn(E * 2 * F, H, device=DEV, generator=g)).to(BF)
    w2 = (0.05 * torch.randn(E * H, F, device=DEV, generator=g)).to(BF)
    q1, _, s1 = bf.quantize_weight_128x128(w1, want_qT=False)
    q2, _, s2 = bf.quantize_weight_128x128(w2, want_qT=False)
    return (z, x, q1, s1.reshape(-1), q2, s2.reshape(-1), E, k, F, H)


def test_layer_on_another_stream_equals_the_current_one():
    args = _layer_inputs(1, 24, 16, 4, 256, 512)
    want = _layer(*args)
    torch.cuda.synchronize()
    for how in ("stream", "handle", "context", "default"):
        s = torch.cuda.default_stream() if how == "default" else torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if how == "default":
            with torch.cuda.stream(torch.cuda.Stream()):       # another stream is current
                got = _layer(*args, stream=s.cuda_stream)
        elif how == "context":
            with torch.cuda.stream(s):
                got = _layer(*args)
        else:
            got = _layer(*args, stream=s if how == "stream" else s.cuda_stream)
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_operators_replay_from_a_graph():
    """The layer's forward and the backward operators captured once and replayed with changed inputs and
    eager work between; every replay equals the eager result."""
    T, E, k, F, H = 600, 16, 8, 128, 256                  # 4800 pairs: the plan takes its counting pass
    args = _layer_inputs(2, T, E, k, F, H)
    z, x = args[0], args[1]
    dy = torch.randn(T, H, device=DEV).to(BF)

    def step():
        weights, ids, e, y, q, s = _layer(*args)
        offsets, slots, rows = bf.moe_plan(ids, E)
        drows, dw = bf.moe_combine_backward(dy, e, slots, weights)
        return [weights, ids, y, q, s, drows, dw, bf.moe_route_backward(z, ids, dw, score="sigmoid")]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        z.copy_(torch.randn(T, E, device=DEV))
        x.copy_(torch.randn(T, H, device=DEV))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (r, i)


def test_repeated_calls_give_the_same_bits():
    args = _layer_inputs(3, 200, 16, 8, 128, 512)
    want = [t.clone() for t in _layer(*args)]
    for _ in range(3):
        for a, b in zip(_layer(*args), want):
            assert torch.equal(a, b)


def _far_slots(T, k, seed):
    """A permutation of the rows as slots: rows of a token lie anywhere."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randperm(T * k, generator=g, device=DEV).to(I32).view(T, k)


def test_dispatch_and_combine_past_4_gib():
    """1.12 million rows of 4096 columns: codes of 4.6e9 bytes, copies of 9.2e9, row offsets past 2^32."""
    T, k, H = 140000, 8, 4096
    x = torch.randn(T, H, device=DEV, dtype=BF)
    slots = _far_slots(T, k, 1)
    q, a_s, copy = bf.moe_dispatch(x, slots, want_copy=True)
    pick = torch.tensor([0, 1, 524287, 524288, 1048575, 1048576, 1048577, T * k - 1], device=DEV)
    owner = torch.empty(T * k, dtype=torch.int64, device=DEV)
    owner[slots.flatten().long()] = torch.arange(T * k, device=DEV) // k
    want_q, want_s = bf.quantize_lhs(x[owner[pick]])
    assert torch.equal(q[pick], want_q) and torch.equal(a_s[:, pick], want_s) and torch.equal(copy[pick], x[owner[pick]])
    del q, a_s
    w = torch.rand(T, k, device=DEV) + 0.5
    y = bf.moe_combine(copy, slots, w)                     # every row is its own token's: y = x * sum of the weights
    t = torch.tensor([0, 1, T // 2, T - 1], device=DEV)
    want = x[t].double() * w[t].double().sum(1, keepdim=True)
    assert torch.all((y[t].double() - want).abs() <= (2.0 ** -8 + 10 * E24) * want.abs() + 2.0 ** -133)
    drows, dw = bf.moe_combine_backward(x, copy, slots, w)
    r = slots[t].long()
    want = w[t].double()[:, :, None] * x[t].double()[:, None, :]
    assert torch.all((drows[r.flatten()].view(4, k, H).double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -10) * want.abs() + 2.0 ** -133)
    norm = (x[t].double() ** 2).sum(1, keepdim=True)       # <dy, row> with dy = x
    assert torch.all((dw[t].double() - norm).abs() <= (H / 64 + 32) * E24 * norm)


@pytest.mark.parametrize("per", [1, 20], ids=["few rows", "tiles"])
def test_routed_product_of_weights_past_4_gib(per):
    """300 experts of 4096 x 4096 codes (5.0e9 bytes); the first and the last ones have rows."""
    E, N, K = 300, 4096, 4096
    b = torch.full((E * N, K), 0x38, dtype=torch.uint8, device=DEV)          # 1.0
    b[(E - 1) * N:] = 0xC0                                                   # -2.0
    b[255 * N:257 * N] = 0x30                                                # 0.5, around 2^32 bytes
    counts = torch.zeros(E, dtype=torch.int64)
    counts[[0, 255, 256, E - 1]] = per
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(DEV)
    M = 4 * per
    a = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)
    a_s = torch.full((K // 128, M), 2.0 ** -6, device=DEV)
    b_s = torch.ones(E * (N // 128) * (K // 128), device=DEV)
    c = bf.gemm_1x128_128x128_routed(a, a_s, b, b_s, off, E, N * K, (N // 128) * (K // 128), K // 128, 1)
    want = torch.tensor([64.0, 32.0, 32.0, -128.0], device=DEV).repeat_interleave(per)
    assert torch.equal(c.float(), want[:, None].expand(M, N))                # exact: powers of two


def test_routed_product_of_the_most_rows():
    """537 million rows, one output column, 64 choices a token: the most tiles of 64 rows that one launch holds.
    Row r is its token's, up to the last one; one row more is refused."""
    k, K = 64, 128
    M = 64 * (2 ** 23 - 3) + 65
    T = (M + k - 1) // k
    a = torch.full((T, K), 0x38, dtype=torch.uint8, device=DEV)                        # 1.0
    a_s = (2.0 ** (torch.arange(T, device=DEV) % 5 - 9).float()).view(1, T).contiguous()
    rows = torch.arange(M + 1, dtype=torch.int32, device=DEV)
    b = torch.full((2, K), 0x38, dtype=torch.uint8, device=DEV)
    b[1] = 0xC0                                                                        # -2.0
    b_s = torch.ones(2, device=DEV)
    c = torch.full((M, 1), float("nan"), dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 1, 2 ** 28 - 1, 2 ** 28, 2 ** 28 + 1, M - 66, M - 65, M - 64, M - 2, M - 1], device=DEV)
    off = torch.tensor([0, 2 ** 28, M], device=DEV)
    bf.gemm_1x128_128x128_routed(a, a_s, b, b_s, off, 2, K, 1, 1, 1, rows=rows[:M], k=k, c=c, N=1)
    want = 2.0 ** ((at // k) % 5 - 2).float() * torch.where(at < 2 ** 28, 1.0, -2.0)
    assert torch.equal(c[at, 0].float(), want)
    assert not any(bool(c[i:i + 2 ** 26].isnan().any()) for i in range(0, M, 2 ** 26))
    with pytest.raises(bf.Bsfp8Error):
        bf.gemm_1x128_128x128_routed(a, a_s, b, b_s, off, 2, K, 1, 1, 1, rows=rows, k=k, N=1)


def _both_ways(f, *args, **kw):
    """A call as users make it and the same with its stream named, which takes the long way of the binding."""
    a, b = f(*args, **kw), f(*args, **kw, stream=torch.cuda.current_stream())
    a, b = (a, b) if isinstance(a, tuple) else ((a,), (b,))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and x.device == y.device
            assert torch.equal(x, y)
    return a


@pytest.mark.parametrize("T,E,k,H", [(1, 8, 1, 128), (1, 256, 8, 1000), (33, 64, 6, 256), (700, 64, 8, 384), (2, 1, 1, 1)])
def test_both_ways_of_a_call_agree(T, E, k, H):
    g = torch.Generator(device=DEV).manual_seed(T)
    z = torch.randn(T, E + 3, device=DEV, generator=g)[:, :E]
    bias = torch.randn(E, device=DEV, generator=g)
    x = torch.randn(T, H, device=DEV, generator=g).to(BF)
    w, ids = _both_ways(bf.moe_route, z, k, score="sigmoid", bias=bias, scale=2)
    _both_ways(bf.moe_route, z.to(BF), k, renormalize=False)
    dw = torch.randn(T, k, device=DEV, generator=g)
    _both_ways(bf.moe_route_backward, z, ids, dw, score="sigmoid")
    _both_ways(bf.moe_route_backward, z.to(BF), ids, dw)
    ids[0, 0] = -1
    _, slots, _ = _both_ways(bf.moe_plan, ids, E)
    q, a_s, none = _both_ways(bf.moe_dispatch, x, slots)
    assert none is None
    rows = _both_ways(bf.moe_dispatch, x, slots, want_copy=True)[2]
    _both_ways(bf.moe_combine, rows, slots, w)
    _both_ways(bf.moe_combine, rows, slots)
    _both_ways(bf.moe_combine_backward, x, rows, slots, w)
    if H % 128 == 0:
        offsets, _, index = bf.moe_plan(ids, E)
        for swiglu in (False, True):
            b = torch.randn(E * 256, H, device=DEV, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
            b_s = torch.rand(E, 2, H // 128, device=DEV, generator=g)
            qx, sx = bf.quantize_lhs(x)
            for rows_given in (dict(rows=index, k=k), {}):
                lhs = (qx, sx) if rows_given else (q, a_s)
                full = offsets.clone()
                full[E] = T * k                             # no row of C left unwritten
                _both_ways(bf.gemm_1x128_128x128_routed, *lhs, b, b_s, full, E, 256 * H, 2 * (H // 128), H // 128, 1, swiglu=swiglu, **rows_given)
    out = torch.zeros(T, H + 5, dtype=BF, device=DEV)
    assert bf.moe_combine(rows, slots, w, y=out[:, :H]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:, :H], bf.moe_combine(rows, slots, w)) and not out[:, H:].any()


def test_one_step_calls_refuse_before_they_launch():
    """Arguments of the wrong type, shape, stride or place on the GPU: the same errors as the long way, outputs as they
    were, and no memory kept."""
    T, E, k, H = 8, 16, 2, 256
    z, x = torch.randn(T, E, device=DEV), torch.randn(T, H, device=DEV).to(BF)
    w, ids = bf.moe_route(z, k)
    _, slots, _ = bf.moe_plan(ids, E)
    rows = bf.moe_dispatch(x, slots, want_copy=True)[2]
    held = torch.full((T, k), 7, dtype=I32, device=DEV)
    wide = torch.empty(T, 2 * k, device=DEV)
    code, scale, edges = torch.zeros(T, H, dtype=torch.uint8, device=DEV), torch.ones(2, T, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    long, long_ids = torch.empty(2 ** 26, 1, dtype=BF, device=DEV), torch.empty(2 ** 26, 1, dtype=I32, device=DEV)       # refused: too many tokens
    before = torch.cuda.memory_allocated()
    for kind, f, args, kw in [
            (ValueError, bf.moe_route, (z, E + 1), {}), (ValueError, bf.moe_route, (z.t(), k), {}), (TypeError, bf.moe_route, (z.double(), k), {}),
            (ValueError, bf.moe_route, (z.cpu(), k), {}), (ValueError, bf.moe_route, (z, k), dict(bias=torch.zeros(E))),
            (ValueError, bf.moe_route, (z, k), dict(ids=held, weights=wide[:, :k])), (TypeError, bf.moe_route, (z, k), dict(ids=held, weights=held)),
            (ValueError, bf.moe_route, (z, k), dict(ids=held, scale=float("inf"))), (ValueError, bf.moe_route, (z, k), dict(ids=held, score="tanh")),
            (ValueError, bf.moe_route, (z, k), dict(ids=held, groups=3)), (ValueError, bf.moe_route, (z, k), dict(ids=held[:4])),
            (TypeError, bf.moe_plan, (ids.long(), E), {}), (ValueError, bf.moe_plan, (ids, 0), {}), (ValueError, bf.moe_plan, (ids, E), dict(rows=held)),
            (ValueError, bf.moe_plan, (ids, E), dict(slots=held.cpu())), (ValueError, bf.moe_dispatch, (x[:4], slots), {}),
            (ValueError, bf.moe_dispatch, (x, slots), dict(q=torch.empty(T, H, dtype=torch.uint8, device=DEV))),
            (ValueError, bf.moe_combine, (rows, slots, wide), {}), (ValueError, bf.moe_combine, (rows, slots.cpu(), w), {}),
            (ValueError, bf.moe_combine_backward, (x, rows[:4], slots, w), {}), (TypeError, bf.moe_combine_backward, (x.float(), rows, slots, w), {}),
            (ValueError, bf.gemm_1x128_128x128_routed, (code, scale, code, scale, edges, 2, 128 * H, 2, 2, 1), {}),
            (TypeError, bf.gemm_1x128_128x128_routed, (code, scale, code, scale, edges.int(), 1, 0, 0, 2, 1), {}),
            (ValueError, bf.gemm_1x128_128x128_routed, (code, scale, code, scale, edges[:1], 1, 0, 0, 2, 1), {}),
            (ValueError, bf.gemm_1x128_128x128_routed, (code, scale, code, scale, edges, 1, 0, 0, 2, 2 ** 62), {}),
            (ValueError, bf.gemm_1x128_128x128_routed, (code, scale, code, scale, edges, 1, 0, 0, 2, 1), dict(ldb=2 ** 62)),
            (bf.Bsfp8Error, bf.moe_route, (long, 1), {}), (bf.Bsfp8Error, bf.moe_route_backward, (long, long_ids, long_ids.float()), {}),
            (ValueError, bf.moe_route_backward, (z[:4], ids, w), {}), (TypeError, bf.moe_route_backward, (z, ids, held), {})]:
        for _ in range(3):
            with pytest.raises(kind):
                f(*args, **kw)
    args = kw = None
    gc.collect()          # what the raised errors' frames held
    torch.cuda.synchronize()
    assert torch.all(held == 7)
    assert torch.cuda.memory_allocated() <= before
