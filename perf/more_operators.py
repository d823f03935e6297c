"""What stands around the 8-bit products of a gated feed-forward layer: cases and plain forms.

Four operators, each one call (or the calls of a training step) of the package:

  norm     rms_norm_quantize: root-mean-square norm with the residual's addition -> e4m3 codes with
           1x128 scales; for training also rms_norm_quantize_rhs (128x1 codes) and rms_norm_backward.
  swiglu   swiglu_quantize: gate and up halves -> e4m3 codes of silu(gate) * up; for training the codes
           of both groupings, forward (swiglu_quantize_lhs_and_rhs) and backward (swiglu_backward_quantize).
  product  gemm_i8: int8 product with a scale a token and a channel, of codes, of bf16 rows
           (quantize_rows_i8), or of rows that come out of the norm (rms_norm_quantize, "int8").
  clip     clip_grads: global norm over many gradients and the clipped copies; grad_norm: the norm alone.

Run where ``own`` is false, the same results come from elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128
FP8_MAX = 448.0
I8_MAX = 127.0
AMAX_FLOOR = 1e-12
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step, before a layer's first product
        dict(name="norm 1 token", op="norm", rows=1, features=4096, residual="bf16", weight="bf16", copy=False, train=False),
        # a prompt; the normed rows are also kept in bf16 (a router reads them)
        dict(name="norm 16384 rows", op="norm", rows=16384, features=5120, residual="bf16", weight="bf16", copy=True, train=False),
        # a training step: codes of both groupings, the residual kept in 32 bits, gradients
        dict(name="norm train 8192", op="norm", rows=8192, features=4096, residual="f32", weight="f32", copy=False, train=True),
        # a decode batch between the two products
        dict(name="swiglu 64 rows", op="swiglu", rows=64, features=5120, copy=False, train=False),
        # a ragged prompt chunk
        dict(name="swiglu 1000 rows", op="swiglu", rows=1000, features=1408, copy=True, train=False),
        # a training step, forward and backward
        dict(name="swiglu train 8192", op="swiglu", rows=8192, features=4096, copy=False, train=True),
        # one token against a wide weight: the weight is read once
        dict(name="product 1 token", op="product", rows=1, n=14336, k=4096, source="codes"),
        # a decode batch whose rows come out of the norm
        dict(name="product 64 after norm", op="product", rows=64, n=5120, k=5120, source="norm"),
        # a ragged prompt chunk: rows quantized, odd width and inner dimension
        dict(name="product 1000 odd", op="product", rows=1000, n=1000, k=1288, source="rows"),
        # a long prompt
        dict(name="product 16384 rows", op="product", rows=16384, n=5120, k=5120, source="codes"),
        # the gradients of one small layer
        dict(name="clip 1 layer", op="clip", layers=1, features=512, hidden=512, experts=8, dtype="bf16", out="bf16", max_norm=1.0),
        # a model's gradients, clipped into the 32-bit ones that the optimizer takes
        dict(name="clip 16 layers", op="clip", layers=16, features=4096, hidden=4096, experts=64, dtype="bf16", out="f32", max_norm=1.0),
    ]


def _between(rng, low, high):
    """A whole number between the two, spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "product", "clip"])
    if op == "norm":
        features = rng.choice([128, 512, 1000, 1001, 1280, 2048, 2056, 4096, 5120, 8192])
        train = rng.random() < 0.5
        most = (8192 * 4096 if train else 16384 * 5120) // features
        return dict(op=op, rows=_between(rng, 1, min(16384, most)), features=features, residual=rng.choice(["none", "bf16", "f32"]),
                    weight=rng.choice(["bf16", "f32"]), copy=rng.random() < 0.5, train=train)
    if op == "swiglu":
        features = rng.choice([128, 512, 1000, 1001, 1280, 1408, 2048, 4096, 5120, 14336])
        train = rng.random() < 0.5
        return dict(op=op, rows=_between(rng, 1, min(16384, 8192 * 4096 // features)), features=features, copy=not train and rng.random() < 0.5, train=train)
    if op == "product":
        n = rng.choice([512, 1000, 1280, 1408, 2048, 4096, 5120, 14336])
        k = rng.choice([512, 1000, 1280, 1408, 2048, 4096, 5120, 8192])
        return dict(op=op, rows=_between(rng, 1, min(16384, 16384 * 5120 * 5120 // (n * k))), n=n, k=k, source=rng.choice(["codes", "rows", "norm"]))
    features, hidden = rng.choice([512, 1000, 2048, 4096]), rng.choice([512, 1001, 1408, 4096])
    dtype, out = rng.choice(["bf16", "f32"]), rng.choice(["none", "bf16", "f32"])
    layers = 16 * 3 * 4096 * 4096 * 6 // ((3 * features * hidden + 65 * features) * (_size(dtype) + _size(out)))
    return dict(op=op, layers=_between(rng, 1, min(24, layers)), features=features, hidden=hidden, experts=rng.choice([8, 64]), dtype=dtype,
                out=out, max_norm=rng.choice([1.0, 1.0, 1e9]))


def _cdiv(a, b):
    return -(-a // b)


def _size(name):
    return {"none": 0, "bf16": 2, "f32": 4}[name]


def _shapes(case):
    """The gradients of a model's layers: norm weight, router, gate and up, down."""
    H, F, E = case["features"], case["hidden"], case["experts"]
    return [(H,), (E, H), (2 * F, H), (H, F)] * case["layers"]


def work(case):
    if case["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        return {"bytes": n * (_size(case["dtype"]) + _size(case["out"])), "flops": 3 * n}
    T = case["rows"]
    if case["op"] == "product":
        N, K, b = case["n"], case["k"], case["n"] * (case["k"] + 4) + 2 * T * case["n"]
        b += {"codes": T * (K + 4), "rows": 2 * T * K, "norm": 6 * T * K + 2 * K}[case["source"]]
        return {"bytes": b, "flops": 2 * T * N * K}
    H = case["features"]
    codes = T * H + 4 * T * _cdiv(H, BLOCK)
    if case["op"] == "norm":
        r, w = _size(case["residual"]), _size(case["weight"])
        hs = r or 2
        b = T * H * (2 + 2 * r + (2 if case["copy"] else 0)) + codes + H * w
        if case["train"]:
            b += 4 * T + T * H + 4 * H * _cdiv(T, BLOCK) + T * H * (2 + 2 * hs) + H * w
        return {"bytes": b, "flops": T * H * (24 if case["train"] else 8)}
    if not case["train"]:
        return {"bytes": 4 * T * H + codes + (2 * T * H if case["copy"] else 0), "flops": 10 * T * H}
    return {"bytes": 4 * T * H + 2 * T * H + 3 * (codes + T * H + 4 * H * _cdiv(T, BLOCK)), "flops": 40 * T * H}


def _rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rows(T, n, dtype=torch.uint8):
    """A [T, n] buffer whose row stride is rounded up to 16 bytes, as the 8-bit products want it."""
    return torch.empty(T, _cdiv(n, 16) * 16, dtype=dtype, device=DEV)[:, :n]


def _scales(groups, n):
    return torch.empty(_cdiv(groups, BLOCK), n, device=DEV)


def _prepare_norm(s, g, T, H, residual, weight):
    x = _normal(g, T, H) * (0.5 + 1.5 * torch.rand(T, 1, generator=g, device=DEV))
    x[:, ::max(1, H // 13)] *= 12                     # a few channels that are always large
    s["x"] = x.to(torch.bfloat16)
    s["residual"] = None if residual == "none" else (2 * _normal(g, T, H)).to(DTYPES[residual])
    s["weight"] = (1 + 0.2 * _normal(g, H)).to(DTYPES[weight])
    s["h"] = None if residual == "none" else torch.empty_like(s["residual"])


def _prepare_clip(s, g, case):
    """Every gradient a view of one buffer, each beginning at a multiple of 128 values."""
    at, n = [], 0
    for shape in _shapes(case):
        at.append(n)
        n += _cdiv(math.prod(shape), BLOCK) * BLOCK
    flat = torch.zeros(n, dtype=DTYPES[case["dtype"]], device=DEV)
    out = None if case["out"] == "none" else torch.zeros(n, dtype=DTYPES[case["out"]], device=DEV)

    def views(buffer):
        return [buffer[a:a + math.prod(shape)].view(shape) for a, shape in zip(at, _shapes(case))]
    s["flat"], s["out"], s["grads"], s["outs"] = flat, out, views(flat), None if out is None else views(out)
    for i, t in enumerate(s["grads"]):
        t.copy_(_normal(g, *t.shape) * (0.002 * (1 + i % 5)))


def prepare(case, seed):
    g, op = _rng(seed), case["op"]
    s = {"case": case}
    if op == "clip":
        _prepare_clip(s, g, case)
        return s
    T = case["rows"]
    if op == "product":
        N, K = case["n"], case["k"]
        w = _normal(g, N, K) * (0.01 + 0.02 * torch.rand(N, 1, generator=g, device=DEV))
        top = w.abs().amax(1)
        s["b"], s["b_s"] = _rows(N, K, torch.int8), top / I8_MAX
        s["b"].copy_((w * (I8_MAX / top)[:, None]).round())
        del w
        s["a"], s["a_s"] = _rows(T, K, torch.int8), torch.empty(T, device=DEV)
        if case["source"] == "norm":
            _prepare_norm(s, g, T, K, "bf16", "bf16")
        else:
            x = (_normal(g, T, K) * (0.5 + 1.5 * torch.rand(T, 1, generator=g, device=DEV))).to(torch.bfloat16)
            if case["source"] == "rows":
                s["x"] = x
            else:
                top = x.float().abs().amax(1)
                s["a_s"].copy_(top / I8_MAX)
                s["a"].copy_((x.float() * (I8_MAX / top)[:, None]).round())
        s["c"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        return s
    H, train = case["features"], case["train"]
    s["q"], s["a_s"] = _rows(T, H), _scales(H, T)
    s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    if train:
        s["qT"], s["s"] = _rows(H, T), _scales(T, H)
        s["dy"] = (0.01 * _normal(g, T, H)).to(torch.bfloat16)
    if op == "swiglu":
        s["gu"] = (_normal(g, T, 2 * H) * (0.5 + 1.5 * torch.rand(T, 1, generator=g, device=DEV))).to(torch.bfloat16)
        if train:
            s["dq"], s["da_s"], s["dqT"], s["ds"] = _rows(T, 2 * H), _scales(2 * H, T), _rows(2 * H, T), _scales(T, 2 * H)
        return s
    _prepare_norm(s, g, T, H, case["residual"], case["weight"])
    s["rstd"] = torch.empty(T, device=DEV) if train else None
    if train:
        like = s["x"] if s["h"] is None else s["h"]
        s["dh"] = (0.01 * _normal(g, T, H)).to(like.dtype)
        s["dx"], s["dweight"] = torch.empty_like(like), torch.empty_like(s["weight"])
    return s


def run(s):
    case = s["case"]
    return (_OWN if own else _PLAIN)[case["op"]](s, case)


# ------------------------------------------------------------------ the package's calls

def _e4m3(q):
    return q.view(torch.float8_e4m3fn)


def _own_norm(s, c):
    import blockwise_scaled_fp8_act_amd as bf
    q, a_s, h, y, rstd = bf.rms_norm_quantize(s["x"], s["weight"], residual=s["residual"], eps=EPS, q=s["q"], s=s["a_s"], h=s["h"], y=s["y"],
                                              rstd=s["rstd"])
    if not c["train"]:
        return _e4m3(q), a_s, h, y
    kept = s["x"] if h is None else h
    qT, sT = bf.rms_norm_quantize_rhs(kept, s["weight"], rstd, qT=s["qT"], s=s["s"])
    dx, dweight = bf.rms_norm_backward(s["dy"], kept, s["weight"], rstd, dh=s["dh"], dx=s["dx"], dweight=s["dweight"])
    return _e4m3(q), a_s, h, y, rstd, _e4m3(qT), sT, dx, dweight


def _own_swiglu(s, c):
    import blockwise_scaled_fp8_act_amd as bf
    if not c["train"]:
        q, a_s, y = bf.swiglu_quantize(s["gu"], q=s["q"], s=s["a_s"], y=s["y"])
        return _e4m3(q), a_s, y
    q, a_s, qT, sT = bf.swiglu_quantize_lhs_and_rhs(s["gu"], q=s["q"], a_s=s["a_s"], qT=s["qT"], s=s["s"])
    dq, da_s, dqT, ds = bf.swiglu_backward_quantize(s["dy"], s["gu"], q=s["dq"], a_s=s["da_s"], qT=s["dqT"], s=s["ds"])
    return _e4m3(q), a_s, _e4m3(qT), sT, _e4m3(dq), da_s, _e4m3(dqT), ds


def _own_product(s, c):
    import blockwise_scaled_fp8_act_amd as bf
    a, a_s, h = s["a"], s["a_s"], None
    if c["source"] == "rows":
        bf.quantize_rows_i8(s["x"], q=a, s=a_s)
    elif c["source"] == "norm":
        h = bf.rms_norm_quantize(s["x"], s["weight"], residual=s["residual"], eps=EPS, fmt="int8", q=a, s=a_s, h=s["h"])[2]
    return bf.gemm_i8(a, a_s, s["b"], s["b_s"], c=s["c"]), h


def _own_clip(s, c):
    import blockwise_scaled_fp8_act_amd as bf
    if s["outs"] is None:
        return bf.grad_norm(s["grads"])
    return bf.clip_grads(s["grads"], c["max_norm"], out=s["outs"], eps=EPS), s["out"]


# ------------------------------------------------------------------ the plain forms

def _plain_lhs(v):
    """Codes and column-major scales of 1x128 groups."""
    T, H = v.shape
    groups = torch.nn.functional.pad(v, (0, -H % BLOCK)).view(T, -1, BLOCK)
    amax = groups.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (groups * (FP8_MAX / amax)[:, :, None]).clamp(-FP8_MAX, FP8_MAX).view(T, -1)[:, :H].to(torch.float8_e4m3fn)
    return q, (amax / FP8_MAX).t().contiguous()


def _plain_rhs(v):
    """Transposed codes and scales of 128x1 groups."""
    return _plain_lhs(v.t().contiguous())


def _plain_i8(v):
    amax = v.abs().amax(1).clamp_min(AMAX_FLOOR)
    return (v * (I8_MAX / amax)[:, None]).round(), amax / I8_MAX


def _plain_normed(s):
    """h as kept (None without a residual), its rows' factors, the normed rows."""
    h = None if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = (s["x"] if h is None else h).float()
    rstd = 1 / (v.square().mean(1) + EPS).sqrt()
    return h, rstd, v * rstd[:, None] * s["weight"].float()


def _plain_norm(s, c):
    h, rstd, v = _plain_normed(s)
    q, a_s = _plain_lhs(v)
    y = v.to(torch.bfloat16) if c["copy"] else None
    if not c["train"]:
        return q, a_s, h, y
    qT, sT = _plain_rhs(v)
    n = (s["x"] if h is None else h).float() * rstd[:, None]
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = s["dh"].float() + rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    return q, a_s, h, y, rstd, qT, sT, dx.to(s["dh"].dtype), (dy * n).sum(0).to(s["weight"].dtype)


def _plain_swiglu(s, c):
    F = c["features"]
    g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
    sig = 1 / (1 + (-g).exp())
    v = g * sig * u
    q, a_s = _plain_lhs(v)
    if not c["train"]:
        return q, a_s, v.to(torch.bfloat16) if c["copy"] else None
    dy = s["dy"].float()
    dgu = torch.cat([dy * u * sig * (1 + g * (1 - sig)), dy * g * sig], dim=1)
    return (q, a_s, *_plain_rhs(v), *_plain_lhs(dgu), *_plain_rhs(dgu))


def _plain_product(s, c):
    h = None
    if c["source"] == "codes":
        a, a_s = s["a"].float(), s["a_s"]
    elif c["source"] == "rows":
        a, a_s = _plain_i8(s["x"].float())
    else:
        h, _, v = _plain_normed(s)
        a, a_s = _plain_i8(v)
    return (a @ s["b"].float().t() * a_s[:, None] * s["b_s"]).to(torch.bfloat16), h


def _plain_clip(s, c):
    flat = s["flat"].float()                          # what lies between the gradients is zero
    norm = flat.square().sum().sqrt().view(1)
    if s["out"] is None:
        return norm
    factor = torch.where(norm.isfinite(), (c["max_norm"] / (norm + EPS)).clamp_max(1.0), 1.0)
    return norm, (flat * factor).to(s["out"].dtype)


_OWN = {"norm": _own_norm, "swiglu": _own_swiglu, "product": _own_product, "clip": _own_clip}
_PLAIN = {"norm": _plain_norm, "swiglu": _plain_swiglu, "product": _plain_product, "clip": _plain_clip}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)


def _exact_e4m3(v):
    """The nearest e4m3 value of numbers within +-448, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -9))).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_groups(v, along):
    """Codes and scales of groups of 128 along a dimension, group by group."""
    codes = torch.empty(v.shape, device=v.device)
    scales = []
    for lo in range(0, v.shape[along], BLOCK):
        part = v.narrow(along, lo, min(BLOCK, v.shape[along] - lo))
        top = torch.maximum(part.max(dim=along, keepdim=True).values, -part.min(dim=along, keepdim=True).values).clamp_min(AMAX_FLOOR)
        codes.narrow(along, lo, part.shape[along]).copy_(_exact_e4m3(part * (FP8_MAX / top)))
        scales.append((top / FP8_MAX).reshape(-1))
    return codes, torch.stack(scales)


def _exact_both(v):
    q, a_s = _exact_groups(v, 1)
    qT, s = _exact_groups(v, 0)
    return q, a_s, qT.t().contiguous(), s


def _exact_normed(s):
    if s["residual"] is None:
        h = None
        kept = s["x"].double()
    else:
        h = s["x"].double() + s["residual"].double()
        kept = h.to(s["residual"].dtype).double()     # the norm is that of the row as it is kept
    rstd = (torch.linalg.vector_norm(kept, dim=1) ** 2 / kept.shape[1] + EPS) ** -0.5
    return h, kept, rstd, kept * torch.outer(rstd, s["weight"].double())


def _exact_norm(s, c):
    h, kept, rstd, v = _exact_normed(s)
    y = v if c["copy"] else None
    if not c["train"]:
        return (*_exact_groups(v, 1), h, y)
    q, a_s, qT, sT = _exact_both(v)
    w, dy, H = s["weight"].double(), s["dy"].double(), kept.shape[1]
    # d rstd / d h = -rstd^3 h / H, by the chain rule through v = h rstd w
    dv = dy * w
    drstd = (dv * kept).sum(dim=1)
    dx = s["dh"].double() + dv * rstd[:, None] - kept * (drstd * rstd ** 3 / H)[:, None]
    return q, a_s, h, y, rstd, qT, sT, dx, torch.einsum("th,th,t->h", dy, kept, rstd)


def _exact_swiglu(s, c):
    gu = s["gu"].double()
    gate, up = gu.chunk(2, dim=1)
    sig = torch.sigmoid(gate)
    v = up * (gate * sig)
    if not c["train"]:
        return (*_exact_groups(v, 1), v if c["copy"] else None)
    dy = s["dy"].double()
    dsilu = sig + gate * sig * torch.sigmoid(-gate)
    return (*_exact_both(v), *_exact_both(torch.cat([dy * up * dsilu, dy * (gate * sig)], dim=1)))


def _exact_rint(v):
    top = v.abs().max(dim=1).values.clamp_min(AMAX_FLOOR)
    return torch.round(v / (top / I8_MAX)[:, None]), top / I8_MAX


def _exact_product(s, c):
    h = None
    if c["source"] == "codes":
        a, a_s = s["a"].double(), s["a_s"].double()
    elif c["source"] == "rows":
        a, a_s = _exact_rint(s["x"].double())
    else:
        h, _, _, v = _exact_normed(s)
        a, a_s = _exact_rint(v)
    return torch.outer(a_s, s["b_s"].double()) * (a @ s["b"].double().t()), h


def _exact_clip(s, c):
    total = np.sqrt(sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"]))
    norm = torch.tensor([total], dtype=torch.float64)
    if s["out"] is None:
        return norm
    factor = min(1.0, c["max_norm"] / (total + EPS))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    start = s["flat"].data_ptr()
    for t in s["grads"]:
        at = (t.data_ptr() - start) // t.element_size()
        out[at:at + t.numel()] = t.reshape(-1).double() * factor
    return norm, out


_EXACT = {"norm": _exact_norm, "swiglu": _exact_swiglu, "product": _exact_product, "clip": _exact_clip}
