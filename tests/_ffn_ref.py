"""References and buffers for the operators between the 8-bit products: plain formulas on the CPU, outputs
with guard bands, and the codes of given fp32 values."""
import torch

BLOCK = 128
U = 2.0 ** -24          # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SENTINEL = {torch.bfloat16: -7.0, torch.float32: -7.0, torch.uint8: 0xA5, torch.int8: 0x5A}


class Guarded:
    """A [rows, cols] view of row stride ld, `shift` elements into its buffer, sentinels all around."""

    def __init__(self, rows, cols, dtype, device, ld=None, shift=0, fill=None):
        ld = cols if ld is None else ld
        self.buf = torch.full((shift + (rows + 2) * ld + 64,), SENTINEL[dtype], dtype=dtype, device=device)
        self.view = self.buf[shift + ld:].as_strided((rows, cols), (ld, 1))
        if fill is not None:
            self.view.copy_(fill)

    def host(self):
        """The view's values, after a look at what surrounds them."""
        inside = torch.zeros(self.buf.shape, dtype=torch.bool)
        inside.as_strided(self.view.shape, self.view.stride(), self.view.storage_offset()).fill_(True)
        around = self.buf.cpu()[~inside]
        assert (around == SENTINEL[self.buf.dtype]).all(), "written outside the output"
        return self.view.cpu()


def lhs_codes(v, fmt="e4m3fn"):
    """(codes uint8 [T, H], scales (Hb, T)) of fp32 values, by the quantizers' arithmetic in fp32."""
    T, H = v.shape
    top = {"e4m3fn": 448.0, "e4m3fnuz": 240.0}[fmt]
    g = torch.nn.functional.pad(v, (0, -H % BLOCK)).view(T, -1, BLOCK)
    amax = g.abs().amax(2).clamp_min(1e-12)
    p = g * (torch.tensor(top) / amax)[:, :, None]
    q = p.clamp(-top, top).view(T, -1)[:, :H]
    q = q.to(torch.float8_e4m3fn if fmt == "e4m3fn" else torch.float8_e4m3fnuz).view(torch.uint8)
    return q, (amax / top).t().contiguous()


def rhs_codes(v, fmt="e4m3fn"):
    return lhs_codes(v.t().contiguous(), fmt)


def i8_codes(v):
    amax = v.abs().amax(1).clamp_min(1e-12) if v.shape[1] else torch.full((v.shape[0],), 1e-12)
    return (v * (torch.tensor(127.0) / amax)[:, None]).round().to(torch.int8), amax / 127.0


def normed(h, rstd, weight):
    """fl(fl(h rstd) weight) of what the kernel kept."""
    return (h.float() * rstd[:, None]) * weight.float()


def swiglu64(gu):
    """silu(gate) up in 64 bits; the gate's sigmoid without overflow."""
    F = gu.shape[1] // 2
    g, u = gu[:, :F].double(), gu[:, F:].double()
    return g * torch.sigmoid(g) * u


def swiglu_grad64(dy, gu):
    F = gu.shape[1] // 2
    g, u, d = gu[:, :F].double(), gu[:, F:].double(), dy.double()
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    return torch.cat([d * u * s * (1 + g * r), d * g * s], dim=1)


def codes_hold(q, s, v, per, top, half, least, slack, names=""):
    """Codes q (as numbers) of the fp64 values v with scales s spread over the elements (``per``): each is a
    nearest code of v / s to `slack` relative, where a step is `half` of the value (at least `least`)."""
    sc = per(s.double())
    p = v / sc
    off = (q.double() - p.clamp(-top, top)).abs()
    bound = torch.maximum(p.abs() * half, torch.full_like(p, least)) + p.abs() * slack + 1e-30
    assert (off <= bound).all(), (names, float((off - bound).max()))
