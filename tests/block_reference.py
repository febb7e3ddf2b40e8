"""Float64 references of the feed-forward block and the norm join, with the error that a float32
computation rounded once to the output type may have (first-order bounds, counted per
operation).  Plain torch on the CPU; nothing of the library is used."""
import math

import torch

U32 = 2.0 ** -24  # unit roundoff of float32
BLOCK = 128


def half_step(dtype):
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def floor_step(dtype):
    """Largest absolute error of one rounding among the subnormals of `dtype`."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def dequantize(codes, scales):
    R, C = codes.shape[1:]
    wide = scales.double().repeat_interleave(BLOCK, 1)[:, :R].repeat_interleave(BLOCK, 2)[:, :, :C]
    return codes.view(torch.float8_e4m3fn).double() * wide


def make_weight(g, E, R, C, lo=-3.0, hi=3.0):
    """Random finite codes (all of them occur) and block scales 2^lo .. 2^hi / (16 sqrt(C))."""
    codes = torch.randint(0, 256, (E, R, C), generator=g, dtype=torch.int16).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    rb, cb = -(-R // BLOCK), -(-C // BLOCK)
    scales = 2.0 ** (torch.rand(E, rb, cb, generator=g) * (hi - lo) + lo) / (64 * C ** 0.5)
    return codes, scales.float()


def make_offsets(g, T, E):
    """Ascending from 0 to T; with more than two experts the second has no rows."""
    cuts = torch.sort(torch.randint(0, T + 1, (E - 1,), generator=g)).values
    if E > 2:
        cuts[1] = cuts[0]
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), T)]).to(torch.int32)


def runs(offsets, T):
    if offsets is None:
        return [(0, 0, T)]
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def grouped(x, w, offsets, transposed):
    """Per expert x w^T (or x w with `transposed`), and the sum of the products' magnitudes."""
    N = w.shape[2] if transposed else w.shape[1]
    out = torch.zeros(x.shape[0], N, dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e, lo, hi in runs(offsets, x.shape[0]):
        m = w[e] if transposed else w[e].t()
        out[lo:hi] = x[lo:hi].double() @ m
        mag[lo:hi] = x[lo:hi].double().abs() @ m.abs()
    return out, mag


def sum_error(mag, n):
    """Of a float32 sum of n products (in any order, each rounding counted twice, and the block
    scales' multiplications)."""
    return (2 * n + 8) * U32 * mag


def act_value(act, h):
    if act == "silu":
        return h * torch.sigmoid(h)
    return h * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3))


def act_slope(act, h):
    h = h.clone().requires_grad_()
    return torch.autograd.grad(act_value(act, h).sum(), h)[0]


def act_error(act, h):
    """Of act(h) and of its slope in float32: the exponential's argument v carries a few roundings,
    which move the logistic function s(v) by s (1 - s) times their size; then a few more."""
    v = h if act == "silu" else 2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)
    s = torch.sigmoid(v)
    dv = torch.ones_like(h) if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * h * h)
    ds = U32 * (8 * v.abs() * s * (1 - s) + 8 * s)
    value = h.abs() * ds + 4 * U32 * (h * s).abs()
    # s(1 - s) also carries the rounding of 1 - s
    slope = ds + h.abs() * dv * (ds + U32 * s + 16 * U32 * s * (1 - s))
    return value, slope + 4 * U32


def rounded(exact, before, dtype):
    """The bound after one rounding to `dtype` of a value within `before` of `exact`."""
    return before + (exact.abs() + before) * half_step(dtype) + floor_step(dtype)


def check(got, exact, bound, what):
    """Every element within its bound; infinities and NaN where the reference has them."""
    got = got.detach().cpu().double()
    assert got.shape == exact.shape, (what, got.shape, exact.shape)
    fine = torch.isfinite(exact)
    assert torch.equal(torch.isnan(got), torch.isnan(exact)), f"{what}: NaN in other places"
    inf = torch.isinf(exact)
    assert torch.equal(got[inf], exact[inf]), f"{what}: infinities"
    if fine.any():
        over = ((got - exact).abs() - bound)[fine]
        i = int(over.argmax())
        assert float(over.max()) <= 0, (what, "off by", float((got - exact).abs()[fine][i]), "allowed",
                                        float(bound.expand_as(exact)[fine][i]), "value", float(exact[fine][i]))
