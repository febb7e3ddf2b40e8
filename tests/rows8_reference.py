"""Rows in 8 bits by plain torch on the CPU: codes and scales of float32 rows, and what they stand for."""
import torch

from tests.block_reference import BLOCK


def groups(x):
    """[T, C] -> [T, ceil(C/128), 128], zeros behind the last column."""
    T, C = x.shape
    wide = torch.zeros(T, -(-C // BLOCK) * BLOCK, dtype=x.dtype)
    wide[:, :C] = x
    return wide.view(T, -1, BLOCK)


def quantize(x, pow2=False):
    """(codes uint8, scales float32) of float32 rows."""
    assert x.dtype == torch.float32
    g = groups(x)
    top = torch.nan_to_num(g.abs(), nan=0.0, posinf=float("inf")).amax(2)
    if pow2:
        e = torch.frexp(top.clamp(max=3.4e38)).exponent - 1 - 8
        scale = torch.where(torch.isinf(top), top, torch.ldexp(torch.ones_like(top), e.clamp(min=-126)))
    else:
        scale = top / 448.0
    scale = torch.where(top == 0, torch.ones_like(top), scale.clamp(min=2.0 ** -126))
    q = (g / scale[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous(), scale


def dequantize(codes, scales):
    wide = scales.double().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).double() * wide


def same_codes(a, b):
    """Equal, a NaN's sign aside."""
    a, b = a.cpu(), b.cpu()
    nan_a, nan_b = (a & 0x7F) == 0x7F, (b & 0x7F) == 0x7F
    return bool(((a == b) | (nan_a & nan_b)).all()) and bool((nan_a == nan_b).all())


def make_rows8(g, T, C, lo=-2.0, hi=2.0):
    """Random finite codes (all of them occur) and group scales 2^lo .. 2^hi / 64."""
    codes = torch.randint(0, 256, (T, C), generator=g, dtype=torch.int16).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    scales = 2.0 ** (torch.rand(T, -(-C // BLOCK), generator=g) * (hi - lo) + lo) / 64
    return codes, scales.float()
