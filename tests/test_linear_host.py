"""CPU: argument errors of the products with an epilogue and of 8-bit rows are found before anything touches a GPU."""
import ctypes as C

import pytest

import blockwise_fp8_zero_fold_amd as fz

EINVAL, ESHAPE = -1, -4
P = 0x1000  # never dereferenced: every call below is refused first


def product(**kw):
    d = dict(T=4, E=2, N=64, K=32, dtype=fz.BF16, x_dtype=fz.E4M3, act=fz.ACT_NONE, reserved=0) | kw
    return C.byref(fz.Product(*d.values()))


def fwd(f, x=P, x_scales=P, codes=P, scales=P, offsets=P, bias=P, res=P, y=P, p=P, ws=None, n=0):
    return fz.lib.fp8z1_linear(f, x, x_scales, codes, scales, offsets, bias, res, y, p, ws, n, None)


def bwd(f, dy=P, p=P, codes=P, scales=P, offsets=P, dp=P, dbias=P, dx=P, ws=P, n=1 << 30):
    return fz.lib.fp8z1_linear_bwd(f, dy, p, codes, scales, offsets, dp, dbias, dx, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), ESHAPE), (dict(T=2 ** 30 + 1), ESHAPE), (dict(E=0), ESHAPE), (dict(E=65536), ESHAPE), (dict(N=0), ESHAPE),
    (dict(K=0), ESHAPE), (dict(N=2 ** 20 + 1), ESHAPE), (dict(K=2 ** 20 + 1), ESHAPE), (dict(dtype=fz.F32), EINVAL),
    (dict(dtype=fz.E4M3), EINVAL), (dict(x_dtype=fz.F16), EINVAL), (dict(x_dtype=fz.F32), EINVAL), (dict(act=3), EINVAL),
    (dict(act=-1), EINVAL)])
def test_product_descriptions(bad, status):
    assert fwd(product(**bad)) == status and bwd(product(**bad)) == status
    n = C.c_size_t()
    assert fz.lib.fp8z1_linear_workspace_bytes(product(**bad), C.byref(n)) == status
    assert fz.lib.fp8z1_linear_bwd_workspace_bytes(product(**bad), C.byref(n)) == status


def test_linear_pointers():
    assert fwd(None) == EINVAL and bwd(None) == EINVAL
    for bad in (dict(x=None), dict(x_scales=None), dict(codes=None), dict(scales=None), dict(offsets=None), dict(y=None),
                dict(x_scales=P + 2), dict(scales=P + 1), dict(offsets=P + 2), dict(bias=P + 2), dict(res=P + 1),
                dict(y=P + 1), dict(p=P + 1), dict(ws=P + 8, n=1 << 30)):
        assert fwd(product(), **bad) == EINVAL, bad
    half = product(x_dtype=fz.BF16)
    assert fwd(half, x=P + 1, x_scales=None) == EINVAL and fwd(half) == EINVAL  # (scales without 8-bit rows)
    assert fwd(half, x=None, x_scales=None) == EINVAL
    for bad in (dict(dy=None), dict(dy=P + 1), dict(codes=None), dict(scales=None), dict(offsets=None), dict(dp=P + 1),
                dict(dx=P + 1), dict(dbias=P + 2), dict(ws=None), dict(n=16), dict(ws=P + 8), dict(dp=None, dbias=None, dx=None)):
        assert bwd(product(), **bad) == EINVAL, bad
    act = product(act=fz.ACT_SILU)
    assert bwd(act, p=None) == EINVAL and bwd(act, dp=None) == EINVAL
    assert fwd(product(T=0), None, None, P, P, P, None, None, None, None) == 0


def test_linear_workspaces():
    n = C.c_size_t()
    for q in (fz.lib.fp8z1_linear_workspace_bytes, fz.lib.fp8z1_linear_bwd_workspace_bytes):
        assert q(None, C.byref(n)) == EINVAL and q(product(), None) == EINVAL
    assert fz.lib.fp8z1_linear_workspace_bytes(product(), C.byref(n)) == 0 and n.value == 0  # nothing to split
    assert fz.lib.fp8z1_linear_workspace_bytes(product(K=7168), C.byref(n)) == 0 and n.value == 0  # few rows: no tiles
    assert fz.lib.fp8z1_linear_workspace_bytes(product(T=100, K=7168), C.byref(n)) == 0 and n.value > 0
    assert fz.lib.fp8z1_linear_workspace_bytes(product(K=7168, x_dtype=fz.BF16), C.byref(n)) == 0 and n.value > 0
    # sums of 16 rows each of the bias's gradient
    assert fz.lib.fp8z1_linear_bwd_workspace_bytes(product(), C.byref(n)) == 0 and n.value == 2 * 64 * 4
    assert fz.lib.fp8z1_linear_bwd_workspace_bytes(product(T=0), C.byref(n)) == 0 and n.value == 0


def ffn(**kw):
    d = dict(T=4, E=2, D=64, F=32, dtype=fz.BF16, act=fz.ACT_SILU) | kw
    return C.byref(fz.Ffn(*d.values()))


def up8(f, x=P, xs=P, codes=P, scales=P, offsets=P, h=P, u=P, a=P, a_scales=P, rule=fz.SCALE_AMAX, ws=None, n=0):
    return fz.lib.fp8z1_ffn_up8(f, x, xs, codes, scales, codes, scales, offsets, h, u, a, a_scales, rule, ws, n, None)


def test_up8_arguments():
    for bad, status in ((dict(T=-1), ESHAPE), (dict(E=0), ESHAPE), (dict(D=0), ESHAPE), (dict(F=2 ** 20 + 1), ESHAPE),
                        (dict(dtype=fz.E4M3), EINVAL), (dict(act=fz.ACT_NONE), EINVAL)):
        assert up8(ffn(**bad)) == status, bad
    assert up8(None) == EINVAL
    for bad in (dict(x=None), dict(xs=None), dict(codes=None), dict(scales=None), dict(offsets=None), dict(a=None),
                dict(a_scales=None), dict(h=None), dict(u=None), dict(xs=P + 2), dict(scales=P + 2), dict(a_scales=P + 1),
                dict(h=P + 1), dict(offsets=P + 2), dict(rule=2), dict(ws=P + 4, n=1 << 30)):
        assert up8(ffn(), **bad) == EINVAL, bad
    n = C.c_size_t()
    q = fz.lib.fp8z1_ffn_up8_workspace_bytes
    assert q(None, C.byref(n)) == EINVAL and q(ffn(), None) == EINVAL and q(ffn(F=0), C.byref(n)) == ESHAPE
    assert q(ffn(), C.byref(n)) == 0 and n.value == 2 * 4 * 4 * 32  # float32 sums of gate and up
    assert up8(ffn(T=0), None, None, P, P, P, None, None, None, None) == 0
