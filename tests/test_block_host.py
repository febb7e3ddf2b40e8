"""CPU: argument errors of the feed-forward and norm calls are found before anything touches a GPU, and
the struct layouts match the header's."""
import ctypes as C

import pytest

import blockwise_fp8_zero_fold_amd as fz

EINVAL, ESHAPE = -1, -4
P = 0x1000  # never dereferenced: every call below is refused first


def ffn(**kw):
    d = dict(T=4, E=2, D=64, F=32, dtype=fz.BF16, act=fz.ACT_SILU) | kw
    return C.byref(fz.Ffn(*d.values()))


def calls(f, offsets=P, codes=P, scales=P, rows=P):
    lib = fz.lib
    return {
        "up": lib.fp8z1_ffn_up(f, rows, codes, scales, codes, scales, offsets, None, None, rows, None, 0, None),
        "down": lib.fp8z1_ffn_down(f, rows, codes, scales, offsets, rows, None, 0, None),
        "down_bwd": lib.fp8z1_ffn_down_bwd(f, rows, codes, scales, rows, rows, offsets, rows, rows, None, None, 0, None),
        "up_bwd": lib.fp8z1_ffn_up_bwd(f, rows, rows, codes, scales, codes, scales, offsets, rows, None, 0, None),
    }


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), ESHAPE), (dict(T=2 ** 30 + 1), ESHAPE), (dict(E=0), ESHAPE), (dict(E=65536), ESHAPE),
    (dict(D=0), ESHAPE), (dict(F=0), ESHAPE), (dict(D=2 ** 20 + 1), ESHAPE), (dict(F=2 ** 20 + 1), ESHAPE),
    (dict(dtype=fz.F32), EINVAL), (dict(dtype=fz.E4M3), EINVAL), (dict(act=2), EINVAL), (dict(act=-1), EINVAL)])
def test_ffn_descriptions(bad, status):
    assert set(calls(ffn(**bad)).values()) == {status}
    assert fz.lib.fp8z1_last_error()


@pytest.mark.parametrize("bad", [dict(offsets=None), dict(codes=None), dict(scales=None), dict(rows=None),
                                 dict(offsets=P + 2), dict(scales=P + 1), dict(rows=P + 1)])
def test_ffn_pointers(bad):
    assert set(calls(ffn(), **bad).values()) == {EINVAL}
    assert set(calls(None).values()) == {EINVAL}


def test_ffn_up_keeps_both_projections_or_none():
    assert fz.lib.fp8z1_ffn_up(ffn(), P, P, P, P, P, P, P, None, P, None, 0, None) == EINVAL
    assert fz.lib.fp8z1_ffn_up(ffn(), P, P, P, P, P, P, None, P, P, None, 0, None) == EINVAL


def test_no_rows_is_no_work():
    f = ffn(T=0)
    assert set(calls(f, rows=None).values()) == {0}


def test_ffn_workspace():
    n = C.c_size_t()
    q = fz.lib.fp8z1_ffn_workspace_bytes
    assert q(None, C.byref(n)) == EINVAL and q(ffn(), None) == EINVAL and q(ffn(D=0), C.byref(n)) == ESHAPE
    assert q(ffn(), C.byref(n)) == 0 and n.value == 0  # sums of 64 and 2 x 32: nothing to split
    assert q(ffn(D=7168), C.byref(n)) == 0 and n.value > 0
    lib = fz.lib
    assert lib.fp8z1_ffn_down(ffn(), P, P, P, P, P, P + 4, 1 << 30, None) == EINVAL  # misaligned workspace


def wgrad(T=8, E=1, M=16, N=16, dtype=fz.BF16, p=P, q=P, offsets=P, out=fz.F32, dw=P, acc=0, ws=None, n=0):
    return fz.lib.fp8z1_ffn_wgrad(T, E, M, N, dtype, p, q, offsets, out, dw, acc, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), ESHAPE), (dict(E=0), ESHAPE), (dict(M=0), ESHAPE), (dict(N=2 ** 20 + 1), ESHAPE),
    (dict(E=65535, M=2 ** 20, N=2 ** 20), ESHAPE),
    (dict(dtype=fz.F32), EINVAL), (dict(out=fz.F16), EINVAL), (dict(out=fz.BF16, acc=1), EINVAL), (dict(p=None), EINVAL),
    (dict(q=None), EINVAL), (dict(dw=None), EINVAL), (dict(E=2, offsets=None), EINVAL), (dict(p=P + 1), EINVAL),
    (dict(dw=P + 2), EINVAL), (dict(offsets=P + 2), EINVAL), (dict(ws=P + 2, n=64), EINVAL)])
def test_wgrad_arguments(bad, status):
    assert wgrad(**bad) == status


def test_three_gradients_arguments():
    def call(f, x=P, offsets=P, out=fz.F32, dw=P, acc=0, ws=None):
        return fz.lib.fp8z1_ffn_bwd_weights(f, x, P, P, P, P, offsets, out, dw, P, P, acc, ws, 0, None)

    assert call(None) == EINVAL
    for bad in (dict(x=None), dict(x=P + 1), dict(offsets=None), dict(offsets=P + 1), dict(out=fz.F16), dict(dw=None),
                dict(dw=P + 2), dict(out=fz.BF16, acc=1), dict(ws=P + 2)):
        assert call(ffn(), **bad) == EINVAL, bad
    for bad in (dict(T=-1), dict(E=0), dict(D=0), dict(F=2 ** 20 + 1), dict(E=65535, D=2 ** 20, F=2 ** 20)):
        assert call(ffn(**bad)) == ESHAPE, bad
    assert call(ffn(dtype=fz.F32)) == EINVAL
    n = C.c_size_t()
    q = fz.lib.fp8z1_ffn_bwd_weights_workspace_bytes
    assert q(None, C.byref(n)) == EINVAL and q(ffn(), None) == EINVAL and q(ffn(D=0), C.byref(n)) == ESHAPE
    assert q(ffn(E=1, T=100000), C.byref(n)) == 0 and n.value and n.value % (3 * 4 * 64 * 32) == 0


def test_wgrad_workspace():
    n = C.c_size_t(7)
    q = fz.lib.fp8z1_ffn_wgrad_workspace_bytes
    assert q(8, 1, 16, 16, None) == EINVAL
    assert q(8, 0, 16, 16, C.byref(n)) == ESHAPE
    assert fz.fp8z1_ffn_wgrad_workspace_bytes(8, 1, 16, 16) == 0
    # a long sum into few tiles is split: whole copies of the float32 output
    b = fz.fp8z1_ffn_wgrad_workspace_bytes(100000, 1, 64, 64)
    assert b > 0 and b % (4 * 64 * 64) == 0


def norm(**kw):
    d = dict(T=4, C=64, dtype=fz.BF16, res_dtype=fz.F32, gate=fz.GATE_NONE, eps=1e-6, res_scale=1.0, block_scale=1.0,
             weight_offset=0.0, reserved=0) | kw
    return C.byref(fz.Norm(*d.values()))


def fwd(f, y=P, res=P, w_post=P, gate=None, w_pre=P, z=P, n=P):
    return fz.lib.fp8z1_norm_join(f, y, res, w_post, gate, w_pre, z, n, None)


def bwd(f, dz=P, dn=P, y=P, z=P, w_post=P, gate=None, w_pre=P, dy=P, dres=P, dw_post=P, dgate=None, dw_pre=P, ws=P,
        n=1 << 30):
    return fz.lib.fp8z1_norm_join_bwd(f, dz, dn, y, z, w_post, gate, w_pre, dy, dres, dw_post, dgate, dw_pre, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), ESHAPE), (dict(C=0), ESHAPE), (dict(C=16385), ESHAPE), (dict(dtype=fz.E4M3), EINVAL),
    (dict(res_dtype=fz.F16), EINVAL), (dict(dtype=fz.F32, res_dtype=fz.BF16), EINVAL), (dict(gate=4), EINVAL),
    (dict(gate=-1), EINVAL), (dict(gate=fz.GATE_CHANNEL), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL)])
def test_norm_descriptions(bad, status):
    assert fwd(norm(**bad)) == status
    assert bwd(norm(**bad)) == status


def test_norm_pointers():
    assert fwd(None) == EINVAL and bwd(None) == EINVAL
    for bad in (dict(res=None), dict(z=None, n=None), dict(gate=P), dict(y=None), dict(y=P + 1), dict(res=P + 2),
                dict(w_post=P + 2), dict(n=P + 1)):
        assert fwd(norm(), **bad) == EINVAL, bad
    for bad in (dict(dz=None, dn=None), dict(z=None), dict(y=None), dict(y=None, w_post=None), dict(w_post=None),
                dict(w_pre=None), dict(dgate=P), dict(ws=None), dict(n=16), dict(ws=P + 4), dict(dres=P + 2)):
        assert bwd(norm(), **bad) == EINVAL, bad
    assert bwd(norm(gate=fz.GATE_CHANNEL), gate=P, dgate=P + 2) == EINVAL


def test_norm_workspace():
    n = C.c_size_t()
    q = fz.lib.fp8z1_norm_join_bwd_workspace_bytes
    assert q(None, C.byref(n)) == EINVAL and q(norm(), None) == EINVAL and q(norm(C=0), C.byref(n)) == ESHAPE
    assert q(norm(), C.byref(n)) == 0 and n.value >= 3 * 4 * 64
    assert fwd(norm(T=0), y=None, res=None, w_post=None, z=None, n=None) == 0
