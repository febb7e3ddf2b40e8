"""CPU: argument errors of the router, the plan and the rows' calls are found before anything touches a GPU."""
import ctypes as C

import pytest

import blockwise_fp8_zero_fold_amd as fz

EINVAL, ESHAPE = -1, -4
P = 0x1000  # never dereferenced: every call below is refused first


def router(**kw):
    d = dict(T=4, E=64, k=8, dtype=fz.F32, score=fz.SCORE_SOFTMAX, normalize=1, scale=1.0) | kw
    return C.byref(fz.Router(*d.values()))


def fwd(f, logits=P, bias=P, experts=P, weights=P):
    return fz.lib.fp8z1_route(f, logits, bias, experts, weights, None)


def bwd(f, logits=P, experts=P, dweights=P, dlogits=P):
    return fz.lib.fp8z1_route_bwd(f, logits, experts, dweights, dlogits, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), ESHAPE), (dict(T=2 ** 30 + 1), ESHAPE), (dict(E=0), ESHAPE), (dict(E=1025), ESHAPE), (dict(k=0), ESHAPE),
    (dict(k=33), ESHAPE), (dict(E=4, k=5), ESHAPE), (dict(dtype=fz.E4M3), EINVAL), (dict(score=2), EINVAL),
    (dict(score=-1), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL)])
def test_router_descriptions(bad, status):
    assert fwd(router(**bad)) == status and bwd(router(**bad)) == status
    assert fz.lib.fp8z1_last_error()


def test_router_pointers():
    assert fwd(None) == EINVAL and bwd(None) == EINVAL
    for bad in (dict(logits=None), dict(experts=None), dict(weights=None), dict(logits=P + 2), dict(bias=P + 2),
                dict(experts=P + 1), dict(weights=P + 2)):
        assert fwd(router(), **bad) == EINVAL, bad
    for bad in (dict(logits=None), dict(experts=None), dict(dweights=None), dict(dlogits=None), dict(dlogits=P + 2),
                dict(dweights=P + 2), dict(experts=P + 3)):
        assert bwd(router(), **bad) == EINVAL, bad
    assert fwd(router(dtype=fz.BF16), logits=P + 1) == EINVAL
    assert fwd(router(T=0), None, None, None, None) == 0 and bwd(router(T=0), None, None, None, None) == 0


def sort(T=4, k=2, E=8, experts=P, offsets=P, row_of=P, ws=None, n=0):
    return fz.lib.fp8z1_sort_tokens(T, k, E, experts, offsets, row_of, ws, n, None)


def test_sort_arguments():
    for bad, status in ((dict(T=-1), ESHAPE), (dict(T=2 ** 30 + 1), ESHAPE), (dict(T=2 ** 29, k=3), ESHAPE),
                        (dict(k=0), ESHAPE), (dict(k=33), ESHAPE), (dict(E=0), ESHAPE), (dict(E=1025), ESHAPE),
                        (dict(experts=None), EINVAL), (dict(offsets=None), EINVAL), (dict(row_of=None), EINVAL),
                        (dict(experts=P + 1), EINVAL), (dict(offsets=P + 2), EINVAL), (dict(row_of=P + 2), EINVAL),
                        (dict(T=100000), EINVAL), (dict(T=100000, ws=P, n=16), EINVAL),
                        (dict(T=100000, ws=P + 8, n=1 << 30), EINVAL)):
        assert sort(**bad) == status, bad
    n = C.c_size_t()
    q = fz.lib.fp8z1_sort_tokens_workspace_bytes
    assert q(4, 2, 8, None) == EINVAL and q(-1, 2, 8, C.byref(n)) == ESHAPE and q(4, 2, 2000, C.byref(n)) == ESHAPE
    assert fz.fp8z1_sort_tokens_workspace_bytes(4, 2, 8) == 0
    b = fz.fp8z1_sort_tokens_workspace_bytes(100000, 8, 256)
    assert b > 0 and b % (4 * 256) == 0
    # the most choices: counts of no more workgroups than the plan has
    assert fz.fp8z1_sort_tokens_workspace_bytes(2 ** 30, 1, 1024) <= 256 * 4 * 1024


def routed(**kw):
    d = dict(T=4, D=64, R=8, k=2, dtype=fz.BF16) | kw
    return C.byref(fz.Routed(*d.values()))


def calls(f, row_of=P, a=P, b=P, c=P):
    lib = fz.lib
    return {"dispatch": lib.fp8z1_dispatch(f, row_of, a, None, b, None, None),
            "combine": lib.fp8z1_combine(f, row_of, a, c, None, b, None),
            "combine_bwd": lib.fp8z1_combine_bwd(f, row_of, a, b, c, b, c, None)}


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), ESHAPE), (dict(T=2 ** 30 + 1), ESHAPE), (dict(D=0), ESHAPE), (dict(D=2 ** 20 + 1), ESHAPE),
    (dict(R=-1), ESHAPE), (dict(R=2 ** 30 + 1), ESHAPE), (dict(k=0), ESHAPE), (dict(k=33), ESHAPE), (dict(dtype=7), EINVAL)])
def test_rows_descriptions(bad, status):
    assert set(calls(routed(**bad)).values()) == {status}


def test_rows_pointers():
    assert set(calls(None).values()) == {EINVAL}
    for bad in (dict(row_of=None), dict(row_of=P + 2), dict(a=None), dict(a=P + 1), dict(b=None), dict(b=P + 1)):
        assert set(calls(routed(), **bad).values()) == {EINVAL}, bad
    lib = fz.lib
    assert lib.fp8z1_combine(routed(), P, P, P + 2, None, P, None) == EINVAL  # weights
    assert lib.fp8z1_combine(routed(), P, P, P, P + 1, P, None) == EINVAL  # base
    assert lib.fp8z1_combine(routed(dtype=fz.E4M3), P, P, P, None, P, None) == EINVAL
    assert lib.fp8z1_combine_bwd(routed(), P, P, P, None, P, P, None) == EINVAL  # no weights
    assert lib.fp8z1_combine_bwd(routed(), P, P, P, P, None, None, None) == EINVAL  # nothing wanted
    assert lib.fp8z1_combine_bwd(routed(), P, P, None, P, P, P, None) == EINVAL  # dweights without rows
    # scales go with 8-bit rows, both of them, and with nothing else
    assert lib.fp8z1_dispatch(routed(), P, P, P, P, None, None) == EINVAL
    assert lib.fp8z1_dispatch(routed(dtype=fz.E4M3), P, P, None, P, P, None) == EINVAL
    assert lib.fp8z1_dispatch(routed(dtype=fz.E4M3), P, P, P, P, None, None) == EINVAL
    assert lib.fp8z1_dispatch(routed(dtype=fz.E4M3), P, P, P + 2, P, P, None) == EINVAL
    assert set(calls(routed(T=0), None, None, None, P).values()) == {0}


def norm(**kw):
    d = dict(T=4, C=64, dtype=fz.BF16, res_dtype=fz.F32, gate=fz.GATE_NONE, eps=1e-6, res_scale=1.0, block_scale=1.0,
             weight_offset=0.0, reserved=0) | kw
    return C.byref(fz.Norm(*d.values()))


def norm8(f, y=P, res=P, w_post=P, gate=None, w_pre=P, z=P, n=P, codes=P, scales=P, rule=fz.SCALE_AMAX):
    return fz.lib.fp8z1_norm_join8(f, y, res, w_post, gate, w_pre, z, n, codes, scales, rule, None)


def test_norm8_arguments():
    assert norm8(None) == EINVAL
    for bad, status in ((dict(T=-1), ESHAPE), (dict(C=0), ESHAPE), (dict(C=16385), ESHAPE), (dict(dtype=fz.E4M3), EINVAL),
                        (dict(gate=fz.GATE_CHANNEL), EINVAL), (dict(eps=-1.0), EINVAL)):
        assert norm8(norm(**bad)) == status, bad
    for bad in (dict(res=None), dict(codes=None), dict(scales=None), dict(scales=P + 2), dict(rule=2), dict(rule=-1),
                dict(y=P + 1), dict(n=P + 1), dict(z=P + 2), dict(gate=P)):
        assert norm8(norm(), **bad) == EINVAL, bad
    assert norm8(norm(T=0), *[None] * 9) == 0
