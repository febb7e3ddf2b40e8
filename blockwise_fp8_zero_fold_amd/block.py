"""The feed-forward block on the shard step's FP8 weights, and the norms around it:
allocation of outputs and call order only; all arithmetic runs in libfp8z1.

A weight is a pair ``(codes [E,R,C] uint8, scales [E,ceil(R/128),ceil(C/128)] float32)`` as
``Shard.unfold`` writes it.  Gate and up weights are [E,F,D], the down weight [E,D,F].
Rows (tokens) are sorted by expert: ``offsets`` [E+1] int32 on the device holds each
expert's first row, from 0 to T; None means one expert.  Outputs' rows that no expert covers hold whatever
their memory held.  Everything runs on torch's current stream.

Products are summed in float32 (but ``linear`` of 8-bit rows, see there); the results, the inner ones too (``a`` between
up and down, ``dh`` and ``du`` before ``dx``), are rounded to the activations' 16 bits.  The sums hold
activation * code before the block's scale: magnitudes of activations and gradients stay below 2^56.

A training step over one block (see ``examples/train_ffn_layer.py``):

    z, x = norm_join(y_before, res, ...)
    y, (h, u, a) = ffn_forward(x, w_gate, w_up, w_down, offsets, save=True)
    ...
    dx, dh, du, a = ffn_backward_data(dy, h, u, w_gate, w_up, w_down, offsets)
    dw_gate, dw_up, dw_down = ffn_backward_weights(x, a, dy, dh, du, n_experts=E, offsets=offsets)
    grads = norm_join_backward(dz, dx, y_before, z, ...)
    shard.step(hp, [dw_gate, dw_up, dw_down], codes, scales)
"""
from __future__ import annotations

import functools
from typing import Dict, Optional, Sequence, Tuple, Union

import torch

from . import _lib as L

Weight = Tuple[torch.Tensor, torch.Tensor]
Rows8 = Tuple[torch.Tensor, torch.Tensor]  # codes [T,C] uint8, scales [T,ceil(C/128)] float32

_ACT = {"silu": L.ACT_SILU, "gelu": L.ACT_GELU}
_CODE = {torch.float32: L.F32, torch.bfloat16: L.BF16, torch.float16: L.F16}
_HALF = (torch.bfloat16, torch.float16)
_SCALE = {"amax": L.SCALE_AMAX, "pow2": L.SCALE_POW2}


def _fail(msg: str):
    raise L.Fp8z1Error(msg)


def _device(x: torch.Tensor, what: str) -> int:
    """The current device's index; the library launches there, on torch's current stream."""
    dev = x.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _fail(f"{what}: tensors must be on the current device, not {x.device}")
    return dev


def _check(x: torch.Tensor, dev: int, dtype: torch.dtype, shape: Tuple[int, ...], what: str) -> int:
    """The address of a contiguous tensor of this type and shape on this device."""
    if x.shape != shape or x.dtype != dtype or x.get_device() != dev or not x.is_contiguous():
        _fail(f"{what}: {x.dtype} {tuple(x.shape)} on {x.device}{'' if x.is_contiguous() else ', not contiguous'}; "
              f"expected a contiguous {dtype} {tuple(shape)} on device {dev}")
    return x.data_ptr()


@functools.lru_cache(maxsize=256)
def _ffn_workspace(T: int, E: int, D: int, F: int) -> int:
    return L.fp8z1_ffn_workspace_bytes(L.Ffn(T, E, D, F, L.BF16, L.ACT_SILU))


@functools.lru_cache(maxsize=256)
def _norm_workspace(T: int, C: int) -> int:
    return L.fp8z1_norm_join_bwd_workspace_bytes(L.Norm(T, C, L.F32, L.F32, L.GATE_NONE, 0.0, 1.0, 1.0, 0.0, 0))


@functools.lru_cache(maxsize=256)
def _weights_workspace(T: int, E: int, D: int, F: int) -> int:
    return L.fp8z1_ffn_bwd_weights_workspace_bytes(L.Ffn(T, E, D, F, L.BF16, L.ACT_SILU))


_wgrad_workspace = functools.lru_cache(maxsize=256)(L.fp8z1_ffn_wgrad_workspace_bytes)


def _weight(w: Weight, dev: int, e: int, r: int, c: int, what: str) -> Tuple[int, int]:
    return (_check(w[0], dev, torch.uint8, (e, r, c), what),
            _check(w[1], dev, torch.float32, (e, -(-r // 128), -(-c // 128)), what))


def _offsets(offsets: Optional[torch.Tensor], dev: int, E: int, what: str) -> Optional[int]:
    if offsets is None:
        if E != 1:
            _fail(f"{what}: {E} experts need offsets")
        return None
    return _check(offsets, dev, torch.int32, (E + 1,), f"{what} offsets")


def _ffn(x: torch.Tensor, w_gate: Weight, act: str, what: str):
    """Device, sizes and their description for the calls; x [T, D], gate codes [E, F, D]."""
    if x.dim() != 2 or w_gate[0].dim() != 3:
        _fail(f"{what}: rows must be [T, D] and codes [E, F, D]")
    if x.dtype not in _HALF:
        _fail(f"{what}: dtype {x.dtype}, expected torch.bfloat16 or torch.float16")
    if act not in _ACT:
        _fail(f"{what}: act {act!r}, expected one of {', '.join(_ACT)}")
    T, D = x.shape
    E, F, _ = w_gate[0].shape
    return _device(x, what), T, D, E, F, L.Ffn(T, E, D, F, _CODE[x.dtype], _ACT[act])


def _empty(like: torch.Tensor, *shape: int) -> torch.Tensor:
    return like.new_empty(shape)


def _scratch(like: torch.Tensor, nbytes: int) -> Optional[torch.Tensor]:
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _empty8(like: torch.Tensor, T: int, C: int) -> Rows8:
    return like.new_empty((T, C), dtype=torch.uint8), like.new_empty((T, -(-C // 128)), dtype=torch.float32)


def _scale_rule(name: str, what: str) -> int:
    if name not in _SCALE:
        _fail(f"{what}: scale_rule {name!r}, expected one of {', '.join(_SCALE)}")
    return _SCALE[name]


def ffn_forward(x: torch.Tensor, w_gate: Weight, w_up: Weight, w_down: Weight,
                offsets: Optional[torch.Tensor] = None, act: str = "silu", save: bool = False):
    """y [T,D] = (act(x Wg^T) * (x Wu^T)) Wd^T.  Returns (y, (h, u, a)) with ``save``, else (y, None)."""
    what = "ffn_forward"
    dev, T, D, E, F, f = _ffn(x, w_gate, act, what)
    px = _check(x, dev, x.dtype, (T, D), what)
    gate, up, down = (_weight(w_gate, dev, E, F, D, "ffn_forward gate"), _weight(w_up, dev, E, F, D, "ffn_forward up"),
                      _weight(w_down, dev, E, D, F, "ffn_forward down"))
    off = _offsets(offsets, dev, E, what)
    a, y = _empty(x, T, F), _empty(x, T, D)
    h, u = (_empty(x, T, F), _empty(x, T, F)) if save else (None, None)
    n = _ffn_workspace(T, E, D, F)
    ws = _scratch(x, n)
    pw, pa, stream = L._ptr(ws), a.data_ptr(), L._current_stream(dev)
    L._check(L.lib.fp8z1_ffn_up(f, px, *gate, *up, off, L._ptr(h), L._ptr(u), pa, pw, n, stream), what)
    L._check(L.lib.fp8z1_ffn_down(f, pa, *down, off, y.data_ptr(), pw, n, stream), what)
    return y, ((h, u, a) if save else None)


def ffn_backward_data(dy: torch.Tensor, h: torch.Tensor, u: torch.Tensor, w_gate: Weight, w_up: Weight,
                      w_down: Weight, offsets: Optional[torch.Tensor] = None, act: str = "silu"):
    """(dx, dh, du, a): the gradients at the block's input and its projections, and a again, from the kept
    (rounded) h and u (what the weight gradients need)."""
    what = "ffn_backward_data"
    dev, T, D, E, F, f = _ffn(dy, w_gate, act, what)
    py = _check(dy, dev, dy.dtype, (T, D), what)
    ph, pu = (_check(v, dev, dy.dtype, (T, F), f"{what} projections") for v in (h, u))
    gate, up, down = (_weight(w_gate, dev, E, F, D, f"{what} gate"), _weight(w_up, dev, E, F, D, f"{what} up"),
                      _weight(w_down, dev, E, D, F, f"{what} down"))
    off = _offsets(offsets, dev, E, what)
    dh, du, a, dx = _empty(dy, T, F), _empty(dy, T, F), _empty(dy, T, F), _empty(dy, T, D)
    n = _ffn_workspace(T, E, D, F)
    ws = _scratch(dy, n)
    pw, pdh, pdu, stream = L._ptr(ws), dh.data_ptr(), du.data_ptr(), L._current_stream(dev)
    L._check(L.lib.fp8z1_ffn_down_bwd(f, py, *down, ph, pu, off, pdh, pdu, a.data_ptr(), pw, n, stream), what)
    L._check(L.lib.fp8z1_ffn_up_bwd(f, pdh, pdu, *gate, *up, off, dx.data_ptr(), pw, n, stream), what)
    return dx, dh, du, a


def ffn_weight_gradient(p: torch.Tensor, q: torch.Tensor, n_experts: int = 1,
                        offsets: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """[E,M,N] = per expert p^T q over its rows.  Given ``out`` (float32), the products are added to it."""
    what = "ffn_weight_gradient"
    if p.dim() != 2 or q.dim() != 2 or p.dtype not in _HALF:
        _fail(f"{what}: p and q must be [T, M] and [T, N] of torch.bfloat16 or torch.float16")
    dev, (T, M), N = _device(p, what), p.shape, q.shape[1]
    pp, pq = _check(p, dev, p.dtype, (T, M), what), _check(q, dev, p.dtype, (T, N), what)
    off = _offsets(offsets, dev, n_experts, what)
    if dtype not in (torch.float32, torch.bfloat16):
        _fail(f"{what}: dtype {dtype}, expected torch.float32 or torch.bfloat16")
    if out is None:
        dw = p.new_empty((n_experts, M, N), dtype=dtype)
    else:
        dw = out
        _check(dw, dev, torch.float32, (n_experts, M, N), f"{what} out")
    n = _wgrad_workspace(T, n_experts, M, N)
    ws = _scratch(p, n)
    L._check(L.lib.fp8z1_ffn_wgrad(T, n_experts, M, N, _CODE[p.dtype], pp, pq, off, _CODE[dw.dtype], dw.data_ptr(),
                                   int(out is not None), L._ptr(ws), n, L._current_stream(dev)), what)
    return dw


def ffn_backward_weights(x: torch.Tensor, a: torch.Tensor, dy: torch.Tensor, dh: torch.Tensor, du: torch.Tensor,
                         n_experts: int = 1, offsets: Optional[torch.Tensor] = None,
                         dtype: torch.dtype = torch.float32, out: Optional[Sequence[torch.Tensor]] = None):
    """(dWg [E,F,D], dWu [E,F,D], dWd [E,D,F]), row-major as the shard step reads its gradients.
    Given ``out`` (three float32 tensors), the products are added to them."""
    what = "ffn_backward_weights"
    if x.dim() != 2 or a.dim() != 2 or x.dtype not in _HALF:
        _fail(f"{what}: rows must be [T, D] and [T, F] of torch.bfloat16 or torch.float16")
    dev, (T, D), F, E = _device(x, what), x.shape, a.shape[1], n_experts
    if dtype not in (torch.float32, torch.bfloat16):
        _fail(f"{what}: dtype {dtype}, expected torch.float32 or torch.bfloat16")
    wide = [_check(v, dev, x.dtype, (T, D), f"{what} {n}") for v, n in ((x, "x"), (dy, "dy"))]
    inner = [_check(v, dev, x.dtype, (T, F), f"{what} {n}") for v, n in ((a, "a"), (dh, "dh"), (du, "du"))]
    off = _offsets(offsets, dev, E, what)
    shapes = ((E, F, D), (E, F, D), (E, D, F))
    if out is None:
        dw = tuple(x.new_empty(s, dtype=dtype) for s in shapes)
    else:
        dtype, dw = torch.float32, tuple(out)
        if len(dw) != len(shapes):
            _fail(f"{what}: out holds {len(dw)} tensors, expected {len(shapes)}")
        for w, s in zip(dw, shapes):
            _check(w, dev, dtype, s, f"{what} out")
    n = _weights_workspace(T, E, D, F)
    ws = _scratch(x, n)
    f = L.Ffn(T, E, D, F, _CODE[x.dtype], L.ACT_SILU)
    L._check(L.lib.fp8z1_ffn_bwd_weights(f, wide[0], inner[0], wide[1], inner[1], inner[2], off, _CODE[dtype],
                                         dw[0].data_ptr(), dw[1].data_ptr(), dw[2].data_ptr(), int(out is not None),
                                         L._ptr(ws), n, L._current_stream(dev)), what)
    return dw


@functools.lru_cache(maxsize=256)
def _linear_workspace(T: int, E: int, N: int, K: int, eight: bool) -> int:
    return L.fp8z1_linear_workspace_bytes(L.Product(T, E, N, K, L.BF16, L.E4M3 if eight else L.BF16, L.ACT_NONE, 0))


@functools.lru_cache(maxsize=256)
def _linear_bwd_workspace(T: int, E: int, N: int, K: int, bias: bool) -> int:
    if bias:
        return L.fp8z1_linear_bwd_workspace_bytes(L.Product(T, E, N, K, L.BF16, L.BF16, L.ACT_NONE, 0))
    return L.fp8z1_linear_workspace_bytes(L.Product(T, E, K, N, L.BF16, L.BF16, L.ACT_NONE, 0))  # (dx = dp W alone)


@functools.lru_cache(maxsize=256)
def _up8_workspace(T: int, E: int, D: int, F: int) -> int:
    return L.fp8z1_ffn_up8_workspace_bytes(L.Ffn(T, E, D, F, L.BF16, L.ACT_SILU))


def _rows8(x: Rows8, dev: int, T: int, C: int, what: str) -> Tuple[int, int]:
    return (_check(x[0], dev, torch.uint8, (T, C), what),
            _check(x[1], dev, torch.float32, (T, -(-C // 128)), f"{what} scales"))


def _linear_act(act: Optional[str], what: str) -> int:
    if act is not None and act not in _ACT:
        _fail(f"{what}: act {act!r}, expected None or one of {', '.join(_ACT)}")
    return L.ACT_NONE if act is None else _ACT[act]


def _half(dtype: Optional[torch.dtype], what: str) -> torch.dtype:
    if dtype not in _HALF:
        _fail(f"{what}: dtype {dtype}, expected torch.bfloat16 or torch.float16")
    return dtype


def linear(x: Union[torch.Tensor, Rows8], w: Weight, offsets: Optional[torch.Tensor] = None,
           bias: Optional[torch.Tensor] = None, act: Optional[str] = None, res: Optional[torch.Tensor] = None,
           save: bool = False, dtype: Optional[torch.dtype] = None):
    """(y, p): y [T,N] = res + act(p), p = x W^T + bias, codes [E,N,K].  x is [T,K] in 16 bits, or a pair (codes,
    scales) in 8; bias float32 [E,N] (one expert: or [N]).  p is None unless ``save``.
    ``dtype`` (of y, p and res): x's own, for 8-bit rows that of res or bfloat16 unless it is given.
    Products of 8-bit rows are summed by 8 consecutive ones with 13 bits below the largest, then in float32
    (see fp8z1.h); those of 16-bit rows in float32 throughout."""
    what = "linear"
    eight = isinstance(x, tuple)
    rows = x[0] if eight else x
    if rows.dim() != 2 or w[0].dim() != 3:
        _fail(f"{what}: rows must be [T, K] and codes [E, N, K]")
    if eight:
        dtype = _half(dtype or (res.dtype if res is not None else torch.bfloat16), what)
    elif dtype not in (None, rows.dtype) or rows.dtype not in _HALF:
        _fail(f"{what}: rows of {rows.dtype} for dtype {dtype}, expected torch.bfloat16 or torch.float16, both alike")
    else:
        dtype = rows.dtype
    dev, (T, K), (E, N, _) = _device(rows, what), rows.shape, w[0].shape
    px, ps = _rows8(x, dev, T, K, what) if eight else (_check(rows, dev, dtype, (T, K), what), None)
    pw = _weight(w, dev, E, N, K, f"{what} weight")
    off = _offsets(offsets, dev, E, what)
    pb = None if bias is None else _check(bias, dev, torch.float32, (E, N) if E > 1 or bias.dim() != 1 else (N,),
                                          f"{what} bias")
    pr = None if res is None else _check(res, dev, dtype, (T, N), f"{what} res")
    y = rows.new_empty((T, N), dtype=dtype)
    p = torch.empty_like(y) if save else None
    f = L.Product(T, E, N, K, _CODE[dtype], L.E4M3 if eight else _CODE[dtype], _linear_act(act, what), 0)
    n = _linear_workspace(T, E, N, K, eight)
    ws = _scratch(rows, n)
    L._check(L.lib.fp8z1_linear(f, px, ps, *pw, off, pb, pr, y.data_ptr(), L._ptr(p), L._ptr(ws), n,
                                L._current_stream(dev)), what)
    return y, p


def linear_backward(dy: torch.Tensor, w: Weight, p: Optional[torch.Tensor] = None,
                    offsets: Optional[torch.Tensor] = None, act: Optional[str] = None,
                    bias: bool = False, dx: bool = True, dp: bool = True) -> Dict[str, Optional[torch.Tensor]]:
    """{"dx" [T,K], "dp" [T,N], "dbias" [E,N] (with ``bias``)} from dy and, with an activation, the kept p.  Without one
    dp is dy itself.  The weight gradient is ffn_weight_gradient(dp, x in 16 bits); res has the gradient dy.
    ``dx`` and ``dp`` False: not wanted, and None (dx needs dp where there is an activation)."""
    what = "linear_backward"
    if dy.dim() != 2 or w[0].dim() != 3:
        _fail(f"{what}: dy must be [T, N] and codes [E, N, K]")
    dtype, kind = _half(dy.dtype, what), _linear_act(act, what)
    dev, (T, N), (E, _, K) = _device(dy, what), dy.shape, w[0].shape
    py = _check(dy, dev, dtype, (T, N), what)
    if (p is None) != (act is None):
        _fail(f"{what}: p is kept where there is an activation, and only there")
    pp = None if p is None else _check(p, dev, dtype, (T, N), f"{what} p")
    pw = _weight(w, dev, E, N, K, f"{what} weight")
    off = _offsets(offsets, dev, E, what)
    dps = None if not dp else dy if p is None else torch.empty_like(dy)
    dxs = dy.new_empty((T, K)) if dx else None
    dbias = dy.new_empty((E, N), dtype=torch.float32) if bias else None
    f = L.Product(T, E, N, K, _CODE[dtype], _CODE[dtype], kind, 0)
    n = _linear_bwd_workspace(T, E, N, K, bias) if bias or dx else 0
    ws = _scratch(dy, n)
    L._check(L.lib.fp8z1_linear_bwd(f, py, pp, *pw, off, None if p is None else L._ptr(dps), L._ptr(dbias), L._ptr(dxs),
                                    L._ptr(ws), n, L._current_stream(dev)), what)
    return {"dx": dxs, "dp": dps, "dbias": dbias}


def ffn_up8(x: Rows8, w_gate: Weight, w_up: Weight, offsets: Optional[torch.Tensor] = None, act: str = "silu",
            save: bool = False, dtype: torch.dtype = torch.bfloat16, scale_rule: str = "amax"):
    """((codes [T,F], scales), (h, u)): a = act(x Wg^T) * (x Wu^T) of rows x in 8 bits, in 8 bits; h and u in ``dtype``
    with ``save``, else None.  ``linear`` of a makes y."""
    what = "ffn_up8"
    if x[0].dim() != 2 or w_gate[0].dim() != 3:
        _fail(f"{what}: rows must be [T, D] and codes [E, F, D]")
    if act not in _ACT:
        _fail(f"{what}: act {act!r}, expected one of {', '.join(_ACT)}")
    dev, (T, D), (E, F, _) = _device(x[0], what), x[0].shape, w_gate[0].shape
    px = _rows8(x, dev, T, D, what)
    gate, up = (_weight(w, dev, E, F, D, f"{what} {n}") for w, n in ((w_gate, "gate"), (w_up, "up")))
    off = _offsets(offsets, dev, E, what)
    f = L.Ffn(T, E, D, F, _CODE[_half(dtype, what)], _ACT[act])
    codes, scales = _empty8(x[0], T, F)
    h, u = (x[0].new_empty((T, F), dtype=dtype) for _ in range(2)) if save else (None, None)
    n = _up8_workspace(T, E, D, F)
    ws = _scratch(x[0], n)
    L._check(L.lib.fp8z1_ffn_up8(f, *px, *gate, *up, off, L._ptr(h), L._ptr(u), codes.data_ptr(), scales.data_ptr(),
                                 _scale_rule(scale_rule, what), L._ptr(ws), n, L._current_stream(dev)), what)
    return (codes, scales), ((h, u) if save else None)


def ffn_forward8(x: Rows8, w_gate: Weight, w_up: Weight, w_down: Weight, offsets: Optional[torch.Tensor] = None,
                 act: str = "silu", save: bool = False, dtype: torch.dtype = torch.bfloat16, scale_rule: str = "amax"):
    """(y [T,D], (h, u)): ffn_forward with x and a in 8 bits, a's scales by ``scale_rule``; y, h and u in ``dtype``.  The
    backward pass is ffn_backward_data of h and u, and ffn_backward_weights of x in 16 bits and the a that it gives."""
    a, kept = ffn_up8(x, w_gate, w_up, offsets, act, save, dtype, scale_rule)
    return linear(a, w_down, offsets, dtype=dtype)[0], kept


def _gate_kind(gate: Optional[torch.Tensor], T: int, C: int) -> int:
    if gate is None:
        return L.GATE_NONE
    shape = tuple(gate.shape)
    if shape == (T, 1) and (C > 1 or gate.dtype == torch.float32):
        return L.GATE_TOKEN
    if shape == (T, C):
        return L.GATE_FULL
    if shape != (C,):
        _fail(f"gate: shape {shape}, expected ({C},), ({T}, 1) or ({T}, {C})")
    return L.GATE_CHANNEL


def _norm(rows_dtype: torch.dtype, res: torch.Tensor, w_post, gate, w_pre, settings, what: str):
    """Device, sizes, description, and the addresses of the weights and the gate."""
    if res.dim() != 2:
        _fail(f"{what}: rows must be [T, C]")
    if rows_dtype not in _CODE or res.dtype not in (rows_dtype, torch.float32):
        _fail(f"{what}: rows of {rows_dtype} with a residual of {res.dtype}")
    T, C = res.shape
    dev, kind = _device(res, what), _gate_kind(gate, T, C)
    wpost, wpre = (None if w is None else _check(w, dev, torch.float32, (C,), f"{what} weight") for w in (w_post, w_pre))
    pg = None if gate is None else _check(gate, dev, rows_dtype if kind == L.GATE_FULL else torch.float32, gate.shape,
                                          f"{what} gate")
    return dev, T, C, L.Norm(T, C, _CODE[rows_dtype], _CODE[res.dtype], kind, *settings, 0), wpost, pg, wpre


def norm_join(y: Optional[torch.Tensor], res: torch.Tensor, w_post: Optional[torch.Tensor] = None,
              gate: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6,
              res_scale: float = 1.0, block_scale: float = 1.0, weight_offset: float = 0.0,
              dtype: Optional[torch.dtype] = None):
    """(z, n): z = res_scale res + block_scale gate norm(y), n = norm(z) (see fp8z1_norm_join).
    The gate is [C] (per channel), [T,1] (per token) or [T,C].
    ``dtype``: type of n where there is no block output y (default: that of res)."""
    what = "norm_join"
    rows = y.dtype if y is not None else dtype or res.dtype
    dev, T, C, f, wpost, pg, wpre = _norm(rows, res, w_post, gate, w_pre, (eps, res_scale, block_scale, weight_offset),
                                          what)
    py = None if y is None else _check(y, dev, rows, (T, C), what)
    pr = _check(res, dev, res.dtype, (T, C), what)
    z, n = res.new_empty((T, C)), res.new_empty((T, C), dtype=rows)
    L._check(L.lib.fp8z1_norm_join(f, py, pr, wpost, pg, wpre, z.data_ptr(), n.data_ptr(), L._current_stream(dev)), what)
    return z, n


def norm_join8(y: Optional[torch.Tensor], res: torch.Tensor, w_post: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6,
               res_scale: float = 1.0, block_scale: float = 1.0, weight_offset: float = 0.0,
               dtype: Optional[torch.dtype] = None, keep: bool = False, scale_rule: str = "amax"):
    """(z, n, (codes, scales)): norm_join with n in 8 bits, a scale for every 128 columns of a row; n itself
    (for a weight gradient) with ``keep``, else None.  Its gradients are norm_join_backward's."""
    what = "norm_join8"
    rows = y.dtype if y is not None else dtype or res.dtype
    dev, T, C, f, wpost, pg, wpre = _norm(rows, res, w_post, gate, w_pre, (eps, res_scale, block_scale, weight_offset),
                                          what)
    py = None if y is None else _check(y, dev, rows, (T, C), what)
    pr = _check(res, dev, res.dtype, (T, C), what)
    z, n = res.new_empty((T, C)), res.new_empty((T, C), dtype=rows) if keep else None
    codes, scales = _empty8(res, T, C)
    L._check(L.lib.fp8z1_norm_join8(f, py, pr, wpost, pg, wpre, z.data_ptr(), L._ptr(n), codes.data_ptr(),
                                    scales.data_ptr(), _scale_rule(scale_rule, what), L._current_stream(dev)), what)
    return z, n, (codes, scales)


def norm_join_backward(dz: Optional[torch.Tensor], dn: Optional[torch.Tensor], y: Optional[torch.Tensor],
                       z: torch.Tensor, w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                       w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6, res_scale: float = 1.0,
                       block_scale: float = 1.0, weight_offset: float = 0.0) -> Dict[str, Optional[torch.Tensor]]:
    """{"dy", "dres", "dw_post", "dgate", "dw_pre"} (None where the forward call had no such input)."""
    what = "norm_join_backward"
    rows = y.dtype if y is not None else dn.dtype if dn is not None else z.dtype
    dev, T, C, f, wpost, pg, wpre = _norm(rows, z, w_post, gate, w_pre, (eps, res_scale, block_scale, weight_offset),
                                          what)
    pdz = None if dz is None else _check(dz, dev, z.dtype, (T, C), f"{what} dz")
    pdn = None if dn is None else _check(dn, dev, rows, (T, C), f"{what} dn")
    py = None if y is None else _check(y, dev, rows, (T, C), f"{what} y")
    pz = _check(z, dev, z.dtype, (T, C), f"{what} z")
    dy, dres = None if y is None else y.new_empty((T, C)), z.new_empty((T, C))
    dw_post, dgate, dw_pre = (None if v is None else v.new_empty(v.shape) for v in (w_post, gate, w_pre))
    n = _norm_workspace(T, C)
    ws = _scratch(z, n)
    L._check(L.lib.fp8z1_norm_join_bwd(f, pdz, pdn, py, pz, wpost, pg, wpre, L._ptr(dy), dres.data_ptr(),
                                       L._ptr(dw_post), L._ptr(dgate), L._ptr(dw_pre), L._ptr(ws), n,
                                       L._current_stream(dev)), what)
    return {"dy": dy, "dres": dres, "dw_post": dw_post, "dgate": dgate, "dw_pre": dw_pre}
