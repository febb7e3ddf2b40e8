"""The router of a mixture of experts, and its tokens sorted by expert and back: allocation of outputs and call order
only; all arithmetic runs in libfp8z1.

A training step over one routed block, with the feed-forward block of block.py on the sorted rows:

    experts, weights = route(logits, k)
    offsets, row_of = sort_tokens(experts, n_experts)
    rows = dispatch(x, row_of)
    y_rows, (h, u, a) = ffn_forward(rows, w_gate, w_up, w_down, offsets, save=True)
    y = combine(y_rows, row_of, weights)
    ...
    dy_rows, dweights = combine_backward(dy, y_rows, row_of, weights)
    dx_rows, dh, du, a = ffn_backward_data(dy_rows, h, u, w_gate, w_up, w_down, offsets)
    dx = combine(dx_rows, row_of)                            # the gradient of dispatch
    dlogits = route_backward(dweights, logits, experts)

``experts``, ``offsets`` and ``row_of`` are int32, weights float32.  The buffer of sorted rows has a row for every
choice; rows behind offsets[-1] hold whatever their memory held.  Everything runs on torch's current stream.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple, Union

import torch

from . import _lib as L
from .block import Rows8, _CODE, _check, _device, _empty8, _fail, _scratch

_SCORE = {"softmax": L.SCORE_SOFTMAX, "sigmoid": L.SCORE_SIGMOID}

_sort_workspace = functools.lru_cache(maxsize=256)(L.fp8z1_sort_tokens_workspace_bytes)


def _choices(k: int, what: str) -> None:
    """(The calls take k in 32 bits, and would see a larger number without its upper ones.)"""
    if not 1 <= k <= L.ROUTE_MAX_CHOICES:
        _fail(f"{what}: {k} choices, expected 1 to {L.ROUTE_MAX_CHOICES}")


def _router(logits: torch.Tensor, k: int, score: str, normalize: bool, scale: float, what: str):
    if logits.dim() != 2 or logits.dtype not in _CODE:
        _fail(f"{what}: logits must be [T, E] of torch.bfloat16, torch.float16 or torch.float32")
    if score not in _SCORE:
        _fail(f"{what}: score {score!r}, expected one of {', '.join(_SCORE)}")
    _choices(k, what)
    T, E = logits.shape
    dev = _device(logits, what)
    return dev, T, E, _check(logits, dev, logits.dtype, (T, E), what), L.Router(T, E, k, _CODE[logits.dtype],
                                                                              _SCORE[score], bool(normalize), scale)


def route(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None, score: str = "softmax",
          normalize: bool = True, scale: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """(experts [T,k], weights [T,k]): each row's k experts of the largest score (plus ``bias`` [E], which decides
    the choice only), largest first, and their scores times ``scale``, with ``normalize`` over their sum.
    An expert whose logit is -inf or NaN is not chosen; choices beyond those left are -1 with weight 0."""
    what = "route"
    dev, T, E, pl, f = _router(logits, k, score, normalize, scale, what)
    pb = None if bias is None else _check(bias, dev, torch.float32, (E,), f"{what} bias")
    experts, weights = logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k), dtype=torch.float32)
    L._check(L.lib.fp8z1_route(f, pl, pb, experts.data_ptr(), weights.data_ptr(), L._current_stream(dev)), what)
    return experts, weights


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, score: str = "softmax",
                   normalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """The logits' gradient from the weights' (``experts`` and the settings as in the forward call)."""
    what = "route_backward"
    if experts.dim() != 2:
        _fail(f"{what}: experts must be [T, k]")
    k = experts.shape[1]
    dev, T, _, pl, f = _router(logits, k, score, normalize, scale, what)
    pe = _check(experts, dev, torch.int32, (T, k), f"{what} experts")
    pd = _check(dweights, dev, torch.float32, (T, k), f"{what} dweights")
    dlogits = torch.empty_like(logits)
    L._check(L.lib.fp8z1_route_bwd(f, pl, pe, pd, dlogits.data_ptr(), L._current_stream(dev)), what)
    return dlogits


def sort_tokens(experts: torch.Tensor, n_experts: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """(offsets [E+1], row_of [T,k]) of experts [T,k]: each expert's first row, and each choice's row among the rows
    sorted by expert, equal ones in the order of the choices; -1 for a choice outside 0..E-1."""
    what = "sort_tokens"
    if experts.dim() != 2:
        _fail(f"{what}: experts must be [T, k]")
    T, k = experts.shape
    _choices(k, what)
    if not 1 <= n_experts <= L.ROUTE_MAX_EXPERTS:
        _fail(f"{what}: {n_experts} experts, expected 1 to {L.ROUTE_MAX_EXPERTS}")
    dev = _device(experts, what)
    pe = _check(experts, dev, torch.int32, (T, k), what)
    n = _sort_workspace(T, k, n_experts)
    offsets, row_of, ws = experts.new_empty(n_experts + 1), torch.empty_like(experts), _scratch(experts, n)
    L._check(L.lib.fp8z1_sort_tokens(T, k, n_experts, pe, offsets.data_ptr(), row_of.data_ptr(), L._ptr(ws), n,
                                     L._current_stream(dev)), what)
    return offsets, row_of


def _plan(row_of: torch.Tensor, dev: int, what: str) -> Tuple[int, int, int]:
    if row_of.dim() != 2:
        _fail(f"{what}: row_of must be [T, k]")
    T, k = row_of.shape
    _choices(k, what)
    return T, k, _check(row_of, dev, torch.int32, (T, k), f"{what} row_of")


def dispatch(x: Union[torch.Tensor, Rows8], row_of: torch.Tensor, out: Union[torch.Tensor, Rows8, None] = None):
    """rows [T k, D] with rows[row_of[t,j]] = x[t]; of 8-bit rows, a pair (codes, scales), both.  Given ``out``
    (of any number of rows) the rows are written there; those that no choice has stay as they were."""
    what = "dispatch"
    eight = isinstance(x, tuple)
    codes = x[0] if eight else x
    if codes.dim() != 2 or (not eight and codes.dtype not in _CODE):
        _fail(f"{what}: x must be [T, D] of torch.bfloat16, torch.float16 or torch.float32, or codes and scales")
    dev, (T, D) = _device(codes, what), codes.shape
    dt = torch.uint8 if eight else codes.dtype
    px = _check(codes, dev, dt, (T, D), what)
    ps = _check(x[1], dev, torch.float32, (T, -(-D // 128)), f"{what} scales") if eight else None
    tokens, k, pr = _plan(row_of, dev, what)
    if tokens != T:
        _fail(f"{what}: row_of of {tokens} tokens for {T}")
    if out is None:
        out = _empty8(codes, T * k, D) if eight else codes.new_empty((T * k, D))
    rows = out[0] if eight else out
    if rows.dim() != 2:
        _fail(f"{what}: out must be [R, D]")
    R = rows.shape[0]
    po = _check(rows, dev, dt, (R, D), f"{what} out")
    pos = _check(out[1], dev, torch.float32, (R, -(-D // 128)), f"{what} out scales") if eight else None
    f = L.Routed(T, D, R, k, L.E4M3 if eight else _CODE[dt])
    L._check(L.lib.fp8z1_dispatch(f, pr, px, ps, po, pos, L._current_stream(dev)), what)
    return out


def _rows(rows: torch.Tensor, what: str):
    if rows.dim() != 2 or rows.dtype not in _CODE:
        _fail(f"{what}: rows must be [R, D] of torch.bfloat16, torch.float16 or torch.float32")
    dev = _device(rows, what)
    return dev, rows.shape[0], rows.shape[1], _check(rows, dev, rows.dtype, rows.shape, what)


def combine(rows: torch.Tensor, row_of: torch.Tensor, weights: Optional[torch.Tensor] = None,
            base: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [T,D] = base + sum over j of weights[t,j] rows[row_of[t,j]]; without weights the gradient of dispatch."""
    what = "combine"
    dev, R, D, px = _rows(rows, what)
    T, k, pr = _plan(row_of, dev, what)
    pw = None if weights is None else _check(weights, dev, torch.float32, (T, k), f"{what} weights")
    pb = None if base is None else _check(base, dev, rows.dtype, (T, D), f"{what} base")
    y = rows.new_empty((T, D))
    L._check(L.lib.fp8z1_combine(L.Routed(T, D, R, k, _CODE[rows.dtype]), pr, px, pw, pb, y.data_ptr(),
                                 L._current_stream(dev)), what)
    return y


def combine_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, weights: torch.Tensor,
                     out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(drows [R,D], dweights [T,k]) from dy [T,D] (which is base's gradient too).  drows go to ``out`` if it is given
    (it may be ``rows`` itself); rows that no choice has are not written."""
    what = "combine_backward"
    dev, R, D, px = _rows(rows, what)
    T, k, pr = _plan(row_of, dev, what)
    py = _check(dy, dev, rows.dtype, (T, D), f"{what} dy")
    pw = _check(weights, dev, torch.float32, (T, k), f"{what} weights")
    drows = torch.empty_like(rows) if out is None else out
    po = _check(drows, dev, rows.dtype, (R, D), f"{what} out")
    dweights = torch.empty_like(weights)
    L._check(L.lib.fp8z1_combine_bwd(L.Routed(T, D, R, k, _CODE[rows.dtype]), pr, py, px, pw, po, dweights.data_ptr(),
                                     L._current_stream(dev)), what)
    return drows, dweights
