"""The feed-forward block on the shard step's FP8 weights, and the norms around it:
allocation of outputs and call order only; all arithmetic runs in libfp8z1.

A weight is a pair ``(codes [E,R,C] uint8, scales [E,ceil(R/128),ceil(C/128)] float32)`` as
``Shard.unfold`` writes it.  Gate and up weights are [E,F,D], the down weight [E,D,F].
Rows (tokens) are sorted by expert: ``offsets`` [E+1] int32 on the device holds each
expert's first row; None means one expert.  Everything runs on torch's current stream.

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

from typing import Dict, Optional, Sequence, Tuple

import torch

from . import _lib as L

Weight = Tuple[torch.Tensor, torch.Tensor]

_ACT = {"silu": L.ACT_SILU, "gelu": L.ACT_GELU}
_CODE = {torch.float32: L.F32, torch.bfloat16: L.BF16, torch.float16: L.F16}


def _fail(msg: str):
    raise L.Fp8z1Error(msg)


def _code(x: torch.Tensor, what: str, allowed=(torch.bfloat16, torch.float16)) -> int:
    if x.dtype not in allowed:
        _fail(f"{what}: dtype {x.dtype}, expected one of {', '.join(map(str, allowed))}")
    return _CODE[x.dtype]


def _same_device(first: torch.Tensor, *xs) -> None:
    """All on the current device: the library launches there, on torch's current stream."""
    if not first.is_cuda or first.device.index != torch.cuda.current_device():
        _fail(f"tensors must be on the current device, not {first.device}")
    for x in xs:
        if x is not None and x.device != first.device:
            _fail(f"tensors on {first.device} and {x.device}")


def _rows(x: torch.Tensor, width: int, T: int, what: str) -> None:
    if tuple(x.shape) != (T, width):
        _fail(f"{what}: shape {tuple(x.shape)}, expected {(T, width)}")


def _weight(w: Weight, shape: Sequence[int], what: str) -> None:
    codes, scales = w
    e, r, c = shape
    if tuple(codes.shape) != (e, r, c):
        _fail(f"{what}: codes {tuple(codes.shape)}, expected {(e, r, c)}")
    if tuple(scales.shape) != (e, -(-r // 128), -(-c // 128)):
        _fail(f"{what}: scales {tuple(scales.shape)}, expected {(e, -(-r // 128), -(-c // 128))}")


def _offsets(offsets: Optional[torch.Tensor], E: int) -> None:
    if offsets is None:
        if E != 1:
            _fail(f"{E} experts need offsets")
    elif tuple(offsets.shape) != (E + 1,):
        _fail(f"offsets: shape {tuple(offsets.shape)}, expected {(E + 1,)}")


def _ffn(x: torch.Tensor, w_gate: Weight, w_up: Weight, w_down: Weight, offsets, act: str, what: str) -> L.Ffn:
    if x.dim() != 2 or w_gate[0].dim() != 3:
        _fail(f"{what}: rows must be [T, D] and codes [E, F, D]")
    if act not in _ACT:
        _fail(f"{what}: act {act!r}, expected one of {', '.join(_ACT)}")
    T, D = x.shape
    E, F = w_gate[0].shape[:2]
    _weight(w_gate, (E, F, D), f"{what} gate")
    _weight(w_up, (E, F, D), f"{what} up")
    _weight(w_down, (E, D, F), f"{what} down")
    _offsets(offsets, E)
    _same_device(x, *w_gate, *w_up, *w_down, offsets)
    return L.Ffn(T, E, D, F, _code(x, what), _ACT[act])


def ffn_forward(x: torch.Tensor, w_gate: Weight, w_up: Weight, w_down: Weight,
                offsets: Optional[torch.Tensor] = None, act: str = "silu", save: bool = False):
    """y [T,D] = (act(x Wg^T) * (x Wu^T)) Wd^T.  Returns (y, (h, u, a)) with ``save``, else (y, None)."""
    f = _ffn(x, w_gate, w_up, w_down, offsets, act, "ffn_forward")
    a = x.new_empty(f.T, f.F)
    h, u = (torch.empty_like(a), torch.empty_like(a)) if save else (None, None)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    L.fp8z1_ffn_up(f, x, *w_gate, *w_up, offsets, h, u, a)
    L.fp8z1_ffn_down(f, a, *w_down, offsets, y)
    return y, ((h, u, a) if save else None)


def ffn_backward_data(dy: torch.Tensor, h: torch.Tensor, u: torch.Tensor, w_gate: Weight, w_up: Weight,
                      w_down: Weight, offsets: Optional[torch.Tensor] = None, act: str = "silu"):
    """(dx, dh, du, a): the gradients at the block's input and its projections, and a again
    (what the weight gradients need)."""
    f = _ffn(dy, w_gate, w_up, w_down, offsets, act, "ffn_backward_data")
    _rows(h, f.F, f.T, "h")
    _rows(u, f.F, f.T, "u")
    _same_device(dy, h, u)
    dh, du, a = (torch.empty_like(h, memory_format=torch.contiguous_format) for _ in range(3))
    dx = torch.empty_like(dy, memory_format=torch.contiguous_format)
    L.fp8z1_ffn_down_bwd(f, dy, *w_down, h, u, offsets, dh, du, a)
    L.fp8z1_ffn_up_bwd(f, dh, du, *w_gate, *w_up, offsets, dx)
    return dx, dh, du, a


def ffn_weight_gradient(p: torch.Tensor, q: torch.Tensor, n_experts: int = 1,
                        offsets: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """[E,M,N] = per expert p^T q over its rows.  Given ``out`` (float32), the products are added to it."""
    if p.dim() != 2 or q.dim() != 2 or p.shape[0] != q.shape[0] or p.dtype != q.dtype:
        _fail("ffn_weight_gradient: p and q must be [T, M] and [T, N] of one type")
    (T, M), N = p.shape, q.shape[1]
    _offsets(offsets, n_experts)
    _same_device(p, q, offsets, out)
    if dtype not in (torch.float32, torch.bfloat16):
        _fail(f"ffn_weight_gradient: dtype {dtype}, expected torch.float32 or torch.bfloat16")
    if out is None:
        dw = p.new_empty(n_experts, M, N, dtype=dtype)
    else:
        dw = out
        if tuple(dw.shape) != (n_experts, M, N) or dw.dtype != torch.float32:
            _fail(f"ffn_weight_gradient: out must be float32 {(n_experts, M, N)}")
    need = L.fp8z1_ffn_wgrad_workspace_bytes(T, n_experts, M, N)
    ws = p.new_empty(need, dtype=torch.uint8) if need else None
    L.fp8z1_ffn_wgrad(T, n_experts, M, N, _code(p, "ffn_weight_gradient"), p, q, offsets, _CODE[dw.dtype], dw,
                      accumulate=out is not None, workspace=ws)
    return dw


def ffn_backward_weights(x: torch.Tensor, a: torch.Tensor, dy: torch.Tensor, dh: torch.Tensor, du: torch.Tensor,
                         n_experts: int = 1, offsets: Optional[torch.Tensor] = None,
                         dtype: torch.dtype = torch.float32, out: Optional[Sequence[torch.Tensor]] = None):
    """(dWg [E,F,D], dWu [E,F,D], dWd [E,D,F]), row-major as the shard step reads its gradients.
    Given ``out`` (three float32 tensors), the products are added to them."""
    og, ou, od = out if out is not None else (None, None, None)
    return (ffn_weight_gradient(dh, x, n_experts, offsets, dtype, og),
            ffn_weight_gradient(du, x, n_experts, offsets, dtype, ou),
            ffn_weight_gradient(dy, a, n_experts, offsets, dtype, od))


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


def _norm(rows: torch.Tensor, res: torch.Tensor, gate, eps, res_scale, block_scale, weight_offset, what) -> L.Norm:
    if rows.dim() != 2 or res.shape != rows.shape:
        _fail(f"{what}: rows must be [T, C], all of one shape")
    T, C = rows.shape
    dt = _code(rows, what, (torch.float32, torch.bfloat16, torch.float16))
    rt = _code(res, what, (torch.float32, rows.dtype))
    return L.Norm(T, C, dt, rt, _gate_kind(gate, T, C), eps, res_scale, block_scale, weight_offset, 0)


def norm_join(y: Optional[torch.Tensor], res: torch.Tensor, w_post: Optional[torch.Tensor] = None,
              gate: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6,
              res_scale: float = 1.0, block_scale: float = 1.0, weight_offset: float = 0.0,
              dtype: Optional[torch.dtype] = None):
    """(z, n): z = res_scale res + block_scale gate norm(y), n = norm(z) (see fp8z1_norm_join).
    The gate is [C] (per channel), [T,1] (per token) or [T,C].
    ``dtype``: type of n where there is no block output y (default: that of res)."""
    n = torch.empty_like(y, memory_format=torch.contiguous_format) if y is not None else torch.empty_like(
        res, dtype=dtype or res.dtype, memory_format=torch.contiguous_format)
    z = torch.empty_like(res, memory_format=torch.contiguous_format)
    f = _norm(n, res, gate, eps, res_scale, block_scale, weight_offset, "norm_join")
    _same_device(res, y, w_post, gate, w_pre)
    L.fp8z1_norm_join(f, y, res, w_post, gate, w_pre, z, n)
    return z, n


def norm_join_backward(dz: Optional[torch.Tensor], dn: Optional[torch.Tensor], y: Optional[torch.Tensor],
                       z: torch.Tensor, w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                       w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6, res_scale: float = 1.0,
                       block_scale: float = 1.0, weight_offset: float = 0.0) -> Dict[str, Optional[torch.Tensor]]:
    """{"dy", "dres", "dw_post", "dgate", "dw_pre"} (None where the forward call had no such input)."""
    rows = y if y is not None else dn if dn is not None else z
    f = _norm(rows, z, gate, eps, res_scale, block_scale, weight_offset, "norm_join_backward")
    _same_device(z, dz, dn, y, w_post, gate, w_pre)
    contiguous = dict(memory_format=torch.contiguous_format)
    out: Dict[str, Optional[torch.Tensor]] = {
        "dy": torch.empty_like(y, **contiguous) if y is not None else None,
        "dres": torch.empty_like(z, **contiguous),
        "dw_post": torch.empty_like(w_post, **contiguous) if w_post is not None else None,
        "dgate": torch.empty_like(gate, **contiguous) if gate is not None else None,
        "dw_pre": torch.empty_like(w_pre, **contiguous) if w_pre is not None else None}
    ws = z.new_empty(L.fp8z1_norm_join_bwd_workspace_bytes(f), dtype=torch.uint8)
    L.fp8z1_norm_join_bwd(f, dz, dn, y, z, w_post, gate, w_pre, *out.values(), workspace=ws)
    return out
