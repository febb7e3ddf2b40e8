"""The feed-forward block and the norms around it, as workloads that can be timed and compared.

Five calls are covered, on row-major weights held as FP8 E4M3 codes with one scale per
128x128 block (what the shard step unfolds):

  forward    y = (act(x Wg^T) * (x Wu^T)) Wd^T, tokens sorted by expert
  data       the same block's gradients with respect to its input and its projections
  weights    the weight gradients, in the row-major layout the shard step reads
  norms      z = alpha res + beta gate * norm(y), n = norm(z)
  norms_bwd  its gradients

`own` chooses between the plain form (elementary torch operations in float32) and the
library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 128


def listed():
    """Twelve calls; the widths 7168 and 2048 are those of the MoE expert workload."""
    return [
        # one token of a request through one expert's weights: latency and the read of 44 MB of codes
        dict(name="forward_one_token", kind="forward", T=1, E=1, D=7168, F=2048, dtype="bf16", act="silu", save=False),
        # a decoding batch spread over 32 experts (some get nothing): the read of 1.4 GB of codes
        dict(name="forward_decode_experts", kind="forward", T=128, E=32, D=7168, F=2048, dtype="bf16", act="silu",
             save=False),
        # ragged widths, three experts, half precision, the projections kept for a backward pass
        dict(name="forward_odd", kind="forward", T=777, E=3, D=1001, F=715, dtype="f16", act="gelu", save=True),
        # a training batch of 8 local experts
        dict(name="forward_train_experts", kind="forward", T=8192, E=8, D=7168, F=2048, dtype="bf16", act="silu",
             save=True),
        # backward of small ragged widths
        dict(name="data_odd", kind="data", T=300, E=5, D=521, F=300, dtype="f16", act="gelu"),
        # backward of the training batch
        dict(name="data_train_experts", kind="data", T=8192, E=8, D=7168, F=2048, dtype="bf16", act="silu"),
        # many tokens on small weights: few output tiles, a long sum
        dict(name="weights_long", kind="weights", T=20000, E=1, D=520, F=300, dtype="bf16", out="bf16"),
        # the training batch's weight gradients as the shard step reads them
        dict(name="weights_train_experts", kind="weights", T=8192, E=8, D=7168, F=2048, dtype="bf16", out="f32"),
        # two tokens while decoding: latency
        dict(name="norms_decode", kind="norms", T=2, C=7168, dtype="bf16", res="bf16", gate="none"),
        # a training batch with a float32 residual stream and a learned gate per channel
        dict(name="norms_train", kind="norms", T=8192, C=7168, dtype="bf16", res="f32", gate="channel"),
        # odd width, a gate per token, half precision
        dict(name="norms_bwd_odd", kind="norms_bwd", T=1003, C=1537, dtype="f16", res="f32", gate="token"),
        # the training batch's backward
        dict(name="norms_bwd_train", kind="norms_bwd", T=8192, C=7168, dtype="bf16", res="f32", gate="channel"),
    ]


def _size(rng, lo, hi):
    """A size from lo to hi, even over its logarithm; half of those over 64 go to a multiple of 16."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n > 64 and rng.random() < 0.5:
        n -= n % 16
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["forward", "forward", "data", "weights", "norms", "norms_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if kind in ("norms", "norms_bwd"):
        return dict(kind=kind, T=_size(rng, 1, 8192), C=_size(rng, 64, 7168), dtype=dtype,
                    res=rng.choice(["same", "f32"]).replace("same", dtype),
                    gate=rng.choice(["none", "channel", "token", "full"]))
    case = dict(kind=kind, T=_size(rng, 1, 8192), E=rng.choice([1, 1, 2, 5, 8, 16]), D=_size(rng, 128, 7168),
                F=_size(rng, 64, 2048), dtype=dtype)
    if kind == "weights":
        case["E"] = min(case["E"], 8)
        case["out"] = rng.choice(["bf16", "f32"])
    else:
        case["act"] = rng.choice(["silu", "gelu"])
        if kind == "forward":
            case["save"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _weight(g, E, R, C):
    """Codes [E,R,C] and scales [E,R/128,C/128] of N(0, 1/C) weights whose size differs from block to block."""
    rb, cb = -(-R // BLOCK), -(-C // BLOCK)
    codes = torch.empty(E, R, C, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, rb, cb, device="cuda")
    for e in range(E):
        w = torch.zeros(rb * BLOCK, cb * BLOCK, device="cuda")
        w[:R, :C] = _randn(g, R, C, std=C ** -0.5)
        t = w.view(rb, BLOCK, cb, BLOCK)
        t *= torch.exp(0.5 * _randn(g, rb, 1, cb, 1))
        scales[e] = t.abs().amax(dim=(1, 3)) / 448.0
        q = (t / scales[e][:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[e] = q.reshape(rb * BLOCK, cb * BLOCK)[:R, :C]
    return codes, scales


def _offsets(seed, T, E):
    """First row of each expert (E + 1 numbers): uneven loads, about one expert in eight without any token."""
    g = torch.Generator().manual_seed(seed)
    load = torch.rand(E, generator=g) + 0.25
    if E > 2:
        load[torch.rand(E, generator=g) < 0.125] = 0.0
        load[int(torch.randint(E, (1,), generator=g))] = 1.0
    picks = torch.multinomial(load, T, replacement=True, generator=g)
    counts = torch.bincount(picks, minlength=E)
    edges = torch.zeros(E + 1, dtype=torch.int32)
    edges[1:] = counts.cumsum(0)
    return edges.cuda(), int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    t, T = _TYPES[case["dtype"]], case["T"]
    if case["kind"] in ("norms", "norms_bwd"):
        C, r = case["C"], _TYPES[case["res"]]
        s["y"] = _randn(g, T, C, dtype=t, std=3.0)
        s["z" if case["kind"] == "norms_bwd" else "x"] = _randn(g, T, C, dtype=r, std=2.0)
        s["w_post"] = 1.0 + _randn(g, C, std=0.2)
        s["w_pre"] = 1.0 + _randn(g, C, std=0.2)
        s["g"] = {"none": lambda: None, "channel": lambda: _randn(g, C), "token": lambda: _randn(g, T, 1),
                  "full": lambda: _randn(g, T, C, dtype=t)}[case["gate"]]()
        s["alpha"], s["beta"] = 1.0, 0.5
        if case["kind"] == "norms_bwd":
            s["dz"], s["dn"] = _randn(g, T, C, dtype=r), _randn(g, T, C, dtype=t)
        return s
    E, D, F = case["E"], case["D"], case["F"]
    s["offsets"], s["cap"] = _offsets(seed, T, E)
    if case["kind"] != "weights":
        s["w_gate"], s["w_up"], s["w_down"] = _weight(g, E, F, D), _weight(g, E, F, D), _weight(g, E, D, F)
    if case["kind"] != "data":
        s["x"] = _randn(g, T, D, dtype=t)
    if case["kind"] != "forward":
        s["dy"] = _randn(g, T, D, dtype=t, std=0.1)
    if case["kind"] == "data":
        s["h"], s["u"] = _randn(g, T, F, dtype=t, std=1.5), _randn(g, T, F, dtype=t)
    if case["kind"] == "weights":
        s["a"] = _randn(g, T, F, dtype=t)
        s["dh"], s["du"] = _randn(g, T, F, dtype=t, std=0.1), _randn(g, T, F, dtype=t, std=0.1)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    kind = s["kind"]
    if own:
        return _own(s)
    if kind == "forward":
        return _forward(s)
    if kind == "data":
        return _data(s)
    if kind == "weights":
        return _weights(s)
    if kind == "norms":
        return _norms(s)
    return _norms_bwd(s)


def _own(s):
    from blockwise_fp8_zero_fold_amd import block

    kind = s["kind"]
    if kind == "forward":
        y, saved = block.ffn_forward(s["x"], s["w_gate"], s["w_up"], s["w_down"], offsets=s["offsets"], act=s["act"],
                                     save=s["save"])
        return (y, *saved) if s["save"] else y
    if kind == "data":
        dx, dh, du, a = block.ffn_backward_data(s["dy"], s["h"], s["u"], s["w_gate"], s["w_up"], s["w_down"],
                                                offsets=s["offsets"], act=s["act"])
        return dx, dh, du, a
    if kind == "weights":
        return block.ffn_backward_weights(s["x"], s["a"], s["dy"], s["dh"], s["du"], n_experts=s["E"],
                                          offsets=s["offsets"], dtype=_TYPES[s["out"]])
    if kind == "norms":
        return block.norm_join(s["y"], s["x"], w_post=s["w_post"], gate=s["g"], w_pre=s["w_pre"], eps=EPS,
                               res_scale=s["alpha"], block_scale=s["beta"])
    grads = block.norm_join_backward(s["dz"], s["dn"], s["y"], s["z"], w_post=s["w_post"], gate=s["g"],
                                     w_pre=s["w_pre"], eps=EPS, res_scale=s["alpha"], block_scale=s["beta"])
    return {k: v for k, v in grads.items() if v is not None}


def _dense(w):
    """The float32 weights that codes and scales stand for."""
    codes, scales = w
    R, C = codes.shape[1:]
    wide = scales.repeat_interleave(BLOCK, 1)[:, :R].repeat_interleave(BLOCK, 2)[:, :, :C]
    return codes.view(torch.float8_e4m3fn).float() * wide


def _spread(s, x):
    """Rows by expert, [E, cap, width] in float32, zeros after each expert's last."""
    at = s["offsets"][:-1, None].long() + torch.arange(s["cap"], device=x.device)
    real = at < s["offsets"][1:, None]
    return x.float()[at.clamp(max=x.shape[0] - 1)] * real[:, :, None]


def _gather(s, y):
    """The rows of [E, cap, width] back in order, in the activations' type."""
    row = torch.arange(s["T"], device=y.device)
    expert = (row[:, None] >= s["offsets"][1:]).sum(dim=1)
    return y[expert, row - s["offsets"][expert]].to(_TYPES[s["dtype"]])


def _act(s, h):
    if s["act"] == "silu":
        return h / (1 + torch.exp(-h))
    return 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))


def _act_grad(s, h):
    if s["act"] == "silu":
        p = 1 / (1 + torch.exp(-h))
        return p * (1 + h * (1 - p))
    t = torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h))
    return 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * h * h)


def _times(x, w):
    return torch.bmm(x, w.transpose(1, 2).contiguous())


def _forward(s):
    x = _spread(s, s["x"])
    h, u = _times(x, _dense(s["w_gate"])), _times(x, _dense(s["w_up"]))
    a = _act(s, h) * u
    y = _times(a, _dense(s["w_down"]))
    if s["save"]:
        return tuple(_gather(s, v) for v in (y, h, u, a))
    return _gather(s, y)


def _data(s):
    dy, h, u = (_spread(s, s[k]) for k in ("dy", "h", "u"))
    da = torch.bmm(dy, _dense(s["w_down"]))
    f = _act(s, h)
    dh, du, a = da * u * _act_grad(s, h), da * f, f * u
    dx = torch.bmm(dh, _dense(s["w_gate"])) + torch.bmm(du, _dense(s["w_up"]))
    return tuple(_gather(s, v) for v in (dx, dh, du, a))


def _weights(s):
    x, dy, a, dh, du = (_spread(s, s[k]) for k in ("x", "dy", "a", "dh", "du"))
    t = _TYPES[s["out"]]

    def product(p, q):
        return torch.bmm(p.transpose(1, 2).contiguous(), q).to(t)

    return product(dh, x), product(du, x), product(dy, a)


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _gate(s):
    return 1.0 if s["g"] is None else s["g"].float()


def _norms(s):
    y, x = s["y"].float(), s["x"].float()
    z = s["alpha"] * x + s["beta"] * (_gate(s) * (y * _rstd(y) * s["w_post"]))
    n = z * _rstd(z) * s["w_pre"]
    return z.to(s["x"].dtype), n.to(s["y"].dtype)


def _norm_grad(d, x, w):
    r = _rstd(x)
    v = d * w
    return r * (v - x * (r * r) * (v * x).mean(dim=1, keepdim=True)), (d * x * r).sum(dim=0)


def _norms_bwd(s):
    y, z, dz, dn = (s[k].float() for k in ("y", "z", "dz", "dn"))
    d, dw_pre = _norm_grad(dn, z, s["w_pre"])
    d = d + dz
    p = y * _rstd(y) * s["w_post"]
    dy, dw_post = _norm_grad(s["beta"] * _gate(s) * d, y, s["w_post"])
    out = {"dy": dy.to(s["y"].dtype), "dres": (s["alpha"] * d).to(s["z"].dtype), "dw_post": dw_post}
    if s["gate"] != "none":
        dg = s["beta"] * d * p
        out["dgate"] = (dg.sum(dim=0) if s["gate"] == "channel" else dg.sum(dim=1, keepdim=True) if s["gate"] == "token"
                        else dg.to(s["y"].dtype))
    out["dw_pre"] = dw_pre
    return out


# --------------------------------------------------------------------------- least work

def work(case):
    el = {"bf16": 2, "f16": 2, "f32": 4}
    b, T = el[case["dtype"]], case["T"]
    if case["kind"] in ("norms", "norms_bwd"):
        C, r = case["C"], el[case["res"]]
        gate = {"none": 0, "channel": 4 * C, "token": 4 * T, "full": b * T * C}[case["gate"]]
        if case["kind"] == "norms":  # y and x in, z and n out
            return {"bytes": 2 * T * C * (b + r) + gate + 8 * C, "flops": 12 * T * C}
        # dz, dn, y, z in; dy, dres out; the weights and the gate with their gradients
        return {"bytes": T * C * (3 * b + 3 * r) + 2 * gate + 16 * C, "flops": 30 * T * C}
    E, D, F = case["E"], case["D"], case["F"]
    flops = 6 * T * D * F
    if case["kind"] == "weights":  # x, dy, a, dh, du in; three gradients out
        return {"bytes": b * T * (2 * D + 3 * F) + 3 * E * D * F * el[case["out"]], "flops": flops}
    codes = 3 * min(E, T) * D * F
    codes += 4 * codes // (BLOCK * BLOCK)
    if case["kind"] == "forward":  # x in, y out, and what is kept
        return {"bytes": codes + b * T * (2 * D + (3 * F if case["save"] else 0)), "flops": flops}
    return {"bytes": codes + b * T * (2 * D + 5 * F), "flops": flops}  # dy, h, u in; dx, dh, du, a out


# --------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("norms", "norms_bwd"):
        return _exact_norms(s) if case["kind"] == "norms" else _exact_norms_bwd(s)
    edges = s["offsets"].tolist()
    parts = [_exact_expert(s, e, slice(edges[e], edges[e + 1])) for e in range(case["E"])]
    if case["kind"] == "weights":
        return tuple(torch.stack(m) for m in zip(*parts))
    whole = tuple(torch.cat(m) for m in zip(*parts))
    return whole[0] if case["kind"] == "forward" and not case["save"] else whole


def _exact_matrix(w, e):
    codes, scales = w
    m = codes[e].view(torch.float8_e4m3fn).double()
    r = torch.arange(m.shape[0], device=m.device) // BLOCK
    c = torch.arange(m.shape[1], device=m.device) // BLOCK
    return m * scales[e].double()[r][:, c]


def _exact_expert(s, e, rows):
    def of(k):
        return s[k][rows].double()

    if s["kind"] == "weights":
        return of("dh").t() @ of("x"), of("du").t() @ of("x"), of("dy").t() @ of("a")
    wg, wu, wd = (_exact_matrix(s[k], e) for k in ("w_gate", "w_up", "w_down"))
    if s["kind"] == "forward":
        h, u = of("x") @ wg.t(), of("x") @ wu.t()
    else:
        h, u = of("h").requires_grad_(), of("u").requires_grad_()
    if s["act"] == "silu":
        f = h * torch.sigmoid(h)
    else:
        f = h * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3))
    a = f * u
    if s["kind"] == "forward":
        return a @ wd.t(), h, u, a
    dh, du = torch.autograd.grad(a, (h, u), of("dy") @ wd)
    return dh @ wg + du @ wu, dh, du, a.detach()


def _exact_join(s, y, x, w_post, gate, w_pre):
    p = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * w_post
    if gate is not None:
        p = p * gate
    z = s["alpha"] * x + s["beta"] * p
    return z, z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * w_pre


def _exact_norms(s):
    gate = None if s["g"] is None else s["g"].double()
    return _exact_join(s, s["y"].double(), s["x"].double(), s["w_post"].double(), gate, s["w_pre"].double())


def _exact_norms_bwd(s):
    """Automatic differentiation of the join; the residual input is the one that gives the kept z."""
    y, z, w_post, w_pre = (s[k].double() for k in ("y", "z", "w_post", "w_pre"))
    gate = None if s["g"] is None else s["g"].double()
    x = (z - _exact_join(s, y, torch.zeros_like(z), w_post, gate, w_pre)[0]) / s["alpha"]
    leaves = dict(dy=y, dres=x, dw_post=w_post, dgate=gate, dw_pre=w_pre)
    leaves = {k: v.clone().requires_grad_() for k, v in leaves.items() if v is not None}
    out = _exact_join(s, leaves["dy"], leaves["dres"], leaves["dw_post"], leaves.get("dgate"), leaves["dw_pre"])
    grads = torch.autograd.grad(out, list(leaves.values()), (s["dz"].double(), s["dn"].double()))
    return dict(zip(leaves, grads))
