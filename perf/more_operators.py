"""A routed layer of experts on rows held in 8 bits, as workloads that can be timed and compared.

What stands around and inside the feed-forward block of a mixture of experts:

  route    each token's k best of E experts and their weights, from router scores; with its gradient
  sort     tokens sorted by expert (each expert's first row, each choice's row) and their rows copied there
  combine  the rows back in the tokens' order, weighted and summed; with its gradients
  norm8    z = alpha res + beta gate * norm(y), and n = norm(z) in 8 bits, a scale for every 128 columns of a row
  linear   y = res + act(x W^T + bias) on FP8 weights, x in 8 bits or 16; or its gradients
  up8      a = act(x Wg^T) * (x Wu^T) on FP8 weights, x and a in 8 bits

Weights are row-major FP8 E4M3 codes with one scale per 128x128 block (what the shard step unfolds); rows in 8
bits are E4M3 codes with one scale per 128 columns, the group's largest magnitude over 448.

`own` chooses between the plain form (elementary torch operations) and the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
TOP = 448.0  # largest E4M3 value


def listed():
    """Twelve calls; the widths 7168 and 2048 and the 64 experts are those of the MoE expert workload."""
    return [
        # four tokens of a decoding batch, scores by the logistic function with a balancing bias: latency
        dict(name="route_decode", kind="route", T=4, E=64, k=8, dtype="bf16", score="sigmoid", bias=True, normalize=True,
             train=False),
        # a training batch over many experts, forward and backward
        dict(name="route_train", kind="route", T=8192, E=256, k=8, dtype="f32", score="softmax", bias=False,
             normalize=True, train=True),
        # three decoding tokens in 8 bits to their experts: latency
        dict(name="sort_decode", kind="sort", T=3, E=64, k=8, D=7168, dtype="e4m3", drop=False),
        # a training batch to 64 experts: 0.94 GB of rows written
        dict(name="sort_train", kind="sort", T=8192, E=64, k=8, D=7168, dtype="bf16", drop=False),
        # odd sizes, some choices dropped, the rows of a shared expert added
        dict(name="combine_odd", kind="combine", T=501, E=7, k=3, D=1537, dtype="f16", drop=True, base=True, train=False),
        # a training batch's rows back, and the gradients of rows and weights
        dict(name="combine_train", kind="combine", T=8192, E=64, k=8, D=7168, dtype="bf16", drop=False, base=False,
             train=True),
        # two tokens while decoding: latency
        dict(name="norm8_decode", kind="norm8", T=2, C=7168, dtype="bf16", res="bf16", gate="none", keep=False),
        # a training batch with a float32 residual stream; the norm's output kept in 16 bits too, for the weight gradient
        dict(name="norm8_train", kind="norm8", T=8192, C=7168, dtype="bf16", res="f32", gate="channel", keep=True),
        # one token through a dense projection with bias and residual: the read of 15 MB of codes
        dict(name="linear_one_token", kind="linear", T=1, E=1, N=2048, K=7168, x="e4m3", dtype="bf16", act="none",
             bias=True, res=True, train=False),
        # the down projection of a training batch over 8 local experts
        dict(name="linear_train_experts", kind="linear", T=8192, E=8, N=7168, K=2048, x="e4m3", dtype="bf16", act="none",
             bias=False, res=False, train=False),
        # backward of a dense projection with bias and activation
        dict(name="linear_bwd_dense", kind="linear", T=4096, E=1, N=4096, K=4096, x="bf16", dtype="bf16", act="gelu",
             bias=True, res=True, train=True),
        # gate and up of the training batch, projections kept for the backward pass
        dict(name="up8_train_experts", kind="up8", T=8192, E=8, D=7168, F=2048, dtype="bf16", act="silu", save=True),
    ]


def _size(rng, lo, hi):
    """A size from lo to hi, even over its logarithm; half of those over 64 go to a multiple of 16."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n > 64 and rng.random() < 0.5:
        n -= n % 16
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["route", "sort", "combine", "norm8", "linear", "linear", "up8"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if kind == "route":
        E = _size(rng, 2, 512)
        return dict(kind=kind, T=_size(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)),
                    dtype=rng.choice(["bf16", "f16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, normalize=rng.random() < 0.5, train=rng.random() < 0.5)
    if kind in ("sort", "combine"):
        E = _size(rng, 2, 512)
        case = dict(kind=kind, T=_size(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), D=_size(rng, 64, 7168),
                    dtype=dtype, drop=rng.random() < 0.3)
        if kind == "sort":
            case["dtype"] = rng.choice([dtype, "e4m3"])
        else:
            case["base"], case["train"] = rng.random() < 0.3, rng.random() < 0.5
        return case
    if kind == "norm8":
        return dict(kind=kind, T=_size(rng, 1, 8192), C=_size(rng, 64, 7168), dtype=dtype,
                    res=rng.choice(["same", "f32"]).replace("same", dtype),
                    gate=rng.choice(["none", "channel", "token", "full"]), keep=rng.random() < 0.5)
    T, E = _size(rng, 1, 8192), rng.choice([1, 1, 2, 5, 8])
    if kind == "up8":
        return dict(kind=kind, T=T, E=E, D=_size(rng, 128, 7168), F=_size(rng, 64, 2048), dtype=dtype,
                    act=rng.choice(["silu", "gelu"]), save=rng.random() < 0.5)
    return dict(kind=kind, T=T, E=E, N=_size(rng, 64, 4096), K=_size(rng, 64, 4096), x=rng.choice(["e4m3", "e4m3", dtype]),
                dtype=dtype, act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.5, res=rng.random() < 0.5,
                train=rng.random() < 0.3)


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
        scales[e] = t.abs().amax(dim=(1, 3)) / TOP
        q = (t / scales[e][:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[e] = q.reshape(rb * BLOCK, cb * BLOCK)[:R, :C]
    return codes, scales


def _rows8(g, T, C, std=1.0):
    """Rows in 8 bits, (codes [T,C], scales [T,C/128]): normal values, one column in a hundred ten times as large."""
    x = _randn(g, T, C, std=std) * torch.where(torch.rand(C, device="cuda", generator=g) < 0.01, 10.0, 1.0)
    return _to8(x)


def _to8(x):
    """Codes and scales of float32 rows: scale = largest magnitude of 128 columns / 448 (1 for zeros)."""
    T, C = x.shape
    cb = -(-C // BLOCK)
    wide = torch.zeros(T, cb * BLOCK, device=x.device)
    wide[:, :C] = x
    t = wide.view(T, cb, BLOCK)
    top = t.abs().amax(dim=2)
    scales = torch.where(top == 0, 1.0, (top / TOP).clamp(min=2.0 ** -126))
    q = (t / scales[:, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return q.view(T, cb * BLOCK)[:, :C].contiguous().view(torch.uint8), scales


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


def _experts(g, T, E, k, drop):
    """k different experts of each token, some liked more; with `drop` one choice in ten is -1 (left out)."""
    like = torch.rand(E, device="cuda", generator=g) + 0.2
    keys = torch.rand(T, E, device="cuda", generator=g) ** (1 / like)
    experts = keys.topk(k, dim=1).indices.to(torch.int32)
    if drop:
        experts[torch.rand(T, k, device="cuda", generator=g) < 0.1] = -1
    return experts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, kind, T = dict(case), case["kind"], case["T"]
    t = _TYPES.get(case["dtype"])
    if kind == "route":
        s["logits"] = _randn(g, T, case["E"], dtype=t, std=1.5)
        s["b"] = _randn(g, case["E"], std=0.05) if case["bias"] else None
        s["scale"] = 2.5
        if case["train"]:
            s["dw"] = _randn(g, T, case["k"])
        return s
    if kind in ("sort", "combine"):
        E, k, D = case["E"], case["k"], case["D"]
        s["experts"] = _experts(g, T, E, k, case["drop"])
        if kind == "sort":
            s["xs"] = _rows8(g, T, D) if case["dtype"] == "e4m3" else _randn(g, T, D, dtype=t)
            # rows behind the last one stay as they are: a program that compares them keeps a buffer
            s["out"] = _zeros(s["xs"], T * k) if case["drop"] else None
            return s
        s["row_of"] = _sort(s["experts"], E)[1]
        s["rows"] = _randn(g, T * k, D, dtype=t)
        s["w"] = torch.rand(T, k, device="cuda", generator=g) + 0.05
        s["add"] = _randn(g, T, D, dtype=t) if case["base"] else None
        if case["train"]:
            s["dy"] = _randn(g, T, D, dtype=t, std=0.1)
            s["out"] = torch.zeros_like(s["rows"]) if case["drop"] else None
        return s
    if kind == "norm8":
        C, r = case["C"], _TYPES[case["res"]]
        s["y"], s["z"] = _randn(g, T, C, dtype=t, std=3.0), _randn(g, T, C, dtype=r, std=2.0)
        s["w_post"], s["w_pre"] = 1.0 + _randn(g, C, std=0.2), 1.0 + _randn(g, C, std=0.2)
        s["g"] = {"none": lambda: None, "channel": lambda: _randn(g, C), "token": lambda: _randn(g, T, 1),
                  "full": lambda: _randn(g, T, C, dtype=t)}[case["gate"]]()
        s["alpha"], s["beta"] = 1.0, 0.5
        return s
    s["offsets"], s["cap"] = _offsets(seed, T, case["E"])
    if kind == "up8":
        E, D, F = case["E"], case["D"], case["F"]
        s["w_gate"], s["w_up"], s["xs"] = _weight(g, E, F, D), _weight(g, E, F, D), _rows8(g, T, D)
        return s
    E, N, K = case["E"], case["N"], case["K"]
    s["w"] = _weight(g, E, N, K)
    s["b"] = _randn(g, E, N, std=0.5) if case["bias"] else None
    if case["train"]:
        s["dy"] = _randn(g, T, N, dtype=t, std=0.1)
        s["p"] = _randn(g, T, N, dtype=t, std=1.5) if case["act"] != "none" else None
        return s
    s["xs"] = _rows8(g, T, K) if case["x"] == "e4m3" else _randn(g, T, K, dtype=t)
    s["add"] = _randn(g, T, N, dtype=t) if case["res"] else None
    return s


def _zeros(x, n):
    if isinstance(x, tuple):
        return tuple(torch.zeros(n, v.shape[1], dtype=v.dtype, device=v.device) for v in x)
    return torch.zeros(n, x.shape[1], dtype=x.dtype, device=x.device)


# --------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"route": _route, "sort": _sort_rows, "combine": _combine, "norm8": _norm8, "linear": _linear,
            "up8": _up8}[s["kind"]](s)


def _values(codes):
    """Codes as the numbers that they stand for."""
    return codes.view(torch.float8_e4m3fn)


def _own(s):
    from blockwise_fp8_zero_fold_amd import block, routing

    kind = s["kind"]
    if kind == "route":
        how = dict(score=s["score"], normalize=s["normalize"], scale=s["scale"])
        experts, weights = routing.route(s["logits"], s["k"], bias=s["b"], **how)
        if s["train"]:
            return experts, weights, routing.route_backward(s["dw"], s["logits"], experts, **how)
        return experts, weights
    if kind == "sort":
        offsets, row_of = routing.sort_tokens(s["experts"], s["E"])
        rows = routing.dispatch(s["xs"], row_of, out=s["out"])
        return (offsets, row_of, _values(rows[0]), rows[1]) if s["dtype"] == "e4m3" else (offsets, row_of, rows)
    if kind == "combine":
        y = routing.combine(s["rows"], s["row_of"], s["w"], base=s["add"])
        if s["train"]:
            return (y, *routing.combine_backward(s["dy"], s["rows"], s["row_of"], s["w"], out=s["out"]))
        return y
    if kind == "norm8":
        z, n, (codes, scales) = block.norm_join8(s["y"], s["z"], w_post=s["w_post"], gate=s["g"], w_pre=s["w_pre"],
                                                 eps=EPS, res_scale=s["alpha"], block_scale=s["beta"], keep=s["keep"])
        return (z, n, _values(codes), scales) if s["keep"] else (z, _values(codes), scales)
    if kind == "up8":
        (codes, scales), kept = block.ffn_up8(s["xs"], s["w_gate"], s["w_up"], offsets=s["offsets"], act=s["act"],
                                              save=s["save"], dtype=_TYPES[s["dtype"]])
        return (_values(codes), scales, *kept) if s["save"] else (_values(codes), scales)
    act = None if s["act"] == "none" else s["act"]
    if s["train"]:
        grads = block.linear_backward(s["dy"], s["w"], s["p"], offsets=s["offsets"], act=act, bias=s["bias"])
        return {k: v for k, v in grads.items() if v is not None}
    y, p = block.linear(s["xs"], s["w"], offsets=s["offsets"], bias=s["b"], act=act, res=s["add"],
                        save=act is not None, dtype=_TYPES[s["dtype"]])
    return y if p is None else (y, p)


def _score(s, logits):
    if s["score"] == "softmax":
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        return e / e.sum(dim=1, keepdim=True)
    return 1 / (1 + torch.exp(-logits))


def _route(s):
    """In 64 bits: a choice between two experts may hang on a difference that 32 do not hold."""
    logits = s["logits"].double()
    p = _score(s, logits)
    by = logits if s["b"] is None else p + s["b"]  # without a bias the scores' order is the logits'
    experts = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    chosen = p.gather(1, experts)
    total = chosen.sum(dim=1, keepdim=True) if s["normalize"] else 1.0
    weights = s["scale"] * chosen / total
    out = (experts.to(torch.int32), weights.float())
    if not s["train"]:
        return out
    d = s["scale"] * s["dw"].double() / total
    if s["normalize"]:
        d = d - (d * chosen).sum(dim=1, keepdim=True) / total
    if s["score"] == "softmax":
        full = torch.zeros_like(p).scatter_(1, experts, d)
        dl = p * (full - (d * chosen).sum(dim=1, keepdim=True))
    else:
        dl = torch.zeros_like(p).scatter_(1, experts, d * chosen * (1 - chosen))
    return (*out, dl.to(s["logits"].dtype))


def _sort(experts, E):
    """First row of each expert, and the row of each choice (-1: none), equal experts in the choices' order."""
    flat = experts.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    row_of = torch.empty_like(flat)
    row_of[order] = torch.arange(flat.numel(), dtype=torch.int32, device=flat.device)
    return offsets, torch.where(key < E, row_of, -1).view(experts.shape)


def _sort_rows(s):
    offsets, row_of = _sort(s["experts"], s["E"])
    to = row_of.reshape(-1).long()
    token = torch.arange(s["T"], device=to.device).repeat_interleave(s["k"])
    if s["drop"]:
        token, to = token[to >= 0], to[to >= 0]

    def rows(x, out):
        out = x.new_empty(s["T"] * s["k"], x.shape[1]) if out is None else out
        out[to] = x[token]
        return out

    if s["dtype"] == "e4m3":
        out = s["out"] or (None, None)
        return offsets, row_of, _values(rows(s["xs"][0], out[0])), rows(s["xs"][1], out[1])
    return offsets, row_of, rows(s["xs"], s["out"])


def _combine(s):
    at, there = s["row_of"].clamp(min=0).long(), (s["row_of"] >= 0).float()
    picked = s["rows"][at].float()
    w = s["w"] * there
    y = (picked * w[:, :, None]).sum(dim=1)
    if s["add"] is not None:
        y = y + s["add"].float()
    t = s["rows"].dtype
    if not s["train"]:
        return y.to(t)
    dy = s["dy"].float()
    drows = torch.empty_like(s["rows"]) if s["out"] is None else s["out"]
    to = s["row_of"] >= 0
    drows[at[to]] = (w[:, :, None] * dy[:, None, :]).to(t)[to]
    dw = (picked * dy[:, None, :]).sum(dim=2) * there
    return y.to(t), drows, dw


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _norm8(s):
    y, res = s["y"].float(), s["z"].float()
    gate = 1.0 if s["g"] is None else s["g"].float()
    z = s["alpha"] * res + s["beta"] * (gate * (y * _rstd(y) * s["w_post"]))
    n = z * _rstd(z) * s["w_pre"]
    codes, scales = _to8(n)
    if s["keep"]:
        return z.to(s["z"].dtype), n.to(s["y"].dtype), _values(codes), scales
    return z.to(s["z"].dtype), _values(codes), scales


def _dense(w):
    """The float32 weights that codes and scales stand for."""
    codes, scales = w
    R, C = codes.shape[1:]
    wide = scales.repeat_interleave(BLOCK, 1)[:, :R].repeat_interleave(BLOCK, 2)[:, :, :C]
    return _values(codes).float() * wide


def _float_rows(x):
    """Rows in float32; of codes and scales, what they stand for."""
    if not isinstance(x, tuple):
        return x.float()
    codes, scales = x
    return _values(codes).float() * scales.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _spread(s, x):
    """Rows by expert, [E, cap, width], zeros after each expert's last."""
    at = s["offsets"][:-1, None].long() + torch.arange(s["cap"], device=x.device)
    real = at < s["offsets"][1:, None]
    return x[at.clamp(max=x.shape[0] - 1)] * real[:, :, None]


def _gather(s, y):
    """The rows of [E, cap, width] back in order."""
    row = torch.arange(s["T"], device=y.device)
    expert = (row[:, None] >= s["offsets"][1:]).sum(dim=1)
    return y[expert, row - s["offsets"][expert]]


def _times(x, w):
    return torch.bmm(x, w.transpose(1, 2).contiguous())


def _act(name, h):
    if name == "silu":
        return h / (1 + torch.exp(-h))
    if name == "gelu":
        return 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))
    return h


def _act_grad(name, h):
    if name == "silu":
        p = 1 / (1 + torch.exp(-h))
        return p * (1 + h * (1 - p))
    t = torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h))
    return 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * h * h)


def _linear(s):
    t = _TYPES[s["dtype"]]
    if s["train"]:
        dp = s["dy"].float()
        out = {}
        if s["act"] != "none":
            dp = dp * _act_grad(s["act"], s["p"].float())
        wide = _spread(s, dp)
        if s["bias"]:
            out["dbias"] = wide.sum(dim=1)
        out["dp"] = dp.to(t)
        # the product takes dp as it is kept, in 16 bits
        out["dx"] = _gather(s, torch.bmm(_spread(s, dp.to(t).float()), _dense(s["w"]))).to(t)
        return out
    p = _times(_spread(s, _float_rows(s["xs"])), _dense(s["w"]))
    if s["b"] is not None:
        p = p + s["b"][:, None]
    y, p = _gather(s, _act(s["act"], p)), _gather(s, p)
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(t) if s["act"] == "none" else (y.to(t), p.to(t))


def _up8(s):
    x = _spread(s, _float_rows(s["xs"]))
    h, u = _times(x, _dense(s["w_gate"])), _times(x, _dense(s["w_up"]))
    h, u = _gather(s, h), _gather(s, u)
    codes, scales = _to8(_act(s["act"], h) * u)
    t = _TYPES[s["dtype"]]
    return (_values(codes), scales, h.to(t), u.to(t)) if s["save"] else (_values(codes), scales)


# --------------------------------------------------------------------------- least work

def work(case):
    el = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1 + 4 / BLOCK}
    kind, b, T = case["kind"], el[case["dtype"]], case["T"]
    if kind == "route":
        E, k = case["E"], case["k"]
        # logits in, experts and weights out; backward: the weights' gradient in, the logits' out
        return {"bytes": int(T * (b * E + 8 * k) + (T * (4 * k + b * E) if case["train"] else 0)),
                "flops": 8 * T * E * (2 if case["train"] else 1)}
    if kind == "sort":  # choices and tokens in, their rows out
        k, D = case["k"], case["D"]
        return {"bytes": int(8 * T * k + 4 * case["E"] + b * T * D * (1 + k)), "flops": T * k}
    if kind == "combine":
        k, D = case["k"], case["D"]
        n = 8 * T * k + b * T * D * (k + 1 + (1 if case["base"] else 0))
        if case["train"]:  # dy and the rows in, the rows' gradients out
            n += b * T * D * (1 + 2 * k) + 12 * T * k
        return {"bytes": int(n), "flops": T * D * k * (5 if case["train"] else 2)}
    if kind == "norm8":  # y and res in, z and n out
        C, r = case["C"], el[case["res"]]
        gate = {"none": 0, "channel": 4 * C, "token": 4 * T, "full": b * T * C}[case["gate"]]
        return {"bytes": int(T * C * (b + 2 * r + el["e4m3"] + (b if case["keep"] else 0)) + gate + 8 * C),
                "flops": 14 * T * C}
    E = min(case["E"], T)
    if kind == "up8":
        D, F = case["D"], case["F"]
        out = el["e4m3"] + (2 * b if case["save"] else 0)
        return {"bytes": int(2 * E * D * F + T * (el["e4m3"] * D + out * F)), "flops": 4 * T * D * F}
    N, K = case["N"], case["K"]
    n = E * N * K + (4 * E * N if case["bias"] else 0)
    keep = case["act"] != "none"
    if case["train"]:  # dy (and p) in, dx and dp out
        return {"bytes": int(n + b * T * (K + N * (3 if keep else 1))), "flops": 2 * T * N * K}
    return {"bytes": int(n + T * (el[case["x"]] * K + b * N * (1 + keep + case["res"]))), "flops": 2 * T * N * K}


# --------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "sort": _exact_sort, "combine": _exact_combine, "norm8": _exact_norm8,
            "linear": _exact_linear, "up8": _exact_up8}[case["kind"]](s)


def _exact_route(s):
    leaf = s["logits"].double().requires_grad_(s["train"])
    score = torch.softmax(leaf, dim=1) if s["score"] == "softmax" else torch.sigmoid(leaf)
    rank = leaf.detach() if s["b"] is None else score.detach() + s["b"].double()
    order = torch.argsort(-rank, dim=1, stable=True)[:, :s["k"]]
    w = torch.take_along_dim(score, order, 1)
    if s["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * s["scale"]
    if not s["train"]:
        return None, w
    return None, w.detach(), torch.autograd.grad(w, leaf, s["dw"].double())[0]


def _exact_sort(s):
    """Row by row: the choices in the order of (expert, choice)."""
    flat = s["experts"].flatten().tolist()
    order = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < s["E"])
    src = torch.tensor([i // s["k"] for _, i in order], dtype=torch.long, device="cuda")

    def of(x):
        full = torch.zeros(len(flat), x.shape[1], dtype=torch.float64, device="cuda")
        full[:len(order)] = x.double()[src]
        return full

    if s["dtype"] == "e4m3":
        return None, None, of(s["xs"][0].view(torch.float8_e4m3fn)), of(s["xs"][1])
    return None, None, of(s["xs"])


def _exact_combine(s):
    T, k, D = s["T"], s["k"], s["D"]
    rows, y = s["rows"], torch.zeros(T, D, dtype=torch.float64, device="cuda")
    if s["add"] is not None:
        y += s["add"].double()
    drows = torch.zeros(rows.shape, dtype=torch.float64, device="cuda") if s["train"] else None
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["row_of"][:, j] >= 0)[:, 0]
        r = s["row_of"][t, j].long()
        w = s["w"][t, j].double()[:, None]
        y[t] += w * rows[r].double()
        if s["train"]:
            dy = s["dy"][t].double()
            drows[r] = w * dy
            dw[t, j] = (rows[r].double() * dy).sum(dim=1)
    return (y, drows, dw) if s["train"] else y


def _exact_to8(x):
    """The codes' values and the scales of float64 rows, group by group."""
    values, scales = torch.empty_like(x), []
    for c in range(0, x.shape[1], BLOCK):
        part = x[:, c:c + BLOCK]
        top = part.abs().amax(dim=1, keepdim=True)
        scale = torch.where(top == 0, torch.ones_like(top), top / TOP).float()
        scales.append(scale)
        # nearest E4M3 value: steps of 2^(exponent - 3), 2^-9 below 2^-6
        q = part / scale.double()
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        values[:, c:c + BLOCK] = (torch.round(q / step) * step).clamp(-TOP, TOP)
    return values, torch.cat(scales, dim=1).double()


def _exact_norm8(s):
    y, z = s["y"].double(), s["z"].double()
    p = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["w_post"].double()
    if s["g"] is not None:
        p = p * s["g"].double()
    z = s["alpha"] * z + s["beta"] * p
    n = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["w_pre"].double()
    return (z, n, *_exact_to8(n)) if s["keep"] else (z, *_exact_to8(n))


def _exact_matrix(w, e):
    codes, scales = w
    m = codes[e].view(torch.float8_e4m3fn).double()
    r = torch.arange(m.shape[0], device=m.device) // BLOCK
    c = torch.arange(m.shape[1], device=m.device) // BLOCK
    return m * scales[e].double()[r][:, c]


def _exact_rows(x, rows):
    if not isinstance(x, tuple):
        return x[rows].double()
    m = x[0][rows].view(torch.float8_e4m3fn).double()
    return m * x[1][rows].double()[:, torch.arange(m.shape[1], device=m.device) // BLOCK]


def _exact_act(name, h):
    if name == "silu":
        return h * torch.sigmoid(h)
    return h * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)) if name == "gelu" else h


def _exact_linear(s):
    edges, ys, ps, dbias = s["offsets"].tolist(), [], [], []
    for e in range(s["E"]):
        rows = slice(edges[e], edges[e + 1])
        w = _exact_matrix(s["w"], e)
        if s["train"]:
            dp = s["dy"][rows].double()
            if s["act"] != "none":
                p = s["p"][rows].double().requires_grad_()
                dp = torch.autograd.grad(_exact_act(s["act"], p), p, dp)[0]
            ps.append(dp)
            ys.append(dp.to(_TYPES[s["dtype"]]).double() @ w)
            dbias.append(dp.sum(dim=0))
            continue
        p = _exact_rows(s["xs"], rows) @ w.t()
        if s["b"] is not None:
            p = p + s["b"][e].double()
        y = _exact_act(s["act"], p)
        ys.append(y if s["add"] is None else y + s["add"][rows].double())
        ps.append(p)
    if s["train"]:
        out = {"dp": torch.cat(ps), "dx": torch.cat(ys)}
        return {**out, "dbias": torch.stack(dbias)} if s["bias"] else out
    return torch.cat(ys) if s["act"] == "none" else (torch.cat(ys), torch.cat(ps))


def _exact_up8(s):
    edges, hs, us = s["offsets"].tolist(), [], []
    for e in range(s["E"]):
        x = _exact_rows(s["xs"], slice(edges[e], edges[e + 1]))
        hs.append(x @ _exact_matrix(s["w_gate"], e).t())
        us.append(x @ _exact_matrix(s["w_up"], e).t())
    h, u = torch.cat(hs), torch.cat(us)
    out = _exact_to8(_exact_act(s["act"], h) * u)
    return (*out, h, u) if s["save"] else out
