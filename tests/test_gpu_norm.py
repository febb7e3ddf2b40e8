"""GPU: the norm join and its gradients against float64 (automatic differentiation), for every
type, gate and width path, rows of zeros, missing inputs, graph replay and refusals."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

fz = block = None


def setup_module(module):
    global fz, block
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import blockwise_fp8_zero_fold_amd as _fz
    from blockwise_fp8_zero_fold_amd import block as _block
    fz, block = _fz, _block


BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def make(T, C, dtype, res, gate, seed=0, post=True, pre=True, scale=1.0):
    g = torch.Generator().manual_seed(T * 31 + C + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shape = {"none": None, "channel": (C,), "token": (T, 1), "full": (T, C)}[gate]
    return dict(y=(3 * scale * r(T, C)).to(dtype), res=(2 * scale * r(T, C)).to(res),
                w_post=0.2 * r(C) if post else None, w_pre=0.2 * r(C) if pre else None,
                gate=None if shape is None else r(*shape).to(dtype if gate == "full" else SF),
                dz=r(T, C).to(res), dn=r(T, C).to(dtype))


OPT = dict(eps=1e-5, res_scale=0.75, block_scale=0.5, weight_offset=1.0)


def f32(x):
    """The value a float argument has as the float32 that the library gets."""
    return float(torch.tensor(x, dtype=SF))


def norm(x, w):
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + f32(OPT["eps"]))
    return n if w is None else n * (w + OPT["weight_offset"])


def join(y, res, w_post, gate, w_pre):
    z = OPT["res_scale"] * res
    if y is not None:
        p = norm(y, w_post) if w_post is not None else y
        z = z + OPT["block_scale"] * (p if gate is None else gate * p)
    return z, norm(z, w_pre)


def dev(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def wide(v):
    return None if v is None else v.double()


SIZES = [(1, 1), (1, 8), (3, 64), (2, 7168), (5, 513), (300, 96), (1030, 264), (40, 1537), (7, 4104), (3, 8192),
         (2, 8200), (3, 16384), (2, 10001)]
KINDS = [(BF, BF, "none"), (BF, SF, "channel"), (HF, SF, "token"), (HF, HF, "full"), (SF, SF, "channel"),
         (SF, SF, "full")]


def check_forward(d, z, n, what):
    args = [wide(d[k]) for k in ("y", "res", "w_post", "gate", "w_pre")]
    ez, en = join(*args)
    y, res, w_post, gate, w_pre = args
    C = d["res"].shape[1]
    # each norm: a sum of C squares (relative error at most C roundings), a root, a division and a few
    # products; then the sum of the two terms.  An error of z moves n by at most twice as much, relatively
    # to z's row.
    rel = (C + 16) * ref.U32
    term = (ez - OPT["res_scale"] * res).abs()
    e_z = rel * term + 2 * ref.U32 * (OPT["res_scale"] * res).abs() + 2 * ref.U32 * ez.abs()
    rms = ez.square().mean(1, keepdim=True).sqrt() + 1e-300
    w = 1.0 if w_pre is None else (w_pre + OPT["weight_offset"]).abs()
    r = torch.rsqrt(ez.square().mean(1, keepdim=True) + f32(OPT["eps"]))
    e_row = e_z.square().mean(1, keepdim=True).sqrt() / rms
    e_n = rel * en.abs() + e_z * r * w + en.abs() * e_row
    if z is not None:
        ref.check(z, ez, ref.rounded(ez, e_z, d["res"].dtype), f"{what}: z")
    if n is not None:
        ref.check(n, en, ref.rounded(en, e_n, d["dn"].dtype), f"{what}: n")


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("dtype,res,gate", KINDS)
def test_join(T, C, dtype, res, gate):
    d = make(T, C, dtype, res, gate)
    what = f"{T} x {C} {dtype} {res} {gate}"
    print("#", what, flush=True)
    g = dev(d)
    z, n = block.norm_join(g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], **OPT)
    check_forward(d, z, n, what)


@pytest.mark.parametrize("C", [72, 1025, 9000])
@pytest.mark.parametrize("missing", ["y", "w_post", "w_pre", "z", "n"])
def test_join_without(C, missing):
    d = make(9, C, BF, SF, "none", post=missing not in ("w_post", "y"), pre=missing != "w_pre")
    if missing == "y":
        d["y"] = None
    g = dev(d)
    if missing in ("z", "n"):
        f = fz.Norm(9, C, fz.BF16, fz.F32, fz.GATE_NONE, *OPT.values(), 0)
        z, n = torch.full_like(g["res"], 7.0), torch.full_like(g["y"], 7.0)
        fz.fp8z1_norm_join(f, g["y"], g["res"], g["w_post"], None, g["w_pre"], None if missing == "z" else z,
                           None if missing == "n" else n)
        assert bool(((z if missing == "z" else n) == 7.0).all())
        z, n = (None, n) if missing == "z" else (z, None)
    else:
        z, n = block.norm_join(g["y"], g["res"], g["w_post"], None, g["w_pre"], dtype=BF, **OPT)
    check_forward(d, z, n, f"without {missing}")


def gradients(d, z):
    """Float64 gradients at the kept z (taken as it is): the join's by automatic differentiation."""
    leaf = {k: wide(d[k]).clone().requires_grad_() for k in ("y", "w_post", "gate", "w_pre") if d[k] is not None}
    zd = wide(z).clone().requires_grad_()
    total = torch.zeros_like(wide(z))
    pre = {}
    if d["dn"] is not None:
        n = norm(zd, leaf.get("w_pre"))
        gs = torch.autograd.grad(n, [zd] + ([leaf["w_pre"]] if "w_pre" in leaf else []), wide(d["dn"]))
        total = total + gs[0]
        pre = {"dw_pre": gs[1]} if len(gs) > 1 else {}
    if d["dz"] is not None:
        total = total + wide(d["dz"])
    out = {"dres": OPT["res_scale"] * total, **pre}
    if d["y"] is not None:
        p = norm(leaf["y"], leaf["w_post"]) if "w_post" in leaf else leaf["y"]
        z2 = OPT["block_scale"] * (p if "gate" not in leaf else leaf["gate"] * p)
        names = [k for k in ("y", "w_post", "gate") if k in leaf]
        for k, v in zip(names, torch.autograd.grad(z2, [leaf[k] for k in names], total)):
            out[{"y": "dy", "w_post": "dw_post", "gate": "dgate"}[k]] = v
    return out, total


def check_backward(d, z, got, what):
    want, total = gradients(d, z)
    T, C = z.shape
    rel = (2 * C + 40) * ref.U32  # the two norms' sums over a row, and the products around them
    rms = lambda x: x.square().mean(1, keepdim=True).sqrt()  # noqa: E731
    zd = wide(z)
    # the size of what is added up in a row of d = dz + rstd (v - z^ mean(v z^))
    size = torch.zeros_like(zd)
    if d["dn"] is not None:
        r = torch.rsqrt(zd.square().mean(1, keepdim=True) + f32(OPT["eps"]))
        w = 1.0 if d["w_pre"] is None else (wide(d["w_pre"]) + OPT["weight_offset"]).abs()
        v = wide(d["dn"]).abs() * w
        size = r * (v + (zd * r).abs() * rms(v))
    if d["dz"] is not None:
        size = size + wide(d["dz"]).abs()
    e_d = rel * size
    bounds = {"dres": OPT["res_scale"] * (e_d + 2 * ref.U32 * total.abs())}
    if "dw_pre" in want:
        t = (wide(d["dn"]) * zd * r).abs()
        bounds["dw_pre"] = ((rel + (2 * T + 8) * ref.U32) * t).sum(0)
    if d["y"] is not None:
        y = wide(d["y"])
        ry = torch.rsqrt(y.square().mean(1, keepdim=True) + f32(OPT["eps"])) if d["w_post"] is not None else 1.0
        wp = 1.0 if d["w_post"] is None else (wide(d["w_post"]) + OPT["weight_offset"]).abs()
        ga = OPT["block_scale"] * (1.0 if d["gate"] is None else wide(d["gate"]).abs())
        sd = size + total.abs()
        dp, yh = ga * sd, (y * ry).abs()
        bounds["dy"] = 2 * rel * ry * (dp * wp + yh * rms(dp * wp) * (1.0 if d["w_post"] is not None else 0.0))
        over = 2 * rel + (2 * T + 8) * ref.U32
        bounds["dw_post"] = (over * dp * yh).sum(0)
        t = OPT["block_scale"] * sd * yh * wp
        if d["gate"] is not None:
            gs = tuple(d["gate"].shape)
            bounds["dgate"] = 2 * rel * t if gs == (T, C) else ((2 * rel + 2 * C * ref.U32) * t).sum(1, keepdim=True) \
                if gs == (T, 1) else (over * t).sum(0)
    for k, v in want.items():
        dtype = {"dy": d["y"], "dres": z, "dgate": d["gate"]}.get(k)
        ref.check(got[k], v, ref.rounded(v, bounds[k], SF if dtype is None else dtype.dtype), f"{what}: {k}")
    return want


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("dtype,res,gate", KINDS)
def test_join_backward(T, C, dtype, res, gate):
    d = make(T, C, dtype, res, gate)
    z = d["res"]
    what = f"{T} x {C} {dtype} {res} {gate}"
    print("#", what, flush=True)
    g = dev(d)
    got = block.norm_join_backward(g["dz"], g["dn"], g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], **OPT)
    check_backward(d, z, got, what)


@pytest.mark.parametrize("C", [72, 1025, 9000])
@pytest.mark.parametrize("missing", ["y", "w_post", "w_pre", "dz", "dn"])
def test_join_backward_without(C, missing):
    d = make(11, C, HF, SF, "none" if missing == "y" else "channel", post=missing not in ("w_post", "y"),
             pre=missing != "w_pre")
    if missing in ("y", "dz", "dn"):
        d[missing] = None
    g = dev(d)
    got = block.norm_join_backward(g["dz"], g["dn"], g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], **OPT)
    if missing == "dn":
        assert not got["dw_pre"].any()
        got["dw_pre"] = None
    want = check_backward(d, d["res"], got, f"without {missing}")
    assert {k for k, v in got.items() if v is not None} == set(want)


def test_no_rows_and_rows_of_zeros():
    d = dev(make(0, 40, BF, SF, "channel"))
    z, n = block.norm_join(d["y"], d["res"], d["w_post"], d["gate"], d["w_pre"], **OPT)
    assert z.shape == n.shape == (0, 40)
    got = block.norm_join_backward(d["dz"], d["dn"], d["y"], d["res"], d["w_post"], d["gate"], d["w_pre"], **OPT)
    assert not got["dw_post"].any() and not got["dw_pre"].any() and not got["dgate"].any()
    d = make(4, 96, BF, SF, "channel")
    d["y"].zero_()
    d["res"].zero_()
    g = dev(d)
    z, n = block.norm_join(g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], **OPT)
    assert not z.any() and not n.any()
    got = block.norm_join_backward(g["dz"], g["dn"], g["y"], z, g["w_post"], g["gate"], g["w_pre"], **OPT)
    check_backward(d, d["res"], got, "zeros")


def test_a_bad_row_stays_alone():
    d = make(6, 200, BF, SF, "channel")
    d["y"][2, 7] = float("inf")
    d["res"][4, 9] = float("nan")
    g = dev(d)
    z, n = block.norm_join(g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], **OPT)
    for t in (z, n):
        fine = torch.isfinite(t).all(1).cpu()
        assert fine.tolist() == [True, True, False, True, False, True]


def test_unaligned_rows_and_in_place():
    """Buffers one element off 16 bytes; z written over res, dres over dz."""
    T, C = 33, 256
    d = make(T, C, BF, SF, "full")

    def shift(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten().cuda()
        return flat[1:].view(t.shape)

    g = {k: shift(v) for k, v in d.items()}
    f = fz.Norm(T, C, fz.BF16, fz.F32, fz.GATE_FULL, *OPT.values(), 0)
    n = shift(torch.zeros(T, C, dtype=BF))
    res = shift(d["res"])
    fz.fp8z1_norm_join(f, g["y"], res, g["w_post"], g["gate"], g["w_pre"], res, n)
    check_forward(d, res, n, "shifted")
    dy, dg = shift(torch.zeros(T, C, dtype=BF)), shift(torch.zeros(T, C, dtype=BF))
    dwp, dwq = shift(torch.zeros(C)), shift(torch.zeros(C))
    ws = torch.empty(fz.fp8z1_norm_join_bwd_workspace_bytes(f), dtype=torch.uint8, device="cuda")
    dz = shift(d["dz"])
    fz.fp8z1_norm_join_bwd(f, dz, g["dn"], g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], dy, dz, dwp, dg, dwq,
                           workspace=ws)
    check_backward(d, d["res"], dict(dy=dy, dres=dz, dw_post=dwp, dgate=dg, dw_pre=dwq), "shifted")


def test_graph_replays_equal_eager():
    d = dev(make(500, 264, BF, SF, "channel"))

    def run():
        z, n = block.norm_join(d["y"], d["res"], d["w_post"], d["gate"], d["w_pre"], **OPT)
        got = block.norm_join_backward(d["dz"], d["dn"], d["y"], z, d["w_post"], d["gate"], d["w_pre"], **OPT)
        return [z, n, *got.values()]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i in range(3):
        d["y"].copy_(torch.randn(500, 264, generator=torch.Generator().manual_seed(i)))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {i}"


def test_gradients_against_differences():
    """Central differences of the float64 join along random directions agree with the float32 gradients
    (relative error of the sums below 1e-4 of the directional derivative's terms)."""
    d = make(20, 70, SF, SF, "channel")
    args = [wide(d[k]) for k in ("y", "res", "w_post", "gate", "w_pre")]
    z, _ = join(*args)
    g = dev(d)
    got = block.norm_join_backward(g["dz"], g["dn"], g["y"], z.float().cuda(), g["w_post"], g["gate"], g["w_pre"],
                                   **OPT)

    def value(*a):
        z, n = join(*a)
        return float((z * wide(d["dz"])).sum() + (n * wide(d["dn"])).sum())

    rng = torch.Generator().manual_seed(4)
    for i, k in enumerate(("dy", "dres", "dw_post", "dgate", "dw_pre")):
        v = torch.randn(args[i].shape, generator=rng, dtype=torch.float64)
        plus, minus = list(args), list(args)
        plus[i], minus[i] = args[i] + 1e-5 * v, args[i] - 1e-5 * v
        slope = (value(*plus) - value(*minus)) / 2e-5
        terms = got[k].cpu().double() * v
        assert abs(float(terms.sum()) - slope) <= 1e-4 * float(terms.abs().sum()), k


def test_refusals():
    d = dev(make(4, 32, BF, SF, "channel"))
    E = fz.Fp8z1Error
    ok = dict(y=d["y"], res=d["res"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    for bad in (dict(gate=d["gate"][:8]), dict(gate=d["gate"].bfloat16()), dict(w_post=d["w_post"].bfloat16()),
                dict(res=d["res"][:2]), dict(res=d["res"].half()), dict(y=None), dict(w_pre=d["w_pre"][:8]),
                dict(y=d["y"].t().contiguous().t()), dict(res=d["res"].cpu()), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(E):
            block.norm_join(**(ok | bad))
    with pytest.raises(E):
        block.norm_join_backward(None, None, d["y"], d["res"], d["w_post"], d["gate"], d["w_pre"])
    wide_rows = torch.zeros(1, 16385, device="cuda")
    with pytest.raises(E):
        block.norm_join(None, wide_rows)


def test_rows_past_four_gigabytes():
    T, C = 310000, 7168
    d = make(60, C, BF, BF, "channel")
    g = dev(d)
    y, res = torch.zeros(T, C, dtype=BF, device="cuda"), torch.zeros(T, C, dtype=BF, device="cuda")
    y[-60:], res[-60:] = g["y"], g["res"]
    z, n = block.norm_join(y, res, g["w_post"], g["gate"], g["w_pre"], **OPT)
    check_forward(d, z[-60:], n[-60:], "far rows")
    assert not z[:-60].any() and not n[:-60].any()
    del z, n
    zero = torch.zeros_like(y)
    dn, dz = zero.clone(), zero.clone()
    dn[-60:], dz[-60:] = g["dn"], g["dz"]
    got = block.norm_join_backward(dz, dn, y, res, g["w_post"], g["gate"], g["w_pre"], **OPT)
    assert not got["dres"][:-60].any() and not got["dy"][:-60].any()
    check_backward(d, d["res"], {k: v[-60:] if v.shape[0] == T else v for k, v in got.items()}, "far rows")
