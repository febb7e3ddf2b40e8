"""GPU: the feed-forward calls against float64, at ragged sizes, for experts without rows, at any
alignment, with special values, under graph replay and on a side stream."""
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


TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    def __init__(self, T, E, D, F, dtype="bf16", act="silu", seed=0, lo=-3.0, hi=3.0, one_run=False):
        g = torch.Generator().manual_seed(1000 * T + 10 * E + D + F + seed)
        self.T, self.E, self.D, self.F, self.act, self.dtype = T, E, D, F, act, TYPES[dtype]
        self.offsets = None if one_run else ref.make_offsets(g, T, E)
        self.gate, self.up = ref.make_weight(g, E, F, D, lo, hi), ref.make_weight(g, E, F, D, lo, hi)
        self.down = ref.make_weight(g, E, D, F, lo, hi)
        r = lambda w, s=1.0: (torch.randn(T, w, generator=g) * s).to(self.dtype)  # noqa: E731
        self.x, self.dy, self.a = r(D), r(D), r(F)
        self.h, self.u, self.dh, self.du = r(F, 2.0), r(F), r(F), r(F)
        self.cfg = fz.Ffn(T, E, D, F, {"bf16": fz.BF16, "f16": fz.F16}[dtype],
                          {"silu": fz.ACT_SILU, "gelu": fz.ACT_GELU}[act])

    def dev(self, name):
        v = getattr(self, name)
        return None if v is None else tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda()

    def out(self, width):
        return torch.full((self.T, width), 7.0, dtype=self.dtype, device="cuda")

    def run_up(self, keep=True):
        h, u, a = (self.out(self.F) for _ in range(3))
        fz.fp8z1_ffn_up(self.cfg, self.dev("x"), *self.dev("gate"), *self.dev("up"), self.dev("offsets"),
                        h if keep else None, u if keep else None, a)
        return h, u, a

    def check_up(self, got, what):
        (h, mh), (u, mu) = (ref.grouped(self.x, ref.dequantize(*w), self.offsets, False) for w in (self.gate, self.up))
        eh, eu = ref.sum_error(mh, self.D), ref.sum_error(mu, self.D)
        f, (ef, _) = ref.act_value(self.act, h), ref.act_error(self.act, h)
        # the activations' slopes stay below 1.2
        ea = (ef + 1.2 * eh) * (u.abs() + eu) + (f.abs() + 1.2 * eh) * eu + 4 * ref.U32 * (f * u).abs()
        for name, t, exact, e in (("h", got[0], h, eh), ("u", got[1], u, eu), ("a", got[2], f * u, ea)):
            if t is not None:
                ref.check(t, exact, ref.rounded(exact, e, self.dtype), f"{what}: {name}")

    def check_down(self, y, what):
        exact, mag = ref.grouped(self.a, ref.dequantize(*self.down), self.offsets, False)
        ref.check(y, exact, ref.rounded(exact, ref.sum_error(mag, self.F), self.dtype), f"{what}: y")

    def check_down_bwd(self, got, what):
        da, mag = ref.grouped(self.dy, ref.dequantize(*self.down), self.offsets, True)
        e = ref.sum_error(mag, self.D)
        h, u = self.h.double(), self.u.double()
        f, s = ref.act_value(self.act, h), ref.act_slope(self.act, h)
        ef, es = ref.act_error(self.act, h)
        want = {"dh": (da * u * s, e * (u * s).abs() + (da.abs() + e) * u.abs() * es + 8 * ref.U32 * (da * u * s).abs()),
                "du": (da * f, e * f.abs() + (da.abs() + e) * ef + 8 * ref.U32 * (da * f).abs()),
                "a": (f * u, ef * u.abs() + 8 * ref.U32 * (f * u).abs())}
        for (name, (exact, err)), t in zip(want.items(), got):
            if t is not None:
                ref.check(t, exact, ref.rounded(exact, err, self.dtype), f"{what}: {name}")

    def check_up_bwd(self, dx, what):
        (a, ma), (b, mb) = (ref.grouped(x, ref.dequantize(*w), self.offsets, True)
                            for x, w in ((self.dh, self.gate), (self.du, self.up)))
        err = ref.sum_error(ma + mb, 2 * self.F)
        ref.check(dx, a + b, ref.rounded(a + b, err, self.dtype), f"{what}: dx")


SIZES = [  # T, E, D, F
    (1, 1, 128, 128), (1, 1, 7, 3), (2, 3, 130, 65), (17, 1, 256, 192), (33, 2, 64, 64), (128, 1, 128, 64),
    (129, 4, 100, 300), (300, 5, 521, 257), (257, 3, 384, 640), (1000, 9, 144, 48), (70, 70, 136, 72),
    (150, 2, 132, 260), (140, 1, 252, 68), (200, 3, 196, 324), (90, 2, 70, 134),
]


@pytest.mark.parametrize("T,E,D,F", SIZES)
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu")])
def test_calls_against_float64(T, E, D, F, dtype, act):
    c = Case(T, E, D, F, dtype, act)
    what = f"{T} rows, {E} experts, {D} x {F}, {dtype}, {act}"
    print("#", what, flush=True)
    c.check_up(c.run_up(), what)
    h, u, a = c.run_up(keep=False)
    assert bool((h == 7.0).all()) and bool((u == 7.0).all())
    c.check_up((None, None, a), what)
    y, dx = c.out(D), c.out(D)
    fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *c.dev("down"), c.dev("offsets"), y)
    c.check_down(y, what)
    for keep in (True, False):
        dh, du, a = (c.out(F) for _ in range(3))
        fz.fp8z1_ffn_down_bwd(c.cfg, c.dev("dy"), *c.dev("down"), c.dev("h"), c.dev("u"), c.dev("offsets"), dh, du,
                              a if keep else None)
        c.check_down_bwd((dh, du, a if keep else None), what)
        assert keep or bool((a == 7.0).all())
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *c.dev("gate"), *c.dev("up"), c.dev("offsets"), dx)
    c.check_up_bwd(dx, what)


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_one_expert_without_offsets(T):
    c = Case(T, 1, 320, 192, one_run=True)
    c.check_up(c.run_up(), f"{T} rows")
    y = c.out(c.D)
    fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *c.dev("down"), None, y)
    c.check_down(y, f"{T} rows")


@pytest.mark.parametrize("T,E,D,F", [(150, 2, 2176, 130), (300, 1, 130, 2300), (100, 2, 2053, 1111), (200, 1, 4096, 1088)])
@pytest.mark.parametrize("far", [False, True])
def test_long_sums_split_over_workgroups(T, E, D, F, far):
    """Few tiles and long sums: with a workspace each call splits its tiles along k."""
    c = Case(T, E, D, F, "bf16", "gelu", lo=-40.0 if far else -3.0, hi=30.0 if far else 3.0)
    what = f"{T} rows, {E} experts, {D} x {F}"
    print("#", what, flush=True)
    ws = torch.empty(fz.fp8z1_ffn_workspace_bytes(c.cfg), dtype=torch.uint8, device="cuda")
    assert ws.numel()
    h, u, a, dh, du, a2 = (c.out(F) for _ in range(6))
    y, dx = c.out(D), c.out(D)
    off = c.dev("offsets")
    fz.fp8z1_ffn_up(c.cfg, c.dev("x"), *c.dev("gate"), *c.dev("up"), off, h, u, a, workspace=ws)
    c.check_up((h, u, a), what)
    fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *c.dev("down"), off, y, workspace=ws)
    c.check_down(y, what)
    fz.fp8z1_ffn_down_bwd(c.cfg, c.dev("dy"), *c.dev("down"), c.dev("h"), c.dev("u"), off, dh, du, a2, workspace=ws)
    c.check_down_bwd((dh, du, a2), what)
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *c.dev("gate"), *c.dev("up"), off, dx, workspace=ws)
    c.check_up_bwd(dx, what)


def wgrad_check(p, q, E, offsets, got, dtype, what, start=None):
    T = p.shape[0]
    exact = torch.zeros(E, p.shape[1], q.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(exact)
    n = 0
    for e, lo, hi in ref.runs(offsets, T):
        exact[e] = p[lo:hi].double().t() @ q[lo:hi].double()
        mag[e] = p[lo:hi].double().abs().t() @ q[lo:hi].double().abs()
        n = max(n, hi - lo)
    err = ref.sum_error(mag, n)
    if start is not None:
        exact += start.double()
        err += ref.U32 * (exact.abs() + err)
    ref.check(got, exact, ref.rounded(exact, err, dtype), what)


@pytest.mark.parametrize("T,E,M,N", [(0, 2, 5, 9), (1, 1, 3, 7), (2, 3, 128, 128), (63, 1, 65, 130), (64, 2, 16, 8),
                                     (129, 4, 200, 136), (1000, 3, 257, 129), (5000, 1, 70, 40), (3000, 2, 33, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weight_gradient(T, E, M, N, dtype):
    g = torch.Generator().manual_seed(T + E + M + N)
    p, q = (torch.randn(T, w, generator=g).to(TYPES[dtype]) for w in (M, N))
    offsets = ref.make_offsets(g, T, E)
    code = {"bf16": fz.BF16, "f16": fz.F16}[dtype]
    need = fz.fp8z1_ffn_wgrad_workspace_bytes(T, E, M, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    print(f"# {T} rows, {E} experts, {M} x {N}, workspace {need}", flush=True)
    dev = [t.cuda() for t in (p, q, offsets)]
    for out, t in ((fz.F32, torch.float32), (fz.BF16, torch.bfloat16)):
        for w in {None, ws}:
            dw = torch.full((E, M, N), float("nan"), dtype=t, device="cuda")
            fz.fp8z1_ffn_wgrad(T, E, M, N, code, dev[0], dev[1], dev[2], out, dw, workspace=w)
            wgrad_check(p, q, E, offsets, dw, t, f"dw {t}, workspace {w is not None}")
    start = torch.randn(E, M, N, generator=g)
    for w in {None, ws}:
        dw = start.cuda()
        fz.fp8z1_ffn_wgrad(T, E, M, N, code, dev[0], dev[1], dev[2], fz.F32, dw, accumulate=True, workspace=w)
        wgrad_check(p, q, E, offsets, dw, torch.float32, "accumulated dw", start)


@pytest.mark.parametrize("T,E,D,F", [(0, 2, 40, 24), (1, 1, 130, 66), (150, 3, 200, 136), (4000, 1, 72, 264),
                                     (3000, 2, 133, 65)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_three_weight_gradients_at_once(T, E, D, F, dtype):
    c = Case(T, E, D, F, dtype)
    dev = [c.dev(n) for n in ("x", "a", "dy", "dh", "du")]
    want = ((c.dh, c.x), (c.du, c.x), (c.dy, c.a))
    for t in (torch.float32, torch.bfloat16):
        dw = block.ffn_backward_weights(*dev, n_experts=E, offsets=c.dev("offsets"), dtype=t)
        for (p, q), got in zip(want, dw):
            wgrad_check(p, q, E, c.offsets, got, t, f"{t}")
    start = [torch.randn(w.shape, generator=torch.Generator().manual_seed(5)) for w in dw]
    out = [s.cuda() for s in start]
    got = block.ffn_backward_weights(*dev, n_experts=E, offsets=c.dev("offsets"), out=out)
    for (p, q), g, s, o in zip(want, got, start, out):
        assert g is o
        wgrad_check(p, q, E, c.offsets, g, torch.float32, "added", s)


def test_rows_and_codes_at_any_alignment():
    """Every buffer one element past a 16-byte boundary, codes at odd addresses."""
    c = Case(150, 2, 192, 160)

    def shift(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten().cuda()
        return flat[1:].view(t.shape)

    gate, up, down = ((shift(w[0]), shift(w[1])) for w in (c.gate, c.up, c.down))
    off = shift(c.offsets)
    h, u, a, dh, du, a2 = (shift(torch.zeros(c.T, c.F, dtype=c.dtype)) for _ in range(6))
    y, dx = (shift(torch.zeros(c.T, c.D, dtype=c.dtype)) for _ in range(2))
    fz.fp8z1_ffn_up(c.cfg, shift(c.x), *gate, *up, off, h, u, a)
    c.check_up((h, u, a), "shifted")
    fz.fp8z1_ffn_down(c.cfg, shift(c.a), *down, off, y)
    c.check_down(y, "shifted")
    fz.fp8z1_ffn_down_bwd(c.cfg, shift(c.dy), *down, shift(c.h), shift(c.u), off, dh, du, a2)
    c.check_down_bwd((dh, du, a2), "shifted")
    fz.fp8z1_ffn_up_bwd(c.cfg, shift(c.dh), shift(c.du), *gate, *up, off, dx)
    c.check_up_bwd(dx, "shifted")
    dw = shift(torch.zeros(c.E, c.F, c.D))
    fz.fp8z1_ffn_wgrad(c.T, c.E, c.F, c.D, fz.BF16, shift(c.dh), shift(c.x), off, fz.F32, dw)
    wgrad_check(c.dh, c.x, c.E, c.offsets, dw, torch.float32, "shifted dw")


@pytest.mark.parametrize("T", [3, 150])
def test_scales_far_apart(T):
    """Block scales from 2^-60 to 2^40 next to each other: each block's partial sum is scaled by its own."""
    c = Case(T, 2, 520, 140, lo=-60.0, hi=40.0)
    c.check_up(c.run_up(), "far scales")
    c = Case(T, 2, 140, 520, lo=-60.0, hi=40.0)
    dx = c.out(c.D)
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *c.dev("gate"), *c.dev("up"), c.dev("offsets"), dx)
    c.check_up_bwd(dx, "far scales")


@pytest.mark.parametrize("T,D,F", [(4, 200, 100), (200, 200, 100), (200, 201, 101), (200, 256, 128)])
def test_special_values_stay_in_their_row(T, D, F):
    """A NaN code reaches only its column, an infinite activation only its row, whatever the
    tile edges: neighbours across a row's end and past the last k stay out of the sums."""
    c = Case(T, 2, D, F)
    c.offsets = torch.tensor([0, T // 2, T], dtype=torch.int32)
    for w, row in ((c.gate, 3), (c.up, F - 1), (c.down, D - 1)):
        w[0][0, row, 0] = 0x7F  # first element of a row: right behind the row before it
        w[0][1, row - 1, -1] = 0xFF
    c.x[1, 0] = float("inf")
    c.a[1, 0] = float("-inf")
    h, u, a = c.run_up()
    hd, ud = (ref.grouped(c.x, ref.dequantize(*w), c.offsets, False)[0] for w in (c.gate, c.up))
    for name, got, exact in (("h", h, hd), ("u", u, ud)):
        assert torch.equal(torch.isfinite(got).cpu(), torch.isfinite(exact)), name
    y = c.out(c.D)
    fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *c.dev("down"), c.dev("offsets"), y)
    yd = ref.grouped(c.a, ref.dequantize(*c.down), c.offsets, False)[0]
    assert torch.equal(torch.isfinite(y).cpu(), torch.isfinite(yd)), "y"
    # transposed products: the codes' rows are summed over
    c.dh[0, 5] = float("nan")
    dx = c.out(c.D)
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *c.dev("gate"), *c.dev("up"), c.dev("offsets"), dx)
    parts = [ref.grouped(x, ref.dequantize(*w), c.offsets, True)[0] for x, w in ((c.dh, c.gate), (c.du, c.up))]
    assert torch.equal(torch.isfinite(dx).cpu(), torch.isfinite(parts[0] + parts[1])), "dx"
    # a token's infinity reaches its expert's gradient only
    dw = torch.empty(2, c.F, c.D, device="cuda")
    fz.fp8z1_ffn_wgrad(T, 2, c.F, c.D, fz.BF16, c.du.cuda(), c.x.cuda(), c.dev("offsets"), fz.F32, dw)
    assert not torch.isfinite(dw[0, :, 0]).any() and torch.isfinite(dw[0, :, 1:]).all() and torch.isfinite(dw[1]).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_at_the_ends(act):
    """h from 0 to the largest bfloat16: finite values give finite gradients of the right size."""
    h = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 16.0, -16.0, 17.0, -17.0, 88.0, -88.0, 104.0, -104.0, 1e4,
                      -1e4, 1e13, -1e13, 3e38, -3e38], dtype=torch.bfloat16)
    T, F, D = h.numel(), 8, 128
    c = Case(T, 1, D, F, act=act, one_run=True)
    c.h = h[:, None].repeat(1, F).contiguous()
    c.u = torch.ones_like(c.h)
    dh, du, a = (c.out(F) for _ in range(3))
    fz.fp8z1_ffn_down_bwd(c.cfg, c.dev("dy"), *c.dev("down"), c.dev("h"), c.dev("u"), None, dh, du, a)
    hd = c.h.double()
    v = hd if act == "silu" else 2 * 0.7978845608028654 * (hd + 0.044715 * hd ** 3)
    dv = torch.ones_like(hd) if act == "silu" else 2 * 0.7978845608028654 * (1 + 3 * 0.044715 * hd ** 2)
    s = torch.sigmoid(v)
    tail = torch.sigmoid(-v)
    f, slope = hd * s, s + hd * dv * s * tail
    slope = torch.where(torch.isfinite(slope), slope, s)
    ref.check(a, f, ref.rounded(f, ref.act_error(act, hd.clamp(-1e4, 1e4))[0] + 8 * ref.U32 * f.abs(), c.dtype), "a")
    da, mag = ref.grouped(c.dy, ref.dequantize(*c.down), None, True)
    e = ref.sum_error(mag, D)
    es = ref.act_error(act, hd.clamp(-1e4, 1e4))[1]
    ref.check(dh, da * slope, ref.rounded(da * slope, e * slope.abs() + (da.abs() + e) * es, c.dtype), "dh")


def test_rows_without_an_expert_are_left_alone():
    """Offsets that leave rows out, and offsets out of range: only covered rows are written."""
    c = Case(300, 3, 136, 72)
    c.offsets = torch.tensor([10, 40, 40, 200], dtype=torch.int32)
    h, u, a = c.run_up()
    for t in (h, u, a):
        assert bool((t[:10] == 7.0).all()) and bool((t[200:] == 7.0).all())
    cover = slice(10, 200)
    d = ref.grouped(c.x, ref.dequantize(*c.gate), c.offsets, False)[0]
    assert float((h[cover].cpu().double() - d[cover]).abs().max()) < 0.05 * float(d.abs().max())
    c.offsets = torch.tensor([-50, 20, 10, 100000], dtype=torch.int32)  # clamped: 0..20, none, 10..300
    h2 = c.run_up()[0]
    assert torch.isfinite(h2).all()


def test_same_bits_every_time():
    c = Case(700, 3, 264, 136)
    g = torch.Generator().manual_seed(3)
    p, q = (torch.randn(9000, 40, generator=g).bfloat16().cuda() for _ in range(2))
    first = None
    for _ in range(3):
        out = [*c.run_up(), block.ffn_weight_gradient(p, q)]
        if first is None:
            first = out
        assert all(torch.equal(x, y) for x, y in zip(first, out))


def _layer(c):
    gate, up, down, off = c.dev("gate"), c.dev("up"), c.dev("down"), c.dev("offsets")

    def run(x, dy):
        y, (h, u, a) = block.ffn_forward(x, gate, up, down, off, c.act, save=True)
        dx, dh, du, a2 = block.ffn_backward_data(dy, h, u, gate, up, down, off, c.act)
        dw = block.ffn_backward_weights(x, a2, dy, dh, du, c.E, off)
        return [y, h, u, a, dx, dh, du, a2, *dw]

    return run


@pytest.mark.parametrize("T,F", [(6, 160), (400, 160), (200, 1200)])
def test_graph_replays_equal_eager(T, F):
    c = Case(T, 3, 264, F)
    run = _layer(c)
    x, dy = c.dev("x"), c.dev("dy")
    run(x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(x, dy)
    for i in range(3):
        g = torch.Generator().manual_seed(50 + i)
        x.copy_(torch.randn(c.T, c.D, generator=g))
        dy.copy_(torch.randn(c.T, c.D, generator=g))
        want = run(x, dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {i}"


def test_side_stream_equals_default_stream():
    c = Case(333, 2, 200, 120)
    run = _layer(c)
    x, dy = c.dev("x"), c.dev("dy")
    want = run(x, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(x * 1, dy * 1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_against_differences():
    """Central differences of the block's float64 value along random directions agree with the
    library's dx and weight gradients, to the size of the 16-bit roundings in between
    (each gradient goes through at most four of them, relative 2^-11 in half precision) and of the
    difference's own error."""
    c = Case(60, 2, 160, 96, "f16", "gelu")
    run = _layer(c)
    y, h, u, a, dx, dh, du, a2, dwg, dwu, dwd = run(c.dev("x"), c.dev("dy"))
    W = [ref.dequantize(*w) for w in (c.gate, c.up, c.down)]
    dy = c.dy.double()

    def value(x, wg, wu, wd):
        h, u = (ref.grouped(x, w, c.offsets, False)[0] for w in (wg, wu))
        return float((ref.grouped(ref.act_value(c.act, h) * u, wd, c.offsets, False)[0] * dy).sum())

    g = torch.Generator().manual_seed(9)
    for i, grad in enumerate((dx, dwg, dwu, dwd)):
        base = [c.x.double(), *W]
        grad = grad.cpu().double()
        d = torch.randn(base[i].shape, generator=g, dtype=torch.float64) * base[i].abs().mean()
        step = 1e-4
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + step * d, base[i] - step * d
        slope = (value(*plus) - value(*minus)) / (2 * step)
        # independent roundings of the elements: four each, so 4 * 2^-11 of the root of the sum of squares
        # would be 1 standard deviation at most; 6 of them are allowed
        allowed = 6 * 4 * 2.0 ** -11 * float((grad * d).norm()) + 1e-5 * abs(slope)
        assert abs(float((grad * d).sum()) - slope) <= allowed, (i, float((grad * d).sum()), slope, allowed)


def test_block_refuses_what_does_not_fit():
    c = Case(8, 2, 64, 32)
    x, gate, up, down, off = (c.dev(n) for n in ("x", "gate", "up", "down", "offsets"))
    E = fz.Fp8z1Error
    for bad in (dict(x=x.float()), dict(x=x[:, :40].contiguous()), dict(w_down=gate), dict(offsets=None),
                dict(offsets=off[:2]), dict(offsets=off.long()), dict(act="relu"), dict(x=x.t().contiguous().t()),
                dict(w_up=(up[0], up[1][:1])), dict(w_gate=(gate[0].float(), gate[1])), dict(x=x.cpu())):
        kw = dict(x=x, w_gate=gate, w_up=up, w_down=down, offsets=off, act="silu") | bad
        with pytest.raises(E):
            block.ffn_forward(**kw)
    with pytest.raises(E):
        block.ffn_weight_gradient(x, c.dev("h")[:4])
    with pytest.raises(E):
        block.ffn_weight_gradient(x, x, n_experts=2)
    with pytest.raises(E):
        block.ffn_weight_gradient(x, x, dtype=torch.float16)


@pytest.mark.parametrize("dtype,value", [("f16", 2.0 ** -20), ("bf16", 2.0 ** -130)])
@pytest.mark.parametrize("T", [3, 150])
def test_subnormal_activations_count(T, dtype, value):
    """Activations below the type's normal range: D equal ones times codes of 1 give D times the value."""
    c = Case(T, 1, 256, 64, dtype, one_run=True)
    c.x = torch.full_like(c.x, value)
    c.gate = (torch.full_like(c.gate[0], 0x38), torch.ones_like(c.gate[1]))
    h, _, _ = c.run_up()
    assert torch.equal(h.cpu(), torch.full((T, c.F), 256 * value, dtype=c.dtype))
    c.du, c.dh = torch.zeros_like(c.du), torch.full_like(c.dh, value)
    dx = c.out(c.D)
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *c.dev("gate"), *c.dev("up"), None, dx)
    assert torch.equal(dx.cpu(), torch.full((T, c.D), 64 * value, dtype=c.dtype))
    dw = torch.empty(1, c.F, c.D, device="cuda")
    ones = torch.ones(T, c.D, dtype=c.dtype, device="cuda")
    fz.fp8z1_ffn_wgrad(T, 1, c.F, c.D, c.cfg.dtype, c.dev("dh"), ones, None, fz.F32, dw)
    assert torch.equal(dw.cpu(), torch.full((1, c.F, c.D), T * value))


def test_no_rows():
    c = Case(0, 2, 64, 32)
    gate, up, down, off = c.dev("gate"), c.dev("up"), c.dev("down"), c.dev("offsets")
    y, (h, u, a) = block.ffn_forward(c.dev("x"), gate, up, down, off, save=True)
    assert y.shape == (0, 64) and h.shape == u.shape == a.shape == (0, 32)
    out = block.ffn_backward_data(c.dev("dy"), h, u, gate, up, down, off)
    assert [tuple(t.shape) for t in out] == [(0, 64), (0, 32), (0, 32), (0, 32)]


@pytest.mark.parametrize("bad", [0.0, -2.0, float("nan"), float("inf"), 2.0 ** -140])
def test_any_scale(bad):
    """One block with a scale that is zero, negative, not finite or subnormal: it counts as it is."""
    for T in (5, 140):
        c = Case(T, 1, 384, 256, one_run=True)
        c.gate[1][0, 0, 1] = bad
        c.down[1][0, 1, 0] = bad
        h, u, _ = c.run_up()
        exact, mag = ref.grouped(c.x, ref.dequantize(*c.gate), None, False)
        err = ref.sum_error(mag, c.D)
        if bad == float("inf"):  # sums of infinities of both signs: no number
            assert not torch.isfinite(h[:, :128]).any() and torch.isfinite(h[:, 128:]).all()
        else:
            ref.check(h, exact, ref.rounded(exact, err, c.dtype), f"h, scale {bad}")
        dh, du, a = (c.out(c.F) for _ in range(3))
        fz.fp8z1_ffn_down_bwd(c.cfg, c.dev("dy"), *c.dev("down"), c.dev("h"), c.dev("u"), None, dh, du, a)
        if bad == bad and abs(bad) != float("inf"):
            c.check_down_bwd((dh, du, a), f"scale {bad}")
        else:
            assert not torch.isfinite(du[:, :128]).any() and torch.isfinite(du[:, 128:]).all()


def test_rows_past_four_gigabytes():
    """Rows whose byte offsets need more than 32 bits, forward and backward."""
    T, D, F = 310000, 7168, 24
    g = torch.Generator().manual_seed(1)
    gate, up, down = (tuple(t.cuda() for t in ref.make_weight(g, 2, *s)) for s in ((F, D), (F, D), (D, F)))
    offsets = torch.tensor([0, 200, T], dtype=torch.int32, device="cuda")
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(150, D, generator=g).bfloat16()
    x[-150:] = tail.cuda()
    y, (h, u, a) = block.ffn_forward(x, gate, up, down, offsets, save=True)
    w = [ref.dequantize(c.cpu()[1:], s.cpu()[1:]) for c, s in (gate, up, down)]
    hd, mag = ref.grouped(tail, w[0], None, False)
    ref.check(h[-150:], hd, ref.rounded(hd, ref.sum_error(mag, D), torch.bfloat16), "far h")
    yd, mag = ref.grouped(a[-150:].cpu(), w[2], None, False)
    ref.check(y[-150:], yd, ref.rounded(yd, ref.sum_error(mag, F), torch.bfloat16), "far y")
    assert not y[:-150].any() and not h[:-150].any()
    dx, dh, du, _ = block.ffn_backward_data(x, h, u, gate, up, down, offsets)
    exact = [ref.grouped(d[-150:].cpu(), m, None, True) for d, m in ((dh, w[0]), (du, w[1]))]
    total, mag = exact[0][0] + exact[1][0], exact[0][1] + exact[1][1]
    ref.check(dx[-150:], total, ref.rounded(total, ref.sum_error(mag, 2 * F), torch.bfloat16), "far dx")
    dw = block.ffn_weight_gradient(dh, x, 2, offsets)
    want = dh[-150:].cpu().double().t() @ tail.double()
    mag = dh[-150:].cpu().double().abs().t() @ tail.double().abs()
    # (rows of zeros add nothing: the sum has 150 terms)
    ref.check(dw[1], want, ref.rounded(want, ref.sum_error(mag, 150), torch.float32), "far dw")
    assert not dw[0].any()


@pytest.mark.parametrize("T,E,D,F", [(40, 1, 2176, 132), (33, 1, 260, 2304), (70, 2, 2176, 132), (129, 1, 2176, 132)])
def test_split_tiles_of_few_rows(T, E, D, F):
    """What the workspace held before is not read: rows past a run have no partial sums."""
    c = Case(T, E, D, F)
    what = f"{T} rows, {E} experts, {D} x {F}"
    print("#", what, flush=True)
    off = c.dev("offsets")

    def ws():
        return torch.full((fz.fp8z1_ffn_workspace_bytes(c.cfg),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN

    h, u, a, dh, du, a2 = (c.out(F) for _ in range(6))
    y, dx = c.out(D), c.out(D)
    fz.fp8z1_ffn_up(c.cfg, c.dev("x"), *c.dev("gate"), *c.dev("up"), off, h, u, a, workspace=ws())
    c.check_up((h, u, a), what)
    fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *c.dev("down"), off, y, workspace=ws())
    c.check_down(y, what)
    fz.fp8z1_ffn_down_bwd(c.cfg, c.dev("dy"), *c.dev("down"), c.dev("h"), c.dev("u"), off, dh, du, a2, workspace=ws())
    c.check_down_bwd((dh, du, a2), what)
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *c.dev("gate"), *c.dev("up"), off, dx, workspace=ws())
    c.check_up_bwd(dx, what)


@pytest.mark.parametrize("T", [31, 32])
def test_few_rows_of_large_weights(T):
    """Either side of where the projections' 52 million codes go from the row kernel to tiles."""
    c = Case(T, 1, 5120, 5120)
    print("#", T, "rows", flush=True)
    ws = torch.full((fz.fp8z1_ffn_workspace_bytes(c.cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    h, u, a = (c.out(c.F) for _ in range(3))
    fz.fp8z1_ffn_up(c.cfg, c.dev("x"), *c.dev("gate"), *c.dev("up"), c.dev("offsets"), h, u, a, workspace=ws)
    c.check_up((h, u, a), f"{T} rows")


@pytest.mark.parametrize("count", [2, 4])
def test_weight_gradients_refuse_another_count_of_outputs(count):
    x, a = (torch.zeros(3, n, dtype=torch.bfloat16, device="cuda") for n in (16, 8))
    out = [torch.zeros(1, 8, 16, device="cuda"), torch.zeros(1, 8, 16, device="cuda"),
           torch.zeros(1, 16, 8, device="cuda"), torch.zeros(1, 16, 8, device="cuda")][:count]
    with pytest.raises(fz.Fp8z1Error, match="expected 3"):
        block.ffn_backward_weights(x, a, x, a, a, out=out)
