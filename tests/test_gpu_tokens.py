"""GPU: the sorted plan, the rows copied to their places and back, and the gradients."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import rows8_reference as r8  # noqa: E402

pytestmark = pytest.mark.gpu
U = ref.U32
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def routing():
    from blockwise_fp8_zero_fold_amd import routing as r
    return r


def plan(experts, E):
    """(offsets, row_of) choice by choice."""
    flat = experts.reshape(-1).tolist()
    count = [0] * E
    for e in flat:
        if 0 <= e < E:
            count[e] += 1
    first = [0]
    for c in count:
        first.append(first[-1] + c)
    at, rows = first[:E], []
    for e in flat:
        if 0 <= e < E:
            rows.append(at[e])
            at[e] += 1
        else:
            rows.append(-1)
    return torch.tensor(first, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32).view(experts.shape)


def make_experts(g, T, k, E, drop=0.1):
    e = (torch.rand(T, k, generator=g) ** 2 * E).to(torch.int32).clamp(max=E - 1)
    e[torch.rand(T, k, generator=g) < drop] = -1
    return e


@pytest.mark.parametrize("T,k,E", [(0, 1, 3), (1, 1, 1), (3, 8, 64), (64, 1, 2), (65, 1, 7), (1000, 4, 1), (1024, 4, 33),
                                   (1365, 3, 1024), (4097, 1, 5), (2050, 2, 1000), (8192, 8, 256), (70001, 5, 64),
                                   (90001, 32, 1024)])
def test_sort(T, k, E):
    g = torch.Generator().manual_seed(T + E)
    e = make_experts(g, T, k, E)
    if T > 2:
        e[1, 0], e[2, 0] = E, 2 ** 31 - 1  # out of range
    offsets, row_of = routing().sort_tokens(e.cuda(), E)
    want = plan(e, E)
    assert torch.equal(offsets.cpu(), want[0]) and torch.equal(row_of.cpu(), want[1])


def test_sort_one_expert_takes_all_and_none():
    r = routing()
    for T in (100, 20000):
        for fill, E in ((5, 9), (-1, 9), (9, 9), (0, 1)):
            e = torch.full((T, 2), fill, dtype=torch.int32)
            offsets, row_of = r.sort_tokens(e.cuda(), E)
            want = plan(e, E)
            assert torch.equal(offsets.cpu(), want[0]) and torch.equal(row_of.cpu(), want[1])


SIZES = [(1, 1, 1, 1), (3, 8, 64, 7168), (5, 2, 3, 7), (17, 3, 4, 8), (33, 4, 9, 15), (9, 1, 2, 129), (50, 6, 5, 1001),
         (7, 32, 40, 520), (11, 9, 12, 4099), (3, 2, 4, 20011), (300, 2, 3, 64), (2, 8, 8, 8193)]


@pytest.mark.parametrize("T,k,E,D", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_dispatch(T, k, E, D, dtype):
    g = torch.Generator().manual_seed(D)
    e = make_experts(g, T, k, E)
    _, row_of = plan(e, E)
    x = torch.randn(T, D, generator=g).to(dtype)
    out = torch.full((T * k + 3, D), 7.0, dtype=dtype)
    want = out.clone()
    for t in range(T):
        for j in range(k):
            if row_of[t, j] >= 0:
                want[row_of[t, j]] = x[t]
    got = routing().dispatch(x.cuda(), row_of.cuda(), out=out.cuda())
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("T,k,E,D", SIZES)
def test_dispatch_8_bits(T, k, E, D):
    g = torch.Generator().manual_seed(D)
    _, row_of = plan(make_experts(g, T, k, E), E)
    codes, scales = r8.make_rows8(g, T, D)
    rows = torch.full((T * k, D), 3, dtype=torch.uint8), torch.full((T * k, scales.shape[1]), 3.0)
    want = tuple(r.clone() for r in rows)
    for t in range(T):
        for j in range(k):
            if row_of[t, j] >= 0:
                want[0][row_of[t, j]], want[1][row_of[t, j]] = codes[t], scales[t]
    got = routing().dispatch((codes.cuda(), scales.cuda()), row_of.cuda(), out=tuple(r.cuda() for r in rows))
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


@pytest.mark.parametrize("T,k,E,D", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_combine(T, k, E, D, dtype):
    g = torch.Generator().manual_seed(D + 1)
    _, row_of = plan(make_experts(g, T, k, E), E)
    rows, base = torch.randn(T * k, D, generator=g).to(dtype), torch.randn(T, D, generator=g).to(dtype)
    used = row_of[row_of >= 0].long()
    left = torch.ones(T * k, dtype=torch.bool)
    left[used] = False
    rows[left] = float("nan")  # rows that no choice has are not read
    w = torch.randn(T, k, generator=g)
    there = row_of >= 0
    picked = torch.where(there[:, :, None], rows.double()[row_of.clamp(min=0).long()], torch.zeros(1, dtype=torch.float64))
    for weights in (w, None):
        for add in (base, None):
            terms = picked * (weights.double()[:, :, None] if weights is not None else 1.0)
            exact, mag = terms.sum(1), terms.abs().sum(1)
            if add is not None:
                exact, mag = exact + add.double(), mag + add.double().abs()
            got = routing().combine(rows.cuda(), row_of.cuda(), None if weights is None else w.cuda(),
                                    None if add is None else base.cuda())
            assert got.dtype == dtype
            ref.check(got, exact, ref.rounded(exact, (2 * k + 2) * U * mag, dtype), "y")


@pytest.mark.parametrize("T,k,E,D", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_combine_backward(T, k, E, D, dtype):
    g = torch.Generator().manual_seed(D + 2)
    _, row_of = plan(make_experts(g, T, k, E), E)
    rows, dy = torch.randn(T * k, D, generator=g).to(dtype), torch.randn(T, D, generator=g).to(dtype)
    w = torch.randn(T, k, generator=g)
    out = torch.full((T * k, D), 5.0, dtype=dtype)
    drows, dw = routing().combine_backward(dy.cuda(), rows.cuda(), row_of.cuda(), w.cuda(), out=out.cuda())
    want, dwant, mag = out.double(), torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    bound = torch.zeros_like(want)
    for t in range(T):
        for j in range(k):
            r = int(row_of[t, j])
            if r < 0:
                continue
            want[r] = w[t, j].double() * dy[t].double()
            bound[r] = ref.rounded(want[r], U * want[r].abs(), dtype)
            terms = dy[t].double() * rows[r].double()
            dwant[t, j], mag[t, j] = terms.sum(), terms.abs().sum()
    ref.check(drows, want, bound, "drows")
    ref.check(dw, dwant, ref.sum_error(mag, D), "dweights")


def test_gradients_against_differences():
    """y is linear in the rows and in the weights: <dy, y> changes by the gradients' products with any step."""
    g = torch.Generator().manual_seed(8)
    T, k, E, D = 6, 3, 4, 40
    _, row_of = plan(make_experts(g, T, k, E), E)
    rows, w, dy = torch.randn(T * k, D, generator=g), torch.randn(T, k, generator=g), torch.randn(T, D, generator=g)
    drows, dw = routing().combine_backward(dy.cuda(), rows.cuda(), row_of.cuda(), w.cuda(),
                                           out=torch.zeros(T * k, D, device="cuda"))

    def loss(r, v):
        return float((routing().combine(r.cuda(), row_of.cuda(), v.cuda()).cpu().double() * dy.double()).sum())

    step_r, step_w = torch.randn(T * k, D, generator=g), torch.randn(T, k, generator=g)
    by_rows = (loss(rows + step_r, w) - loss(rows - step_r, w)) / 2
    by_w = (loss(rows, w + step_w) - loss(rows, w - step_w)) / 2
    assert abs(by_rows - float((drows.cpu().double() * step_r.double()).sum())) < 1e-3
    assert abs(by_w - float((dw.cpu().double() * step_w.double()).sum())) < 1e-3


@pytest.mark.parametrize("T,k,D,dtype", [(50, 3, 7168, torch.bfloat16), (9, 20, 1001, torch.float16), (300, 2, 63, torch.float32)])
def test_gradient_in_place_of_the_rows(T, k, D, dtype):
    g = torch.Generator().manual_seed(T)
    _, row_of = routing().sort_tokens(make_experts(g, T, k, 40).cuda(), 40)
    rows, dy = torch.randn(T * k, D, generator=g).to(dtype).cuda(), torch.randn(T, D, generator=g).to(dtype).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    out = rows.clone()  # (rows that no choice has stay)
    drows, dw = routing().combine_backward(dy, rows, row_of, w, out=out)
    same, dw2 = routing().combine_backward(dy, rows, row_of, w, out=rows)
    assert same is rows and torch.equal(rows, drows) and torch.equal(dw, dw2)


def test_nan_and_infinite_rows():
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([[nan], [1.0], [inf]], device="cuda")
    row_of = torch.tensor([[0, -1], [1, -1], [2, 1], [-1, -1], [3, -5]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, nan], [2.0, inf], [1.0, 1.0], [nan, nan], [nan, nan]], device="cuda")
    y = routing().combine(rows, row_of, w).cpu()[:, 0].tolist()
    assert y[0] != y[0] and y[1] == 2.0 and y[2] == inf and y[3] == 0.0 and y[4] == 0.0


def test_base_in_place_unaligned_and_no_rows():
    import blockwise_fp8_zero_fold_amd as fz
    r = routing()
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(1 + 12 * 33, generator=g).bfloat16().cuda()[1:].view(12, 33)
    row_of = torch.arange(12, dtype=torch.int32).view(6, 2).cuda()
    base = torch.randn(6, 33, generator=g).bfloat16().cuda()
    want = r.combine(rows.clone(), row_of, None, base)
    y = base.clone()
    fz.fp8z1_combine(fz.Routed(6, 33, 12, 2, fz.BF16), row_of, rows, None, y, y)
    assert torch.equal(y, want)
    none = torch.zeros(0, 33, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(r.combine(none, row_of, None, base), base)  # no row is there
    empty = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert r.combine(rows, empty).shape == (0, 33) and r.dispatch(none, empty).shape == (0, 33)
    dr, dw = r.combine_backward(none, rows, empty, torch.zeros(0, 2, device="cuda"))
    assert dr.shape == rows.shape and dw.shape == (0, 2)


def test_the_whole_way_there_and_back_in_a_graph():
    """Sort, dispatch, combine and their gradients captured once, replayed with other choices."""
    r = routing()
    g = torch.Generator().manual_seed(6)
    T, k, E, D = 3000, 4, 40, 264
    e, x = make_experts(g, T, k, E).cuda(), torch.randn(T, D, generator=g).bfloat16().cuda()
    w, dy = torch.rand(T, k, generator=g).cuda(), torch.randn(T, D, generator=g).bfloat16().cuda()

    def step():
        offsets, row_of = r.sort_tokens(e, E)
        rows = r.dispatch(x, row_of, out=torch.zeros(T * k, D, dtype=torch.bfloat16, device="cuda"))
        y = r.combine(rows, row_of, w)
        drows, dw = r.combine_backward(dy, rows, row_of, w, out=torch.zeros_like(rows))
        return offsets, row_of, rows, y, drows, dw, r.combine(drows, row_of)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        e.copy_(make_experts(g, T, k, E))
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))
        # y = sum of w x over the choices that are there
        s = (w * (kept[1] >= 0)).sum(1, keepdim=True)
        assert float((kept[3].float() - s * x.float()).abs().max()) <= 2.0 ** -7 * float((s * x.float()).abs().max())


def test_refusals():
    import blockwise_fp8_zero_fold_amd as fz
    r = routing()
    x, row_of = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    rows, w = torch.zeros(8, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    for call in (lambda: r.sort_tokens(row_of, 0), lambda: r.sort_tokens(row_of, 1025), lambda: r.sort_tokens(row_of.long(), 4),
                 lambda: r.sort_tokens(row_of[0], 4), lambda: r.sort_tokens(row_of.cpu(), 4),
                 lambda: r.dispatch(x, row_of[:3]), lambda: r.dispatch(x.double(), row_of), lambda: r.dispatch(x, row_of.long()),
                 lambda: r.dispatch(x.t(), row_of), lambda: r.dispatch(x, row_of, out=rows.half()),
                 lambda: r.dispatch((x.to(torch.uint8), x), row_of), lambda: r.combine(rows, row_of, w[:2]),
                 lambda: r.combine(rows, row_of, w.half()), lambda: r.combine(rows, row_of, w, x.half()),
                 lambda: r.combine(rows.t(), row_of), lambda: r.combine_backward(x[:2], rows, row_of, w),
                 lambda: r.combine_backward(x, rows, row_of, w, out=rows[:2]),
                 lambda: r.combine(rows, torch.zeros(4, 33, dtype=torch.int32, device="cuda"))):
        with pytest.raises(fz.Fp8z1Error):
            call()
