"""GPU: the router against float64, choices exactly, weights and gradients within bounds counted per rounding."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
U = ref.U32


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def routing():
    from blockwise_fp8_zero_fold_amd import routing as r
    return r


def scores(l, score):
    return torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)


def choose(l, bias, k, score):
    """Choices by float64 ranks, the lowest index among equals; -1 where nothing is left."""
    rank = l if bias is None else scores(l, score) + bias.double()
    rank = torch.where(torch.isnan(l) | (l == -float("inf")), torch.full_like(l, -float("inf")), rank)
    v, i = torch.sort(rank, dim=1, descending=True, stable=True)
    return torch.where(v[:, :k] == -float("inf"), -1, i[:, :k])


def weights_of(l, experts, score, normalize, scale):
    """Weights of given choices as a function of the logits (the chosen ones alone where softmax is normalized)."""
    there = experts >= 0
    at = experts.clamp(min=0)
    chosen = l.gather(1, at)
    if normalize:
        log = chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen)
        w = torch.softmax(torch.where(there, log, torch.full_like(log, -float("inf"))), 1)
        w = torch.where(there.any(1, keepdim=True), w, torch.zeros_like(w))
    else:
        w = scores(l, score).gather(1, at)
    return scale * torch.where(there, w, torch.zeros_like(w))


def relative(l, experts, score):
    """Of a weight: the difference to the largest logit, rounded once, moves its exponential by that size;
    exponentials (2 ulp), sums of positive terms (at most 16 + 6 deep), divisions and the scale come to 64 half steps."""
    fin = torch.where(torch.isfinite(l), l, torch.zeros_like(l))
    far = (fin.amax(1, keepdim=True) - fin).amax(1, keepdim=True) if score == "softmax" else fin.abs().amax(1, keepdim=True)
    return (64 + 4 * far) * U


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (33, 64, 8), (17, 65, 6), (9, 128, 32), (130, 200, 8),
                                   (6, 256, 1), (7, 500, 5), (4, 1024, 32), (2, 1000, 8), (4099, 16, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_route(T, E, k, score, normalize, dtype):
    g = torch.Generator().manual_seed(T * 1000 + E)
    for bias in (None, (torch.randn(E, generator=g) * 0.1)):
        logits = (torch.randn(T, E, generator=g) * 3).to(dtype)
        experts, w = routing().route(logits.cuda(), k, None if bias is None else bias.cuda(), score, normalize, 1.5)
        l = logits.double()
        want = choose(l, bias, k, score)
        assert experts.dtype == torch.int32 and torch.equal(experts.cpu().long(), want), "choices"
        leaf = l.requires_grad_()
        exact = weights_of(leaf, want, score, normalize, 1.5)
        rel = relative(l.detach(), want, score)
        ref.check(w, exact.detach(), exact.detach().abs() * rel + 1e-37, "weights")
        dw = torch.randn(T, k, generator=g)
        got = routing().route_backward(dw.cuda(), logits.cuda(), experts, score, normalize, 1.5)
        dl = torch.autograd.grad(exact, leaf, dw.double())[0]
        # each entry is a sum of products of weights, scores and dw: the sums' magnitudes times the roundings
        ws = exact.detach().abs()
        mag = (ws * dw.double().abs()).sum(1, keepdim=True)
        per = torch.zeros_like(l.detach()).scatter_add_(1, want, ws * (dw.double().abs() + mag / 1.5))
        if score == "softmax" and not normalize:
            per = per + scores(l.detach(), score) * mag
        assert got.dtype == dtype
        ref.check(got, dl, ref.rounded(dl, per * rel + 1e-37, dtype), "dlogits")


def test_ties_go_to_the_lowest_index():
    r = routing()
    for E in (1, 5, 64, 130, 1024):
        k = min(E, 8)
        logits = torch.zeros(3, E, device="cuda")
        want = torch.arange(k, dtype=torch.int32).expand(3, k)
        for bias in (None, torch.zeros(E, device="cuda")):
            for score in ("softmax", "sigmoid"):
                experts, w = r.route(logits, k, bias, score)
                assert torch.equal(experts.cpu(), want)
                assert torch.allclose(w.cpu(), torch.full((3, k), 1.0 / k))
    # equal logits at far places, and a bias that makes sums meet
    logits = torch.tensor([[0.0, 2.0, 1.0, 2.0, 1.0]], device="cuda")
    assert r.route(logits, 4)[0].cpu().tolist() == [[1, 3, 2, 4]]


def test_ranks_closer_than_a_float32_step():
    """Scores that are the same in float32 but not in float64."""
    l = torch.tensor([[20.0, 20.0 + 2.0 ** -18, 19.0, 20.0 + 2.0 ** -17]])
    bias = torch.zeros(4)
    p = torch.sigmoid(l.double())
    assert (p.float()[0, [0, 1, 3]] == p.float()[0, 0]).all() and p[0, 3] > p[0, 1] > p[0, 0]
    assert routing().route(l.cuda(), 3, bias.cuda(), "sigmoid")[0].cpu().tolist() == [[3, 1, 0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(score, normalize, with_bias):
    r, inf, nan = routing(), float("inf"), float("nan")
    bias = torch.zeros(4, device="cuda") if with_bias else None
    l = torch.tensor([[-inf, 1.0, -inf, 2.0], [-inf] * 4, [0.0, -inf, -inf, -inf], [-3.4e38] * 4], device="cuda")
    experts, w = r.route(l, 3, bias, score, normalize)
    assert experts.cpu().tolist() == [[3, 1, -1], [-1, -1, -1], [0, -1, -1], [0, 1, 2]]
    w = w.cpu()
    assert torch.isfinite(w).all() and (w[0, 2] == 0) and (w[1] == 0).all() and (w[2, 1:] == 0).all()
    if normalize:
        assert abs(float(w[0].sum()) - 1) < 1e-6 and float(w[2, 0]) == 1
        assert torch.allclose(w[3], torch.full((3,), 1 / 3))
    elif score == "softmax":
        assert torch.allclose(w[3], torch.full((3,), 0.25))
    d = r.route_backward(torch.ones(4, 3, device="cuda"), l, experts, score, normalize).cpu()
    assert torch.isfinite(d).all() and (d[1] == 0).all() and (d[0, [0, 2]] == 0).all()
    # NaN and infinities: not hidden by softmax, and never chosen if NaN
    l = torch.tensor([[nan, 1.0, 0.5, 2.0], [inf, 1.0, 0.5, 2.0]], device="cuda")
    experts, w = r.route(l, 2, bias, score, normalize)
    assert 0 not in experts[0].cpu().tolist() and experts[0].cpu().tolist() == [3, 1]
    if score == "softmax":
        assert torch.isnan(w[0]).all() and torch.isnan(w[1]).all()
    else:
        assert torch.isfinite(w).all() and experts[1, 0] == 0


def test_sizes_of_logits_that_leave_float32():
    """Normalized weights of scores too small for float32, of either kind."""
    for top in (-300.0, -80.0, 300.0, 3e38):
        l = torch.tensor([[top, top - 1, top - 2, top - 3]]) if abs(top) < 1e30 else torch.tensor([[top, top, -top, 0.0]])
        for score in ("softmax", "sigmoid"):
            experts, w = routing().route(l.cuda(), 3, None, score, True)
            exact = weights_of(l.double(), experts.cpu().long(), score, True, 1.0)
            assert torch.allclose(w.cpu().double(), exact, rtol=1e-6, atol=1e-30), (top, score)
            dw = torch.tensor([[1.0, -2.0, 0.5]])
            leaf = l.double().requires_grad_()
            want = torch.autograd.grad(weights_of(leaf, experts.cpu().long(), score, True, 1.0), leaf, dw.double())[0]
            got = routing().route_backward(dw.cuda(), l.cuda(), experts, score, True)
            assert torch.allclose(got.cpu().double(), want, rtol=1e-5, atol=1e-6), (top, score)


def test_gradient_against_differences():
    """Central differences of the float64 weights, at the framework's own choices."""
    g = torch.Generator().manual_seed(3)
    logits, dw = torch.randn(4, 12, generator=g), torch.randn(4, 3, generator=g)
    for score in ("softmax", "sigmoid"):
        for normalize in (False, True):
            experts, _ = routing().route(logits.cuda(), 3, None, score, normalize)
            got = routing().route_backward(dw.cuda(), logits.cuda(), experts, score, normalize).cpu().double()
            e, l, h = experts.cpu().long(), logits.double(), 1e-5
            for c in range(12):
                step = torch.zeros(4, 12, dtype=torch.float64)
                step[:, c] = h
                diff = (weights_of(l + step, e, score, normalize, 1.0) - weights_of(l - step, e, score, normalize, 1.0))
                assert torch.allclose(got[:, c], (diff * dw.double()).sum(1) / (2 * h), rtol=1e-4, atol=1e-5)


def test_choices_given_by_the_caller():
    """The same expert twice adds up; choices outside 0..E-1 have no gradient."""
    logits = torch.tensor([[1.0, 2.0, 3.0]], device="cuda")
    dw = torch.tensor([[1.0, 2.0]], device="cuda")
    r = routing()
    one = r.route_backward(torch.tensor([[3.0]], device="cuda"), logits, torch.tensor([[1]], dtype=torch.int32, device="cuda"),
                           normalize=False)
    two = r.route_backward(dw, logits, torch.tensor([[1, 1]], dtype=torch.int32, device="cuda"), normalize=False)
    assert torch.allclose(one, two)
    bad = r.route_backward(dw, logits, torch.tensor([[-1, 3]], dtype=torch.int32, device="cuda"), normalize=False)
    assert (bad == 0).all()


def test_refusals():
    import blockwise_fp8_zero_fold_amd as fz
    r, l = routing(), torch.zeros(2, 8, device="cuda")
    e = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    d = torch.zeros(2, 2, device="cuda")
    for call in (lambda: r.route(l, 0), lambda: r.route(l, 9), lambda: r.route(l, -1), lambda: r.route(l.cpu(), 2),
                 lambda: r.route(l.double(), 2), lambda: r.route(l[0], 2), lambda: r.route(l.t(), 2),
                 lambda: r.route(l, 2, torch.zeros(7, device="cuda")), lambda: r.route(l, 2, score="relu"),
                 lambda: r.route(torch.zeros(2, 1025, device="cuda"), 2), lambda: r.route(l, 2, scale=float("nan")),
                 lambda: r.route_backward(d, l, e.long()), lambda: r.route_backward(d[:1], l, e),
                 lambda: r.route_backward(d, l, e[0]), lambda: r.route_backward(d.half(), l, e)):
        with pytest.raises(fz.Fp8z1Error):
            call()
    experts, w = r.route(torch.zeros(0, 8, device="cuda"), 2)
    assert experts.shape == (0, 2) and w.shape == (0, 2)
    assert r.route_backward(w, torch.zeros(0, 8, device="cuda"), experts).shape == (0, 8)


def test_unaligned_rows_side_stream_and_graph():
    """Logits that start two bytes off a 4-byte boundary; on a side stream; captured and replayed."""
    r = routing()
    g = torch.Generator().manual_seed(1)
    base = torch.randn(1 + 37 * 70, generator=g).bfloat16().cuda()
    logits = base[1:].view(37, 70)
    want = r.route(logits.clone(), 4)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = r.route(logits, 4)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = logits.clone()
    dw = torch.ones(37, 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        e, w = r.route(x, 4)
        d = r.route_backward(dw, x, e)
    for i in range(4):
        x.copy_(torch.randn(37, 70, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        we, ww = r.route(x, 4)
        assert torch.equal(e, we) and torch.equal(w, ww) and torch.equal(d, r.route_backward(dw, x, we))
