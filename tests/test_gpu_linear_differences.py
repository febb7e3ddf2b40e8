"""GPU: gradients of a product by central differences, in several directions, held to what the roundings can do."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests.test_gpu_linear import act_error, block, pair, value  # noqa: E402

U, H = ref.U32, 1e-4
T, N, K = 6, 20, 24
DIRECTIONS = 8


def problem(act):
    g = torch.Generator().manual_seed(4)
    w, b = ref.make_weight(g, 1, N, K), torch.randn(1, N, generator=g)
    x, dy = torch.randn(T, K, generator=g).half(), torch.randn(T, N, generator=g).half()
    s = [(torch.randn(T, K, generator=g).double(), torch.randn(1, N, generator=g).double()) for _ in range(DIRECTIONS)]
    return w, b, x, dy, s


def curve(act, h, err):
    """A bound on |act''| within err of h: the value there, and the third derivative (at most 0.31 of h s(h), 0.78 of the tanh
    form of GELU) times err."""
    if act is None:
        return torch.zeros_like(h)
    v = h.clone().requires_grad_()
    first, = torch.autograd.grad(ref.act_value(act, v).sum(), v, create_graph=True)
    return torch.autograd.grad(first.sum(), v)[0].abs() + err


def differences(act):
    """By direction: the differences of <dy, y> in x and in the bias, and what the gradients may be off by along it."""
    w, b, x, dy, directions = problem(act)
    wd = ref.dequantize(*w)[0]

    def loss(xx, bb):
        return float((value(act, xx @ wd.t() + bb) * dy.double()).sum())

    # p is rounded to float16 and moves the slope; the slope's own error, dp's and dx's roundings, and dx's sum
    half = ref.half_step(torch.float16)
    tiny = ref.floor_step(torch.float16)
    p = x.double() @ wd.t() + b.double()
    mag = x.double().abs() @ wd.t().abs() + b.double().abs()
    perr = ref.rounded(p, ref.sum_error(mag, K + 1), torch.float16) if act else torch.zeros_like(p)
    slope = ref.act_slope(act, p) if act else torch.ones_like(p)
    serr = curve(act, p, perr) * perr + (act_error(act, p)[1] if act else 0.0)
    dp = dy.double() * slope
    before = dy.double().abs() * serr + 2 * U * dp.abs()  # of dp before it is rounded (and of dbias's terms)
    dperr = before + ((dp.abs() + before) * half + tiny if act else 0.0)
    dx = dp @ wd
    dxerr = dperr @ wd.abs() + ref.sum_error((dp.abs() + dperr) @ wd.abs(), N)
    dxerr = dxerr + (dx.abs() + dxerr) * half + tiny
    dberr = before.sum(0) + ref.sum_error(dp.abs().sum(0), T)
    out = []
    for sx, sb in directions:
        by = [(loss(x.double() + H * a, b.double() + H * c) - loss(x.double() - H * a, b.double() - H * c)) / (2 * H)
              for a, c in ((sx, 0 * sb), (0 * sx, sb))]
        # central differences: h^2 / 6 of the third derivative (below 1 for both activations), and float64's cancellation
        step = [float(dy.double().abs().mul(d.abs() ** 3).sum()) * H * H * (act is not None) + 1e-9
                for d in (sx @ wd.t(), sb.expand(T, N))]
        out.append((sx, sb, by, (float((dxerr * sx.abs()).sum()) + step[0], float((dberr * sb.abs()).sum()) + step[1])))
    return (w, b, x, dy), out


def misses(dx, db, out):
    """How many directions the gradients are off in, by x and by the bias."""
    return [sum(abs(by[i] - float((grad * s[i]).sum())) > tol[i] for *s, by, tol in out) for i, grad in enumerate((dx, db))]


@pytest.mark.parametrize("act", ["silu", "gelu", None])
def test_the_bound_tells_wrong_gradients(act):
    """The float64 gradients are within the bounds; halved and doubled ones, and ones that are a tenth too small or lack a term, are
    outside in half of the directions at least (one would tell)."""
    (w, b, x, dy), out = differences(act)
    wd = ref.dequantize(*w)[0]
    p = x.double() @ wd.t() + b.double()
    dp = dy.double() * (ref.act_slope(act, p) if act else 1.0)
    dx, db = dp @ wd, dp.sum(0, keepdim=True)
    assert misses(dx, db, out) == [0, 0]
    for wrong in (dx / 2, dx * 2, 0.9 * dx, dp[:, :-1] @ wd[:-1]):
        assert misses(wrong, db, out)[0] >= DIRECTIONS // 2
    for wrong in (db / 2, 0.95 * db, dp[:-1].sum(0, keepdim=True)):
        assert misses(dx, wrong, out)[1] >= DIRECTIONS // 2


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", None])
def test_gradients(act):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    (w, b, x, dy), out = differences(act)
    _, p = block().linear(x.cuda(), pair(w), bias=b.cuda(), act=act, save=True)
    got = block().linear_backward(dy.cuda(), pair(w), p if act else None, act=act, bias=True)
    assert misses(got["dx"].cpu().double(), got["dbias"].cpu().double(), out) == [0, 0]
