"""GPU: how exactly products of 8-bit rows are summed.  The residual takes the rounded result away, so that y is what the sums
are off by (and what the rounding took), held in 16 bits of its own size."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import rows8_reference as r8  # noqa: E402
from tests.test_gpu_linear import block, pair  # noqa: E402

pytestmark = pytest.mark.gpu
U = ref.U32


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def exact_and_bound(x, w):
    """p = x W^T in float64, and what the sums may be off by.  Each 8 consecutive products are added as fixed-point numbers with
    13 bits below the power of two of the largest: less than 2^-13 of the largest is cut off of each of the 7 others.
    The rest is a float32 sum."""
    (xc, xs), (wc, ws) = x, (w[0][0], w[1][0])
    T, K = xc.shape
    N, kb = wc.shape[0], xs.shape[1]
    xv, wv = torch.zeros(T, kb * 128, dtype=torch.float64), torch.zeros(N, kb * 128, dtype=torch.float64)
    xv[:, :K], wv[:, :K] = values(xc), values(wc)
    wide = ws.double().repeat_interleave(128, 0)[:N]
    p, mag, cut = (torch.zeros(T, N, dtype=torch.float64) for _ in range(3))
    for q in range(kb):
        s = xs[:, q].double()[:, None] * wide[:, q][None]
        a, b = xv[:, q * 128:q * 128 + 128], wv[:, q * 128:q * 128 + 128]
        p += s * (a @ b.t())
        mag += s.abs() * (a.abs() @ b.abs().t())
        top = (a.abs().view(T, 1, 16, 8) * b.abs().view(1, N, 16, 8)).amax(3).sum(2)
        cut += s.abs() * 7 * 2.0 ** -13 * top
    return p, cut + ref.sum_error(mag, K)


def check(x, w, dtype=torch.float16):
    p, bound = exact_and_bound(x, w)
    res = -p.to(dtype)
    y, _ = block().linear(pair(x), pair(w), res=res.cuda())
    left = p + res.double()
    bound = bound + U * (p.abs() + bound) + U * left.abs()  # (the sum of both, in float32)
    ref.check(y, left, ref.rounded(left, bound, dtype), "y")
    return y.cpu().double() - left, p


# few rows by 16 and by 4 waves, the smaller tiles and the larger ones, whole and split along k
@pytest.mark.parametrize("T,N,K", [(1, 64, 512), (20, 40, 1000), (40, 2100, 96), (100, 200, 640), (300, 260, 2048),
                                   (2200, 4100, 24)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_random_rows(T, N, K, dtype):
    g = torch.Generator().manual_seed(T + K)
    x = r8.quantize(torch.randn(T, K, generator=g))
    w = r8.quantize(torch.randn(N, K, generator=g) / 16)[0][None], torch.rand(1, -(-N // 128), -(-K // 128), generator=g) + 0.5
    check(x, (w[0], w[1] / 64), dtype)


@pytest.mark.parametrize("T", [2, 70, 300])
def test_large_products_that_cancel(T):
    """448 * 448 and -448 * 448 among each 8, and 6 small ones that are all that is left."""
    g = torch.Generator().manual_seed(T)
    N, K = 200, 640
    codes = []
    for rows in (T, N):
        v = (2.0 ** torch.randint(-6, 6, (rows, K), generator=g).double() * (1 + torch.randint(0, 8, (rows, K), generator=g) / 8))
        v = v * (1 - 2 * torch.randint(0, 2, (rows, K), generator=g))
        v[:, 0::8] = 448.0
        v[:, 5::8] = 448.0 if rows is T else -448.0
        codes.append(v.float().to(torch.float8_e4m3fn).view(torch.uint8))
    x = codes[0], 2.0 ** torch.randint(-3, 3, (T, 5), generator=g).float()
    w = codes[1][None], 2.0 ** torch.randint(-12, -8, (1, 2, 5), generator=g).float()
    check(x, w)
