"""GPU: rows behind the first 4 GiB of a tensor (offsets past 32 bits)."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import rows8_reference as r8  # noqa: E402

pytestmark = pytest.mark.gpu
GIB4 = 2 ** 32


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_rows_of_tokens():
    """2400 rows of 2 MiB: the copies, their weighted sums and the gradients, on the rows that lie last."""
    from blockwise_fp8_zero_fold_amd import routing
    g = torch.Generator(device="cuda").manual_seed(0)
    T, k, D, E = 300, 8, 2 ** 20, 8
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    experts = torch.stack([torch.randperm(E, generator=g, device="cuda") for _ in range(T)]).to(torch.int32)
    offsets, row_of = routing.sort_tokens(experts, E)
    rows = routing.dispatch(x, row_of)
    assert rows.numel() * 2 > GIB4 and int(offsets[-1]) == T * k
    late = torch.nonzero(row_of.reshape(-1) >= T * k - 40).reshape(-1)
    assert len(late) == 40
    for i in late.tolist():
        assert torch.equal(rows[row_of.reshape(-1)[i]], x[i // k])
    w = torch.rand(T, k, generator=g, device="cuda")
    y = routing.combine(rows, row_of, w)
    for t in sorted({i // k for i in late.tolist()})[:6]:
        want = (x[t].double() * w[t].double().sum()).cpu()
        ref.check(y[t].cpu(), want, ref.rounded(want, (k + 1) * ref.U32 * want.abs(), torch.bfloat16), "y")
    drows, dw = routing.combine_backward(x, rows, row_of, w)
    norm = x.double().square().sum(1)
    assert ((dw.double() - norm[:, None]).abs() <= ref.sum_error(norm, D)[:, None]).all()
    for i in late[:6].tolist():
        want = (x[i // k].double() * w.reshape(-1)[i].double()).cpu()
        ref.check(drows[row_of.reshape(-1)[i]].cpu(), want, ref.rounded(want, ref.U32 * want.abs(), torch.bfloat16), "drows")


def test_norm():
    """Codes, z and n of 265000 rows of 16384: the last rows are what a call of them alone gives."""
    from blockwise_fp8_zero_fold_amd import block
    g = torch.Generator(device="cuda").manual_seed(1)
    T, C = 265000, 16384
    y = torch.randn(T, C, generator=g, device="cuda", dtype=torch.bfloat16)
    z, n, (codes, scales) = block.norm_join8(y, y, keep=True)
    assert codes.numel() > GIB4
    few, few_n, (few_codes, few_scales) = block.norm_join8(y[-70:].contiguous(), y[-70:].contiguous(), keep=True)
    assert torch.equal(z[-70:], few) and torch.equal(n[-70:], few_n)
    assert torch.equal(codes[-70:], few_codes) and torch.equal(scales[-70:], few_scales)


def check_last(y, x, w, K):
    last = tuple(v[-40:].cpu() for v in x)
    p, mag = ref.grouped(r8.dequantize(*last), ref.dequantize(*(v.cpu() for v in w)), None, False)
    ref.check(y[-40:].cpu(), p, ref.rounded(p, ref.sum_error(mag, K) + 7 * 2.0 ** -13 * mag, torch.bfloat16), "y")


@pytest.mark.parametrize("T,N,K", [(4200, 130, 2 ** 20), (36000, 2 ** 16, 128), (36000, 2 ** 16, 130)])
def test_product(T, N, K):
    """x, or y, of more than 4 GiB."""
    from blockwise_fp8_zero_fold_amd import block
    g = torch.Generator().manual_seed(K)
    few = r8.make_rows8(g, 300, K)
    x = tuple(v.cuda().repeat(T // 300, 1) for v in few)
    assert max(x[0].numel(), 2 * T * N) > GIB4
    w = tuple(v.cuda() for v in ref.make_weight(g, 1, N, K))
    y, _ = block.linear(x, w)
    check_last(y, x, w, K)


@pytest.mark.parametrize("T,F,D", [(4200, 130, 2 ** 20), (66000, 2 ** 16, 128)])
def test_up8(T, F, D):
    """x, or the codes, of more than 4 GiB: equal rows give equal codes."""
    from blockwise_fp8_zero_fold_amd import block
    g = torch.Generator().manual_seed(D)
    few = r8.make_rows8(g, 300, D)
    x = tuple(v.cuda().repeat(T // 300, 1) for v in few)
    assert max(x[0].numel(), T * F) > GIB4
    wg, wu = (tuple(v.cuda() for v in ref.make_weight(g, 1, F, D)) for _ in range(2))
    (codes, scales), _ = block.ffn_up8(x, wg, wu)
    assert torch.equal(codes[-300:], codes[:300]) and torch.equal(scales[-300:], scales[:300])
