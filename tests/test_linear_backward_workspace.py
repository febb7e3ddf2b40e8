"""The workspace of a product's backward pass: as much as the gradients that are wanted need."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402

KB, PARTS = 128, 64 << 20  # at most, for the partial sums of split tiles


def block():
    from blockwise_fp8_zero_fold_amd import block as b
    return b


@pytest.mark.parametrize("T,E,N,K", [(65536, 1, 7168, 2048), (1 << 20, 8, 7168, 512), (4096, 1, 4096, 4096), (100, 2, 64, 7168)])
def test_without_the_bias_its_sums_take_no_room(T, E, N, K):
    n = block()._linear_bwd_workspace(T, E, N, K, False)
    assert n <= PARTS and (n == 0) == (N <= 2 * KB)
    assert block()._linear_bwd_workspace(T, E, N, K, True) >= max(n, 4 * (E + T // 512) * N)
    assert block()._linear_bwd_workspace(0, E, N, K, False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", [None, "gelu"])
def test_memory_of_a_call(act):
    """200,000 rows of 256 columns, whose sums by 8 rows would take 25 MB: dp and dx are all that a call without the bias's
    gradient allocates, and they are as with it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(0)
    T, N, K = 200000, 256, 16
    w = tuple(v.cuda() for v in ref.make_weight(g, 1, N, K))
    dy = torch.randn(T, N, generator=g).bfloat16().cuda()
    p = torch.randn(T, N, generator=g).bfloat16().cuda() if act else None
    with_bias = block().linear_backward(dy, w, p, act=act, bias=True)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = block().linear_backward(dy, w, p, act=act)
    outputs = 2 * T * K + (2 * T * N if act else 0)
    assert torch.cuda.max_memory_allocated() - before <= outputs + (1 << 20)
    assert got["dbias"] is None and torch.equal(got["dx"], with_bias["dx"]) and torch.equal(got["dp"], with_bias["dp"])


@pytest.mark.gpu
def test_split_tiles_without_the_bias():
    """Tiles that are split along N use the same partial sums either way."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(1)
    T, N, K = 500, 2048, 300
    w = tuple(v.cuda() for v in ref.make_weight(g, 1, N, K))
    dy = torch.randn(T, N, generator=g).bfloat16().cuda()
    a, b = (block().linear_backward(dy, w, bias=bias)["dx"] for bias in (False, True))
    assert torch.equal(a, b)
