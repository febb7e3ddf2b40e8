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


@pytest.mark.parametrize("T,E,N,rows", [(100, 2, 64, 8), (37, 1, 40, 8), (4096, 1, 4096, 8), (48828, 3, 2048, 8), (48829, 3, 2048, 64),
                                        (65536, 8, 7168, 64), (1 << 20, 1, 2047, 64), (1 << 20, 1, 2048, 512),
                                        (1 << 24, 1, 7168, 512), (1 << 30, 5, 1, 64)])
def test_the_biass_sums(T, E, N, rows):
    """A float32 sum of each column for every group of rows; an expert's rows may begin and end inside a group.  They take no more than
    134 MB, or 1/256 of dy, and a row for each expert."""
    n, sums = block()._linear_bwd_workspace(T, E, N, 16, True), 4 * (E + T // rows) * N
    assert n == -(-max(sums, block()._linear_bwd_workspace(T, E, N, 16, False)) // 16) * 16
    assert sums <= max(2 ** 27, 2 * T * N // 256) + 4 * E * N


# groups of 8, 64 and 512 rows; experts that end inside a group, with one row, without one, and all rows with one
@pytest.mark.gpu
@pytest.mark.parametrize("T,N,cuts", [(700, 130, (3, 3, 11, 500)), (60000, 2048, (1, 65, 65, 30000)), (400001, 1001, (64, 128, 200, 399999)),
                                      (1100000, 2047, (513, 514, 1024, 700001))])
def test_bias_gradient_of_many_rows(T, N, cuts):
    """dy of small whole numbers, so that every sum is exact in float32."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import blockwise_fp8_zero_fold_amd as fz
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randint(-3, 4, (T, N), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    for off in ((0, *cuts, T), (0, 0, 0, 0, 0, T), (0, T, T, T, T, T)):
        E, f = 5, fz.Product(T, 5, N, 16, fz.BF16, fz.BF16, fz.ACT_NONE, 0)
        n = fz.fp8z1_linear_bwd_workspace_bytes(f)
        db = torch.full((E, N), 7.0, device="cuda")
        fz.fp8z1_linear_bwd(f, dy, None, None, None, torch.tensor(off, dtype=torch.int32, device="cuda"), None, db, None,
                            torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n)
        for e in range(E):
            want = torch.zeros(N, dtype=torch.float64, device="cuda")
            for lo in range(off[e], off[e + 1], 1 << 16):
                want += dy[lo:min(lo + (1 << 16), off[e + 1])].float().sum(0)
            assert torch.equal(db[e].double(), want), (off, e)


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
