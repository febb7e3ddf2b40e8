"""GPU: gate and up on 8-bit rows where a tile is summed block by block, because the scales of one of its rows lie too far
apart: what the other rows get must not hang on when each wave leaves its last block for the results."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import rows8_reference as r8  # noqa: E402
from tests.test_gpu_linear import block, check_up8, pair  # noqa: E402

pytestmark = pytest.mark.gpu

# (T, D, F): tiles of 64 and of 256 rows, whole ones and ones split along k; the last block of k whole and partial
SHAPES = [(300, 256, 700), (300, 200, 700), (300, 2048, 300), (300, 2000, 130), (2600, 384, 4000), (2600, 300, 4000),
          (1500, 1152, 1500)]
FAR = (3, 40, 77)  # rows of one tile of either size, or of its neighbour


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def far_row(x, row):
    codes, scales = x[0].clone(), x[1].clone()
    scales[row] = 2.0 ** -90
    scales[row, -1] = 2.0 ** 25
    return codes, scales


@pytest.mark.parametrize("T,D,F", SHAPES)
@pytest.mark.parametrize("save", [True, False])
def test_sound_rows_do_not_depend_on_the_row_that_is_far(T, D, F, save):
    """A far row in every tile; the sums of the others are the same sums wherever it is, bit for bit."""
    g = torch.Generator().manual_seed(T + D + F)
    x, wg, wu = r8.make_rows8(g, T, D), pair(ref.make_weight(g, 1, F, D)), pair(ref.make_weight(g, 1, F, D))
    lows = torch.arange(0, T, 64)
    sound = torch.ones(T, dtype=torch.bool)
    places = [(lows + k).clamp(max=T - 1) for k in (3, 40, 61)]  # (in the last tile, which may be short, too)
    for p in places:
        sound[p] = False
    want = None
    for _ in range(4):
        for p in places:
            (codes, scales), kept = block().ffn_up8(pair(far_row(x, p)), wg, wu, save=save)
            got = [v.cpu()[sound] for v in (codes, scales, *(kept or ()))]
            if want is None:
                want = got
            for name, a, b in zip(("codes", "scales", "h", "u"), got, want):
                assert torch.equal(a, b), name


@pytest.mark.parametrize("T,D,F", SHAPES[:4])
@pytest.mark.parametrize("row", FAR)
def test_one_far_row_among_sound_ones(T, D, F, row):
    """Against float64: the far row, the rows of its tile and those of the others."""
    g = torch.Generator().manual_seed(row + D)
    x = far_row(r8.make_rows8(g, T, D), row)
    wg, wu = ref.make_weight(g, 1, F, D), ref.make_weight(g, 1, F, D)
    check_up8(x, r8.dequantize(*x), wg, wu, None, T, D, F, torch.bfloat16, "silu", "amax")


@pytest.mark.parametrize("T,D,F", SHAPES[:5])
def test_nan_and_infinite_rows_among_sound_ones(T, D, F):
    """A scale of NaN, of infinity and of 0 each send their tile through the same sums: the rest within float64's bounds."""
    g = torch.Generator().manual_seed(F)
    x, wg, wu = r8.make_rows8(g, T, D), ref.make_weight(g, 1, F, D), ref.make_weight(g, 1, F, D)
    x[1][2, 0], x[1][70, 1], x[1][130, 0] = float("nan"), float("inf"), 0.0
    (codes, scales), (h, u) = block().ffn_up8(pair(x), pair(wg), pair(wu), save=True)
    rest = torch.ones(T, dtype=torch.bool)
    rest[[2, 70]] = False
    assert torch.isnan(h[2].float()).all() and not torch.isfinite(h[70].float()).any()
    xd = r8.dequantize(*x)[rest]
    for got, w in ((h, wg), (u, wu)):
        exact, mag = ref.grouped(xd, ref.dequantize(*w), None, False)
        ref.check(got.cpu()[rest], exact, ref.rounded(exact, ref.sum_error(mag, D), torch.bfloat16), "projection")


@pytest.mark.parametrize("T,D,F", [(300, 128, 700), (300, 256, 700), (9000, 100, 1300), (4100, 128, 2100)])
@pytest.mark.parametrize("far", [False, True])
def test_whole_tiles_give_the_same_without_kept_projections(T, D, F, far):
    """Tiles of few blocks, whose waves go straight from the sums to the rows' largest magnitudes where h and u are not kept:
    whether a tile is summed again is decided alike by all of them, call after call."""
    g = torch.Generator().manual_seed(T + F)
    x = r8.make_rows8(g, T, D)
    if far:
        x[1][torch.arange(0, T, 130), 0] = 2.0 ** -90
    x, wg, wu = pair(x), pair(ref.make_weight(g, 1, F, D)), pair(ref.make_weight(g, 1, F, D))
    (codes, scales), _ = block().ffn_up8(x, wg, wu, save=True)
    for _ in range(10):
        (c, s), none = block().ffn_up8(x, wg, wu)
        assert none is None and torch.equal(c, codes) and torch.equal(s, scales)
