"""GPU: the block on 8-bit rows with power-of-two scales between its products."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import rows8_reference as r8  # noqa: E402
from tests.test_gpu_linear import block, pair  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("rule", ["amax", "pow2"])
def test_the_rule_is_that_of_the_inner_rows(T, rule):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(T)
    b, x = block(), pair(r8.make_rows8(g, T, 256))
    wg, wu, wd = (pair(ref.make_weight(g, 2, n, k)) for n, k in ((200, 256), (200, 256), (256, 200)))
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    y, kept = b.ffn_forward8(x, wg, wu, wd, off, "gelu", True, torch.float16, rule)
    a, inner = b.ffn_up8(x, wg, wu, off, "gelu", True, torch.float16, rule)
    assert torch.equal(y, b.linear(a, wd, off, dtype=torch.float16)[0]) and all(map(torch.equal, kept, inner))
    if rule == "pow2":
        assert (torch.frexp(a[1]).mantissa == 0.5).all()
    with pytest.raises(Exception, match="scale_rule"):
        b.ffn_forward8(x, wg, wu, wd, off, scale_rule="none")
