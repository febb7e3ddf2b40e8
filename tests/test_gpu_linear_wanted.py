"""GPU: a product's backward pass without the gradients that are not wanted."""
import pytest

torch = pytest.importorskip("torch")
import blockwise_fp8_zero_fold_amd as fz  # noqa: E402
from tests import block_reference as ref  # noqa: E402
from tests.test_gpu_linear import block, pair  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("T", [9, 300])
def test_each_alone_is_as_with_the_others(T, act):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(T)
    N, K = 520, 260
    w, dy = pair(ref.make_weight(g, 1, N, K)), torch.randn(T, N, generator=g).bfloat16().cuda()
    p = torch.randn(T, N, generator=g).bfloat16().cuda() if act else None
    every = block().linear_backward(dy, w, p, act=act, bias=True)
    for bias in (False, True):
        for dx in (False, True):
            for dp in (False, True):
                call = lambda: block().linear_backward(dy, w, p, act=act, bias=bias, dx=dx, dp=dp)
                if (dx and act and not dp) or not (bias or dx or (dp and act)):
                    with pytest.raises(fz.Fp8z1Error):
                        call()
                    continue
                got = call()
                for name, wanted in (("dx", dx), ("dp", dp), ("dbias", bias)):
                    assert (got[name] is not None) == wanted
                    assert not wanted or torch.equal(got[name], every[name]), name
