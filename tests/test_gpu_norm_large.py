"""GPU: the norm join and its gradients where every workgroup takes several rows of every width path, and on both
sides of the output size up to which the forward pass stores with the non-temporal hint.  The bounds
are those of the small sizes' tests."""
import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_norm as small  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    small.setup_module(None)


BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
SIZES = [(600, 6656), (600, 8192), (560, 8193), (600, 10001), (530, 16384), (2731, 1024), (2730, 1024)]


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("dtype,res,gate", [(BF, SF, "channel"), (HF, HF, "token"), (SF, SF, "full")])
def test_join_of_many_rows(T, C, dtype, res, gate):
    d = small.make(T, C, dtype, res, gate)
    what = f"{T} x {C} {dtype} {res} {gate}"
    print("#", what, flush=True)
    g = small.dev(d)
    z, n = small.block.norm_join(g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"], **small.OPT)
    small.check_forward(d, z, n, what)
    got = small.block.norm_join_backward(g["dz"], g["dn"], g["y"], g["res"], g["w_post"], g["gate"], g["w_pre"],
                                         **small.OPT)
    small.check_backward(d, d["res"], got, what)
