"""GPU: the 256-column tiles that large weight gradients take, against float64, at sizes just above those
where they begin, ragged on every side.  The bounds are those of the small sizes' tests."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import test_gpu_ffn as small  # noqa: E402

pytestmark = pytest.mark.gpu

fz = block = None


def setup_module(module):
    global fz, block
    small.setup_module(None)
    fz, block = small.fz, small.block


def wgrad_reference(p, q, E, offsets, start=None):
    """Per expert p^T q in float64 on the GPU, and the bound of a float32 sum."""
    exact = torch.zeros(E, p.shape[1], q.shape[1], dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(exact)
    p, q = p.cuda().double(), q.cuda().double()
    for e, lo, hi in ref.runs(offsets, p.shape[0]):
        if hi > lo:
            exact[e] = p[lo:hi].t().contiguous() @ q[lo:hi]
            bound[e] = p[lo:hi].abs().t().contiguous() @ q[lo:hi].abs()
            bound[e] *= (2 * (hi - lo) + 8) * ref.U32
    if start is not None:
        exact += start.double()
        bound += ref.U32 * (exact.abs() + bound)
    return exact, bound


def wgrad_compare(got, exact, bound, what):
    allowed = ref.rounded(exact, bound, got.dtype)
    over = (got.double() - exact).abs() - allowed
    assert bool((over <= 0).all()), (what, float(over.max()))  # (a NaN is not <= 0)


@pytest.mark.parametrize("T,E,M,N", [(100, 2, 4098, 8330), (300, 3, 2052, 5636), (33, 1, 4098, 8196)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wide_weight_gradient(T, E, M, N, dtype):
    """At least 1024 tiles of 128 x 256, the last of which hold 2 or 4 rows and 4 or 138 columns."""
    assert E * (-(-M // 128)) * (-(-N // 256)) >= 1024
    g = torch.Generator().manual_seed(T + E + M + N)
    p, q = (torch.randn(T, w, generator=g).to(small.TYPES[dtype]) for w in (M, N))
    offsets = ref.make_offsets(g, T, E)
    code = {"bf16": fz.BF16, "f16": fz.F16}[dtype]
    assert fz.fp8z1_ffn_wgrad_workspace_bytes(T, E, M, N) == 0
    print(f"# {T} rows, {E} experts, {M} x {N}, {dtype}", flush=True)
    dev = [t.cuda() for t in (p, q, offsets)]
    exact, bound = wgrad_reference(p, q, E, offsets)
    for out, t in ((fz.F32, torch.float32), (fz.BF16, torch.bfloat16)):
        dw = torch.full((E, M, N), float("nan"), dtype=t, device="cuda")
        fz.fp8z1_ffn_wgrad(T, E, M, N, code, *dev, out, dw)
        wgrad_compare(dw, exact, bound, f"dw {t}")
    start = torch.randn(E, M, N, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    exact, bound = wgrad_reference(p, q, E, offsets, start)
    fz.fp8z1_ffn_wgrad(T, E, M, N, code, *dev, fz.F32, start, accumulate=True)
    wgrad_compare(start, exact, bound, "accumulated dw")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_three_wide_weight_gradients(dtype):
    T, E, D, F = 333, 2, 4110, 2050
    assert E * (2 * 17 * 17 + 33 * 9) >= 1024
    g = torch.Generator().manual_seed(8)
    x, dy = (torch.randn(T, D, generator=g).to(small.TYPES[dtype]) for _ in range(2))
    a, dh, du = (torch.randn(T, F, generator=g).to(small.TYPES[dtype]) for _ in range(3))
    offsets = torch.tensor([0, 201, T], dtype=torch.int32)
    dev = [t.cuda() for t in (x, a, dy, dh, du)]
    pairs = ((dh, x), (du, x), (dy, a))
    for t in (torch.float32, torch.bfloat16):
        for (p, q), dw in zip(pairs, block.ffn_backward_weights(*dev, n_experts=E, offsets=offsets.cuda(), dtype=t)):
            wgrad_compare(dw, *wgrad_reference(p, q, E, offsets), f"{t}")
    out = [torch.full(s, 0.5, device="cuda") for s in ((E, F, D), (E, F, D), (E, D, F))]
    block.ffn_backward_weights(*dev, n_experts=E, offsets=offsets.cuda(), out=out)
    for (p, q), dw in zip(pairs, out):
        wgrad_compare(dw, *wgrad_reference(p, q, E, offsets, torch.full_like(dw, 0.5)), "added")
