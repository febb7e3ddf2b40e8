"""GPU: the norm join with its output in 8 bits: z and n are those of the plain join bit for bit, and the codes and
scales those of the float32 n."""
import pytest

torch = pytest.importorskip("torch")
from tests import rows8_reference as r8  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def block():
    from blockwise_fp8_zero_fold_amd import block as b
    return b


def inputs(T, C, dtype, res_dtype, gate, seed=0):
    g = torch.Generator().manual_seed(seed + T + C)
    y, res = (torch.randn(T, C, generator=g) * 2).to(dtype), (torch.randn(T, C, generator=g) * 3).to(res_dtype)
    # groups of very different size, and one of zeros
    res *= torch.exp2(torch.randint(-9, 9, (T, 1), generator=g)).to(res_dtype)
    kw = dict(w_post=(1 + 0.2 * torch.randn(C, generator=g)).cuda(), w_pre=(1 + 0.2 * torch.randn(C, generator=g)).cuda())
    kw["w_pre"][:128] = 0.0
    kw["gate"] = {"none": None, "channel": torch.randn(C, generator=g), "token": torch.randn(T, 1, generator=g),
                  "full": torch.randn(T, C, generator=g).to(dtype)}[gate]
    if kw["gate"] is not None:
        kw["gate"] = kw["gate"].cuda()
    return y.cuda(), res.cuda(), kw


@pytest.mark.parametrize("T,C", [(1, 1), (1, 7), (2, 8), (3, 100), (5, 128), (4, 129), (9, 136), (3, 255), (7, 1000), (2, 1537),
                                 (5, 4096), (2, 7168), (3, 8192), (2, 8200), (2, 16384), (2500, 264)])
@pytest.mark.parametrize("dtype,res_dtype", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                             (torch.float16, torch.float16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("gate,rule", [("none", "amax"), ("channel", "pow2"), ("token", "amax"), ("full", "amax")])
def test_codes_of_the_join(T, C, dtype, res_dtype, gate, rule):
    b = block()
    y, res, kw = inputs(T, C, dtype, res_dtype, gate)
    args = dict(eps=1e-6, res_scale=0.9, block_scale=0.5, weight_offset=0.0)
    z, n, (codes, scales) = b.norm_join8(y, res, **kw, **args, keep=True, scale_rule=rule)
    wz, wn = b.norm_join(y, res, **kw, **args)
    assert torch.equal(z, wz) and torch.equal(n, wn)
    # the same join on the widened inputs has the float32 n that the codes are taken from
    wide = dict(kw)
    if gate == "full":
        wide["gate"] = kw["gate"].float()
    _, n32 = b.norm_join(y.float(), res.float(), **wide, **args)
    want = r8.quantize(n32.cpu(), rule == "pow2")
    assert torch.equal(scales.cpu(), want[1]) and r8.same_codes(codes, want[0])
    z2, none, again = b.norm_join8(y, res, **kw, **args, scale_rule=rule)
    assert none is None and torch.equal(z2, z) and torch.equal(again[0], codes) and torch.equal(again[1], scales)


def test_no_block_output_and_only_the_codes():
    import blockwise_fp8_zero_fold_amd as fz
    b = block()
    _, res, kw = inputs(33, 300, torch.bfloat16, torch.bfloat16, "none")
    z, n, (codes, scales) = b.norm_join8(None, res, w_pre=kw["w_pre"], keep=True)
    wz, wn = b.norm_join(None, res, w_pre=kw["w_pre"])
    assert torch.equal(z, wz) and torch.equal(n, wn)
    c2, s2 = torch.zeros_like(codes), torch.zeros_like(scales)
    f = fz.Norm(33, 300, fz.BF16, fz.BF16, fz.GATE_NONE, 1e-6, 1.0, 1.0, 0.0, 0)
    fz.fp8z1_norm_join8(f, None, res, None, None, kw["w_pre"], None, None, c2, s2)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_zeros_infinities_nan_and_tiny_values():
    b = block()
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(2))
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3] *= 1e-38
    w = torch.ones(300)
    w[:128] = 1e-38  # a group whose scale would be subnormal
    for rule in ("amax", "pow2"):
        _, n32 = b.norm_join(None, x.cuda(), w_pre=w.cuda())
        _, _, (codes, scales) = b.norm_join8(None, x.cuda(), w_pre=w.cuda(), scale_rule=rule)
        want = r8.quantize(n32.cpu(), rule == "pow2")
        assert torch.equal(scales.cpu(), want[1]) and r8.same_codes(codes, want[0]), rule
    assert (scales[0].cpu() == 1).all() and (codes[0].cpu() & 0x7F == 0).all()


def test_every_rounding_border():
    """Values on and next to the borders between codes, through a join that leaves them as they are up to one factor."""
    b = block()
    q = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (q[1:] + q[:-1]) / 2
    v = torch.cat([q, mid, mid * (1 + 2.0 ** -22), mid * (1 - 2.0 ** -22), -mid])
    v = torch.cat([v, torch.zeros(-len(v) % 127)]).view(-1, 127)
    v = torch.cat([v, torch.full((v.shape[0], 1), 448.0)], 1)  # the group's largest: scale 1 after the norm's factor
    _, n32 = b.norm_join(None, v.cuda())
    _, _, (codes, scales) = b.norm_join8(None, v.cuda())
    want = r8.quantize(n32.cpu())
    assert torch.equal(scales.cpu(), want[1]) and r8.same_codes(codes, want[0])


def test_unaligned_outputs_graph_and_refusals():
    import blockwise_fp8_zero_fold_amd as fz
    b = block()
    y, res, kw = inputs(50, 264, torch.bfloat16, torch.float32, "token")
    want = b.norm_join8(y, res, **kw)
    codes = torch.zeros(3 + 50 * 264, dtype=torch.uint8, device="cuda")[3:].view(50, 264)
    scales = torch.zeros(50, 3, device="cuda")
    f = fz.Norm(50, 264, fz.BF16, fz.F32, fz.GATE_TOKEN, 1e-6, 1.0, 1.0, 0.0, 0)
    fz.fp8z1_norm_join8(f, y, res, kw["w_post"], kw["gate"], kw["w_pre"], None, None, codes, scales)
    assert torch.equal(codes, want[2][0]) and torch.equal(scales, want[2][1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        z, n, (c, s) = b.norm_join8(y, res, **kw, keep=True)
    for _ in range(3):
        y.normal_()
        graph.replay()
        torch.cuda.synchronize()
        wz, wn, (wc, ws) = b.norm_join8(y, res, **kw, keep=True)
        assert all(torch.equal(p, q) for p, q in ((z, wz), (n, wn), (c, wc), (s, ws)))
    for call in (lambda: b.norm_join8(y, res, scale_rule="max"), lambda: b.norm_join8(y[:1], res),
                 lambda: b.norm_join8(y, res.double()), lambda: fz.fp8z1_norm_join8(f, y, res, None, kw["gate"], None, None, None, codes[:3], scales)):
        with pytest.raises(fz.Fp8z1Error):
            call()
    assert b.norm_join8(None, torch.zeros(0, 64, device="cuda"))[2][0].shape == (0, 64)
