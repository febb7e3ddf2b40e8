"""GPU: the forward and backward tiles that large problems take (four matrix columns per wave), whole and
split along k, against float64, at sizes just above those where they begin, ragged on every side.
The bounds are those of the small sizes' tests."""
import copy

import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import test_gpu_ffn as small  # noqa: E402

pytestmark = pytest.mark.gpu

fz = None


def setup_module(module):
    global fz
    small.setup_module(None)
    fz = small.fz


def some_rows(offsets, T, n=150):
    """Rows around every expert's ends and around the edges of its row tiles and waves, and some others."""
    rows = set(torch.randint(0, T, (n,), generator=torch.Generator().manual_seed(T)).tolist()) if T else set()
    for _, lo, hi in ref.runs(offsets, T):
        last = lo + (max(hi - lo, 1) - 1) // 128 * 128
        for edge in (lo, lo + 32, lo + 64, lo + 128, last, last + 64, hi):
            rows |= {r for r in (edge - 1, edge) if lo <= r < hi}
    return torch.tensor(sorted(rows))


def sampled(c):
    """The case of these rows alone (its checks hold them against float64), and the rows."""
    rows = some_rows(c.offsets, c.T)
    s = copy.copy(c)
    for k in ("x", "dy", "a", "h", "u", "dh", "du"):
        setattr(s, k, getattr(c, k)[rows])
    s.T = rows.numel()
    s.offsets = torch.searchsorted(rows, c.offsets.long()).to(torch.int32)
    return s, rows


def all_calls(c, what, workspace):
    """The four calls on the case, every element finite and a sample of rows checked."""
    s, rows = sampled(c)
    n = fz.fp8z1_ffn_workspace_bytes(c.cfg) if workspace else 0

    def ws():
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None  # NaN

    off, gate, up, down = (c.dev(k) for k in ("offsets", "gate", "up", "down"))

    def check(test, outs):
        assert all(bool(torch.isfinite(t).all()) for t in outs), what
        test([t[rows.cuda()] for t in outs] if len(outs) > 1 else outs[0][rows.cuda()], what)

    outs = [c.out(c.F) for _ in range(3)]
    fz.fp8z1_ffn_up(c.cfg, c.dev("x"), *gate, *up, off, *outs, workspace=ws())
    check(s.check_up, outs)
    y = c.out(c.D)
    fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *down, off, y, workspace=ws())
    check(s.check_down, [y])
    outs = [c.out(c.F) for _ in range(3)]
    fz.fp8z1_ffn_down_bwd(c.cfg, c.dev("dy"), *down, c.dev("h"), c.dev("u"), off, *outs, workspace=ws())
    check(s.check_down_bwd, outs)
    dx = c.out(c.D)
    fz.fp8z1_ffn_up_bwd(c.cfg, c.dev("dh"), c.dev("du"), *gate, *up, off, dx, workspace=ws())
    check(s.check_up_bwd, [dx])


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu")])
def test_wide_tiles(dtype, act, workspace):
    """67 row tiles by 9 or 17 wide columns; with the workspace the tiles past the last full round are
    split along their 17 (34) blocks."""
    c = small.Case(8200, 3, 2052, 2052, dtype, act)
    what = f"wide tiles, {dtype}, workspace {workspace}"
    print("#", what, flush=True)
    all_calls(c, what, workspace)


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wide_tiles_of_far_scales(dtype, workspace):
    """Scales far apart and scales of zero: every tile column is summed in a pass of its own."""
    far = dict(lo=-60.0, hi=40.0 if dtype == "bf16" else 3.0)  # (half precision ends at 65,504)
    c = small.Case(8200, 3, 2052, 2052, dtype, **far)
    for w in (c.gate, c.up, c.down):
        w[1][:, 1, 2] = 0.0
        w[1][0, -1, -1] = 0.0
    what = f"wide tiles, far scales, {dtype}, workspace {workspace}"
    print("#", what, flush=True)
    all_calls(c, what, workspace)
