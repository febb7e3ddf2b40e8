"""GPU: the feed-forward calls where one of many experts takes nearly all rows, and in several threads and
streams at once."""
import copy
import threading

import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_ffn as small  # noqa: E402
from tests import test_gpu_ffn_large as large  # noqa: E402
from tests.test_gpu_wgrad_large import wgrad_compare, wgrad_reference  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    large.setup_module(None)


@pytest.mark.parametrize("T,E,D,F", [(1500, 64, 512, 384), (1500, 64, 510, 386), (2500, 64, 256, 320), (40, 200, 128, 160)])
def test_nearly_all_rows_on_one_expert(T, E, D, F):
    """64 experts and more: one in the middle takes nearly all rows, some a single row, the others none (the
    average load chooses the kernel: rows for the first, second and last sizes, tiles for the third)."""
    c = small.Case(T, E, D, F)
    cuts = torch.zeros(E + 1, dtype=torch.int32)
    cuts[3:] = 1
    cuts[E // 2 + 1:] = T - 2
    cuts[E - 1:] = T - 1
    cuts[E] = T
    c.offsets = cuts
    what = f"{T} rows on one of {E} experts"
    print("#", what, flush=True)
    large.all_calls(c, what, True)
    x, a, dy, dh, du = (c.dev(n) for n in ("x", "a", "dy", "dh", "du"))
    dw = small.block.ffn_backward_weights(x, a, dy, dh, du, E, c.dev("offsets"))
    for (p, q), got in zip(((c.dh, c.x), (c.du, c.x), (c.dy, c.a)), dw):
        wgrad_compare(got, *wgrad_reference(p, q, E, c.offsets), what)


def test_streams_and_threads_at_once():
    """Two threads, each on a stream of its own, run blocks of different sizes over and over: each gets what it
    gets alone."""
    cases = [small.Case(500, 3, 264, 136), small.Case(20, 4, 192, 1200, "f16", "gelu")]
    runs = [small._layer(c) for c in cases]
    rows = [(c.dev("x"), c.dev("dy")) for c in cases]
    want = [run(*r) for run, r in zip(runs, rows)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        torch.cuda.set_device(0)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for turn in range(20):
                got = runs[i](*rows[i])
                side.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append((i, turn))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


@pytest.mark.parametrize("T,E,D,F", [(300, 5000, 16, 24), (70000, 65535, 8, 16)])
def test_thousands_of_experts(T, E, D, F):
    """More experts than one or two looks of a wave find, and more groups of rows than a grid has in y."""
    c = small.Case(T, E, D, F)
    what = f"{T} rows, {E} experts"
    print("#", what, flush=True)
    s, rows = large.sampled(c)
    outs = c.run_up()
    s.check_up([t[rows.cuda()] for t in outs], what)
    y = c.out(D)
    small.fz.fp8z1_ffn_down(c.cfg, c.dev("a"), *c.dev("down"), c.dev("offsets"), y)
    s.check_down(y[rows.cuda()], what)
    assert all(bool(torch.isfinite(t).all()) for t in (*outs, y))


def test_rows_of_few_experts_without_cover():
    """Few rows (the row kernel): rows that no expert covers are left alone, offsets out of range and out
    of order write within the tensor."""
    c = small.Case(90, 5, 136, 72)
    c.offsets = torch.tensor([20, 40, 40, 41, 75, 75], dtype=torch.int32)
    outs = c.run_up()
    s = copy.copy(c)
    rows = torch.arange(20, 75)
    for k in ("x", "dy", "a", "h", "u", "dh", "du"):
        setattr(s, k, getattr(c, k)[rows])
    s.T, s.offsets = rows.numel(), c.offsets - 20
    s.check_up([t[rows.cuda()] for t in outs], "covered rows")
    for t in outs:
        assert bool((t[:20] == 7.0).all()) and bool((t[75:] == 7.0).all())
    for bad in ([-50, 20, 10, 100000, 3, 90], [90, 80, 60, 40, 20, 0], [2 ** 31 - 1] * 6, [-2 ** 31] * 6):
        c.offsets = torch.tensor(bad, dtype=torch.int64).to(torch.int32)
        assert all(bool(torch.isfinite(t).all()) for t in c.run_up()), bad


def test_a_load_on_one_expert_takes_no_longer_than_an_even_one():
    """All of 8192 rows on one of 256 experts, and evenly on all: the groups of rows run side by side either
    way (one after another they took 7 times as long; 3 are allowed)."""
    T, E, D, F = 8192, 256, 510, 510

    def weight(r, c):
        return (torch.full((E, r, c), 0x30, dtype=torch.uint8, device="cuda"),
                torch.full((E, -(-r // 128), -(-c // 128)), 1e-3, device="cuda"))

    gate, up, down = weight(F, D), weight(F, D), weight(D, F)
    x = torch.ones(T, D, dtype=torch.bfloat16, device="cuda")
    even = (torch.arange(E + 1, device="cuda") * T // E).to(torch.int32)
    one = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    one[E // 2 + 1:] = T

    def least(offsets):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                small.block.ffn_forward(x, gate, up, down, offsets)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    t_even, t_one = least(even), least(one)
    assert t_one <= 3 * t_even, (t_one, t_even)
