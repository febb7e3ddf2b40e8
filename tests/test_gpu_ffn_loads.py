"""GPU: the feed-forward calls where one of many experts takes nearly all rows, and in several threads and
streams at once."""
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
