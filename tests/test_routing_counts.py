"""Numbers of choices and experts that 32 bits do not hold are refused, not cut off."""
import pytest

import blockwise_fp8_zero_fold_amd as fz

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T,k,E", [(50000, 2 ** 32 + 1, 8), (50000, 1, 2 ** 32 + 8), (2 ** 64 + 4, 1, 8), (4, -2 ** 32 + 2, 8),
                                   (4, 2, 2 ** 31)])
def test_sort_tokens_counts(T, k, E):
    with pytest.raises(fz.Fp8z1Error):
        fz.fp8z1_sort_tokens_workspace_bytes(T, k, E)
    with pytest.raises(fz.Fp8z1Error):
        fz.fp8z1_sort_tokens(T, k, E, None, None, None)


@pytest.mark.gpu
def test_the_tensor_layer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from blockwise_fp8_zero_fold_amd import routing as r
    l, e = torch.zeros(1, 64, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for k in (2 ** 32 + 8, 2 ** 31, 33, 0, -1, -2 ** 32 + 8):
        with pytest.raises(fz.Fp8z1Error):
            r.route(l, k)
    for n in (2 ** 32 + 8, 2 ** 31, 1025, 0, -1):
        with pytest.raises(fz.Fp8z1Error):
            r.sort_tokens(e, n)
    wide = torch.zeros(1, 33, dtype=torch.int32, device="cuda")
    for call in (lambda: r.sort_tokens(wide, 4), lambda: r.dispatch(l, wide), lambda: r.combine(l, wide),
                 lambda: r.combine_backward(l, l, wide, wide.float()), lambda: r.route_backward(wide.float(), l, wide)):
        with pytest.raises(fz.Fp8z1Error):
            call()


@pytest.mark.gpu
def test_plans_of_another_shape():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from blockwise_fp8_zero_fold_amd import routing as r
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    for shape in ((), (4,), (3, 2), (4, 2, 1), (4, 0)):
        plan = torch.zeros(shape, dtype=torch.int32, device="cuda")
        for call in (lambda: r.dispatch(x, plan), lambda: r.combine(x, plan, w), lambda: r.combine_backward(x, x, plan, w)):
            with pytest.raises(fz.Fp8z1Error):
                call()
