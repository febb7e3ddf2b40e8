"""GPU: the example's layer -- norms, feed-forward block and shard step together.  Its gradients equal
float64 ones of the same layer, the step consumes them, and training lowers the loss."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _layer(E, D, F, seed=5):
    import blockwise_fp8_zero_fold_amd as fz
    from examples.train_ffn_layer import Layer

    hp = fz.Hparams(1e-3, 0.9, 0.95, 1e-8, 0.0, 1.0, 0, 1.0, 2.0, 0.5, 1000, 0, 0, 0.0, None)
    return Layer(E, D, F, hp, seed)


def test_layer_gradients_against_float64():
    """All gradients of the layer against automatic differentiation in float64 on the dequantized weights.
    Between them lie a few 16-bit tensors (x, h, u, a, y, dy, dh, du, dx; relative 2^-9 each in bfloat16),
    whose roundings are independent: the norm of the difference stays within 16 of them."""
    E, D, F, T = 3, 264, 136, 200
    layer = _layer(E, D, F)
    g = torch.Generator().manual_seed(0)
    tokens = torch.randn(T, D, generator=g).bfloat16()
    offsets = torch.tensor([0, 70, 70, T], dtype=torch.int32)
    dz = torch.randn(T, D, generator=g).bfloat16()
    z, kept = layer.forward(tokens.cuda(), offsets.cuda())
    dtok, small = layer.backward(dz.cuda(), tokens.cuda(), offsets.cuda(), kept)

    w = [ref.dequantize(c.cpu(), s.cpu()).requires_grad_() for c, s in layer.weights]
    par = {k: getattr(layer, k).cpu().double().requires_grad_() for k in ("w_pre", "w_post", "gate")}
    t = tokens.double().requires_grad_()

    def norm(x, k):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * par[k]

    x = norm(t, "w_pre")
    rows = []
    for e, lo, hi in ref.runs(offsets, T):
        h, u = x[lo:hi] @ w[0][e].t(), x[lo:hi] @ w[1][e].t()
        rows.append((h * torch.sigmoid(h) * u) @ w[2][e].t())
    zd = t + 0.5 * par["gate"] * norm(torch.cat(rows), "w_post")
    leaves = [t, *w, *par.values()]
    want = torch.autograd.grad(zd, leaves, dz.double())
    got = [dtok, *layer.grads, *(small[k] for k in par)]

    def close(a, b, what):
        a, b = a.detach().cpu().double(), b.detach()
        assert float((a - b).norm()) <= 16 * 2.0 ** -9 * float(b.norm()), what

    close(z, zd, "z")
    for a, b, what in zip(got, want, ("tokens", "gate weight", "up weight", "down weight", *par)):
        close(a, b, what)


def test_step_moves_the_codes_and_masters():
    layer = _layer(2, 256, 128)
    before = [c.clone() for c in layer.codes]
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randn(96, 256, device="cuda", generator=g).bfloat16()
    offsets = torch.tensor([0, 50, 96], dtype=torch.int32, device="cuda")
    z, kept = layer.forward(tokens, offsets)
    _, small = layer.backward(z, tokens, offsets, kept)
    layer.step(small, 1e-3)
    assert layer.shard.read_state()["step"] == 1
    assert all(bool((a != b).any()) for a, b in zip(before, layer.codes))


def test_training_lowers_the_loss():
    from examples.train_ffn_layer import main

    losses = main(["--steps", "30", "--experts", "2", "--width", "256", "--inner", "128", "--tokens", "512"])
    assert losses[-1] < 0.7 * losses[0], losses
