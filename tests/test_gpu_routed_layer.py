"""GPU: a routed feed-forward layer with 8-bit rows, forward and backward, as a training step calls it: every call's
results against 64 bits from that call's own inputs, the rows' gradient against the layer's, and the step in a graph."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_reference as ref  # noqa: E402
from tests import rows8_reference as r8  # noqa: E402
from tests.test_gpu_tokens import plan  # noqa: E402

pytestmark = pytest.mark.gpu
U = ref.U32
EPS = 1e-6


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(T, D, F, E, dtype, seed):
    """Inputs of a step, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    weights = dict(router=ref.make_weight(g, 1, E, D), gate=ref.make_weight(g, E, F, D), up=ref.make_weight(g, E, F, D),
                   down=ref.make_weight(g, E, D, F))
    for name, width in (("router", D), ("gate", D), ("up", D), ("down", F)):
        codes, scales = weights[name]
        rms = ref.dequantize(codes, scales).square().mean().sqrt()
        weights[name] = codes, (scales / float(rms) / width ** 0.5).float()
    rows = {n: torch.randn(T, D, generator=g).to(dtype) for n in ("y", "res", "dy")}
    return weights, dict(rows, norm=torch.rand(D, generator=g) + 0.5)


def step(weights, x, k, score):
    """The layer and its gradients; everything that a call gave."""
    from blockwise_fp8_zero_fold_amd import block, routing
    dtype = x["y"].dtype
    out = {}
    out["z"], out["n"], n8 = block.norm_join8(x["y"], x["res"], w_pre=x["norm"], eps=EPS, keep=True)
    out["n8"] = n8
    out["logits"], _ = block.linear(n8, weights["router"], dtype=dtype)
    out["experts"], out["weights"] = routing.route(out["logits"], k, score=score)
    E = weights["gate"][0].shape[0]
    out["offsets"], out["row_of"] = off, row_of = routing.sort_tokens(out["experts"], E)
    out["rows8"] = rows8 = routing.dispatch(n8, row_of)
    out["a8"], (h, u) = block.ffn_up8(rows8, weights["gate"], weights["up"], off, save=True, dtype=dtype)
    out["h"], out["u"] = h, u
    out["rows"], _ = block.ffn_forward8(rows8, weights["gate"], weights["up"], weights["down"], off, dtype=dtype)
    out["out"] = routing.combine(out["rows"], row_of, out["weights"], base=out["z"])
    out["drows"], out["dweights"] = routing.combine_backward(x["dy"], out["rows"], row_of, out["weights"])
    dx_rows, dh, du, a = block.ffn_backward_data(out["drows"], h, u, weights["gate"], weights["up"], weights["down"], off)
    out["dlogits"] = routing.route_backward(out["dweights"], out["logits"], out["experts"], score=score)
    out["dn_router"] = block.linear_backward(out["dlogits"], weights["router"])["dx"]
    out["dn"] = routing.combine(dx_rows, row_of, base=out["dn_router"])
    rows16 = routing.dispatch(out["n"], row_of)
    out["dw"] = block.ffn_backward_weights(rows16, a, out["drows"], dh, du, n_experts=E, offsets=off)
    out["dw_router"] = block.ffn_weight_gradient(out["dlogits"], out["n"])
    grads = block.norm_join_backward(x["dy"], out["dn"], x["y"], out["z"], w_pre=x["norm"], eps=EPS)
    out["dy_in"], out["dres"], out["dnorm"] = grads["dy"], grads["dres"], grads["dw_pre"]
    return out


def to(v, device):
    return tuple(to(t, device) for t in v) if isinstance(v, tuple) else v.to(device)


def flat(out):
    """(name, tensor) of everything, rows that no expert has cleared."""
    used = int(out["offsets"][-1])
    for name, v in out.items():
        for i, t in enumerate(v if isinstance(v, tuple) else (v,)):
            rows = name in ("rows8", "a8", "h", "u", "rows", "drows")
            yield f"{name}{i}", t[:used] if rows else t


def layer(n, experts, weights, W, score):
    """sum over the choices of weights times the expert's rows, and the weights, in 64 bits; `weights` of the logits'
    scores if None."""
    T, k = experts.shape
    chosen = experts.clamp(min=0).long()
    logits = n @ W["router"][0].T
    if weights is None:
        s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
        s = s.gather(1, chosen) * (experts >= 0)
        weights = s / s.sum(1, keepdim=True)
    y = torch.zeros(T, n.shape[1], dtype=torch.float64)
    for e in range(W["gate"].shape[0]):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        if len(t):
            x = n[t]
            a = torch.nn.functional.silu(x @ W["gate"][e].T) * (x @ W["up"][e].T)
            y = y.index_add(0, t, weights[t, j][:, None] * (a @ W["down"][e].T))
    return y, weights


SIZES = [(1, 256, 128, 4, 2), (37, 300, 200, 5, 3), (700, 384, 260, 8, 2), (500, 130, 129, 64, 6)]


@pytest.mark.parametrize("T,D,F,E,k", SIZES)
@pytest.mark.parametrize("dtype,score", [(torch.bfloat16, "softmax"), (torch.float16, "sigmoid")])
def test_layer(T, D, F, E, k, dtype, score):
    W, x = make(T, D, F, E, dtype, T + D)
    out = step({n: to(w, "cuda") for n, w in W.items()}, {n: v.cuda() for n, v in x.items()}, k, score)
    used = int(out["offsets"][-1])
    c = {n: to(v, "cpu") for n, v in out.items()}
    V = {n: ref.dequantize(*w) for n, w in W.items()}
    half = ref.half_step(dtype)

    z = x["y"].double() + x["res"].double()
    ref.check(c["z"], z, ref.rounded(z, 2 * U * z.abs(), dtype), "z")
    n = c["n"].double()
    nd = r8.dequantize(*c["n8"])
    wide = c["n8"][1].double().repeat_interleave(128, 1)[:, :D]
    # n in 8 bits and in 16, each rounded from the same float32 value
    assert ((nd - n).abs() <= n.abs() * (1 + 2 * half) * (2.0 ** -4 + half) + wide * 2.0 ** -10 + 1e-7).all()

    logits, mag = ref.grouped(nd, V["router"], None, False)
    ref.check(c["logits"], logits, ref.rounded(logits, ref.sum_error(mag, D) + 7 * 2.0 ** -13 * mag, dtype), "logits")
    got = c["logits"].double()
    assert torch.equal(c["experts"].long(), torch.sort(got, dim=1, descending=True, stable=True).indices[:, :k])
    s = torch.softmax(got, 1) if score == "softmax" else torch.sigmoid(got)
    s = s.gather(1, c["experts"].long())
    want = s / s.sum(1, keepdim=True)
    # the exponential's argument to U of its size and 2 ulp of its own, sums of E, two divisions
    slack = (2 * got.abs().amax(1, keepdim=True) + E + 12) * U
    ref.check(c["weights"], want, slack * want, "weights")

    offsets, row_of = plan(c["experts"], E)
    assert torch.equal(c["offsets"], offsets) and torch.equal(c["row_of"], row_of) and used == T * k
    token = torch.empty(used, dtype=torch.int64)
    token[row_of.reshape(-1).long()] = torch.arange(T).repeat_interleave(k)
    for i in range(2):
        assert torch.equal(c["rows8"][i], c["n8"][i][token])

    rows = nd[token]
    for name, w in (("h", "gate"), ("u", "up")):
        p, mag = ref.grouped(rows, V[w], offsets, False)
        ref.check(c[name], p, ref.rounded(p, ref.sum_error(mag, D), dtype), name)
    ad = r8.dequantize(*c["a8"])
    p, mag = ref.grouped(ad, V["down"], offsets, False)
    ref.check(c["rows"], p, ref.rounded(p, ref.sum_error(mag, F) + 7 * 2.0 ** -13 * mag, dtype), "rows")

    picked, w = c["rows"].double()[row_of.long()], c["weights"].double()
    y = c["z"].double() + (w[:, :, None] * picked).sum(1)
    mag = c["z"].double().abs() + (w[:, :, None] * picked.abs()).sum(1)
    ref.check(c["out"], y, ref.rounded(y, (k + 2) * U * mag, dtype), "out")
    dy = x["dy"].double()
    want = torch.zeros(used, D, dtype=torch.float64)
    want[row_of.reshape(-1).long()] = (w[:, :, None] * dy[:, None]).reshape(-1, D)
    ref.check(c["drows"], want, ref.rounded(want, U * want.abs(), dtype), "drows")
    want = (picked * dy[:, None]).sum(2)
    ref.check(c["dweights"], want, ref.sum_error((picked * dy[:, None]).abs().sum(2), D), "dweights")

    # The gradient of the rows that the experts and the router have read.  Through the experts: the weights of 16-bit
    # logits, drows, h, u, dh and du, dx and its sum are rounded, each to half a step of its own (six halves at bfloat16
    # are under 2^-5).  Through the weights: y's rows come of a in 8 bits (2^-4), and the softmax takes a difference.
    leaf = nd.clone().requires_grad_()
    y, _ = layer(leaf, c["experts"], layer(nd, c["experts"], None, V, score)[1], V, score)
    through, = torch.autograd.grad((y * dy).sum(), leaf)
    leaf = nd.clone().requires_grad_()
    y, _ = layer(leaf, c["experts"], None, V, score)
    whole, = torch.autograd.grad((y * dy).sum(), leaf)
    error = (c["dn"].double() - whole).norm()
    assert float(error) <= 2.0 ** -5 * float(through.norm()) + 2.0 ** -3 * float((whole - through).norm())

    for name, v in flat(c):
        assert torch.isfinite(v.float()).all(), name


@pytest.mark.parametrize("T,D,F,E,k", SIZES[1:3])
def test_layer_in_a_graph(T, D, F, E, k):
    """The step captured once and replayed on other inputs, with eager work between the replays."""
    W, x = make(T, D, F, E, torch.bfloat16, 1)
    W = {n: to(w, "cuda") for n, w in W.items()}
    held = {n: v.cuda() for n, v in x.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(W, held, k, "softmax")
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(W, held, k, "softmax")
    for seed in (2, 3, 2, 4):
        _, x = make(T, D, F, E, torch.bfloat16, seed)
        for n, v in x.items():
            held[n].copy_(v)
        graph.replay()
        got = {n: to(v, "cpu") for n, v in captured.items()}
        eager = {n: to(v, "cpu") for n, v in step(W, {n: v.cuda() for n, v in x.items()}, k, "softmax").items()}
        for (name, a), (_, b) in zip(flat(got), flat(eager)):
            assert torch.equal(a, b), (seed, name)


def test_two_threads_on_streams_of_their_own():
    """Steps of two threads at once give what they give alone."""
    import threading
    T, D, F, E, k = SIZES[2]
    jobs = []
    for seed in (1, 2):
        W, x = make(T, D, F, E, torch.bfloat16, seed)
        jobs.append(({n: to(w, "cuda") for n, w in W.items()}, {n: v.cuda() for n, v in x.items()}))
    alone = [{n: to(v, "cpu") for n, v in step(W, x, k, "softmax").items()} for W, x in jobs]
    torch.cuda.synchronize()
    together, failures = [None, None], []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    out = step(*jobs[i], k, "softmax")
                stream.synchronize()
                together[i] = {n: to(v, "cpu") for n, v in out.items()}
        except Exception as e:  # (shown by the assertion below)
            failures.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures
    for a, b in zip(alone, together):
        for (name, u), (_, v) in zip(flat(a), flat(b)):
            assert torch.equal(u, v), name
