"""The mixture-of-experts operators together, as a layer uses them: few tokens
and a prompt, a training step, captured graphs, other streams, and what the
conveniences refuse."""
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import moe_util as M
from test_gpu_streams import late_writes, ordered

sys.path.insert(0, str(Path(__file__).resolve().parents[1] / "examples"))
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_layer(fp4, fmt, score, tokens):
    """Both ways of the example against its formula in 64 bits over the same
    packed weights. few: bf16 rounds three times (2^-8 relative each, on both
    halves of the gate and on its product, then at the experts' results and the
    sum); every rounding is bounded by the magnitudes that meet there. many:
    also quantizes activations to 4 bits, and is checked where that is exact."""
    import moe_layer as ex
    hidden, inter, E, k = 128, 64, 8, 2
    layer = ex.MoeLayer(hidden, inter, E, k, fmt, score)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(tokens)).bfloat16().cuda()
    w, ids = layer.route(x)
    W13, W2 = M.values(layer.w13), M.values(layer.w2)
    x64, i, w64 = x.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy()
    h = np.einsum("th,tknh->tkn", x64, W13[i])
    mag = np.einsum("th,tknh->tkn", np.abs(x64), np.abs(W13[i])) * 2 * hidden * U
    a, b = h[..., :inter], h[..., inter:]
    silu = a / (1 + np.exp(-a))
    g = silu * b
    # errors: of a and b (sum, one rounding), silu' <= 1.1, two roundings of the gate
    ea, eb = mag[..., :inter] + 2.0 ** -8 * np.abs(a), mag[..., inter:] + 2.0 ** -8 * np.abs(b)
    eg = 1.1 * ea * (np.abs(b) + eb) + (np.abs(silu) + 1.1 * ea) * eb + 2 * 2.0 ** -8 * (np.abs(silu) + 1.1 * ea) * (np.abs(b) + eb)
    y = np.einsum("tki,tkhi->tkh", g, W2[i])
    ey = np.einsum("tki,tkhi->tkh", eg + 2 * inter * U * np.abs(g), np.abs(W2[i]))
    ey = ey + 2.0 ** -8 * (np.abs(y) + ey)
    out = (y * w64[..., None]).sum(1)
    tol = (ey * w64[..., None]).sum(1)
    tol = tol + 2.0 ** -8 * (np.abs(out) + tol) + 8 * U * (np.abs(y) * w64[..., None]).sum(1)
    got = layer.few(x)
    err = np.abs(got.double().cpu().numpy() - out)
    assert got.dtype == BF and (err <= tol).all(), (err / tol).max()
    # the grouped way: its own 4-bit activations, so compare what its steps make of them
    groups = fp4.moe_group(ids, E)
    rows = fp4.moe_dispatch(fp4.quantize(x, fmt, four_over_six=True), groups)
    c = fp4.gemm_grouped(rows, layer.w13, groups.offsets, torch.float32).double().cpu().numpy()
    A = M.values(rows)
    at = groups.place.cpu().numpy()
    want = np.einsum("tkh,tknh->tkn", A[at], W13[i])
    size = np.einsum("tkh,tknh->tkn", np.abs(A[at]), np.abs(W13[i]))
    assert (np.abs(c[at] - want) <= (2 * hidden + 4) * U * size).all()
    many = layer.many(x)
    assert many.shape == x.shape and many.isfinite().all()


def test_example_runs(fp4, capsys):
    import moe_layer as ex
    ex.main("nvfp4", hidden=256, inter=128, experts=8, top_k=2, prompt=100, batch=3, steps=3)
    assert "us a step" in capsys.readouterr().out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step(fp4, score):
    """Gradients of sum(out * g), out = sum_j w_j W_e x with fp32 experts, for
    x, the experts and the router, against 64 bits. Every sum in the chain has at
    most H + F + T + k terms, so the result is within (sum of their lengths + 64)
    2^-24 of the same chain over magnitudes."""
    T, H, F, E, k = 24, 64, 48, 8, 3
    gen = torch.Generator().manual_seed(4)
    x, R, W, g = (torch.randn(*s, generator=gen) for s in ((T, H), (E, H), (E, F, H), (T, F)))
    dev = lambda t: t.cuda()
    logits = dev(x) @ dev(R).T
    w, ids = fp4.moe_route(logits, k, score=score, scale=1.5)
    groups = fp4.moe_group(ids, E)
    rows = fp4.moe_dispatch(dev(x), groups)
    offs = groups.offsets.tolist()
    part = [slice(offs[e], offs[e + 1]) for e in range(E)]
    y = torch.cat([rows[p] @ dev(W[e]).T for e, p in enumerate(part)])
    out = fp4.moe_combine(y, w, groups)
    gy, gw = fp4.moe_combine_backward(dev(g), y, w, groups)
    gW = torch.stack([gy[p].T @ rows[p] for p in part])
    grows = torch.cat([gy[p] @ dev(W[e]) for e, p in enumerate(part)])
    glogits = fp4.moe_route_backward(gw, logits, ids, score=score, scale=1.5)
    gx = fp4.moe_combine(grows, None, groups) + glogits @ dev(R)
    gR = glogits.T @ dev(x)

    z, i = logits.double().cpu().numpy(), ids.cpu().numpy()
    X, Rn, Wn, G = (t.double().numpy() for t in (x, R, W, g))

    def chain(X, Rn, Wn, G, w, back):
        Y = np.einsum("th,tkfh->tkf", X, Wn[i])
        dw = np.einsum("tkf,tf->tk", Y, G)
        dl = back(dw)
        dW = np.zeros_like(Wn)
        for t in range(T):
            for j in range(k):
                dW[i[t, j]] += w[t, j] * np.outer(G[t], X[t])
        dX = np.einsum("tk,tkfh,tf->th", w, Wn[i], G) + dl @ Rn
        return (Y * w[..., None]).sum(1), dW, dX, dl.T @ X

    w64 = M.weights(z, i, score, True, 1.5)
    want = chain(X, Rn, Wn, G, w64, lambda d: M.route_gradient(d, z, i, score, True, 1.5))

    def spread(d):  # magnitudes of what enters a logit's gradient
        o = np.zeros((T, E))
        np.put_along_axis(o, i, w64 * (d + (d * w64 / 1.5).sum(1, keepdims=True)), 1)
        return o
    size = chain(np.abs(X), np.abs(Rn), np.abs(Wn), np.abs(G), w64, spread)
    tol = (2 * (H + F + T) + 8 * k + 64) * U
    for name, got, a, b in zip(("out", "W", "x", "router"), (out, gW, gx, gR), want, size):
        err = np.abs(got.double().cpu().numpy() - a)
        assert (err <= tol * b + 1e-30).all(), (name, (err / (tol * b + 1e-30)).max())


def steps(fp4, T, E, k, H, seed):
    """Operands on the GPU and a pass of every operator on them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    z, x, grad = rnd(T, E), rnd(T, H).bfloat16(), rnd(T, H).bfloat16()
    q = fp4.quantize(rnd(E, 96, H), "nvfp4")
    bias = 0.1 * rnd(E)

    def run(stream=None):
        w, ids = fp4.moe_route(z, k, score="sigmoid", bias=bias, groups=4, top_groups=2, group_best=2, stream=stream)
        gr = fp4.moe_group(ids, E, stream=stream)
        rows = fp4.moe_dispatch(x, gr, stream=stream)
        out = fp4.moe_combine(rows, w, gr, stream=stream)
        dr, dw = fp4.moe_combine_backward(grad, rows, w, gr, stream=stream)
        dz = fp4.moe_route_backward(dw, z, ids, score="sigmoid", stream=stream)
        res = [w, ids, gr.offsets, gr.order, gr.place, rows, out, dr, dw, dz]
        if T * k <= 4096:
            res += [fp4.matvec(x, q, ids, stream=stream),
                    fp4.matvec(x[:3], fp4.Quantized(q.fmt, q.codes[0], q.scales[0], q.tensor_scale[:1]), stream=stream)]
        return res
    return (z, x, grad), run


@pytest.mark.parametrize("T", [5, 300, 4000])
def test_graph_replays_match_eager(fp4, T):
    inputs, run = steps(fp4, T, 16, 4, 160, 1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    other = torch.cuda.CUDAGraph()  # a second graph of the same calls, replayed in between
    with torch.cuda.graph(other):
        again = run()
    for n in range(4):
        for t in inputs:
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(10 * T + n)).to(t.dtype))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        eager = run()
        for a, b, c in zip(captured, again, eager):
            assert torch.equal(a, c) and torch.equal(b, c)


@pytest.mark.parametrize("T", [6, 5000])
def test_on_another_stream(fp4, T):
    """Outputs and workspace belong to the stream named: late writes of the
    current stream over freed memory do not reach them."""
    E, k, H = 16, 4, 96
    inputs, run = steps(fp4, T, E, k, H, 2)
    want = [t.cpu() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late_writes([T * k * 4, T * k * 4, (E + 1) * 4, T * k * H * 2, T * H * 2, T * E * 4, T * k * 96 * 2, 5 * 17 * 4, 20 * 17 * 4])
    got = ordered(side, lambda s: tuple(run(s)))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_packed_dispatch_on_another_stream(fp4):
    x = fp4.quantize(torch.randn(40, 64).bfloat16().cuda(), "nvfp4")
    g = fp4.moe_group(torch.randint(0, 4, (40, 2), dtype=torch.int32).cuda(), 4)
    want = fp4.moe_dispatch(x, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late_writes([80 * 128, 80 * 16])
    got = fp4.moe_dispatch(x, g, stream=side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    assert got.tensor_scale is x.tensor_scale


def test_refusals(fp4):
    """What the conveniences check before the library does."""
    F = fp4
    z, w, ids = torch.zeros(4, 8).cuda(), torch.zeros(4, 2).cuda(), torch.zeros(4, 2, dtype=torch.int32).cuda()
    g = F.moe_group(ids, 8)
    q = F.quantize(torch.zeros(3, 16, 64).cuda(), "mxfp4")
    x = torch.zeros(4, 64).cuda()
    bad = [lambda: F.moe_route(z, 2, score="max"), lambda: F.moe_route(z.double(), 2), lambda: F.moe_route(z[0], 2),
           lambda: F.moe_route(z.T, 2), lambda: F.moe_route(z, 2, bias=torch.zeros(7).cuda()),
           lambda: F.moe_route(z, 2, bias=torch.zeros(8)), lambda: F.moe_route(z, 2, scale="x"),
           lambda: F.moe_route_backward(w, z, ids.long()), lambda: F.moe_route_backward(w[:, :1], z, ids),
           lambda: F.moe_route_backward(w, z, ids[:2]), lambda: F.moe_group(ids.long(), 8), lambda: F.moe_group(ids.T, 8),
           lambda: F.moe_dispatch(z[:3], g), lambda: F.moe_dispatch(z.T, g), lambda: F.moe_dispatch(z.double(), g),
           lambda: F.moe_combine(z, w, g, out=torch.zeros(3, 8).cuda()), lambda: F.moe_combine(z[:3], w),
           lambda: F.moe_combine(torch.zeros(8, 8).cuda(), w, g, out=torch.zeros(4, 8).cuda().bfloat16()),
           lambda: F.moe_combine(torch.zeros(8, 8).cuda(), w.double(), g), lambda: F.moe_combine(torch.zeros(8, 8).cuda()),
           lambda: F.moe_combine_backward(z, torch.zeros(7, 8).cuda(), w, g),
           lambda: F.moe_combine_backward(z[:, :5], torch.zeros(8, 8).cuda(), w, g),
           lambda: F.matvec(x, q), lambda: F.matvec(x[:, :32], q, ids), lambda: F.matvec(x, q, ids.long()),
           lambda: F.matvec(x[:3], q, ids), lambda: F.matvec(x.half(), q, ids),
           lambda: F.matvec(x, q, ids, out=torch.zeros(4, 2, 15).cuda()),
           lambda: F.matvec(x, F.Quantized(q.fmt, q.codes[0], q.scales[0].cpu(), None)),
           lambda: F.matvec(x, F.Quantized(1, q.codes[0], q.scales[0].repeat(1, 2), None))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} passed")
    for call, status in ((lambda: F.moe_route(z, 9), F.FP4_ERR_INVALID), (lambda: F.moe_group(ids, 0), F.FP4_ERR_INVALID),
                         (lambda: F.moe_group(ids, 2000), F.FP4_ERR_UNSUPPORTED),
                         (lambda: F.moe_route(z, 2, groups=3), F.FP4_ERR_INVALID)):
        with pytest.raises(F.Fp4Error) as e:
            call()
        assert e.value.status == status
