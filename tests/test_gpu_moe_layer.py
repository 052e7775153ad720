"""The example's layer of experts end to end: each step's operands and results
against the 64-bit oracle, the gradients against the formula's differences, and the
layer captured into a graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import experts as ox
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    return t.double().cpu().numpy()


def rows_of(r):
    kp = -(-r.cols // 128) * 128
    return ox.dequant_rows(r.q.cpu().numpy().reshape(r.rows, kp), r.scale.cpu().numpy().reshape(-1, r.rows))[:, :r.cols]


def weights_of(w, transposed=False):
    n, k = (w.n_in, w.n_out) if transposed else (w.n_out, w.n_in)
    q, s = (w.qt, w.scale_t) if transposed else (w.q, w.scale)
    np_, kp = -(-n // 128) * 128, -(-k // 128) * 128
    q, s = q.cpu().numpy().reshape(w.experts, n, kp), s.cpu().numpy().reshape(w.experts, np_ // 128, kp // 128)
    return np.stack([ox.dequant_weights(a, b) for a, b in zip(q, s)])[:, :, :k]


def near(got, ref, terms, k, half):
    """A product to bf16: fp32 sums, and each eight products of e4m3 cut at 2^-13 of
    their largest, 2^-10 of their magnitudes at most."""
    bound = (k / 32 * 2.0 ** -22 + 8 * U + 2.0 ** -10) * terms
    assert np.all(np.abs(got - ref) <= bound + (np.abs(ref) + bound) * half + 2.0 ** -134)


def make(tokens, topk, experts, hidden, inner, seed):
    g = torch.Generator(device="cuda:0").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda:0") * scale).bfloat16()
    layer = example().Experts(config(), normal(experts, 2 * inner, hidden, scale=hidden ** -0.5),
                              normal(experts, hidden, inner, scale=inner ** -0.5))
    top = torch.randn((tokens, experts + 2), generator=g, device="cuda:0").topk(topk, 1)
    ids = torch.where(top.indices < experts, top.indices, -1)  # two experts are elsewhere
    return layer, normal(tokens, hidden), ids, torch.softmax(top.values, 1), normal(tokens, hidden)


@pytest.mark.parametrize("tokens,topk,experts,hidden,inner", [(1, 4, 6, 200, 128), (37, 2, 3, 384, 256), (400, 3, 4, 260, 128)])
def test_layer_step_by_step(tokens, topk, experts, hidden, inner):
    note(f"layer of experts {tokens} {topk} {experts} {hidden} {inner}")
    layer, x, ids, w, dy = make(tokens, topk, experts, hidden, inner, tokens)
    y = layer.forward(x, ids, w)
    dx, dw, dW13, dW2 = layer.backward(dy)
    sync()
    place, order, offsets = ox.sort(ids.cpu().numpy(), experts)
    n = offsets[-1]
    assert np.array_equal(layer.place.cpu(), place) and np.array_equal(layer.offsets.cpu(), offsets)
    a = rows_of(layer.A)[:n]
    tok = order[:n] // topk
    q, s = ox.quant_rows(host(x)[tok])
    assert np.array_equal(a, ox.dequant_rows(q, s)[:, :hidden])
    # gate and up as the layer's own kept codes have them: each within the product's error, then e4m3's half step
    g, terms = ox.product(a, weights_of(layer.W13)[:, :, :hidden], offsets)
    kept = rows_of(layer.G)[:n]
    err = ((hidden / 32 + 2) * 2.0 ** -22 + 2.0 ** -10) * terms[:n] * 1.01 + 2.0 ** -8 * np.abs(g[:n])
    top = np.abs(kept).reshape(n, -1, 128).max(-1).repeat(128, 1)
    assert np.all(np.abs(kept - g[:n]) <= err + np.maximum(np.abs(g[:n]) * 2.0 ** -4, top * 2.0 ** -16) * 1.01)
    b = rows_of(layer.B)[:n]
    near(host(layer.Y)[:n], *(t[:n] for t in ox.product(b, weights_of(layer.W2)[:, :, :inner], offsets)), inner, 2.0 ** -8)
    Y = np.zeros((tokens * topk, hidden))
    Y[:n] = host(layer.Y)[:n]
    ref, mag = ox.combine(Y, place, host(w), host(x))
    bound = (topk + 1) * U * mag
    assert np.all(np.abs(host(y) - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8)
    ref_dx, ref_dw, mag = ox.combine_grad(host(dy), Y, place, host(w))
    assert np.all(np.abs(host(dw) - ref_dw) <= (hidden + 1) * U * mag)
    # the weight gradients, from the rows that the oracle quantises itself
    dY = np.zeros((tokens * topk, hidden))
    dY[:n] = (host(dy).astype(np.float32)[tok] * host(w).astype(np.float32).reshape(-1)[order[:n]][:, None])
    dYq = ox.dequant_rows(*ox.quant_rows(dY))[:, :hidden]
    full = np.zeros((tokens * topk, inner))
    full[:n] = b
    ref, mag = ox.wgrad(dYq, full, offsets)
    assert np.all(np.abs(host(dW2) - ref) <= (n / 32 + 3) * 2.0 ** -22 * mag)


def test_gradients_against_differences():
    """The layer's own function is a staircase (e4m3), so differences are taken of
    the function without quantisation, with the gradients' error bounded by what 8
    bits do to each factor: a relative step of 2^-4 at most in each of a product's
    chain of six roundings, far less in the norm of a sum of many; the direction has
    to agree."""
    layer, x, ids, w, dy = make(50, 2, 3, 256, 128, 5)
    W13, W2 = (torch.from_numpy(weights_of(t)).cuda() for t in (layer.W13, layer.W2))
    layer.forward(x, ids, w)
    got = layer.backward(dy)
    sync()

    def f(xv, wv, a, b):
        y = xv.clone()
        for j in range(2):
            for e in range(3):
                at = (ids[:, j] == e).nonzero().view(-1)
                g, u = (xv[at] @ a[e].t()).split(128, 1)
                y.index_add_(0, at, (g * torch.sigmoid(g) * u) @ b[e].t() * wv[at, j:j + 1])
        return (y * dy.double()).sum()
    at = [x.double(), w.double(), W13, W2]
    gen = torch.Generator(device="cuda:0").manual_seed(9)
    for i, grad in enumerate(got):
        h = 1e-5 * torch.randn(at[i].shape, generator=gen, device="cuda:0", dtype=torch.float64)
        h = h + 1e-4 * grad.double() / grad.double().norm()  # mostly along the gradient: no cancellation in the difference
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - h, at[i] + h
        want = (f(*hi) - f(*lo)) / 2
        have = (grad.double() * h).sum()
        size = grad.double().norm() * h.norm()
        assert abs((have - want).item()) <= 6 * 2.0 ** -4 * size.item(), i


def test_layer_captured_while_an_eager_one_lives():
    """Forward and backward captured into a graph, replayed with other inputs and
    other routing, against the eager layer on the same inputs."""
    layer, x, ids, w, dy = make(130, 3, 5, 256, 128, 11)
    eager = example().Experts.__new__(example().Experts)
    eager.__dict__.update(layer.__dict__)
    layer.forward(x, ids, w)
    layer.backward(dy)
    sync()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        out = (layer.forward(x, ids, w), *layer.backward(dy))
    for i in range(4):
        _, x2, ids2, w2, dy2 = make(130, 3, 5, 256, 128, 20 + i)
        for a, b in ((x, x2), (ids, ids2 if i else torch.full_like(ids2, -1)), (w, w2), (dy, dy2)):
            a.copy_(b)
        want = (eager.forward(x, ids, w), *eager.backward(dy))
        sync()
        graph.replay()
        again = (eager.forward(x, ids, w), *eager.backward(dy))
        sync()
        for a, b, c in zip(out, want, again):
            assert torch.equal(a, b) and torch.equal(a, c), i


def test_two_layers_on_two_streams_at_once():
    """No workspace is shared: two streams run the same calls of one config."""
    a, b = make(300, 3, 5, 256, 128, 31), make(280, 2, 5, 256, 128, 32)
    want = []
    for layer, x, ids, w, dy in (a, b):
        want.append((layer.forward(x, ids, w), *layer.backward(dy)))
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, (layer, x, ids, w, dy) in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append((layer.forward(x, ids, w), *layer.backward(dy)))
        for s in streams:
            s.synchronize()
        for g, r in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, r))
