"""Every step of the example's backward against the 64-bit oracle, from the layer's own
operands of that step: the quantised gradient rows, both products by the transposed
weights, the activation's gradient, the tokens' gradient and both weight gradients.

Tolerances are those of the single operators: a product to bf16 as test_gpu_gemm_experts
has it, the activation's gradient as test_gpu_glu, sums of topk + 1 terms 2^-24 of their
magnitudes for each, a weight gradient 2^-22 for each 32 rows, and half a step of the
result's type."""
import numpy as np
import pytest

from oracle import experts as ox
from tests.gpu_util import note, sync
from tests.test_gpu_glu import near_e4m3
from tests.test_gpu_moe_layer import U, host, make, near, rows_of, weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,topk,experts,hidden,inner", [(1, 4, 6, 200, 128), (37, 2, 3, 384, 256), (400, 3, 4, 260, 128),
                                                              (900, 4, 5, 512, 384)])
def test_every_step(tokens, topk, experts, hidden, inner):
    note(f"backward of the layer of experts {tokens} {topk} {experts} {hidden} {inner}")
    layer, x, ids, w, dy = make(tokens, topk, experts, hidden, inner, 40 + tokens)
    steps, product = [], layer.product

    def kept(a, *args):
        steps.append((a, product(a, *args)))
        return steps[-1][1]
    layer.product = kept
    layer.forward(x, ids, w)
    dx, dw, dW13, dW2 = layer.backward(dy)
    sync()
    (A, _), (B, Y), (dY, dB), (dG, dA) = steps
    place, order, offsets = ox.sort(ids.cpu().numpy(), experts)
    slots, n = tokens * topk, offsets[-1]
    tok = order[:n] // topk

    def full(v):  # rows of no slot are not read: zeros here
        out = np.zeros((slots, v.shape[1]))
        out[:n] = v[:n]
        return out

    rows = host(dy).astype(np.float32)[tok] * host(w).astype(np.float32).reshape(-1)[order[:n]][:, None]
    assert np.array_equal(rows_of(dY)[:n], ox.dequant_rows(*ox.quant_rows(rows))[:, :hidden])
    ref, mag = ox.product(full(rows_of(dY)), weights_of(layer.W2, True)[:, :, :hidden], offsets)
    near(host(dB)[:n], ref[:n], mag[:n], hidden, 2.0 ** -8)
    ref, mag = ox.glu_grad(host(dB)[:n], rows_of(layer.G)[:n])
    near_e4m3(np.ascontiguousarray(dG.q.cpu().numpy().reshape(slots, -1)[:n]),
              np.ascontiguousarray(dG.scale.cpu().numpy().reshape(-1, slots)[:, :n]), ref, 16 * U * mag + 2.0 ** -126)
    ref, mag = ox.product(full(rows_of(dG)), weights_of(layer.W13, True)[:, :, :2 * inner], offsets)
    near(host(dA)[:n], ref[:n], mag[:n], 2 * inner, 2.0 ** -8)
    ref, mag = ox.combine(full(host(dA)), place, None, host(dy))
    bound = (topk + 1) * U * mag
    assert np.all(np.abs(host(dx) - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8)
    _, ref, mag = ox.combine_grad(host(dy), full(host(Y)), place, host(w))
    assert np.all(np.abs(host(dw) - ref) <= (hidden + 1) * U * mag)
    for got, d, a in ((dW13, dG, A), (dW2, dY, B)):
        ref, mag = ox.wgrad(full(rows_of(d)), full(rows_of(a)), offsets)
        assert np.all(np.abs(host(got) - ref) <= (n / 32 + 3) * 2.0 ** -22 * mag)
