"""The example's residual layer end to end: every product of the forward and
the backward against the 64-bit oracle of the operators it is made of, on the
operands those produce (each operator by itself is tested elsewhere)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import mx
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("mxfp4_layer", os.path.join(ROOT, "examples", "mxfp4_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    return t.double().cpu().numpy()


def tensor(v):
    return torch.from_numpy(np.asarray(v, np.float32)).bfloat16().to("cuda:0")


def near(got, ref, terms, k, half):
    """A product over k values: fp32 sums (k / 128 instructions, 2^-22 of the
    magnitudes each) and the result's own rounding."""
    bound = k / 128 * 2.0 ** -22 * terms
    bound = bound + (np.abs(ref) + bound) * half
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("tokens,n_in,n_out", [(1, 200, 260), (37, 384, 130), (300, 256, 520)])
def test_layer_forward_and_backward(tokens, n_in, n_out):
    rng = np.random.default_rng(tokens)
    W, w = tensor(rng.standard_normal((n_out, n_in)) / np.sqrt(n_in)), tensor(1 + 0.2 * rng.standard_normal(n_in))
    x, r, dh = (tensor(rng.standard_normal((tokens, n_in))) for _ in range(3))
    dc = tensor(rng.standard_normal((tokens, n_out)))
    note(f"layer {tokens} {n_in} {n_out}")
    layer = example().ResidualLinear(config(), W, w, tokens + 3)
    c, h = layer.forward(x, r)
    dx, dw, dW = layer.backward(dc, dh)
    sync()
    assert torch.equal(h, x + r)
    y, rstd = mx.rms(host(h), host(w), layer.eps)
    k = mx.padded(n_in)
    near(host(c), *mx.gemm_mxfp4(*mx.quant_mxfp4(y), *mx.quant_mxfp4(host(W))), k, 2.0 ** -8)
    # dy as the layer computes it, rounded to bf16, feeds the norm's gradient
    qd, sd = mx.quant_mxfp4(host(dc))
    dy, dy_abs = mx.gemm_mxfp4(qd, sd, *mx.quant_mxfp4(host(W), transpose=True))
    ko = mx.padded(n_out)
    dy_err = ko / 128 * 2.0 ** -22 * dy_abs
    dy_err = dy_err + (np.abs(dy) + dy_err) * 2.0 ** -8
    want, want_w, _, _ = mx.rms_grad(dy, host(h), host(w), rstd, host(dh))
    # what an error of dy does to dx and dw, linear in it, and the gradient's
    # own fp32 sums over n_in and over the tokens (2^-24 a term and operation),
    # with rstd itself off by half an fp32 step
    n = np.abs(host(h)) * rstd[:, None]
    ge, ga = dy_err * np.abs(host(w)), np.abs(dy * host(w))
    u = 2.0 ** -24
    lin = rstd[:, None] * (ge + n * (ge * n).mean(1, keepdims=True))
    own = rstd[:, None] * (8 * u * ga + (n_in + 10) * u * n * (ga * n).mean(1, keepdims=True)) + 2 * u * np.abs(host(dh))
    bound = (lin + own) * (1 + 1e-2)
    assert np.all(np.abs(host(dx) - want) <= bound + (np.abs(want) + bound) * 2.0 ** -8)
    bound = ((dy_err * n).sum(0) + (tokens + 6) * u * (np.abs(dy) * n).sum(0)) * (1 + 1e-2)
    assert np.all(np.abs(host(dw) - want_w) <= bound + 2.0 ** -149)
    # y in bf16 before it is quantised along the tokens
    yb = torch.empty_like(h)
    import tile_scheduling_persistent_amd as pg
    pg.prms_run(config(), h, w, yb, tokens, n_in, eps=layer.eps)
    sync()
    kt = mx.padded(tokens)
    near(host(dW), *mx.gemm_mxfp4(*mx.quant_mxfp4(host(dc), transpose=True), *mx.quant_mxfp4(host(yb), transpose=True)),
         kt, 2.0 ** -24)


def test_one_token_equals_its_row_of_many():
    """A token alone and among others: quantisation is by row and the products
    differ only in the order of their sums."""
    rng = np.random.default_rng(3)
    n_in, n_out = 640, 700
    W, w = tensor(rng.standard_normal((n_out, n_in))), tensor(1 + 0.2 * rng.standard_normal(n_in))
    x, r = tensor(rng.standard_normal((90, n_in))), tensor(rng.standard_normal((90, n_in)))
    layer = example().ResidualLinear(config(), W, w, 90)
    many, _ = layer.forward(x, r)
    one, h = layer.forward(x[41:42], r[41:42])
    sync()
    y, _ = mx.rms(host(h), host(w), layer.eps)
    ref, terms = mx.gemm_mxfp4(*mx.quant_mxfp4(y), *mx.quant_mxfp4(host(W)))
    near(host(one), ref, terms, n_in, 2.0 ** -8)
    near(host(many)[41:42], ref, terms, n_in, 2.0 ** -8)
