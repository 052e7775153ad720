"""The oracle of the layers of experts: hand-made cases, the gradients against
differences, and the refusals that need no device."""
import ctypes

import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import experts as ox
from tile_scheduling_persistent_amd import _abi


def test_sort_by_hand():
    place, order, offsets = ox.sort([[2, 0], [0, 5], [2, -1], [1, 0]], 3)
    assert offsets.tolist() == [0, 3, 4, 6]
    assert order.tolist() == [1, 2, 7, 6, 0, 4, -1, -1]
    assert place.tolist() == [[4, 0], [1, -1], [5, -1], [3, 2]]


def test_weight_blocks_by_hand():
    w = np.zeros((130, 129))
    w[0, 0], w[127, 127] = 3.0, -448.0 * 2
    w[129, 128] = 0.5
    q, s = ox.quant_weights(w)
    assert q.shape == (130, 256) and s.shape == (2, 2)
    assert s.tolist() == [[128, 0], [0, 127 - 9]]
    assert ox.dequant_weights(q, s)[:, :129].tolist() == w.tolist()
    w[5, 5] = np.inf
    q, s = ox.quant_weights(w)
    assert s[0, 0] == 255 and not q[:128, :128].any() and np.isnan(ox.dequant_weights(q, s)[:128, :128]).all()
    # a block of 128 x 128 is the transposed matrix's block
    rng = np.random.default_rng(0)
    w = rng.standard_normal((200, 300))
    q, s = ox.quant_weights(w)
    qt, st = ox.quant_weights(w.T)
    assert np.array_equal(st, s.T) and np.array_equal(qt[:, :200], q[:, :300].T)


def differences(f, x, h=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


def test_glu_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, dy = 2 * rng.standard_normal((3, 10)), rng.standard_normal((3, 5))
    want = differences(lambda v: (ox.glu(v) * dy).sum(), x)
    assert np.allclose(ox.glu_grad(dy, x)[0], want, atol=1e-8)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(2)
    place, order, offsets = ox.sort([[1, 0], [3, 1], [0, 0]], 2)
    x, w, dy = rng.standard_normal((6, 4)), rng.standard_normal((3, 2)), rng.standard_normal((3, 4))
    dx, dw, _ = ox.combine_grad(dy, x, place, w)
    assert np.allclose(dx, differences(lambda v: (ox.combine(v, place, w)[0] * dy).sum(), x), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: (ox.combine(x, place, v)[0] * dy).sum(), w), atol=1e-8)
    # without weights it is the gradient of the gather
    g = rng.standard_normal((6, 4))
    toks = rng.standard_normal((3, 4))

    def gathered(v):
        return (v[np.maximum(order, 0) // 2] * (order >= 0)[:, None] * g).sum()
    assert np.allclose(ox.combine(g * (order >= 0)[:, None], place)[0], differences(gathered, toks), atol=1e-8)


def test_weight_gradient_against_differences():
    rng = np.random.default_rng(3)
    a, b, d = rng.standard_normal((7, 3)), rng.standard_normal((2, 4, 3)), rng.standard_normal((7, 4))
    offsets = [0, 5, 7]
    want = differences(lambda v: (ox.product(a, v, offsets)[0] * d).sum(), b)
    assert np.allclose(ox.wgrad(d, a, offsets)[0], want, atol=1e-8)


def test_calls_without_a_config_are_refused():
    L = _abi.lib()
    n = None
    assert L.pmoe_sort_run(n, n, 0, 1, 1, 1, n, n, n, n) == _abi.ERR_INVALID
    assert L.pmoe_gather_run(n, n, 0, 8, n, 1, 1, 8, 0, n, 8, n, n) == _abi.ERR_INVALID
    assert L.pmoe_combine_run(n, n, 0, 8, n, n, n, 8, n, 0, 8, 1, 1, 8, n) == _abi.ERR_INVALID
    assert L.pmoe_combine_grad_run(n, n, 0, 8, n, 8, n, n, n, 1, 1, 8, 0, n, 8, n, n, n) == _abi.ERR_INVALID
    assert L.pfp8_quant_run(n, n, 0, 1, 8, 8, n, n, n) == _abi.ERR_INVALID
    assert L.pfp8_quant_weights_run(n, n, 0, 1, 8, 8, n, n, n, n, n) == _abi.ERR_INVALID
    assert L.pgemm_run_experts(n, n, n, n, n, n, 0, 1, 8, 128, 1, n, n) == _abi.ERR_INVALID
    assert L.pgemm_run_experts_wgrad(n, n, 1, 8, n, n, n, n, n, 0, 1, 8, 128, 1, n, n) == _abi.ERR_INVALID
    assert L.pglu_run(n, n, 0, 16, 1, 8, n, 0, n, 8, n, n, n, n) == _abi.ERR_INVALID
    assert L.pglu_grad_run(n, n, 0, 8, n, 16, n, 1, 8, n, 0, n, 16, n, n) == _abi.ERR_INVALID


class NoDevice:
    handle, device = ctypes.c_void_p(), 0


def test_binding_refuses_before_any_device_call():
    """Wrong types, short buffers, missing scales and host tensors, without a GPU."""
    cfg, u8 = NoDevice(), torch.uint8
    i32 = torch.zeros(8, dtype=torch.int32)
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ids"):
        pg.pmoe_sort_run(cfg, torch.zeros(8), i32, i32, i32, 4, 2, 3)
    with pytest.raises(ValueError, match="ids"):
        pg.pmoe_sort_run(cfg, torch.zeros(7, dtype=torch.int32), i32, i32, i32, 4, 2, 3)
    with pytest.raises(ValueError, match="GPU"):
        pg.pmoe_gather_run(cfg, x, i32, torch.zeros((8, 8), dtype=torch.bfloat16), 4, 2, 8)
    with pytest.raises(ValueError):
        pg.pfp8_quant_run(cfg, torch.zeros(4, 8, dtype=torch.int32), torch.zeros(512, dtype=u8), torch.zeros(4, dtype=u8), 4, 8)
    with pytest.raises(ValueError, match="bytes|GPU"):
        pg.pgemm_run_experts(cfg, torch.zeros(4 * 128 - 1, dtype=u8), torch.zeros(8 * 128, dtype=u8),
                             torch.zeros((4, 8)), 4, 8, 128, torch.zeros(4, dtype=u8), torch.zeros(1, dtype=u8))
    with pytest.raises(ValueError):
        pg._rows_out(_abi.PRMS_OUT_SAME, torch.zeros((4, 8)), "Y", _abi.PMX_BF16, None, 4, 8)
    with pytest.raises(ValueError, match="scales"):
        pg._rows_out(_abi.PRMS_OUT_FP8_B128, torch.zeros(512, dtype=u8), "Y", _abi.PMX_BF16, None, 4, 8)
    with pytest.raises(KeyError):
        pg.pglu_run(cfg, x, x, 4, 4, out="fp16")
