"""Pins of the MXFP4 / RMS-norm oracle on small cases worked by hand or by
brute force, and the host-side checks of the new entry points' binding."""
import itertools

import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tile_scheduling_persistent_amd import _abi


def test_e2m1_rounding_by_hand():
    t = np.array([0.0, 0.25, 0.2500001, 0.75, 0.7499, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 6.0, 7.9, 100.0])
    want = [0, 0, 0.5, 1.0, 0.5, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0, 6.0]
    assert np.array_equal(mx.E2M1_MAGNITUDES[mx.nearest_code(t, mx.E2M1_MAGNITUDES)], want)


@pytest.mark.parametrize("mag", [mx.E2M1_MAGNITUDES, mx.E4M3_MAGNITUDES])
def test_nearest_code_by_brute_force(mag):
    t = np.concatenate([mag, (mag[1:] + mag[:-1]) / 2, np.random.default_rng(1).uniform(0, mag[-1] * 1.2, 500)])
    for v, c in zip(t, mx.nearest_code(t, mag)):
        d = np.abs(mag - min(v, mag[-1]))
        best = np.flatnonzero(d == d.min())
        assert c == (best[0] if len(best) == 1 else best[best % 2 == 0][0])


def test_scale_exponents_by_hand():
    a = np.array([6.0, 6.0001, 3.0, 3.0001, 1.5 * 2.0 ** -140, 0.0, 2.0 ** 120, 7.99])
    assert mx.scale_exponent(a, 6.0, 2, "ceil").tolist() == [0, 1, -1, 0, -127, -127, 118, 1]
    assert mx.scale_exponent(a, 6.0, 2, "floor").tolist() == [0, 0, -1, -1, -127, -127, 118, 0]
    assert mx.scale_exponent(np.array([448.0, 449.0, 224.0]), 448.0, 8, "ceil").tolist() == [0, 1, -1]


def test_quant_layout_and_round_trip():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 200)) * np.exp(rng.standard_normal((5, 1)))
    q, s = mx.quant_mxfp4(x)
    assert q.shape == (5, 128) and s.shape == (2, 5, 4)
    assert np.all(s[1, :, 3] == 0) and np.all(q[:, 100:] == 0)   # the block of 224..255 is padding
    v = mx.dequant_mxfp4(q, s, 200)
    scale = 2.0 ** (s.transpose(1, 0, 2).reshape(5, -1).astype(float) - 127).repeat(32, 1)[:, :200]
    assert np.all(np.abs(v - x) <= scale)             # half the largest step, 2, in units of the scale
    q2, s2 = mx.quant_mxfp4(v)
    assert np.array_equal(mx.dequant_mxfp4(q2, s2, 200), v)
    qt, st = mx.quant_mxfp4(x, transpose=True)
    assert qt.shape == (200, 64) and st.shape == (1, 200, 4)
    # element (k = 3, n = 1): low / high nibble
    q, s = mx.quant_mxfp4(np.array([[1.0, 2.0, 3.0, 6.0]]))
    assert q[0, :2].tolist() == [0x42, 0x75] and s[0, 0, 0] == 127


def test_special_blocks():
    x = np.zeros((1, 128))
    x[0, 5], x[0, 40] = np.nan, -np.inf
    x[0, 70] = 1.0
    q, s = mx.quant_mxfp4(x)
    assert s[0, 0].tolist() == [255, 255, 125, 0]
    v = mx.dequant_mxfp4(q, s, 128)
    assert np.all(np.isnan(v[0, :64])) and v[0, 70] == 1.0 and np.all(v[0, 96:] == 0)


def test_gradient_against_differences():
    """The oracle's gradient against central differences of its norm: with step
    d and values of order one the difference's own error is of order d**2 and
    2**-53 / d, 1e-8 at d = 1e-5 within two orders."""
    rng = np.random.default_rng(3)
    rows, cols, eps, d = 3, 7, 1e-3, 1e-5
    x, r, w = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols)), rng.standard_normal(cols)
    dy, dh = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))

    def loss(x, w):
        return (mx.rms(x + r, w, eps)[0] * dy).sum() + ((x + r) * dh).sum()

    dx, dw, _, _ = mx.rms_grad(dy, x + r, w, mx.rms(x + r, w, eps)[1], dh)
    for i, j in itertools.product(range(rows), range(cols)):
        e = np.zeros_like(x)
        e[i, j] = d
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - dx[i, j]) < 1e-6
    for j in range(cols):
        e = np.zeros(cols)
        e[j] = d
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - dw[j]) < 1e-6


# ---- refusals that need no device ------------------------------------------


def test_entry_points_refuse_null_config():
    L = _abi.lib()
    assert L.pmx_quant_run(None, None, 1, 1, 1, 1, 0, 0, None, None, None) == _abi.ERR_INVALID
    assert L.pmx_dequant_run(None, None, None, 1, 1, None, 1, 1, None) == _abi.ERR_INVALID
    assert L.prms_run(None, None, 1, 1, None, 1, 1, None, 1, 1e-6, 1, 1, None, 1, 0, None, 1, None, None,
                      None) == _abi.ERR_INVALID
    assert L.prms_grad_run(None, None, 1, 1, None, 1, 1, None, 1, None, 1, None, 1, 1, None, 1, None,
                           None) == _abi.ERR_INVALID


class _NoDevice:
    """Stands for a config: the binding's own checks come before the library."""
    handle = None
    device = 0


def test_binding_checks_shapes_and_types():
    cfg = _NoDevice()
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros(4, 200, dtype=torch.bfloat16)
    assert pg.mxfp4_bytes(4, 200) == {"Q": 4 * 128, "scale": 2 * 4 * 4}
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        pg.pmx_quant_run(cfg, x.double(), u8(512), u8(32), 4, 200)
    with pytest.raises(ValueError, match="X"):
        pg.pmx_quant_run(cfg, x[:3], u8(512), u8(32), 4, 200)
    with pytest.raises(KeyError):
        pg.pmx_quant_run(cfg, 4096, u8(512), u8(32), 4, 200, rule="nearest", x_type=1)
    with pytest.raises(ValueError, match="Q"):
        pg.pmx_quant_run(cfg, 4096, u8(511), u8(32), 4, 200, x_type=1)
    with pytest.raises(ValueError, match="scale"):
        pg.pmx_dequant_run(cfg, 4096, u8(31), 4096, 4, 200, y_type=1)
    w = torch.zeros(200, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        pg.prms_run(cfg, x, w, x, 4, 200)
    nb = pg.gemm_bytes(3, 5, 256, "mxfp4_out_f32")
    assert nb == {"A": 384, "B": 640, "C": 60, "a_scale": 24, "b_scale": 40}
    with pytest.raises(ValueError, match="C"):
        pg._gemm_ptrs(u8(384), u8(640), torch.zeros(14), 3, 5, 256, "mxfp4_out_f32", None)
    with pytest.raises(ValueError, match="dtype"):
        pg._gemm_ptrs(u8(384), u8(640).to(torch.int32), torch.zeros(15), 3, 5, 256, "mxfp4_out_f32", None)
