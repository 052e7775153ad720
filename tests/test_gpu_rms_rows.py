"""The RMS norm where rows end inside vectors while they fill the device, where
the order of row groups is permuted, and where a workgroup takes several groups,
against the 64-bit oracle.  h, codes and scale bytes equal; y and rstd to half a
step of their type, plus 1e-9 relative for the 64-bit sums."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tests.gpu_util import config, note, sync
from tests.test_gpu_mx import Bytes
from tests.test_gpu_rms import EPS, U, h_of, half_step, host, inputs, strided
from tests.test_gpu_rms_grad_rows import Banded, normal

pytestmark = pytest.mark.gpu

# ends inside a vector with rows past the CUs or columns past 8192; ranges of
# permuted row groups and a rest of them, for both scale layouts
NORM = [(1061, 1003), (2500, 131), (300, 8201), (1100, 1024)]


@pytest.mark.parametrize("x,r,w", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f16", "f16", "f32"),
                                   ("f32", "f32", "f32"), ("bf16", None, "bf16"), ("f16", None, "f16"),
                                   ("f32", None, "f32")])
@pytest.mark.parametrize("out", ["same", "fp8_b128", "mxfp4"])
@pytest.mark.parametrize("rows,cols", NORM)
def test_norm_of_many_rows_equals_the_oracle(rows, cols, out, x, r, w):
    X, R, W = inputs(rows, cols, x, r, w, rows)
    h = h_of(X, R)
    y, rstd = mx.rms(host(h), host(W), EPS)
    H = Banded((rows, cols), R.dtype) if r else None
    T = torch.zeros(rows, device="cuda:0")
    kw = dict(eps=EPS, R=R, H=H.t if r else None, rstd=T)
    kp = mx.padded(cols)
    note(f"prms_run {rows}x{cols} {x} {r} {w} {out}")
    if out == "same":
        Y = Banded((rows, cols), X.dtype)
        pg.prms_run(config(), X, W, Y.t, rows, cols, **kw)
        sync()
        assert Y.intact()
        assert np.all(np.abs(host(Y.t) - y) <= half_step(y, x) + 1e-9 * np.abs(y))
    else:
        n = 2 if out == "mxfp4" else 1
        Y, S = Bytes(rows * kp // n), Bytes(kp // 128 * rows * (4 if n == 2 else 1))
        pg.prms_run(config(), X, W, Y.view, rows, cols, out=out, y_scale=S.view, **kw)
        sync()
        qr, sr = mx.quant_mxfp4(y) if n == 2 else mx.quant_e4m3(y)
        assert np.array_equal(S.get().reshape(sr.shape), sr)
        assert np.array_equal(Y.get().reshape(qr.shape), qr)
    assert np.all(np.abs(host(T) - rstd) <= rstd * (U * (1 + 1e-6) + 1e-9))
    if r:
        assert H.intact() and torch.equal(H.t, h)


@pytest.mark.parametrize("rows,cols", [(1061, 1003), (300, 8201)])
def test_norm_of_many_strided_rows_and_in_place(rows, cols):
    X, R, W = inputs(rows, cols, "bf16", "bf16", "bf16", 6)
    h = h_of(X, R)
    y, _ = mx.rms(host(h), host(W), EPS)
    (xs, xb), (rs, rb) = strided(X, cols + 4, 3), strided(R, cols + 9, 1)
    note(f"in place {rows}x{cols}")
    pg.prms_run(config(), xs, W, xs, rows, cols, eps=EPS, R=rs, H=rs)      # y over x, h over r
    sync()
    assert torch.equal(rs, h)
    assert np.all(np.abs(host(xs) - y) <= half_step(y, "bf16") + 1e-9 * np.abs(y))
    for big, t in ((xb, xs), (rb, rs)):
        gaps = torch.ones(big.numel(), dtype=torch.bool, device="cuda:0")
        gaps.as_strided((rows, cols), t.stride(), t.storage_offset()).fill_(False)
        assert torch.isnan(big[gaps]).all()


@pytest.mark.parametrize("rows,cols", [(16 * (1 << 20) + 37, 16), (2 * (1 << 20) + 5, 2056)])
def test_norm_of_more_row_groups_than_a_grid_holds(rows, cols):
    """Past 2^20 groups of rows a workgroup takes several, in turn (16 rows of
    16 lanes a group; 2 rows of 128 lanes, whose sums pass through LDS)."""
    g = torch.Generator(device="cuda:0")
    g.manual_seed(cols)
    X = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda:0").normal_(generator=g)
    W = (1 + 0.3 * normal(g, cols)).bfloat16()
    Y, T = torch.full_like(X, -9.0), torch.zeros(rows, device="cuda:0")
    note(f"prms_run {rows}x{cols}")
    pg.prms_run(config(), X, W, Y, rows, cols, eps=EPS, rstd=T)
    sync()
    for a in range(0, rows, 1 << 17):
        x = X[a:a + (1 << 17)].double()
        r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        y = x * r * W.double()
        assert bool(((Y[a:a + (1 << 17)].double() - y).abs() <= y.abs() * (2.0 ** -8 * (1 + 1e-6) + 1e-9) + 2.0 ** -133).all()), a
        assert bool(((T[a:a + (1 << 17)].double() - r[:, 0]).abs() <= r[:, 0] * (U * (1 + 1e-6) + 1e-9)).all()), a
