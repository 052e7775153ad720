"""The norm's e4m3 output as the A operand of the block-scaled fp8 product: the
same C, bit for bit, as from the oracle's quantisation of the oracle's norm, and
within the fp8 product's tolerance of the 64-bit product of that operand."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import gemm as og
from oracle import mx
from synthetic import fp8_blockscaled
from tests.gpu_util import FP8_TOL, Guarded, assert_abs_bound, config, dev_u8, note, sync
from tests.test_gpu_rms import EPS, h_of, host, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,n", [(1, 200, 64), (37, 1000, 272), (300, 1024, 400), (600, 131, 256)])
def test_norm_feeds_the_fp8_product(rows, cols, n):
    X, R, W = inputs(rows, cols, "bf16", "bf16", "bf16", rows)
    kp = mx.padded(cols)
    qb, sb = fp8_blockscaled(n, kp, 5, 6, k_major=False)
    B, SB = dev_u8(qb), dev_u8(sb)
    H = torch.empty_like(R)
    A = torch.empty((rows, kp), dtype=torch.uint8, device="cuda:0")
    SA = torch.empty((kp // 128, rows), dtype=torch.uint8, device="cuda:0")
    C, D = Guarded(rows * n, "bf16"), Guarded(rows * n, "bf16")
    args = lambda s: pg.make_args(tile=(128, 128, 128), a_scale=s, b_scale=SB)  # noqa: E731
    note(f"norm {rows}x{cols} to e4m3, product with {n} columns")
    pg.prms_run(config(), X, W, A, rows, cols, eps=EPS, R=R, H=H, out="fp8_b128", y_scale=SA)
    pg.pgemm_run(config(), A, B, C.view, rows, n, kp, "fp8_b128_out_bf16", "grouped", args(SA))
    sync()
    qa, sa = mx.quant_e4m3(mx.rms(host(h_of(X, R)), host(W), EPS)[0])
    pg.pgemm_run(config(), dev_u8(qa), B, D.view, rows, n, kp, "fp8_b128_out_bf16", "grouped", args(dev_u8(sa)))
    sync()
    assert C.guards_intact()
    assert np.array_equal(C.body_bits(), D.body_bits())
    assert_abs_bound(C.as_f64().reshape(rows, n), *og.gemm_fp8_b128(qa, sa, qb, sb), FP8_TOL, (rows, cols, n))
