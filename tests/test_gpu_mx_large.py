"""MXFP4 and RMS norm calls whose buffers pass 4 GiB: rows at the start, around
the 2 GiB and 4 GiB marks and at the end against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

ROWS, COLS = 140000, 16384                      # 4.59 GB of bf16
PICK = [0, 1, 65535, 65536, 65537, 131071, 131072, 139998, 139999]


@pytest.fixture(scope="module")
def big():
    g = torch.Generator(device="cuda:0")
    g.manual_seed(5)
    x = torch.empty((ROWS, COLS), dtype=torch.bfloat16, device="cuda:0")
    x.normal_(generator=g)
    yield x


def host(t):
    return t.double().cpu().numpy()


def test_quantise_and_back(big):
    nb = pg.mxfp4_bytes(ROWS, COLS)
    Q = torch.empty(nb["Q"], dtype=torch.uint8, device="cuda:0")
    S = torch.empty(nb["scale"], dtype=torch.uint8, device="cuda:0")
    Y = torch.empty((ROWS, COLS), dtype=torch.bfloat16, device="cuda:0")
    note("quantise and dequantise 140000x16384")
    pg.pmx_quant_run(config(), big, Q, S, ROWS, COLS)
    pg.pmx_dequant_run(config(), Q, S, Y, ROWS, COLS)
    sync()
    q, s = mx.quant_mxfp4(host(big[PICK]))
    assert np.array_equal(Q.view(ROWS, -1)[PICK].cpu().numpy(), q)
    assert np.array_equal(S.view(COLS // 128, ROWS, 4)[:, PICK].cpu().numpy(), s)
    assert np.array_equal(host(Y[PICK]), mx.dequant_mxfp4(q, s, COLS))


def test_quantise_transposed(big):
    nb = pg.mxfp4_bytes(COLS, ROWS)
    Q = torch.empty(nb["Q"], dtype=torch.uint8, device="cuda:0")
    S = torch.empty(nb["scale"], dtype=torch.uint8, device="cuda:0")
    note("quantise 140000x16384 transposed")
    pg.pmx_quant_run(config(), big, Q, S, ROWS, COLS, transpose=True)
    sync()
    pick = [0, 9999, COLS - 1]
    q, s = mx.quant_mxfp4(host(big[:, pick]), transpose=True)
    assert np.array_equal(Q.view(COLS, -1)[pick].cpu().numpy(), q)
    assert np.array_equal(S.view(-1, COLS, 4)[:, pick].cpu().numpy(), s)


def test_norm_and_gradient(big):
    W = torch.ones(COLS, dtype=torch.bfloat16, device="cuda:0")
    H, Y = torch.empty_like(big), torch.empty_like(big)
    T = torch.empty(ROWS, device="cuda:0")
    note("norm 140000x16384")
    pg.prms_run(config(), big, W, Y, ROWS, COLS, R=big, H=H, rstd=T)
    sync()
    h = host(big[PICK]) * 2
    y, rstd = mx.rms(h, np.ones(COLS), 1e-6)
    assert np.array_equal(host(H[PICK]), h)                     # doubling is exact in bf16
    assert np.all(np.abs(host(Y[PICK]) - y) <= np.abs(y) * (2.0 ** -8 + 1e-6) + 2.0 ** -133)
    note("gradient 140000x16384")
    dW = torch.empty(COLS, device="cuda:0")
    pg.prms_grad_run(config(), big, H, W, T, Y, dW, ROWS, COLS)  # dy = h / 2: g and n are parallel
    sync()
    dx, _, _, _ = mx.rms_grad(host(big[PICK]), h, np.ones(COLS), T[PICK].double().cpu().numpy())
    # rstd * (dy - n * mean): both near 1/4 of n, so the difference is of the
    # rounding's size: COLS + 10 fp32 roundings of their magnitudes and a bf16 one
    size = np.abs(h * rstd[:, None]) * rstd[:, None]
    assert np.all(np.abs(host(Y[PICK]) - dx) <= np.abs(dx) * 2.0 ** -8 + (COLS + 10) * 2.0 ** -24 * size + 2.0 ** -133)
    # dw = sum over the rows of h^2 rstd / 2; rows differ in rstd by 1 / sqrt(2 COLS)
    # = 0.55% (one deviation), so its mean over the rows is within 5% for any of them
    want = (H.float().square().sum(0, dtype=torch.float64) * 0.5 * T.double().mean()).cpu().numpy()
    assert np.all(np.abs(dW.double().cpu().numpy() / want - 1) < 0.05)


def test_product_past_4_gib():
    M, N, K = 20000, 60000, 128                  # 4.8 GB of fp32
    rng = np.random.default_rng(1)
    a, b = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    qa, sa = mx.quant_mxfp4(a)
    qb, sb = mx.quant_mxfp4(b)
    up = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to("cuda:0")  # noqa: E731
    C = torch.zeros((M, N), device="cuda:0")
    note("mxfp4 20000x60000x128")
    A, B, SA, SB = up(qa), up(qb), up(sa), up(sb)
    pg.pgemm_run(config(), A, B, C, M, N, K, "mxfp4_out_f32", "grouped", pg.make_args(a_scale=SA, b_scale=SB))
    sync()
    pick = [0, 8947, 8948, 17895, 17896, M - 1]
    ref, terms = mx.gemm_mxfp4(qa[pick], sa[:, pick], qb, sb)
    assert np.all(np.abs(host(C[pick]) - ref) <= 2.0 ** -22 * terms)
