"""MXFP4 quantisation and dequantisation where the tiles fill the device (eight
rows a wave, the wide side non-temporal), on sizes that end inside tiles both
ways and on rows that start anywhere; all codes, scales and values against the
64-bit oracle, for equality."""
import functools

import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tests.gpu_util import config, dev_u8, note, sync
from tests.test_gpu_mx import TYPES, make, quant

pytestmark = pytest.mark.gpu

ROWS, COLS = 3001, 3003   # 94 x 6 tiles of 32 rows by 512 columns, both with a rest


@functools.lru_cache(maxsize=1)
def data(kind):
    v, x = make(ROWS, COLS, kind, 21, special=True)
    return x, {rule: mx.quant_mxfp4(v, rule) for rule in ("ceil", "floor")}


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_quant_of_many_rows(kind):
    x, want = data(kind)
    for rule, (qr, sr) in want.items():
        q, s = quant(x, ROWS, COLS, False, rule)
        assert np.array_equal(s, sr) and np.array_equal(q, qr), rule
    for ld, off in ((COLS, 1), (COLS + 4, 3)):
        big = torch.full((off + ROWS * ld,), float("nan"), dtype=TYPES[kind], device="cuda:0")
        view = big.as_strided((ROWS, COLS), (ld, 1), off)
        view.copy_(x)
        q, s = quant(view, ROWS, COLS, False, "ceil")
        assert np.array_equal(s, want["ceil"][1]) and np.array_equal(q, want["ceil"][0]), (ld, off)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_quant_of_many_rows_that_start_on_lines(kind):
    cols, ld = COLS - 3, 3008
    x, _ = data(kind)
    big = torch.full((ROWS, ld), float("nan"), dtype=TYPES[kind], device="cuda:0")
    big[:, :cols] = x[:, :cols]
    assert big.data_ptr() % 128 == 0
    v = x[:, :cols].double().cpu().numpy()
    for rule in ("ceil", "floor"):
        q, s = quant(big[:, :cols], ROWS, cols, False, rule)
        qr, sr = mx.quant_mxfp4(v, rule)
        assert np.array_equal(s, sr) and np.array_equal(q, qr), rule


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_dequant_of_many_rows(kind):
    _, want = data(kind)
    q, s = want["ceil"]
    Q, S = dev_u8(q), dev_u8(s)
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(mx.dequant_mxfp4(q, s, COLS)).to(TYPES[kind]).to("cuda:0")
    for ld, off in ((COLS, 0), (COLS + 4, 3)):
        big = torch.full((off + ROWS * ld + 64,), -7.0, dtype=TYPES[kind], device="cuda:0")
        y = big.as_strided((ROWS, COLS), (ld, 1), off)
        note(f"pmx_dequant_run {ROWS}x{COLS} ld={ld} off={off} {kind}")
        pg.pmx_dequant_run(config(), Q, S, y, ROWS, COLS)
        sync()
        nan = torch.isnan(ref)
        assert torch.equal(torch.isnan(y), nan)
        bits = torch.int32 if kind == "f32" else torch.int16
        assert torch.equal(y.contiguous().view(bits)[~nan], ref.view(bits)[~nan])
        gaps = torch.ones(big.numel(), dtype=torch.bool, device="cuda:0")
        gaps.as_strided((ROWS, COLS), (ld, 1), off).fill_(False)
        assert torch.all(big[gaps] == -7.0)
