"""Refused calls of the experts' entry points: a status, nothing written."""
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from tests.gpu_util import config, sync
from tile_scheduling_persistent_amd import _abi

pytestmark = pytest.mark.gpu

INVALID, UNSUPPORTED = _abi.ERR_INVALID, _abi.ERR_UNSUPPORTED


def u8(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda:0")


def i32(n):
    return torch.zeros(n, dtype=torch.int32, device="cuda:0")


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device="cuda:0")


def refused(code, f, *a, **k):
    with pytest.raises(pg.PgemmError) as e:
        f(config(), *a, **k)
    assert e.value.code == code


def test_sort():
    refused(UNSUPPORTED, pg.pmoe_sort_run, i32(8), i32(8), i32(8), i32(1026), 4, 2, 1025)
    refused(INVALID, pg.pmoe_sort_run, i32(8), i32(8), i32(8), i32(4), 4, 2, 0)
    refused(INVALID, pg.pmoe_sort_run, i32(8), i32(8), i32(8), i32(4), 4, 0, 3)
    a = i32(8)
    refused(INVALID, pg.pmoe_sort_run, a, a, i32(8), i32(4), 4, 2, 3)          # place on ids
    refused(INVALID, pg.pmoe_sort_run, i32(8), a, a, i32(4), 4, 2, 3)          # place on order
    whole = i32(12)
    refused(INVALID, pg.pmoe_sort_run, whole.data_ptr() + 2 ** 40, a, i32(8), i32(4), 4, 2, 3)
    with pytest.raises(ValueError):
        pg.pmoe_sort_run(config(), i32(8), i32(8), i32(8), i32(3), 4, 2, 3)     # offsets too short


def test_gather_and_combine():
    x, y, o = bf(4, 128), bf(8, 128), i32(8)
    refused(UNSUPPORTED, pg.pmoe_gather_run, x, o, u8(8 * 128 + 4)[4:], 4, 2, 128, out="fp8_b128", y_scale=u8(8))
    with pytest.raises(ValueError, match="scales"):
        pg.pmoe_gather_run(config(), x, o, u8(8 * 128), 4, 2, 128, out="fp8_b128")
    refused(UNSUPPORTED, lambda c, *a: pg._check("x", _abi.lib().pmoe_gather_run(c.handle, *a)), x.data_ptr(), 1, 128,
            o.data_ptr(), 4, 2, 128, _abi.PRMS_OUT_MXFP4, y.data_ptr(), 128, None, None)
    refused(INVALID, pg.pmoe_gather_run, y[:4], o, y, 4, 2, 128)                 # Y on X
    refused(INVALID, pg.pmoe_combine_run, y, o, y[:4], 4, 2, 128)                # Y on X
    refused(UNSUPPORTED, pg.pmoe_combine_run, y, o, torch.zeros((4, 128), dtype=torch.float16, device="cuda:0"), 4, 2, 128)
    r = bf(5, 128)
    refused(INVALID, pg.pmoe_combine_run, y, o, r[1:], 4, 2, 128, R=r[:4])       # Y partly on R
    with pytest.raises(ValueError):
        pg.pmoe_combine_run(config(), y, o, x, 4, 2, 128, weights=torch.zeros(7, device="cuda:0"))
    refused(INVALID, pg.pmoe_combine_grad_run, x, y, o, i32(8), y, 4, 2, 128, dW=torch.zeros(8, device="cuda:0"))  # dX on X
    with pytest.raises(ValueError):
        pg.pmoe_combine_grad_run(config(), x, None, o, o, y, 4, 2, 128, dW=torch.zeros(8, device="cuda:0"))


def test_quant():
    refused(UNSUPPORTED, pg.pfp8_quant_run, bf(3, 100), u8(3 * 128 + 4)[4:], u8(3), 3, 100)
    q = u8(3 * 128)
    refused(INVALID, pg.pfp8_quant_run, bf(3, 100), q, q[:3], 3, 100)            # scales on codes
    with pytest.raises(ValueError):
        pg.pfp8_quant_run(config(), bf(3, 100), u8(3 * 128 - 1), u8(3), 3, 100)
    refused(INVALID, pg.pfp8_quant_weights_run, bf(2, 100, 100), u8(2 * 100 * 128), u8(2), 2, 100, 100, Qt=u8(2 * 100 * 128))
    refused(INVALID, pg.pfp8_quant_weights_run, bf(2, 100, 100), u8(2 * 100 * 128), u8(2), 0, 100, 100)


def test_products():
    A, B, C, sa, sb, off = u8(10 * 256), u8(2 * 20 * 256), bf(10, 20), u8(20), u8(4), i32(3)
    ok = (A, B, C, 10, 20, 256, sa, sb)
    refused(INVALID, pg.pgemm_run_experts, A, B, C, 10, 20, 200, sa, sb, experts=2, offsets=off)   # K
    refused(INVALID, pg.pgemm_run_experts, *ok, experts=2)                                          # no offsets
    refused(UNSUPPORTED, pg.pgemm_run_experts, A, B, torch.zeros((10, 20), dtype=torch.float16, device="cuda:0"), *ok[3:],
            experts=2, offsets=off)
    refused(UNSUPPORTED, pg.pgemm_run_experts, u8(10 * 256 + 8)[8:], *ok[1:], experts=2, offsets=off)
    refused(INVALID, pg.pgemm_run_experts, B.data_ptr(), B, B[:400].view(torch.bfloat16).view(10, 20), *ok[3:], experts=2,
            offsets=off)                                                                            # C on B
    with pytest.raises(ValueError):
        pg.pgemm_run_experts(config(), *ok, experts=3, offsets=off)
    D, dB = bf(10, 20), torch.zeros((2, 20, 256), device="cuda:0")
    w = (D, A, dB, 10, 20, 256, sa)
    refused(INVALID, pg.pgemm_run_experts_wgrad, *w, experts=2)
    refused(UNSUPPORTED, pg.pgemm_run_experts_wgrad, torch.zeros((10, 20), device="cuda:0"), *w[1:], experts=2, offsets=off)
    refused(UNSUPPORTED, pg.pgemm_run_experts_wgrad, u8(10 * 128 + 8)[8:], *w[1:], d_scale=u8(10), experts=2, offsets=off)
    big = torch.zeros(2 * 20 * 256 + 8, device="cuda:0")
    refused(INVALID, pg.pgemm_run_experts_wgrad, D, A, big[8:].view(2, 20, 256), 10, 20, 256, sa, experts=2, offsets=off,
            base=big[:-8].view(2, 20, 256))
    with pytest.raises(ValueError):
        pg.pgemm_run_experts_wgrad(config(), *w, experts=2, offsets=off, base=bf(2, 20, 256))


def test_glu():
    X, Y = bf(6, 200), bf(6, 100)
    refused(INVALID, pg.pglu_run, X, Y, 6, 100, kept=u8(6 * 256))
    refused(UNSUPPORTED, pg.pglu_run, X, Y, 6, 100, kept=u8(6 * 256 + 4)[4:], kept_scale=u8(12))
    refused(INVALID, pg.pglu_run, X, X.view(-1)[:600].view(6, 100), 6, 100)
    refused(UNSUPPORTED, pg.pglu_grad_run, Y, X, u8(6 * 256), 6, 100, out="fp8_b128", dx_scale=u8(12))
    refused(INVALID, pg.pglu_grad_run, Y, X, X, 6, 100)
    with pytest.raises(ValueError):
        pg.pglu_grad_run(config(), Y, X.float(), bf(6, 200), 6, 100)


def test_nothing_was_written_and_empty_calls():
    """Calls without rows are no errors and write nothing but offsets."""
    off = torch.full((4,), 7, dtype=torch.int32, device="cuda:0")
    e = i32(0)
    pg.pmoe_sort_run(config(), e, e, e, off, 0, 2, 3)
    pg.pmoe_gather_run(config(), bf(0, 64), e, bf(0, 64), 0, 2, 64)
    pg.pmoe_combine_run(config(), bf(0, 64), e, bf(0, 64), 0, 2, 64)
    pg.pmoe_combine_grad_run(config(), bf(0, 64), None, e, e, bf(0, 64), 0, 2, 64)
    pg.pfp8_quant_run(config(), bf(0, 64), u8(0), u8(0), 0, 64)
    pg.pgemm_run_experts(config(), u8(0), u8(64 * 128), bf(0, 64), 0, 64, 128, u8(0), u8(1))
    pg.pglu_run(config(), bf(0, 64), bf(0, 32), 0, 32)
    pg.pglu_grad_run(config(), bf(0, 32), bf(0, 64), bf(0, 64), 0, 32)
    sync()
    assert off.tolist() == [0, 0, 0, 0]
