"""An output of the experts' entry points may be the one input that its documentation
names, and no other buffer at that address."""
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from tests.gpu_util import config, sync
from tile_scheduling_persistent_amd import _abi

pytestmark = pytest.mark.gpu


def refused(f, *a, **k):
    with pytest.raises(pg.PgemmError) as e:
        f(config(), *a, **k)
    assert e.value.code == _abi.ERR_INVALID


@pytest.mark.parametrize("topk", [1, 2])
def test_combine_of_rows_in_place(topk):
    """X, R and Y one tensor: rows are read while others are written."""
    tokens, cols = 8, 256
    rows = torch.randn((tokens * topk, cols), device="cuda:0")
    place = torch.arange(tokens * topk, dtype=torch.int32, device="cuda:0").flip(0)
    before, t = rows.clone(), rows[:tokens]
    refused(pg.pmoe_combine_run, rows, place, t, tokens, topk, cols, R=t)
    sync()
    assert torch.equal(rows, before)
    r = before[:tokens].clone()  # R and X at one address are both read only
    y = torch.empty_like(r)
    pg.pmoe_combine_run(config(), rows, place, y, tokens, topk, cols, R=t)
    pg.pmoe_combine_run(config(), rows, place, r, tokens, topk, cols, R=r)
    sync()
    want = before[:tokens] + before[place.long()].view(tokens, topk, cols).sum(1)
    assert torch.allclose(y, want, rtol=1e-6, atol=1e-6) and torch.equal(r, y)


@pytest.mark.parametrize("which", ["D", "A", "e4m3 D"])
def test_weight_gradient_onto_an_operand(which):
    rows, n, k = 128, 128, 128
    dB = torch.zeros((n, k), device="cuda:0")
    D = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda:0")
    A = torch.zeros((rows, k), dtype=torch.uint8, device="cuda:0")
    sa = torch.full((rows,), 127, dtype=torch.uint8, device="cuda:0")
    kw = {}
    if which == "D":
        D = dB.view(torch.bfloat16).view(-1)[:rows * n].view(rows, n)
    elif which == "A":
        A = dB.view(torch.uint8).view(-1)[:rows * k].view(rows, k)
    else:
        D, kw["d_scale"] = dB.view(torch.uint8).view(-1)[:rows * n].view(rows, n), sa
    refused(pg.pgemm_run_experts_wgrad, D, A, dB, rows, n, k, sa, base=dB, **kw)
    refused(pg.pgemm_run_experts_wgrad, D, A, dB, rows, n, k, sa, **kw)
