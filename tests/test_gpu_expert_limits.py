"""Sizes past what the experts' product counts are refused before any buffer is
looked at (none of that size exists here)."""
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from tests.gpu_util import config, sync
from tile_scheduling_persistent_amd import _abi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2 ** 31 - 256, 2 ** 31 - 64, 2 ** 31 - 1])
@pytest.mark.parametrize("c_type", [_abi.PMX_BF16, _abi.PMX_F32])
def test_columns_next_to_the_limit(n, c_type):
    p = torch.zeros(4096, dtype=torch.uint8, device="cuda:0")
    code = _abi.lib().pgemm_run_experts(config().handle, p.data_ptr(), p.data_ptr(), p.data_ptr(), p.data_ptr(), p.data_ptr(),
                                        c_type, 1, n, 128, 1, None, None)
    assert code == _abi.ERR_UNSUPPORTED, pg.status_str(code)
    sync()
    assert not p.any()
