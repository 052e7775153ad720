"""e4m3 rows and weights against the 64-bit oracle, bit for bit: a power of two
divides exactly, and one rounding to e4m3 is left."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import experts as ox
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def values(rng, shape, dtype):
    """Blocks of very different size, zeros, ties, infinities and NaN."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-12, 6, shape[:-1] + (1,)))
    flat = x.reshape(-1)
    flat[rng.random(flat.size) < 0.05] = 0.0
    flat[rng.random(flat.size) < 0.05] = 17.0  # halfway between e4m3 values where the scale is 2^0
    t = torch.from_numpy(x).to(dtype)
    if x.size > 3000:
        t.view(-1)[1500] = float("inf")
        t.view(-1)[2900] = float("nan")
    return t.to("cuda:0")


def buffers(nb, *names):
    return [torch.full((nb[k] + 32,), 0x55, dtype=torch.uint8, device="cuda:0") for k in names]


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 128), (5, 129), (64, 520), (67, 2000), (513, 1100), (2500, 3001)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_rows(rows, cols, x):
    note(f"fp8 rows {rows} {cols} {x}")
    X = values(np.random.default_rng(rows), (rows, cols + 1), TYPES[x])[:, :cols]
    nb = pg.fp8_bytes(rows, cols)
    Q, S = buffers(nb, "Q", "scale")
    pg.pfp8_quant_run(config(), X, Q, S, rows, cols)
    sync()
    q, s = ox.quant_rows(X.double().cpu().numpy())
    assert np.array_equal(Q[:nb["Q"]].cpu().numpy().reshape(q.shape), q)
    assert np.array_equal(S[:nb["scale"]].cpu().numpy().reshape(s.shape), s)
    assert bool((Q[nb["Q"]:] == 0x55).all()) and bool((S[nb["scale"]:] == 0x55).all())


@pytest.mark.parametrize("experts,rows,cols", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (1, 127, 640), (5, 300, 100), (2, 1000, 900)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("both", [True, False])
def test_weights(experts, rows, cols, x, both):
    note(f"fp8 weights {experts} {rows} {cols} {x} {both}")
    W = values(np.random.default_rng(rows), (experts, rows, cols), TYPES[x])
    nb = pg.fp8_weight_bytes(experts, rows, cols)
    out = buffers(nb, "Q", "scale", "Qt", "scale_t")
    pg.pfp8_quant_weights_run(config(), W, *out[:2], experts, rows, cols, **(dict(Qt=out[2], scale_t=out[3]) if both else {}))
    sync()
    w = W.double().cpu().numpy()
    a, b = [ox.quant_weights(v) for v in w], [ox.quant_weights(v.T) for v in w]
    want = [np.stack(t) for t in (*zip(*a), *zip(*b))]
    for i, (t, k) in enumerate(zip(out, ("Q", "scale", "Qt", "scale_t"))):
        if both or i < 2:
            assert np.array_equal(t[:nb[k]].cpu().numpy().reshape(want[i].shape), want[i]), k
        assert bool((t[nb[k] if both or i < 2 else 0:] == 0x55).all()), k


def test_smallest_and_largest_magnitudes():
    """Scales at both ends of e8m0, and magnitudes around the largest code."""
    X = torch.zeros((6, 256), device="cuda:0")
    X[0, :3] = torch.tensor([1.0, 448.0, 448.0000305])
    X[1, 0] = 3.4028234663852886e38
    X[2, :2] = torch.tensor([2.0 ** -149, 2.0 ** -140])
    X[3, :2] = torch.tensor([2.0 ** -126, -2.0 ** -126])
    X[4, 5] = -float("inf")
    X[5, 128] = -0.0
    nb = pg.fp8_bytes(6, 256)
    Q, S = buffers(nb, "Q", "scale")
    pg.pfp8_quant_run(config(), X, Q, S, 6, 256)
    sync()
    q, s = ox.quant_rows(X.double().cpu().numpy())
    assert np.array_equal(S[:nb["scale"]].cpu().numpy().reshape(s.shape), s)
    assert np.array_equal(Q[:nb["Q"]].cpu().numpy().reshape(q.shape), q)
