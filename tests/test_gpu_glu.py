"""The gated activation and its gradient against the 64-bit oracle.

Tolerances (u = 2^-24).  s = 1 / (1 + exp(-g)): exp and the reciprocal within 1 ulp
(2 u each), the sum u: 5 u, y two products more: 8 u of |y|.  du the same.  dg =
dy u_ (s + gs (1 - s)): s and gs within 6 u, 1 - s off by 5 u at most, the products
and the sum 5 u more: 16 u of |dy u_| (s + |gs|).  Then the result's own rounding."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import experts as ox
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def host(t):
    return t.double().cpu().numpy()


def near(got, want, bound, dtype):
    half = torch.finfo(dtype).eps / 2
    least = {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -134)
    assert np.all(np.abs(host(got) - want) <= bound + (np.abs(want) + bound) * half + least)


def near_e4m3(q, s, want, bound):
    """Codes and scales of values off by at most `bound`: a scale that the block's
    largest magnitude allows within the bound, and codes within half a step."""
    rows, cols = want.shape
    kp = -(-cols // 128) * 128
    w, b = np.zeros((rows, kp)), np.zeros((rows, kp))
    w[:, :cols], b[:, :cols] = want, bound
    w, b = w.reshape(rows, -1, 128), b.reshape(rows, -1, 128)
    lo, hi = np.maximum(np.abs(w) - b, 0).max(-1), (np.abs(w) + b).max(-1)
    s = s.reshape(kp // 128, rows).T.astype(np.int64)
    least = ox.scale_exponent(lo, 448.0, 8, "ceil") + 127
    most = ox.scale_exponent(hi, 448.0, 8, "ceil") + 127
    assert np.all((least <= s) & (s <= most))
    v = ox.dequant_rows(q.reshape(rows, kp), np.ascontiguousarray(s.T.astype(np.uint8))).reshape(w.shape)
    scale = np.exp2(s - 127.0)[..., None]
    step = np.maximum((np.abs(w) + b) * 2.0 ** -4, scale * 2.0 ** -10)
    assert np.all(np.abs(v - w) <= b + step)


def u8(n):
    return torch.full((n,), 0x55, dtype=torch.uint8, device="cuda:0")


SHAPES = [(1, 1), (1, 128), (3, 130), (40, 512), (67, 1000), (300, 2056), (2100, 1025), (3001, 1600)]


def inputs(rows, cols, x, seed):
    rng = np.random.default_rng(seed)
    v = 3 * rng.standard_normal((rows, 2 * cols + 3))
    v[0, 0] = -60.0  # far into the tail
    return torch.from_numpy(v).to("cuda:0", TYPES[x])[:, :2 * cols]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["same", "fp8_b128"])
@pytest.mark.parametrize("kept", [True, False])
def test_glu(rows, cols, x, out, kept):
    note(f"glu {rows} {cols} {x} {out} {kept}")
    X = inputs(rows, cols, x, rows)
    want = ox.glu(host(X))
    bound = 8 * U * np.abs(want) + 2.0 ** -126
    kp = -(-cols // 128) * 128
    kw = dict(kept=u8(rows * 2 * kp), kept_scale=u8(2 * kp // 128 * rows)) if kept else {}
    if out == "same":
        Y = torch.empty((rows, cols + 1), dtype=TYPES[x], device="cuda:0")[:, :cols]
        pg.pglu_run(config(), X, Y, rows, cols, **kw)
        sync()
        near(Y, want, bound, TYPES[x])
    else:
        Q, S = u8(rows * kp), u8(kp // 128 * rows)
        pg.pglu_run(config(), X, Q, rows, cols, out=out, y_scale=S, **kw)
        sync()
        near_e4m3(Q.cpu().numpy(), S.cpu().numpy(), want, bound)
    if kept:
        (qg, sg), (qu, su) = (ox.quant_rows(v) for v in np.split(host(X), 2, axis=1))
        assert np.array_equal(kw["kept"].cpu().numpy().reshape(rows, 2 * kp), np.concatenate([qg, qu], 1))
        assert np.array_equal(kw["kept_scale"].cpu().numpy().reshape(-1, rows), np.concatenate([sg, su]))


GRAD = [(s, out) for s in SHAPES + [(33, 640), (1500, 1024), (4100, 768)] for out in ("same", "fp8_b128")
        if out == "same" or s[1] % 128 == 0]


@pytest.mark.parametrize("shape,out", GRAD)
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kept", [True, False])
def test_glu_grad(shape, x, out, kept):
    rows, cols = shape
    note(f"glu_grad {rows} {cols} {x} {out} {kept}")
    X = inputs(rows, cols, x, rows)
    dY = torch.from_numpy(np.random.default_rng(7).standard_normal((rows, cols + 1))).to("cuda:0", TYPES[x])[:, :cols]
    kp = -(-cols // 128) * 128
    used = host(X)
    kw, src = {}, X
    if kept:
        parts = [ox.quant_rows(v) for v in np.split(used, 2, axis=1)]
        used = np.concatenate([ox.dequant_rows(*p)[:, :cols] for p in parts], 1)
        src = torch.from_numpy(np.concatenate([p[0] for p in parts], 1)).to("cuda:0")
        kw["x_scale"] = torch.from_numpy(np.concatenate([p[1] for p in parts])).to("cuda:0")
    want, terms = ox.glu_grad(host(dY), used)
    bound = 16 * U * terms + 2.0 ** -126
    if out == "same":
        dX = torch.empty((rows, 2 * cols + 1), dtype=TYPES[x], device="cuda:0")[:, :2 * cols]
        pg.pglu_grad_run(config(), dY, src, dX, rows, cols, **kw)
        sync()
        near(dX, want, bound, TYPES[x])
    else:
        Q, S = u8(rows * 2 * cols), u8(2 * cols // 128 * rows)
        pg.pglu_grad_run(config(), dY, src, Q, rows, cols, out=out, dx_scale=S, **kw)
        sync()
        near_e4m3(Q.cpu().numpy(), S.cpu().numpy(), want, bound)
    assert kp >= cols


@pytest.mark.parametrize("valid", [-3, 0, 1, 37, 90, 91, 2 ** 31 - 1])
def test_rows_behind_the_valid_ones_are_left(valid):
    note(f"glu valid {valid}")
    rows, cols = 90, 256
    X = inputs(rows, cols, "bf16", 3)
    n = min(max(valid, 0), rows)
    X[n:] = float("nan")
    v = torch.tensor([valid], dtype=torch.int32, device="cuda:0")
    Y = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda:0")
    K, KS, Q, S = u8(rows * 2 * cols), u8(4 * rows), u8(rows * 2 * cols), u8(4 * rows)
    dY = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda:0")
    pg.pglu_run(config(), X, Y, rows, cols, kept=K, kept_scale=KS, valid=v)
    pg.pglu_grad_run(config(), dY, K, Q, rows, cols, x_scale=KS, out="fp8_b128", dx_scale=S, valid=v)
    sync()
    assert bool((Y[n:] == 7.0).all()) and bool(torch.isfinite(Y[:n].float()).all())
    for t in (K, Q):
        assert bool((t.view(rows, -1)[n:] == 0x55).all())
    for t in (KS, S):
        assert bool((t.view(4, rows)[:, n:] == 0x55).all()) and bool((t.view(4, rows)[:, :n] != 0x55).all())


@pytest.mark.parametrize("kept", [True, False])
def test_gates_whose_exponential_is_past_fp32(kept):
    """silu(g) is a normal number down to g = -91 or so, where exp(-g) is infinite."""
    rows, cols = 3, 128
    X = torch.ones((rows, 2 * cols), device="cuda:0")
    X[:, :cols] = -torch.linspace(80, 104, rows * cols, device="cuda:0").reshape(rows, cols)
    Y, dY, dX = torch.empty((rows, cols), device="cuda:0"), torch.ones((rows, cols), device="cuda:0"), torch.empty_like(X)
    K, KS = u8(rows * 2 * cols), u8(2 * rows)
    pg.pglu_run(config(), X, Y, rows, cols, kept=K, kept_scale=KS)
    src, kw, used = (K, dict(x_scale=KS), host(X)) if kept else (X, {}, host(X))
    if kept:
        used = ox.dequant_rows(K.cpu().numpy().reshape(rows, -1), KS.cpu().numpy().reshape(2, rows))
    pg.pglu_grad_run(config(), dY, src, dX, rows, cols, **kw)
    sync()
    want = ox.glu(host(X))
    near(Y, want, 8 * U * np.abs(want) + 2.0 ** -126, torch.float32)
    want, terms = ox.glu_grad(host(dY), used)
    near(dX, want, 16 * U * terms + 2.0 ** -126, torch.float32)


def test_infinities_and_nan_stay_in_their_block():
    rows, cols = 4, 384
    X = inputs(rows, cols, "f32", 4)
    X[1, 130], X[2, cols + 5] = float("inf"), float("nan")
    Q, S, K, KS = u8(rows * cols), u8(3 * rows), u8(rows * 2 * cols), u8(6 * rows)
    pg.pglu_run(config(), X, Q, rows, cols, out="fp8_b128", y_scale=S, kept=K, kept_scale=KS)
    sync()
    bad = S.view(3, rows).cpu() == 255
    assert bad.nonzero().tolist() == [[0, 2], [1, 1]]
    bad = KS.view(6, rows).cpu() == 255
    assert bad.nonzero().tolist() == [[1, 1], [3, 2]]


def test_many_rows_equal_few():
    """Inputs past the size that is loaded through the caches: the bits of calls on
    1000 rows each."""
    rows, cols = 8200, 8192
    note("glu past the caches")
    g = torch.Generator(device="cuda:0").manual_seed(1)
    X = torch.randn((rows, 2 * cols), generator=g, device="cuda:0").bfloat16()
    dY = torch.randn((rows, cols), generator=g, device="cuda:0").bfloat16()

    def run(x, dy):
        n = len(x)
        out = [u8(n * cols), u8(cols // 128 * n), u8(n * 2 * cols), u8(2 * cols // 128 * n), u8(n * 2 * cols),
               u8(2 * cols // 128 * n), torch.empty((n, 2 * cols), dtype=torch.bfloat16, device="cuda:0")]
        pg.pglu_run(config(), x, out[0], n, cols, out="fp8_b128", y_scale=out[1], kept=out[2], kept_scale=out[3])
        pg.pglu_grad_run(config(), dy, out[2], out[4], n, cols, x_scale=out[3], out="fp8_b128", dx_scale=out[5])
        pg.pglu_grad_run(config(), dy, x, out[6], n, cols)
        return [t.view(n, -1) if i % 2 == 0 else t.view(-1, n).t() for i, t in enumerate(out)]
    many = run(X, dY)
    sync()
    for lo in range(0, rows, 1000):
        few = run(X[lo:lo + 1000], dY[lo:lo + 1000])
        sync()
        for a, b in zip(many, few):
            assert torch.equal(a[lo:lo + 1000], b)
