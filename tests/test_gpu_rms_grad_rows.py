"""The RMS norm's gradient where a workgroup walks many rows, against the formula
in 64 bits.

Tolerances.  u = 2^-24.  dW: an fp32 product and its factor n = h * rstd are two
roundings; a term then passes through at most `depth` fp32 additions (the rows
that its thread walks, the rows the workgroup takes side by side, the rows of
partial sums that one of 32 threads adds, ten more to join those), so dW is off
by at most (depth + 2) u sum |dy n|.  A row left out, taken twice or scaled by
another row's rstd is 1/rows of that sum, far more.  dX: a row's sum c of g n has
at most 8 * ceil(cols / 8192) + 22 additions per term and three roundings in
each; the mean, its product with n, the difference, the factor rstd and dh's
addition are a rounding each; then half a step of dX's type."""
import functools

import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tests.gpu_util import config, note, sync
from tests.test_gpu_rms import EPS, TYPES, strided

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"), ("bf16", "f32", "f32"),
         ("f16", "f16", "f16"), ("f16", "f16", "f32"), ("f16", "f32", "f16"), ("f16", "f32", "f32"),
         ("f32", "f32", "f32")]
# rows side by side in a workgroup 1, 8, 64, 1 (two vectors per thread), 1 (long rows)
GRAD = [(1100, 4099), (5003, 1000), (40000, 96), (600, 9001), (150, 20000)]


class Banded:
    """A dense tensor with bands of NaN before and after it."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.full = torch.full((n + 512,), float("nan"), dtype=dtype, device="cuda:0")
        self.t = self.full[256:256 + n].view(shape)

    def intact(self):
        return bool(torch.isnan(self.full[:256]).all() and torch.isnan(self.full[-256:]).all())


def lanes(kp, vpt):
    need = -(-(kp // 8) // vpt)
    return 16 if need <= 16 else 32 if need <= 32 else -(-need // 64) * 64


def depth(rows, cols):
    """Additions that a term of dW passes through, at most."""
    kp, cus = mx.padded(cols), config().info["num_cus"]
    if kp > 16384:
        per, programs = 1, min(rows, 64)
    else:
        per = 1024 // lanes(kp, 1) if kp <= 8192 else 1
        programs = min(-(-rows // per), cus)
    return -(-rows // (per * programs)) + per + -(-programs // 32) + 10


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda:0")


@functools.lru_cache(maxsize=1)
def grad_inputs(rows, cols, y, h, w, with_dh):
    """Rows of different size, and a part of dY along H that differs by row, so
    that the mean of a row is large and no other row's will do."""
    g = torch.Generator(device="cuda:0")
    g.manual_seed(rows + cols)
    size = torch.exp(0.5 * normal(g, rows, 1))
    H = (normal(g, rows, cols) * size).to(TYPES[h])
    W = (1 + 0.3 * normal(g, cols)).to(TYPES[w])
    dY = (0.1 * (normal(g, rows, cols) + normal(g, rows, 1) * H.float() / size)).to(TYPES[y])
    dH = (0.1 * normal(g, rows, cols)).to(TYPES[h]) if with_dh else None
    T = torch.rsqrt(H.double().square().mean(1) + EPS).float()
    return dY, H, W, T, dH


def check(dX, dW, dY, H, W, T, dH, what):
    rows, cols = H.shape
    dy, h, w, r = dY.double(), H.double(), W.double(), T.double()[:, None]
    n, g = h * r, dy * w
    c = (g * n).sum(1, keepdim=True)
    want = r * (g - n * c / cols)
    size = r * (4 * g.abs() + n.abs() / cols * ((8 * -(-cols // 8192) + 25) * (g * n).abs().sum(1, keepdim=True) + 8 * c.abs()))
    if dH is not None:
        want = want + dH.double()
        size = size + 2 * dH.double().abs()
    t = torch.finfo(dX.dtype)
    bound = (want.abs() + size * U) * (t.eps / 2) + size * U * (1 + 1e-3) + t.smallest_normal * t.eps
    bad = ~((dX.double() - want).abs() <= bound)
    assert not bad.any(), (what, "dX", int(bad.sum()), bad.nonzero()[:4].tolist())
    if dW is not None:
        terms = dy * n
        bad = ~((dW.double() - terms.sum(0)).abs() <= (depth(rows, cols) + 2) * U * (1 + 1e-3) * terms.abs().sum(0))
        assert not bad.any(), (what, "dW", int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("y,h,w", KINDS)
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("rows,cols", GRAD)
def test_gradient_over_many_rows(rows, cols, with_dh, y, h, w):
    dY, H, W, T, dH = grad_inputs(rows, cols, y, h, w, with_dh)
    dX, dW = Banded((rows, cols), H.dtype), Banded((cols,), torch.float32)
    note(f"prms_grad_run {rows}x{cols} {y} {h} {w} dh={with_dh}")
    pg.prms_grad_run(config(), dY, H, W, T, dX.t, dW.t, rows, cols, dH=dH)
    sync()
    assert dX.intact() and dW.intact()
    check(dX.t, dW.t, dY, H, W, T, dH, (rows, cols))


@pytest.mark.parametrize("rows,cols", GRAD)
def test_gradient_has_the_same_bits_in_place_strided_and_without_dw(rows, cols):
    """The order of every sum depends on the sizes only."""
    dY, H, W, T, dH = grad_inputs(rows, cols, "bf16", "bf16", "bf16", True)
    cfg = config()
    dX, dW = torch.empty_like(H), torch.empty(cols, device="cuda:0")
    note(f"prms_grad_run {rows}x{cols} in place and strided")
    pg.prms_grad_run(cfg, dY, H, W, T, dX, dW, rows, cols, dH=dH)
    alone = torch.empty_like(dX)
    pg.prms_grad_run(cfg, dY, H, W, T, alone, None, rows, cols, dH=dH)
    sync()
    check(dX, dW, dY, H, W, T, dH, (rows, cols))
    assert torch.equal(alone, dX)
    over = [torch.empty_like(dW) for _ in range(3)]
    on_dh, on_dy = dH.clone(), dY.clone()
    pg.prms_grad_run(cfg, dY, H, W, T, on_dh, over[0], rows, cols, dH=on_dh)
    pg.prms_grad_run(cfg, on_dy, H, W, T, on_dy, over[1], rows, cols, dH=dH)
    ys, hs, ds, xs = (strided(t, cols + k, k)[0] for k, t in ((3, dY), (5, H), (8, dH), (1, dX)))
    xs.zero_()
    pg.prms_grad_run(cfg, ys, hs, W, T, xs, over[2], rows, cols, dH=ds)
    sync()
    for got, w in zip((on_dh, on_dy, xs), over):
        assert torch.equal(got, dX) and torch.equal(w, dW)


def test_gradient_of_calls_past_4_gib():
    """Every row of dX and the whole of dW against 64 bits, by chunks of rows.  547
    rows a workgroup; the first and the last round of rows are 64 times as large
    in dY, so that one row of them left out is more than dW's bound."""
    rows, cols = 140000, 16384                      # 4.59 GB of bf16
    g = torch.Generator(device="cuda:0")
    g.manual_seed(8)
    cus = config().info["num_cus"]
    H = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda:0").normal_(generator=g)
    dY = torch.empty_like(H).normal_(generator=g)
    dY[:cus] *= 64
    dY[-cus:] *= 64
    W = (1 + 0.3 * normal(g, cols)).bfloat16()
    T, step = torch.empty(rows, device="cuda:0"), 1 << 14
    for a in range(0, rows, step):
        T[a:a + step] = torch.rsqrt(H[a:a + step].double().square().mean(1) + EPS).float()
    dX, dW = torch.full_like(H, float("nan")), torch.empty(cols, device="cuda:0")
    note(f"prms_grad_run {rows}x{cols}")
    pg.prms_grad_run(config(), dY, H, W, T, dX, dW, rows, cols, dH=H)
    sync()
    total, size = torch.zeros(cols, dtype=torch.float64, device="cuda:0"), 0.0
    for a in range(0, rows, step):
        dy, h, t = dY[a:a + step], H[a:a + step], T[a:a + step]
        check(dX[a:a + step], None, dy, h, W, t, h, a)
        terms = dy.double() * (h.double() * t.double()[:, None])
        total += terms.sum(0)
        size = size + terms.abs().sum(0)
    assert bool(((dW.double() - total).abs() <= (depth(rows, cols) + 2) * U * (1 + 1e-3) * size).all())
