"""The RMS norm with residual and quantised outputs, and its gradient, on the
GPU against the 64-bit oracle.

Tolerances.  The norm is computed in 64 bits and rounded once, so h, the
quantised codes and the scale bytes are compared for equality (a value would
have to lie within 1e-13 of a rounding border to differ), and y and rstd to
half a step of their type, plus 1e-9 relative for the 64-bit sums.  The
gradient sums in fp32 (u = 2^-24): a sum of n terms in any order is off by at
most n * u * sum |terms|, and the few operations around it by u each."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tile_scheduling_persistent_amd import _abi
from tests.gpu_util import config, note, sync
from tests.test_gpu_mx import Bytes

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
U = 2.0 ** -24


def tensor(v, kind):
    return torch.from_numpy(np.asarray(v, np.float32)).to(TYPES[kind]).to("cuda:0")


def host(t):
    return t.double().cpu().numpy()


def inputs(rows, cols, x, r, w, seed):
    rng = np.random.default_rng(seed)
    X = tensor(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))), x)
    R = tensor(rng.standard_normal((rows, cols)) * 3, r) if r else None
    W = tensor(1 + 0.3 * rng.standard_normal(cols), w)
    return X, R, W


def h_of(X, R):
    return X if R is None else (X.float() + R.float()).to(R.dtype)


def half_step(y, kind):
    return np.abs(y) * (torch.finfo(TYPES[kind]).eps / 2) * (1 + 1e-6) + torch.finfo(TYPES[kind]).smallest_normal * \
        torch.finfo(TYPES[kind]).eps


SHAPES = [(1, 1), (1, 128), (3, 31), (2, 130), (5, 255), (9, 1024), (17, 1000), (4, 4099), (33, 2048), (1, 8192),
          (3, 8200), (2, 20000), (1, 70001)]


@pytest.mark.parametrize("x,r,w", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f16", "f16", "f32"),
                                   ("f32", "f32", "f32"), ("bf16", None, "bf16"), ("f16", None, "f16"),
                                   ("f32", None, "f32")])
@pytest.mark.parametrize("out", ["same", "fp8_b128", "mxfp4"])
def test_norm_equals_the_oracle(x, r, w, out):
    for i, (rows, cols) in enumerate(SHAPES):
        X, R, W = inputs(rows, cols, x, r, w, 100 + i)
        h = h_of(X, R)
        y, rstd = mx.rms(host(h), host(W), EPS)
        H = torch.full_like(R, -9.0) if r else None
        T = torch.zeros(rows, device="cuda:0")
        kp = mx.padded(cols)
        note(f"prms_run {rows}x{cols} {x} {r} {w} {out}")
        if out == "same":
            Y = torch.full_like(X, -9.0)
            pg.prms_run(config(), X, W, Y, rows, cols, eps=EPS, R=R, H=H, rstd=T)
            sync()
            assert np.all(np.abs(host(Y) - y) <= half_step(y, x) + 1e-9 * np.abs(y)), (rows, cols)
        else:
            n = 2 if out == "mxfp4" else 1
            Y, S = Bytes(rows * kp // n), Bytes(kp // 128 * rows * (4 if n == 2 else 1))
            pg.prms_run(config(), X, W, Y.view, rows, cols, eps=EPS, R=R, H=H, rstd=T, out=out, y_scale=S.view)
            sync()
            qr, sr = mx.quant_mxfp4(y) if n == 2 else mx.quant_e4m3(y)
            assert np.array_equal(S.get().reshape(sr.shape), sr), (rows, cols)
            assert np.array_equal(Y.get().reshape(qr.shape), qr), (rows, cols)
        assert np.all(np.abs(host(T) - rstd) <= rstd * (U * (1 + 1e-6) + 1e-9)), (rows, cols)
        if r:
            assert torch.equal(H, h), (rows, cols)


@pytest.mark.parametrize("out", ["same", "fp8_b128", "mxfp4"])
def test_special_rows(out):
    """A row of zeros, of the smallest and largest values, with an infinity,
    with a NaN: other rows are untouched by them."""
    rows, cols = 12, 384
    X, R, W = inputs(rows, cols, "bf16", None, "bf16", 7)
    X[1] = 0.0
    X[2] = 2.0 ** -130
    X[3] = 3e38
    X[4, 200] = float("inf")
    X[5, 10] = float("nan")
    X[6] = -0.0
    X[7, :] = 0.0
    X[7, 300] = 1.0
    h = host(X)
    with np.errstate(all="ignore"):
        y, rstd = mx.rms(h, host(W), EPS)
    T = torch.zeros(rows, device="cuda:0")
    note(f"special rows {out}")
    with np.errstate(all="ignore"):
        if out == "same":
            Y = torch.zeros_like(X)
            pg.prms_run(config(), X, W, Y, rows, cols, eps=EPS, rstd=T)
            sync()
            got = host(Y)
            assert np.array_equal(np.isnan(got), np.isnan(y))
            ok = ~np.isnan(y)
            assert np.all(np.abs(got - y)[ok] <= (half_step(y, "bf16") + 1e-9 * np.abs(y))[ok])
        else:
            n = 2 if out == "mxfp4" else 1
            Y, S = Bytes(rows * 384 // n), Bytes(3 * rows * (4 if n == 2 else 1))
            pg.prms_run(config(), X, W, Y.view, rows, cols, eps=EPS, rstd=T, out=out, y_scale=S.view)
            sync()
            qr, sr = mx.quant_mxfp4(y) if n == 2 else mx.quant_e4m3(y)
            assert np.array_equal(S.get().reshape(sr.shape), sr)
            assert np.array_equal(Y.get().reshape(qr.shape), qr)
    t = host(T)
    assert np.isnan(t[5]) and t[4] == 0.0
    ok = [i for i in range(rows) if i not in (4, 5)]
    assert np.all(np.abs(t - rstd)[ok] <= (rstd * (U * (1 + 1e-6) + 1e-9) + 2.0 ** -149)[ok])


def strided(v, ld, off=0):
    rows, cols = v.shape
    big = torch.full((off + rows * ld,), float("nan"), dtype=v.dtype, device="cuda:0")
    t = big.as_strided((rows, cols), (ld, 1), off)
    t.copy_(v)
    return t, big


@pytest.mark.parametrize("cols,ld,off", [(256, 264, 0), (256, 259, 0), (1000, 1008, 8), (1000, 1003, 5)])
def test_strided_rows_and_in_place(cols, ld, off):
    rows = 21
    X, R, W = inputs(rows, cols, "bf16", "bf16", "bf16", 3)
    h = h_of(X, R)
    y, _ = mx.rms(host(h), host(W), EPS)
    xs, xb = strided(X, ld, off)
    rs, rb = strided(R, ld, off)
    note(f"in place {cols} ld={ld} off={off}")
    pg.prms_run(config(), xs, W, xs, rows, cols, eps=EPS, R=rs, H=rs)      # y over x, h over r
    sync()
    assert torch.equal(rs, h)
    assert np.all(np.abs(host(xs) - y) <= half_step(y, "bf16") + 1e-9 * np.abs(y))
    for big in (xb, rb):                                                   # the gaps stay NaN
        gaps = torch.ones(big.numel(), dtype=torch.bool, device="cuda:0")
        gaps.as_strided((rows, cols), (ld, 1), off).fill_(False)
        assert torch.isnan(big[gaps]).all()
    X2, _ = strided(X, ld, off)
    S, Y = Bytes(mx.padded(cols) // 128 * rows), Bytes(rows * mx.padded(cols))
    pg.prms_run(config(), X2, W, Y.view, rows, cols, eps=EPS, R=R, H=X2, out="fp8_b128", y_scale=S.view)  # h over x
    sync()
    assert torch.equal(X2, h)
    qr, sr = mx.quant_e4m3(y)
    assert np.array_equal(Y.get().reshape(qr.shape), qr) and np.array_equal(S.get().reshape(sr.shape), sr)


# ---- gradient ---------------------------------------------------------------


def check_grad(got_dx, got_dw, dy, h, w, rstd, dh, y_kind, h_kind, what):
    rows, cols = h.shape
    dx, dw, terms, wterms = mx.rms_grad(dy, h, w, rstd, dh)
    r = rstd[:, None]
    c = np.abs((dy * w * h).sum(1, keepdims=True))
    # sum of g * h: cols terms, each product rounded twice; then r^3 c / cols * h
    # (6 roundings), r * g (2), two additions of at most the terms' magnitudes
    hk = np.abs(h) * r ** 3 / cols
    err = hk * ((cols + 2) * U * terms + 6 * U * c) + 3 * U * np.abs(r * dy * w) + \
        2 * U * (np.abs(r * dy * w) + hk * c + (0 if dh is None else np.abs(dh)))
    assert np.all(np.abs(got_dx - dx) <= half_step(dx, h_kind) + err * (1 + 1e-3) + 2.0 ** -149), what
    if got_dw is not None:
        assert np.all(np.abs(got_dw - dw) <= (rows + 3) * U * wterms * (1 + 1e-3) + 2.0 ** -149), what


@pytest.mark.parametrize("y,h,w", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f16", "f16", "f32"),
                                   ("f32", "f32", "f32")])
@pytest.mark.parametrize("with_dh", [False, True])
def test_gradient_equals_the_oracle(y, h, w, with_dh):
    for i, (rows, cols) in enumerate(SHAPES + [(300, 520), (1025, 96)]):
        rng = np.random.default_rng(200 + i)
        H = tensor(rng.standard_normal((rows, cols)) * 2, h)
        W = tensor(1 + 0.3 * rng.standard_normal(cols), w)
        dY = tensor(rng.standard_normal((rows, cols)) * 0.1, y)
        dH = tensor(rng.standard_normal((rows, cols)) * 0.1, h) if with_dh else None
        T = tensor(mx.rms(host(H), host(W), EPS)[1], "f32")
        dX, dW = torch.full_like(H, -9.0), torch.full((cols,), -9.0, device="cuda:0")
        note(f"prms_grad_run {rows}x{cols} {y} {h} {w} dh={with_dh}")
        pg.prms_grad_run(config(), dY, H, W, T, dX, dW, rows, cols, dH=dH)
        sync()
        check_grad(host(dX), host(dW), host(dY), host(H), host(W), host(T), None if dH is None else host(dH), y, h,
                   (rows, cols))


@pytest.mark.parametrize("cols,ld,off", [(256, 264, 0), (1000, 1003, 5)])
def test_gradient_in_place_strided_and_repeatable(cols, ld, off):
    rows = 77
    rng = np.random.default_rng(9)
    H, dY, dH = (tensor(rng.standard_normal((rows, cols)), "bf16") for _ in range(3))
    W = tensor(1 + 0.3 * rng.standard_normal(cols), "bf16")
    T = tensor(mx.rms(host(H), host(W), EPS)[1], "f32")
    dX, dW = torch.empty_like(H), torch.empty(cols, device="cuda:0")
    pg.prms_grad_run(config(), dY, H, W, T, dX, dW, rows, cols, dH=dH)
    sync()
    hs, ds, ys = strided(H, ld, off)[0], strided(dH, ld, off)[0], strided(dY, ld, off)[0]
    dW2, dW3 = torch.empty_like(dW), torch.empty_like(dW)
    pg.prms_grad_run(config(), ys, hs, W, T, ds, dW2, rows, cols, dH=ds)     # dX over dH
    pg.prms_grad_run(config(), ys, hs, W, T, ys, dW3, rows, cols, dH=dH)     # dX over dY
    sync()
    # the same sizes with other strides may add in another order: formula's bounds
    for got, w in ((ds, dW2), (ys, dW3)):
        check_grad(host(got), host(w), host(dY), host(H), host(W), host(T), host(dH), "bf16", "bf16", (cols, ld))
    again, dWa = torch.empty_like(H), torch.empty_like(dW)
    pg.prms_grad_run(config(), dY, H, W, T, again, dWa, rows, cols, dH=dH)
    pg.prms_grad_run(config(), dY, H, W, T, torch.empty_like(H), None, rows, cols, dH=dH)
    sync()
    assert torch.equal(again, dX) and torch.equal(dWa, dW)


@pytest.mark.parametrize("exponent", [-90, -60, 50, 62])
def test_gradient_of_very_small_and_large_rows(exponent):
    """rstd of 2^90 or 2^-62: its third power and sums of h leave the range of
    fp32, the gradient (of order rstd) does not."""
    for rows, cols in [(3, 200), (2, 20000)]:
        rng = np.random.default_rng(exponent + 100)
        H = tensor(rng.standard_normal((rows, cols)) * 2.0 ** exponent, "f32")
        W, dY = tensor(1 + 0.3 * rng.standard_normal(cols), "f32"), tensor(rng.standard_normal((rows, cols)), "f32")
        T = tensor(mx.rms(host(H), host(W), 0.0)[1], "f32")
        dX, dW = torch.empty_like(H), torch.empty(cols, device="cuda:0")
        note(f"prms_grad_run {rows}x{cols} 2^{exponent}")
        pg.prms_grad_run(config(), dY, H, W, T, dX, dW, rows, cols)
        sync()
        check_grad(host(dX), host(dW), host(dY), host(H), host(W), host(T), None, "f32", "f32", (rows, cols))


def test_gradient_against_differences():
    """dX and dW of an fp32 call against central differences of the forward
    (computed in 64 bits from perturbed inputs): step 1e-4 on values of order
    one leaves 1e-7 from the third derivative and 1e-11 from rounding."""
    rows, cols, d = 2, 24, 1e-4
    rng = np.random.default_rng(4)
    h, w = rng.standard_normal((rows, cols)).astype(np.float32), rng.standard_normal(cols).astype(np.float32)
    dy = rng.standard_normal((rows, cols)).astype(np.float32)
    H, W, dY = (torch.from_numpy(v).to("cuda:0") for v in (h, w, dy))
    T, Y = torch.empty(rows, device="cuda:0"), torch.empty_like(H)
    dX, dW = torch.empty_like(H), torch.empty_like(W)
    pg.prms_run(config(), H, W, Y, rows, cols, eps=EPS, rstd=T)
    pg.prms_grad_run(config(), dY, H, W, T, dX, dW, rows, cols)
    sync()
    f = lambda h, w: (mx.rms(h, w, EPS)[0] * dy).sum()  # noqa: E731
    h, w = h.astype(np.float64), w.astype(np.float64)
    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(h)
            e[i, j] = d
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * d) - dX[i, j].item()) < 2e-5
    for j in range(cols):
        e = np.zeros_like(w)
        e[j] = d
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * d) - dW[j].item()) < 2e-5


def test_no_rows():
    e = torch.zeros((0, 64), device="cuda:0")
    W, dW = torch.ones(64, device="cuda:0"), torch.full((64,), 5.0, device="cuda:0")
    pg.prms_run(config(), e, W, e, 0, 64)
    pg.prms_grad_run(config(), e, e, W, torch.zeros(0, device="cuda:0"), e, dW, 0, 64)
    sync()
    assert torch.all(dW == 0)


def test_graph_replays():
    """Forward and gradient captured on a stream of the caller's; replays on
    new data, with eager work between, equal eager calls."""
    rows, cols = 60, 512
    X, R, W = inputs(rows, cols, "bf16", "bf16", "bf16", 1)
    dY = tensor(np.random.default_rng(2).standard_normal((rows, cols)), "bf16")
    H, Y, dX = torch.empty_like(X), torch.empty_like(X), torch.empty_like(X)
    T, dW = torch.empty(rows, device="cuda:0"), torch.empty(cols, device="cuda:0")

    def both(st=None):
        pg.prms_run(config(), X, W, Y, rows, cols, R=R, H=H, rstd=T, stream=st)
        pg.prms_grad_run(config(), dY, H, W, T, dX, dW, rows, cols, dH=dY, stream=st)

    both()
    sync()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        both()
    for seed in range(3):
        X.copy_(inputs(rows, cols, "bf16", "bf16", "bf16", 30 + seed)[0])
        both()
        sync("eager")
        want = [t.clone() for t in (H, Y, T, dX, dW)]
        for t in (H, Y, T, dX, dW):
            t.zero_()
        sync("cleared")
        g.replay()
        sync("replay")
        assert all(torch.equal(a, b) for a, b in zip(want, (H, Y, T, dX, dW)))


def test_refusals():
    L, hd = _abi.lib(), config().handle
    rows, cols = 16, 128
    mk = lambda: torch.full((rows * cols,), 7.0, device="cuda:0")  # noqa: E731
    x, r, h, y, w, t = mk(), mk(), mk(), mk(), torch.ones(cols, device="cuda:0"), torch.zeros(rows, device="cuda:0")
    s = torch.zeros(rows * 4, dtype=torch.uint8, device="cuda:0")
    p = {k: v.data_ptr() for k, v in dict(x=x, r=r, h=h, y=y, w=w, t=t, s=s).items()}

    def fwd(X=p["x"], xt=0, ldx=cols, R=p["r"], rt=0, ldr=cols, W=p["w"], wt=0, eps=1e-6, n=rows, c=cols, H=p["h"],
            ldh=cols, out=0, Y=p["y"], ldy=cols, S=None, T=p["t"]):
        return L.prms_run(hd, X, xt, ldx, R, rt, ldr, W, wt, eps, n, c, H, ldh, out, Y, ldy, S, T, None)

    I, V = _abi.ERR_INVALID, _abi.ERR_UNSUPPORTED  # noqa: E741
    for bad in (dict(X=None), dict(W=None), dict(Y=None), dict(H=None), dict(R=None), dict(xt=5), dict(wt=-1),
                dict(rt=9), dict(n=-1), dict(c=0), dict(ldx=127), dict(ldr=127), dict(ldh=1), dict(ldy=5),
                dict(eps=-1.0), dict(eps=float("nan")), dict(out=3), dict(out=1), dict(n=1 << 24),
                dict(Y=p["r"]), dict(Y=p["h"]), dict(Y=p["x"] + 4), dict(H=p["x"] + 512, ldh=cols, n=8),
                dict(T=p["x"]), dict(out=1, S=p["x"]), dict(out=2, S=p["y"]), dict(T=p["t"] + 2)):
        assert fwd(**bad) == I, bad
    assert fwd(xt=1, rt=2, n=8) == V and fwd(xt=1, rt=1, wt=2, n=8) == V
    assert fwd(out=1, Y=p["y"] + 4, S=p["s"], n=8) == V and fwd(out=2, S=p["s"] + 1, n=8) == V

    def bwd(Y=p["y"], yt=0, ldy=cols, H=p["h"], ht=0, ldh=cols, D=None, ldd=cols, W=p["w"], wt=0, T=p["t"], n=rows,
            c=cols, X=p["x"], ldx=cols, G=p["r"]):
        return L.prms_grad_run(hd, Y, yt, ldy, H, ht, ldh, D, ldd, W, wt, T, n, c, X, ldx, G, None)

    for bad in (dict(Y=None), dict(H=None), dict(W=None), dict(T=None), dict(X=None), dict(yt=4), dict(n=-2),
                dict(c=0), dict(ldy=3), dict(ldh=3), dict(ldx=3), dict(D=p["r"], ldd=3), dict(X=p["h"]),
                dict(G=p["x"]), dict(G=p["h"]), dict(X=p["y"] + 4), dict(n=1 << 24), dict(G=p["r"] + 2)):
        assert bwd(**bad) == I, bad
    assert bwd(yt=1, ht=2, n=8) == V and bwd(yt=1, ht=1, wt=2, n=8) == V
    sync()
    assert all(torch.all(v == 7.0) for v in (x, r, h, y))
