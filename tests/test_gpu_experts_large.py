"""The experts' row operators on rows of more than 128 MiB in every type and on rows
that start anywhere, and their matrices past the fourth gibibyte.

A call's rows are worked on one by one, so a large call has the bits of calls on a part
of its rows, which the tests of small calls hold against the 64-bit oracle; the weight
gradient is compared with a call for the one expert alone (the same rows in the same
order; equal bits on the same tile)."""
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOKENS, TOPK = 2110, 8
SLOTS = TOKENS * TOPK
PART = 61  # tokens of a part


def i32(*s):
    return torch.empty(s, dtype=torch.int32, device="cuda:0")


def u8(n):
    return torch.full((n,), 0x55, dtype=torch.uint8, device="cuda:0")


def randn(seed, rows, cols, dtype, stride):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return torch.randn((rows, stride), generator=g, device="cuda:0").to(dtype)[:, :cols]


# the row strides of the inputs and of the outputs: whole lines, and odd
COLS = [(4096, 4096, 4096), (4095, 4099, 4097), (8200, 8200, 8208)]


@pytest.fixture(scope="module")
def routed():
    g = torch.Generator(device="cuda:0").manual_seed(3)
    ids = torch.randint(-1, 16, (TOKENS, TOPK), generator=g, device="cuda:0", dtype=torch.int32)
    place, order, offsets = i32(TOKENS, TOPK), i32(SLOTS), i32(17)
    pg.pmoe_sort_run(config(), ids, place, order, offsets, TOKENS, TOPK, 16)
    w = torch.rand((TOKENS, TOPK), generator=g, device="cuda:0")
    sync()
    return place, order, offsets, w


def part_of(place, lo, n):
    """Tokens lo .. lo + n alone: the large call's rows of their slots, one after the
    other, and place and order that point at those."""
    p = place[lo:lo + n].reshape(-1)
    on = p >= 0
    rows = p[on].long()
    small = torch.full_like(p, -1)
    small[on] = torch.arange(len(rows), dtype=torch.int32, device="cuda:0")
    order = torch.full_like(p, -1)
    order[:len(rows)] = on.nonzero().view(-1).int()
    return rows, small.view(n, -1).contiguous(), order


def take(x, rows, total):
    """The rows of x, padded to a part's slots."""
    out = torch.zeros((total, x.shape[1]), dtype=x.dtype, device="cuda:0")
    out[:len(rows)] = x[rows]
    return out


@pytest.mark.parametrize("cols,ldx,ldy", COLS)
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_combine(routed, cols, ldx, ldy, x, y):
    note(f"combine, large, {cols} {ldx} {x} {y}")
    place, _, _, w = routed
    X, R = randn(1, SLOTS, cols, TYPES[x], ldx), randn(2, TOKENS, cols, TYPES[y], ldy)
    out = torch.full((TOKENS, ldy), 7.0, dtype=TYPES[y], device="cuda:0")
    pg.pmoe_combine_run(config(), X, place, out[:, :cols], TOKENS, TOPK, cols, weights=w, R=R)
    sync()
    assert bool((out[:, cols:] == 7.0).all())
    for lo in (0, 777, TOKENS - PART):
        rows, p, _ = part_of(place, lo, PART)
        want = torch.empty((PART, cols), dtype=TYPES[y], device="cuda:0")
        pg.pmoe_combine_run(config(), take(X, rows, PART * TOPK), p, want, PART, TOPK, cols, weights=w[lo:lo + PART].contiguous(),
                            R=R[lo:lo + PART])
        sync()
        assert torch.equal(out[lo:lo + PART, :cols], want), lo


@pytest.mark.parametrize("cols,ldx,ldy", COLS)
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "fp8_b128"])
def test_gather_and_combine_grad(routed, cols, ldx, ldy, x, out):
    note(f"gather and combine's gradient, large, {cols} {ldx} {x} {out}")
    place, order, offsets, w = routed
    n = int(offsets[-1])
    X, dY = randn(4, SLOTS, cols, TYPES[x], ldx), randn(5, TOKENS, cols, TYPES[x], ldx)
    nb = pg.fp8_bytes(SLOTS, cols)

    def outputs(slots, stride):
        if out == "same":
            return torch.full((slots, stride), 7.0, dtype=TYPES[x], device="cuda:0"), None
        b = pg.fp8_bytes(slots, cols)
        return u8(b["Q"]).view(slots, -1), u8(b["scale"]).view(-1, slots)

    def call(dy, xs, p, o, wt, tokens, stride):
        """(gathered rows, their scales, dX, its scales, dW)"""
        (y, ys), (d, ds) = outputs(tokens * TOPK, stride), outputs(tokens * TOPK, stride)
        dw = torch.full((tokens, TOPK), 7.0, device="cuda:0")
        yv, dv = (y[:, :cols], d[:, :cols]) if out == "same" else (y, d)
        pg.pmoe_gather_run(config(), dy, o, yv, tokens, TOPK, cols, out=out, y_scale=ys)
        pg.pmoe_combine_grad_run(config(), dy, xs, p, o, dv, tokens, TOPK, cols, weights=wt, dW=dw, out=out, dx_scale=ds)
        sync()
        return y, ys, d, ds, dw
    got = call(dY, X, place, order, w, TOKENS, ldy)
    assert nb["Q"] >= 16 << 20
    for i in (0, 2):
        untouched = 7.0 if out == "same" else 0x55
        assert bool((got[i][n:] == untouched).all()) and (out != "same" or bool((got[i][:, cols:] == 7.0).all()))
        assert got[i + 1] is None or bool((got[i + 1][:, n:] == 0x55).all())
    for lo in (0, 1201, TOKENS - PART):
        rows, p, o = part_of(place, lo, PART)
        want = call(dY[lo:lo + PART], take(X, rows, PART * TOPK), p, o, w[lo:lo + PART].contiguous(), PART, cols)
        m = len(rows)
        for i in (0, 2):
            width = cols if out == "same" else want[i].shape[1]
            assert torch.equal(got[i][rows][:, :width], want[i][:m]), (lo, i)
            assert want[i + 1] is None or torch.equal(got[i + 1][:, rows], want[i + 1][:, :m]), (lo, i)
        assert torch.equal(got[4][lo:lo + PART], want[4]), lo


@pytest.mark.parametrize("rows,cols,extra", [(9000, 2048, 0), (8900, 2055, 3), (9000, 4104, 8), (33000, 2048, 64)])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "fp8_b128"])
def test_glu(rows, cols, extra, x, out):
    note(f"activation, large, {rows} {cols} {extra} {x} {out}")
    X, dY = randn(6, rows, 2 * cols, TYPES[x], 2 * cols + extra), randn(7, rows, cols, TYPES[x], cols + extra)
    kp = -(-cols // 128) * 128
    back = out if cols % 128 == 0 else "same"

    def call(xs, dy, stride):
        n = len(xs)
        kept, ks = u8(n * 2 * kp), u8(2 * kp // 128 * n)
        y, ys = (torch.full((n, cols + stride), 7.0, dtype=TYPES[x], device="cuda:0"), None) if out == "same" else \
            (u8(n * kp).view(n, kp), u8(kp // 128 * n))
        pg.pglu_run(config(), xs, y[:, :cols] if out == "same" else y, n, cols, out=out, y_scale=ys, kept=kept, kept_scale=ks)
        res = [y[:, :cols] if out == "same" else y, ys, kept.view(n, -1), ks]
        for src, scale in ((kept, ks), (xs, None)):
            d, ds = (torch.full((n, 2 * cols + stride), 7.0, dtype=TYPES[x], device="cuda:0"), None) if back == "same" else \
                (u8(n * 2 * kp).view(n, -1), u8(2 * kp // 128 * n))
            dv = d[:, :2 * cols] if back == "same" else d
            pg.pglu_grad_run(config(), dy, src, dv, n, cols, x_scale=scale, out=back, dx_scale=ds)
            res += [dv, ds]
        sync()
        return res
    got = call(X, dY, extra)
    for lo in (0, 5003, rows - 300):
        want = call(X[lo:lo + 300], dY[lo:lo + 300], 0)
        for i, (a, b) in enumerate(zip(got, want)):
            if b is None:
                continue
            if i % 2:  # scales [groups][rows]
                a, b = a.view(-1, rows)[:, lo:lo + 300], b.view(-1, 300)
            else:
                a = a[lo:lo + 300]
            assert torch.equal(a, b), (lo, i)


def test_weights_past_four_gib():
    """65 matrices of 8192 x 8192: the last one's bytes, in both orientations, start
    past the fourth gibibyte of every matrix buffer."""
    note("weights' quantisation past 4 GiB")
    experts, n = 65, 8192
    W = torch.zeros((experts, n, n), dtype=torch.bfloat16, device="cuda:0")
    g = torch.Generator(device="cuda:0").manual_seed(8)
    W[-1] = torch.randn((n, n), generator=g, device="cuda:0")
    Q, S, Qt, St = (u8(pg.fp8_weight_bytes(experts, n, n)[k]) for k in ("Q", "scale", "Qt", "scale_t"))
    q, s, qt, st = (u8(pg.fp8_weight_bytes(1, n, n)[k]) for k in ("Q", "scale", "Qt", "scale_t"))
    pg.pfp8_quant_weights_run(config(), W, Q, S, experts, n, n, Qt=Qt, scale_t=St)
    pg.pfp8_quant_weights_run(config(), W[-1], q, s, 1, n, n, Qt=qt, scale_t=st)
    sync()
    for a, b in ((Q, q), (S, s), (Qt, qt), (St, st)):
        a = a.view(experts, -1)
        assert torch.equal(a[-1], b) and not bool(a[:-1].any())


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weight_gradient_past_four_gib(out):
    note(f"weight gradient past 4 GiB {out}")
    experts, n, rows = (70 if out == "f32" else 140), 4096, 640
    g = torch.Generator(device="cuda:0").manual_seed(9)
    A = torch.randint(0, 0x60, (rows, n), generator=g, device="cuda:0", dtype=torch.uint8)
    SA = torch.randint(120, 130, (n // 128, rows), generator=g, device="cuda:0", dtype=torch.uint8)
    D = torch.randn((rows, n), generator=g, device="cuda:0").bfloat16()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda:0")
    offsets[-1:] = rows
    dB = torch.full((experts, n, n), 7.0, dtype=TYPES[out], device="cuda:0")
    one = torch.empty((n, n), dtype=TYPES[out], device="cuda:0")
    pg.pgemm_run_experts_wgrad(config(), D, A, dB, rows, n, n, SA, experts=experts, offsets=offsets)
    pg.pgemm_run_experts_wgrad(config(), D, A, one, rows, n, n, SA)
    sync()
    assert torch.equal(dB[-1], one) and not bool(dB[:-1].any())
