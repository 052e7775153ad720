"""Tokens sorted to experts and back: the sort, gather, combine and combine's
gradient against the 64-bit oracle.

Tolerances: an operation in fp32 is off by at most 2^-24 of its value, so a sum of
n terms by n * 2^-24 of the sum of magnitudes; the result's own rounding adds half
a step of its type (eps / 2 of the value)."""
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


def gpu(v, dtype=None):
    return torch.as_tensor(v).to("cuda:0") if dtype is None else torch.as_tensor(v).to("cuda:0", dtype)


def rounded(got, want, bound, dtype):
    """got is want, off by at most bound, rounded to dtype."""
    half = torch.finfo(dtype).eps / 2
    return np.all(np.abs(host(got) - want) <= bound + (np.abs(want) + bound) * half + 2.0 ** -149)


def run_sort(ids, experts):
    tokens, topk = ids.shape
    slots = tokens * topk
    place = torch.full((tokens, topk), -7, dtype=torch.int32, device="cuda:0")
    order = torch.full((slots,), -7, dtype=torch.int32, device="cuda:0")
    offsets = torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda:0")
    pg.pmoe_sort_run(config(), ids, place, order, offsets, tokens, topk, experts)
    return place, order, offsets


def routed(rng, tokens, topk, experts, dropped=0.2):
    """Distinct experts per token, some slots without one."""
    ids = np.stack([rng.permutation(max(experts, topk))[:topk] for _ in range(tokens)]) if tokens else np.zeros((0, topk))
    ids = np.where(ids < experts, ids, -1)
    return np.where(rng.random(ids.shape) < dropped, rng.choice([-1, experts, -2 ** 31, 2 ** 31 - 1], ids.shape), ids)


@pytest.mark.parametrize("tokens,topk,experts", [(0, 2, 3), (1, 1, 1), (1, 8, 64), (7, 3, 2), (64, 8, 64), (333, 6, 160),
                                                 (2048, 8, 1024), (16384, 1, 5), (16385, 1, 5), (5000, 8, 256),
                                                 (65536, 1, 70), (65537, 1, 1024), (131072 + 5, 2, 1024),
                                                 (300000, 1, 3)])
@pytest.mark.parametrize("wide", [False, True])
def test_sort(tokens, topk, experts, wide):
    note(f"sort {tokens} {topk} {experts} {wide}")
    rng = np.random.default_rng(tokens + experts)
    ids = rng.integers(-1, experts + 1, (tokens, topk))
    if wide and tokens:
        ids[0, 0] = 2 ** 32  # an id whose low half is an expert
    place, order, offsets = run_sort(gpu(ids, torch.int64 if wide else torch.int32), experts)
    sync()
    want = ox.sort(ids, experts)
    assert np.array_equal(offsets.cpu(), want[2])
    assert np.array_equal(place.cpu(), want[0]) and np.array_equal(order.cpu(), want[1])


@pytest.mark.parametrize("tokens", [100, 30000, 140000])
@pytest.mark.parametrize("what", ["one expert", "no rows", "last expert"])
def test_sort_when_slots_agree(tokens, what):
    note(f"sort {tokens} {what}")
    ids = np.full((tokens, 2), {"one expert": 3, "no rows": -1, "last expert": 8}[what])
    place, order, offsets = run_sort(gpu(ids, torch.int32), 9)
    sync()
    want = ox.sort(ids, 9)
    for got, ref in zip((place, order, offsets), want):
        assert np.array_equal(got.cpu(), ref)


SHAPES = [(1, 1, 1, 1), (1, 8, 16, 130), (5, 2, 3, 127), (33, 3, 4, 512), (64, 8, 64, 1000), (700, 6, 9, 520), (3000, 2, 8, 640),
          (9000, 2, 8, 1300)]


@pytest.mark.parametrize("tokens,topk,experts,cols", SHAPES)
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["same", "fp8_b128"])
def test_gather(tokens, topk, experts, cols, x, out):
    note(f"gather {tokens} {topk} {experts} {cols} {x} {out}")
    rng = np.random.default_rng(cols + tokens)
    ids = routed(rng, tokens, topk, experts)
    place, order, offsets = ox.sort(ids, experts)
    slots, n = tokens * topk, offsets[-1]
    X = gpu(rng.standard_normal((tokens, cols + 3)), TYPES[x])[:, :cols]  # a row stride of its own
    rows = host(X)[np.maximum(order, 0) // topk]
    if out == "same":
        Y = torch.full((slots, cols + 5), 7.0, dtype=TYPES[x], device="cuda:0")
        pg.pmoe_gather_run(config(), X, gpu(order), Y[:, :cols], tokens, topk, cols)
        sync()
        assert np.array_equal(host(Y)[:n, :cols], rows[:n])
        assert np.all(host(Y)[n:] == 7.0) and np.all(host(Y)[:, cols:] == 7.0)
        return
    nb = pg.fp8_bytes(slots, cols)
    Q = torch.full((nb["Q"],), 0x55, dtype=torch.uint8, device="cuda:0")
    S = torch.full((nb["scale"],), 0x55, dtype=torch.uint8, device="cuda:0")
    pg.pmoe_gather_run(config(), X, gpu(order), Q, tokens, topk, cols, out="fp8_b128", y_scale=S)
    sync()
    q, s = ox.quant_rows(rows)
    Q, S = Q.cpu().numpy().reshape(q.shape), S.cpu().numpy().reshape(s.shape)
    assert np.array_equal(Q[:n], q[:n]) and np.array_equal(S[:, :n], s[:, :n])
    assert np.all(Q[n:] == 0x55) and np.all(S[:, n:] == 0x55)


@pytest.mark.parametrize("tokens,topk,experts,cols", SHAPES + [(40, 11, 30, 300)])
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("form", ["weights", "weights and residual", "sum", "in place"])
def test_combine(tokens, topk, experts, cols, x, y, form):
    note(f"combine {tokens} {topk} {experts} {cols} {x} {y} {form}")
    rng = np.random.default_rng(cols + tokens)
    place, order, offsets = ox.sort(routed(rng, tokens, topk, experts), experts)
    X = gpu(rng.standard_normal((tokens * topk, cols + 1)), TYPES[x])[:, :cols]
    X[int(offsets[-1]):] = float("nan")  # rows that no slot has are not read
    w = None if form == "sum" else rng.standard_normal((tokens, topk)).astype(np.float32)
    R = gpu(rng.standard_normal((tokens, cols + 2)), TYPES[y])[:, :cols] if form in ("weights and residual", "in place") else None
    want, terms = ox.combine(host(X), place, w, None if R is None else host(R))
    Y = R if form == "in place" else torch.empty((tokens, cols), dtype=TYPES[y], device="cuda:0")
    pg.pmoe_combine_run(config(), X, gpu(place), Y, tokens, topk, cols, weights=None if w is None else gpu(w), R=R)
    sync()
    assert rounded(Y, want, (topk + 1) * U * terms, TYPES[y])


@pytest.mark.parametrize("tokens,topk,experts,cols", SHAPES)
@pytest.mark.parametrize("x,out", [("bf16", "same"), ("f16", "fp8_b128"), ("f32", "same"), ("f32", "fp8_b128"),
                                   ("bf16", "fp8_b128")])
@pytest.mark.parametrize("form", ["weights", "ones", "no dW"])
def test_combine_grad(tokens, topk, experts, cols, x, out, form):
    note(f"combine_grad {tokens} {topk} {experts} {cols} {x} {out} {form}")
    rng = np.random.default_rng(cols + tokens)
    place, order, offsets = ox.sort(routed(rng, tokens, topk, experts), experts)
    slots, n = tokens * topk, offsets[-1]
    dY = gpu(rng.standard_normal((tokens, cols + 1)), TYPES[x])[:, :cols]
    X = gpu(rng.standard_normal((slots, cols + 3)), TYPES[x])[:, :cols]
    X[int(n):] = float("nan")
    w = None if form == "ones" else rng.standard_normal((tokens, topk)).astype(np.float32)
    dW = None if form == "no dW" else torch.full((tokens, topk), 7.0, device="cuda:0")
    Xn = np.nan_to_num(host(X))
    want, want_w, terms = ox.combine_grad(host(dY), Xn, place, w)
    # one fp32 product, which is what is quantised
    prod = host(dY).astype(np.float32)[np.maximum(order, 0) // topk]
    if w is not None:
        prod = prod * w.reshape(-1)[np.maximum(order, 0)][:, None]
    kw = dict(weights=None if w is None else gpu(w), dW=dW)
    if out == "same":
        dX = torch.full((slots, cols + 5), 7.0, dtype=TYPES[x], device="cuda:0")
        pg.pmoe_combine_grad_run(config(), dY, None if dW is None else X, gpu(place), gpu(order), dX[:, :cols], tokens, topk,
                                 cols, **kw)
        sync()
        assert rounded(dX[:n, :cols], want[:n], U * np.abs(want[:n]), TYPES[x])
        assert np.all(host(dX)[n:] == 7.0) and np.all(host(dX)[:, cols:] == 7.0)
    else:
        nb = pg.fp8_bytes(slots, cols)
        Q = torch.full((nb["Q"],), 0x55, dtype=torch.uint8, device="cuda:0")
        S = torch.full((nb["scale"],), 0x55, dtype=torch.uint8, device="cuda:0")
        pg.pmoe_combine_grad_run(config(), dY, None if dW is None else X, gpu(place), gpu(order), Q, tokens, topk, cols,
                                 out="fp8_b128", dx_scale=S, **kw)
        sync()
        q, s = ox.quant_rows(prod)
        Q, S = Q.cpu().numpy().reshape(q.shape), S.cpu().numpy().reshape(s.shape)
        assert np.array_equal(Q[:n], q[:n]) and np.array_equal(S[:, :n], s[:, :n])
        assert np.all(Q[n:] == 0x55) and np.all(S[:, n:] == 0x55)
    if dW is not None:
        assert rounded(dW, want_w, cols * U * terms, torch.float32)
        assert np.all(host(dW)[place < 0] == 0.0)


def test_indices_outside_the_call_leave_rows_out():
    """Device memory that holds no sort's result: such rows and slots count as
    absent, nothing is read or written for them."""
    rng = np.random.default_rng(5)
    tokens, topk, cols = 40, 3, 256
    slots = tokens * topk
    place, order, _ = ox.sort(rng.integers(0, 6, (tokens, topk)), 6)
    bad = np.array([slots, 2 ** 31 - 1, -2 ** 31, -1], np.int32)
    order[::7], place.reshape(-1)[::5] = bad[np.arange(len(order[::7])) % 4], bad[np.arange(len(place.reshape(-1)[::5])) % 4]
    X, D = gpu(rng.standard_normal((tokens, cols)), torch.float32), gpu(rng.standard_normal((slots, cols)), torch.float32)
    Y = torch.full((slots, cols), 7.0, device="cuda:0")
    Z, G = torch.empty_like(X), torch.full((slots, cols), 7.0, device="cuda:0")
    dW = torch.full((tokens, topk), 7.0, device="cuda:0")
    pg.pmoe_gather_run(config(), X, gpu(order), Y, tokens, topk, cols)
    pg.pmoe_combine_run(config(), D, gpu(place), Z, tokens, topk, cols)
    pg.pmoe_combine_grad_run(config(), X, D, gpu(place), gpu(order), G, tokens, topk, cols, dW=dW)
    sync()
    on = (order >= 0) & (order < slots)
    want = np.where(on[:, None], host(X)[np.where(on, order, 0) // topk], 7.0)
    assert np.array_equal(host(Y), want) and np.array_equal(host(G), want)
    ref, terms = ox.combine(host(D), place)
    assert rounded(Z, ref, topk * U * terms, torch.float32)
    gone = (place < 0) | (place >= slots)
    left_out = np.setdiff1d(np.flatnonzero(gone), order[on])
    assert np.all(host(dW).reshape(-1)[left_out] == 0.0)


def test_rows_past_four_gib():
    """Offsets past 32 bits: rows of 64 KiB behind the fourth gibibyte."""
    tokens, topk, cols = 40000, 2, 32768
    note("rows past 4 GiB")
    ids = torch.arange(tokens, device="cuda:0", dtype=torch.int32)[:, None].expand(tokens, 2).contiguous() % 2
    ids[:, 1] = 1 - ids[:, 0]
    place, order, offsets = run_sort(ids, 2)
    X = torch.arange(tokens, device="cuda:0", dtype=torch.float32)[:, None].bfloat16().expand(tokens, cols).contiguous()
    Y = torch.empty((tokens * topk, cols), dtype=torch.bfloat16, device="cuda:0")
    pg.pmoe_gather_run(config(), X, order, Y, tokens, topk, cols)
    Z = torch.empty_like(X)
    pg.pmoe_combine_run(config(), Y, place, Z, tokens, topk, cols, weights=torch.full((tokens, topk), 0.5, device="cuda:0"))
    sync()
    assert torch.equal(Y[:, ::4093], X[order.long() // topk][:, ::4093]) and torch.equal(Z, X)


def test_rows_past_the_caches():
    """Rows of more than 128 MiB, which are loaded and stored past the caches."""
    tokens, topk, cols = 2100, 8, 4096
    slots = tokens * topk
    note("combine past the caches")
    g = torch.Generator(device="cuda:0").manual_seed(2)
    ids = torch.randint(-1, 16, (tokens, topk), generator=g, device="cuda:0", dtype=torch.int32)
    place, order, offsets = run_sort(ids, 16)
    X = torch.randn((slots, cols), generator=g, device="cuda:0").bfloat16()
    dY = torch.randn((tokens, cols), generator=g, device="cuda:0").bfloat16()
    w = torch.rand((tokens, topk), generator=g, device="cuda:0")
    Y, dX, dW = torch.empty_like(dY), torch.zeros_like(X), torch.empty_like(w)
    Q, S = torch.zeros((slots, cols), dtype=torch.uint8, device="cuda:0"), torch.zeros(cols // 128 * slots, dtype=torch.uint8, device="cuda:0")
    Q2, S2 = torch.zeros_like(Q), torch.zeros_like(S)
    pg.pmoe_combine_run(config(), X, place, Y, tokens, topk, cols, weights=w, R=dY)
    pg.pmoe_combine_grad_run(config(), dY, X, place, order, dX, tokens, topk, cols, weights=w, dW=dW)
    pg.pmoe_combine_grad_run(config(), dY, None, place, order, Q, tokens, topk, cols, weights=w, out="fp8_b128", dx_scale=S)
    sync()
    on, slot = order >= 0, order.clamp(min=0).long()
    prod = dY.float()[slot // topk] * w.view(-1)[slot][:, None]
    assert torch.equal(dX, (prod * on[:, None]).bfloat16())
    pg.pfp8_quant_run(config(), prod, Q2, S2, slots, cols)
    sync()
    n = int(offsets[-1])
    assert torch.equal(Q[:n], Q2[:n]) and torch.equal(S.view(-1, slots)[:, :n], S2.view(-1, slots)[:, :n])
    for lo in range(0, tokens, 300):
        p = place[lo:lo + 300].long()
        rows = X[p.clamp(min=0)].double() * (p >= 0)[..., None]
        ref = (rows * w[lo:lo + 300].double()[..., None]).sum(1) + dY[lo:lo + 300].double()
        mag = (rows.abs() * w[lo:lo + 300].double()[..., None]).sum(1) + dY[lo:lo + 300].double().abs()
        bound = (topk + 1) * U * mag
        assert bool(((Y[lo:lo + 300].double() - ref).abs() <= bound + (ref.abs() + bound) * 2.0 ** -8).all())
        ref = (rows * dY[lo:lo + 300, None].double()).sum(-1)
        mag = (rows * dY[lo:lo + 300, None].double()).abs().sum(-1)
        assert bool(((dW[lo:lo + 300].double() - ref).abs() <= (cols + 1) * U * mag).all())
