"""The experts' product and its weight gradient against the 64-bit oracle.

Tolerances.  Product to fp32: sums of exact products by the bf16 MFMA, an
instruction of 32 within 2^-22 of the magnitudes it adds (k / 32 instructions), then
the sums of up to eight waves (8 * 2^-24).  To bf16, the e4m3 MFMA cuts each product
at 2^-13 of the largest of the eight that it adds first: the eight's cuts are at most
8 * 2^-13 of that one, and so 2^-10 of the sum of their magnitudes (measured on
operands of two equal and opposite products 2^16 and a third, 2^e: it is lost from
e = 2 on down beside them, from -8 on in another eight).  Then the result's
rounding.  Weight gradient: a sum over n rows in fp32,
32 products to an instruction: (n / 32 + 2) * 2^-22 of the magnitudes; the base's
addition 2^-24 of both; the result's rounding."""
import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import experts as ox
from tests.gpu_util import config, note, sync

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gpu(v):
    return torch.from_numpy(np.ascontiguousarray(v)).to("cuda:0")


def host(t):
    return t.double().cpu().numpy()


def split(rng, rows, experts, how):
    """Offsets of `rows` rows: spread, all of one expert's, or with experts that
    have none and rows behind the last."""
    if how == "one":
        n = np.zeros(experts, int)
        n[experts // 2] = rows
    else:
        p = rng.dirichlet(np.full(experts, 0.6))
        n = rng.multinomial(rows if how == "all" else rows - rows // 5, p)
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def operands(rng, rows, n, k, experts):
    a = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
    qa, sa = ox.quant_rows(a)
    parts = [ox.quant_weights(rng.standard_normal((n, k)) * 2.0 ** rng.integers(-4, 5)) for _ in range(experts)]
    return qa, sa, np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


def check(C, offsets, ref, terms, k, dtype):
    n = offsets[-1]
    bound = (k / 32 * 2.0 ** -22 + 8 * 2.0 ** -24 + (2.0 ** -10 if dtype == torch.bfloat16 else 0.0)) * terms
    bound = bound + (np.abs(ref) + bound) * torch.finfo(dtype).eps / 2
    got = host(C)
    assert np.all(np.abs(got[:n] - ref[:n]) <= bound[:n])
    assert np.all(got[n:] == 7.0)


# rows per expert from none to many: every kernel and tile
SHAPES = [(1, 128, 128, 1), (24, 300, 1280, 1), (50, 1100, 384, 20), (60, 4100, 256, 6), (1, 70, 256, 5), (8, 256, 384, 64), (17, 129, 128, 2), (40, 1000, 640, 3), (64, 513, 1024, 1),
          (130, 300, 1152, 4), (200, 256, 2048, 6), (700, 300, 512, 3), (1100, 777, 256, 2), (2000, 512, 384, 9),
          (3000, 1030, 128, 5), (5000, 4200, 256, 3), (4000, 3000, 128, 20), (2000, 150, 128, 1024), (13000, 130, 128, 1000)]


@pytest.mark.parametrize("rows,n,k,experts", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["all", "one", "some"])
def test_product(rows, n, k, experts, out, how):
    note(f"product {rows} {n} {k} {experts} {out} {how}")
    rng = np.random.default_rng(rows + n)
    offsets = split(rng, rows, experts, how)
    qa, sa, qb, sb = operands(rng, rows, n, k, experts)
    a = ox.dequant_rows(qa, sa)
    qa[offsets[-1]:], sa[:, offsets[-1]:] = 0x7f, 255  # rows of no expert: NaN that reaches nothing
    C = torch.full((rows, n), 7.0, dtype=TYPES[out], device="cuda:0")
    pg.pgemm_run_experts(config(), gpu(qa), gpu(qb), C, rows, n, k, gpu(sa), gpu(sb), experts=experts, offsets=gpu(offsets))
    sync()
    b = np.stack([ox.dequant_weights(q, s) for q, s in zip(qb, sb)])
    check(C, offsets, *ox.product(a, b, offsets), k, TYPES[out])


@pytest.mark.parametrize("rows,n,k", [(1, 300, 512), (50, 130, 256), (300, 400, 384), (1030, 520, 640)])
def test_one_matrix_without_offsets(rows, n, k):
    note(f"product {rows} {n} {k}, no offsets")
    rng = np.random.default_rng(rows)
    qa, sa, qb, sb = operands(rng, rows, n, k, 1)
    C = torch.full((rows, n), 7.0, device="cuda:0")
    pg.pgemm_run_experts(config(), gpu(qa), gpu(qb), C, rows, n, k, gpu(sa), gpu(sb))
    sync()
    ref, terms = ox.product(ox.dequant_rows(qa, sa), ox.dequant_weights(qb[0], sb[0])[None], [0, rows])
    check(C, [rows], ref, terms, k, torch.float32)


@pytest.mark.parametrize("rows", [30, 600])
def test_offsets_outside_the_rows(rows):
    """Offsets that no sort writes: ranges are cut to the call's rows, nothing is
    read or written outside."""
    rng = np.random.default_rng(rows)
    n, k = 200, 256
    qa, sa, qb, sb = operands(rng, rows, n, k, 4)
    bad = np.array([-5, rows // 3, rows // 4, rows + 7, 2 ** 31 - 1], np.int32)
    C = torch.full((rows, n), 7.0, device="cuda:0")
    dB = torch.empty((4, n, k), device="cuda:0")
    D = gpu(rng.standard_normal((rows, n)).astype(np.float32)).bfloat16()
    pg.pgemm_run_experts(config(), gpu(qa), gpu(qb), C, rows, n, k, gpu(sa), gpu(sb), experts=4, offsets=gpu(bad))
    pg.pgemm_run_experts_wgrad(config(), D, gpu(qa), dB, rows, n, k, gpu(sa), experts=4, offsets=gpu(bad))
    sync()
    a = ox.dequant_rows(qa, sa)
    ranges = [(0, rows // 3), (0, 0), (rows // 4, rows), (0, 0)]
    for e, (lo, hi) in enumerate(ranges):
        ref = host(D)[lo:hi].T @ a[lo:hi]
        terms = np.abs(host(D)[lo:hi]).T @ np.abs(a[lo:hi])
        assert np.all(np.abs(host(dB)[e] - ref) <= (rows / 32 + 3) * 2.0 ** -22 * terms)
    ref = a[rows // 3:] @ ox.dequant_weights(qb[2], sb[2]).T
    assert np.allclose(host(C)[rows // 3:], ref, rtol=1e-5, atol=1e-5 * np.abs(ref).max())


@pytest.mark.parametrize("rows", [20, 300, 1200])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_nan_codes_and_scales_stay_in_their_rows(rows, out):
    rng = np.random.default_rng(8)
    n, k = 260, 384
    qa, sa, qb, sb = operands(rng, rows, n, k, 2)
    qa[3, 200], sa[1, 7] = 0x7f, 255
    sb[1, 1, 0] = 255  # expert 1's columns 128 .. 255
    offsets = np.array([0, rows - 6, rows], np.int32)
    C = torch.empty((rows, n), dtype=TYPES[out], device="cuda:0")
    pg.pgemm_run_experts(config(), gpu(qa), gpu(qb), C, rows, n, k, gpu(sa), gpu(sb), experts=2, offsets=gpu(offsets))
    sync()
    want = np.zeros((rows, n), bool)
    want[[3, 7]] = True
    want[rows - 6:, 128:256] = True
    assert np.array_equal(np.isnan(host(C)), want)


WGRAD = [(1, 1, 1, 1), (5, 130, 100, 3), (64, 128, 128, 1), (100, 260, 390, 4), (300, 72, 513, 2), (700, 256, 256, 5),
         (2000, 520, 260, 3), (1000, 640, 1100, 2),
         (1500, 1032, 1100, 14), (600, 64, 130, 300), (40, 130, 8, 1024),
         (4600, 2064, 2050, 4), (3300, 130, 260, 1)]  # several stretches of 512 rows, on both tiles


@pytest.mark.parametrize("rows,n,k,experts", WGRAD)
@pytest.mark.parametrize("d", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("base", ["none", "other", "same"])
@pytest.mark.parametrize("how", ["all", "some"])
def test_wgrad(rows, n, k, experts, d, out, base, how):
    note(f"wgrad {rows} {n} {k} {experts} {d} {out} {base} {how}")
    rng = np.random.default_rng(rows + n)
    offsets = split(rng, rows, experts, how)
    last = offsets[-1]
    qa, sa = ox.quant_rows(rng.standard_normal((rows, k)) * np.exp2(rng.integers(-6, 7, (rows, 1))))
    a = ox.dequant_rows(qa, sa)[:, :k]
    qa[last:], sa[:, last:] = 0x7f, 255
    kw = {}
    if d == "bf16":
        D = gpu(rng.standard_normal((rows, n + 3)).astype(np.float32)).bfloat16()[:, :n]
        D[int(last):] = float("nan")
        dv = np.nan_to_num(host(D))
    else:
        qd, sd = ox.quant_rows(rng.standard_normal((rows, n)) * np.exp2(rng.integers(-6, 7, (rows, 1))))
        dv = ox.dequant_rows(qd, sd)[:, :n]
        qd[last:], sd[:, last:] = 0x7f, 255
        D, kw["d_scale"] = gpu(qd), gpu(sd)
    ref, terms = ox.wgrad(dv, a, offsets)
    counts = (offsets[1:] - offsets[:-1])[:, None, None]
    bound = (counts / 32 + 2) * 2.0 ** -22 * terms
    dB = torch.full((experts, n, k), 3.0, dtype=TYPES[out], device="cuda:0")
    if base != "none":
        B = dB if base == "same" else gpu(rng.standard_normal((experts, n, k)).astype(np.float32)).to(TYPES[out])
        ref = ref + host(B)
        bound = bound + 2.0 ** -24 * (np.abs(ref) + bound)
        kw["base"] = B
    pg.pgemm_run_experts_wgrad(config(), D, gpu(qa), dB, rows, n, k, gpu(sa), experts=experts, offsets=gpu(offsets), **kw)
    sync()
    bound = bound + (np.abs(ref) + bound) * torch.finfo(TYPES[out]).eps / 2
    assert np.all(np.abs(host(dB) - ref) <= bound)


@pytest.mark.parametrize("rows,n,k,experts", [(3, 5, 130, 1), (70, 131, 260, 3), (700, 2053, 2050, 4), (1300, 4095, 1030, 5)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("ldd", ["n to 8", "more"])
def test_wgrad_rows_on_vectors(rows, n, k, experts, out, ldd):
    """bf16 rows that start on 16 bytes and end inside a vector, on both tiles; the last
    row ends where the memory that belongs to the matrix does."""
    note(f"wgrad rows on vectors {rows} {n} {k} {experts} {out} {ldd}")
    rng = np.random.default_rng(n)
    ld = (n + 7) // 8 * 8 + (16 if ldd == "more" else 0)
    offsets = split(rng, rows, experts, "all")
    qa, sa = ox.quant_rows(rng.standard_normal((rows, k)) * np.exp2(rng.integers(-6, 7, (rows, 1))))
    a = ox.dequant_rows(qa, sa)[:, :k]
    D = gpu(rng.standard_normal((rows, ld)).astype(np.float32)).bfloat16()
    D[:, n:] = float("nan")
    D = D[:, :n]
    ref, terms = ox.wgrad(host(D), a, offsets)
    counts = (offsets[1:] - offsets[:-1])[:, None, None]
    bound = (counts / 32 + 2) * 2.0 ** -22 * terms
    dB = torch.full((experts, n, k), 3.0, dtype=TYPES[out], device="cuda:0")
    pg.pgemm_run_experts_wgrad(config(), D, gpu(qa), dB, rows, n, k, gpu(sa), experts=experts, offsets=gpu(offsets))
    sync()
    bound = bound + (np.abs(ref) + bound) * torch.finfo(TYPES[out]).eps / 2
    assert np.all(np.abs(host(dB) - ref) <= bound)


@pytest.mark.parametrize("d", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,k", [(260, 390), (2064, 2050)])
def test_wgrad_nan_rows_stay_in_their_expert(n, k, d):
    """A row whose block is NaN makes its expert's gradient NaN in that block's columns
    and leaves the experts before and after it, which share slabs of 64 rows."""
    note(f"wgrad nan {n} {k} {d}")
    rng = np.random.default_rng(9)
    rows, experts = 640, 5
    offsets = np.array([0, 100, 230, 500, 540, 640], np.int32)
    qa, sa = ox.quant_rows(rng.standard_normal((rows, k)))
    sa[1, 230] = 255  # expert 2's first row, columns 128 .. 255
    qa[539, 0] = 0x7f  # expert 3's last row
    kw = {}
    D = gpu(rng.standard_normal((rows, n)).astype(np.float32)).bfloat16()
    if d == "bf16":
        D[99, 5] = float("nan")  # expert 0's last row
    else:
        qd, sd = ox.quant_rows(host(D))
        qd[99, 5] = 0x7f
        D, kw["d_scale"] = gpu(qd), gpu(sd)
    dB = torch.zeros((experts, n, k), device="cuda:0")
    pg.pgemm_run_experts_wgrad(config(), D, gpu(qa), dB, rows, n, k, gpu(sa), experts=experts, offsets=gpu(offsets), **kw)
    sync()
    want = np.zeros((experts, n, k), bool)
    want[0, 5] = want[2, :, 128:256] = want[3, :, 0] = True
    assert np.array_equal(np.isnan(host(dB)), want)


def test_wgrad_without_rows():
    """No rows at all: zeros, or the base."""
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    A = torch.empty(0, dtype=torch.uint8, device="cuda:0")
    D = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda:0")
    dB = torch.full((3, 40, 130), 7.0, device="cuda:0")
    base = torch.randn((3, 40, 130), device="cuda:0")
    pg.pgemm_run_experts_wgrad(config(), D, A, dB, 0, 40, 130, A, experts=3, offsets=offsets)
    sync()
    assert bool((dB == 0).all())
    pg.pgemm_run_experts_wgrad(config(), D, A, dB, 0, 40, 130, A, experts=3, offsets=offsets, base=base)
    sync()
    assert torch.equal(dB, base)


@pytest.mark.parametrize("rows", [3, 700])
def test_operands_past_four_gib(rows):
    """Weights behind the fourth gibibyte: expert 300 of 301 matrices of 16 MiB; the
    rows' products are those of the matrix alone."""
    note(f"product past 4 GiB, {rows} rows")
    n = k = 4096
    experts = 301
    B = torch.zeros((experts, n, k), dtype=torch.uint8, device="cuda:0")
    SB = torch.full((experts, n // 128, k // 128), 127, dtype=torch.uint8, device="cuda:0")
    g = torch.Generator(device="cuda:0").manual_seed(1)
    B[300] = torch.randint(0, 0x60, (n, k), generator=g, device="cuda:0", dtype=torch.uint8)
    A = torch.randint(0, 0x60, (rows, k), generator=g, device="cuda:0", dtype=torch.uint8)
    SA = torch.randint(120, 130, (k // 128, rows), generator=g, device="cuda:0", dtype=torch.uint8)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda:0")
    offsets[301:] = rows
    C, C1 = torch.empty((rows, n), device="cuda:0"), torch.empty((rows, n), device="cuda:0")
    pg.pgemm_run_experts(config(), A, B, C, rows, n, k, SA, SB, experts=experts, offsets=offsets)
    pg.pgemm_run_experts(config(), A, B[300], C1, rows, n, k, SA, SB[300])
    sync()
    # positive terms: any order of sums is within k / 32 * 2^-22 of the value
    assert bool(((C - C1).abs() <= 2 * k / 32 * 2.0 ** -22 * C1).all())


@pytest.mark.parametrize("rows", [6, 900])
def test_replayed_on_another_stream(rows):
    """A captured product and gradient whose offsets and operands change between the
    replays, beside eager calls on the current stream."""
    note(f"captured product {rows}")
    rng = np.random.default_rng(3)
    n, k, experts = 384, 512, 4
    qa, sa, qb, sb = operands(rng, rows, n, k, experts)
    A, SA, B, SB = gpu(qa), gpu(sa), gpu(qb), gpu(sb)
    D = gpu(rng.standard_normal((rows, n)).astype(np.float32)).bfloat16()
    offsets = gpu(split(rng, rows, experts, "all"))
    C, dB = torch.zeros((rows, n), device="cuda:0"), torch.empty((experts, n, k), device="cuda:0")

    def call(c, g):
        pg.pgemm_run_experts(config(), A, B, c, rows, n, k, SA, SB, experts=experts, offsets=offsets)
        pg.pgemm_run_experts_wgrad(config(), D, A, g, rows, n, k, SA, experts=experts, offsets=offsets)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    call(C, dB)
    sync()
    with torch.cuda.graph(graph, stream=side):
        call(C, dB)
    for i in range(4):
        offsets.copy_(gpu(split(rng, rows, experts, ("all", "one", "some", "all")[i])))
        A.copy_(gpu(np.roll(qa, i, 0)))
        C.zero_()
        want, want_b = torch.zeros_like(C), torch.empty_like(dB)
        sync()
        graph.replay()
        call(want, want_b)
        sync()
        assert torch.equal(C, want) and torch.equal(dB, want_b), i
