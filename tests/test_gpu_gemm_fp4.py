"""MXFP4 GEMM on the GPU against the 64-bit oracle.

Tolerance: the products of two e2m1 values and a power of two are exact; one
matrix instruction adds a row's 128 products to the fp32 accumulator, which is
taken to cost at most 2^-22 (four fp32 roundings, one per block) of the
magnitudes added so far, so |C - C_ref| <= K/128 * 2^-22 * (|A|.|B|)_ij, and a
bf16 C half a step more."""
import ctypes

import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from oracle import sched_model as sm  # noqa: F401
from tile_scheduling_persistent_amd import _abi
from tests.gpu_util import Guarded, config, dev_u8, note, sync

pytestmark = pytest.mark.gpu

SCHEDS = ["blocked", "interleaved", "grouped", "work_stealing", "blocked_grouped", "work_stealing_xcc"]
OUTS = {"mxfp4_out_bf16": "bf16", "mxfp4_out_f32": "f32"}


def operand(rows, K, seed):
    """Codes of normal values with rows of different size, one row of zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1)))
    x[:, : K // 4] *= np.exp2(rng.integers(-8, 9, (rows, 1)))
    x[rows // 2] = 0.0 if rows > 2 else x[rows // 2]
    return mx.quant_mxfp4(x)


def run(qa, sa, qb, sb, M, N, K, dtype, sched, fn=None, **kw):
    C = Guarded(M * N, OUTS[dtype])
    note(f"mxfp4 M={M} N={N} K={K} {dtype} {sched} {kw}")
    (fn or pg.pgemm_run)(config(), dev_u8(qa), dev_u8(qb), C.view, M, N, K, dtype, sched,
                         pg.make_args(a_scale=dev_u8(sa), b_scale=dev_u8(sb), **kw))
    sync()
    assert C.guards_intact(), (M, N, K, dtype, sched, kw)
    return C


def check(C, Cref, Abs, K, dtype, what):
    got = C.as_f64().reshape(Cref.shape)
    bound = K / 128 * 2.0 ** -22 * Abs
    if OUTS[dtype] == "bf16":
        bound = bound + (np.abs(Cref) + bound) * 2.0 ** -8
    bad = ~(np.abs(got - Cref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], Cref[bad][:3])


SHAPES = [(1, 1, 128), (1, 100, 256), (2, 17, 384), (3, 4096, 512), (15, 33, 640), (16, 64, 1024), (17, 130, 2048),
          (33, 257, 128), (64, 96, 896), (65, 1000, 256), (100, 112, 1152), (129, 127, 384), (255, 300, 512),
          (256, 272, 256), (257, 520, 640), (300, 513, 1280)]


@pytest.mark.parametrize("dtype", list(OUTS))
def test_default_tile_any_shape(dtype):
    for i, (M, N, K) in enumerate(SHAPES):
        qa, sa = operand(M, K, 300 + i)
        qb, sb = operand(N, K, 400 + i)
        Cref, Abs = mx.gemm_mxfp4(qa, sa, qb, sb)
        check(run(qa, sa, qb, sb, M, N, K, dtype, "grouped"), Cref, Abs, K, dtype, (M, N, K))


TILES = [(256, 256), (256, 128), (128, 128), (64, 32), (32, 32), (16, 32), (16, 16)]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("dtype", list(OUTS))
def test_every_tile_on_ragged_shapes(tile, dtype):
    """Every built tile: edges in M and N, one to six K groups (odd ones end
    inside a slab), C rows that start on a line (N = 512) or not, and eight
    programs, so that each walks several tiles and the loads run on across
    them."""
    for i, (M, N, K) in enumerate([(5, 7, 128), (259, 263, 384), (513, 512, 256), (270, 512, 640), (600, 777, 768)]):
        if tile[0] <= 64 and M > 300:
            M = M // 8
        qa, sa = operand(M, K, 500 + i)
        qb, sb = operand(N, K, 600 + i)
        Cref, Abs = mx.gemm_mxfp4(qa, sa, qb, sb)
        for sched, grid in (("grouped", 0), ("interleaved", 8), ("work_stealing", 8)):
            C = run(qa, sa, qb, sb, M, N, K, dtype, sched, tile=tile + (256,), grid=grid)
            check(C, Cref, Abs, K, dtype, (tile, M, N, K, sched))


def test_more_tiles_than_cus_and_fewer_give_the_same_bits():
    """128 x 128 tiles take another ring depth where no CU gets two of them: the
    columns that both launches share have the same sums in the same order."""
    M, K, wide, few = 260, 640, 16500, 900
    qa, sa = operand(M, K, 1)
    qb, sb = operand(wide, K, 2)
    A = run(qa, sa, qb, sb, M, wide, K, "mxfp4_out_f32", "grouped", tile=(128, 128, 256))
    B = run(qa, sa, qb[:few].copy(), sb[:, :few].copy(), M, few, K, "mxfp4_out_f32", "grouped", tile=(128, 128, 256))
    a, b = A.as_f64().reshape(M, wide), B.as_f64().reshape(M, few)
    assert np.array_equal(a[:, :few], b)
    Cref, Abs = mx.gemm_mxfp4(qa, sa, qb[-few:].copy(), sb[:, -few:].copy())
    assert np.all(np.abs(a[:, -few:] - Cref) <= K / 128 * 2.0 ** -22 * Abs)


@pytest.mark.parametrize("tile", TILES)
def test_grouped_problems_on_every_tile(tile):
    shapes = [(70, 130, 256), (1, 257, 640), (290, 512, 384)]
    ops, outs = [], []
    for i, (M, N, K) in enumerate(shapes):
        qa, sa = operand(M, K, 70 + i)
        qb, sb = operand(N, K, 80 + i)
        C = Guarded(M * N, "bf16")
        outs.append((C, qa, sa, qb, sb, M, N, K))
        ops.append((dev_u8(qa), dev_u8(qb), C.view, M, N, K, dev_u8(sa), dev_u8(sb)))
    note(f"grouped mxfp4 {tile}")
    pg.pgemm_run_grouped(config(), ops, "mxfp4_out_bf16", "work_stealing", pg.make_args(tile=tile + (256,)))
    sync()
    for C, qa, sa, qb, sb, M, N, K in outs:
        assert C.guards_intact()
        check(C, *mx.gemm_mxfp4(qa, sa, qb, sb), K, "mxfp4_out_bf16", (tile, M, N, K))


@pytest.mark.parametrize("sched", SCHEDS)
def test_schedulers_agree(sched):
    for M, N, K in [(1, 700, 512), (40, 2100, 384), (700, 1100, 640)]:
        qa, sa = operand(M, K, 1)
        qb, sb = operand(N, K, 2)
        Cref, Abs = mx.gemm_mxfp4(qa, sa, qb, sb)
        for dtype in OUTS:
            C = run(qa, sa, qb, sb, M, N, K, dtype, sched)
            check(C, Cref, Abs, K, dtype, (M, N, K, sched))
            D = run(qa, sa, qb, sb, M, N, K, dtype, sched, fn=pg.pgemm_run_noalloc)
            assert np.array_equal(C.body_bits(), D.body_bits())


def test_closed_form_scales():
    """Codes all 1.0, scale bytes 127 + (g + i + 2 b) % 5 - 2 and 127 - (j + b) % 3:
    C is a sum of powers of two times 32, exact in fp32."""
    M, N, K = 150, 70, 768
    G = K // 128
    qa, qb = np.full((M, K // 2), 0x22, np.uint8), np.full((N, K // 2), 0x22, np.uint8)
    g, i, b = np.meshgrid(np.arange(G), np.arange(M), np.arange(4), indexing="ij")
    sa = (127 + (g + i + 2 * b) % 5 - 2).astype(np.uint8)
    g, j, b = np.meshgrid(np.arange(G), np.arange(N), np.arange(4), indexing="ij")
    sb = (127 - (j + b) % 3).astype(np.uint8)
    fa, fb = 2.0 ** (sa.astype(float) - 127), 2.0 ** (sb.astype(float) - 127)
    want = 32.0 * np.einsum("gmb,gnb->mn", fa, fb)
    for sched in SCHEDS:
        C = run(qa, sa, qb, sb, M, N, K, "mxfp4_out_f32", sched)
        assert np.array_equal(C.as_f64().reshape(M, N), want), sched


@pytest.mark.parametrize("M", [1, 20, 200])
def test_nan_scales_reach_their_rows_and_columns_only(M):
    N, K = 150, 512
    qa, sa = operand(M, K, 11)
    qb, sb = operand(N, K, 12)
    sa, sb = sa.copy(), sb.copy()
    sa[1, M // 2, 2] = 255
    sb[3, 77, 0] = 255
    C = run(qa, sa, qb, sb, M, N, K, "mxfp4_out_f32", "grouped")
    nan = np.isnan(C.as_f64().reshape(M, N))
    want = np.zeros((M, N), bool)
    want[M // 2], want[:, 77] = True, True
    assert np.array_equal(nan, want)


def test_scale_extremes():
    """Bytes 0 (2^-127) and 254 (2^127) whose products are in range."""
    M, N, K = 5, 40, 256
    qa, _ = operand(M, K, 1)
    qb, _ = operand(N, K, 2)
    sa, sb = np.zeros((2, M, 4), np.uint8), np.full((2, N, 4), 254, np.uint8)
    Cref, Abs = mx.gemm_mxfp4(qa, sa, qb, sb)
    check(run(qa, sa, qb, sb, M, N, K, "mxfp4_out_f32", "blocked"), Cref, Abs, K, "mxfp4_out_f32", "extremes")


@pytest.mark.parametrize("dtype", list(OUTS))
def test_grouped_problems(dtype):
    shapes = [(70, 130, 256), (0, 64, 128), (1, 257, 640), (300, 90, 384)]
    ops, outs = [], []
    for i, (M, N, K) in enumerate(shapes):
        qa, sa = operand(max(M, 1), K, 20 + i)
        qb, sb = operand(N, K, 30 + i)
        C = Guarded(max(M * N, 1), OUTS[dtype])
        outs.append((C, qa, sa, qb, sb, M, N, K))
        ops.append((dev_u8(qa), dev_u8(qb), C.view, M, N, K, dev_u8(sa), dev_u8(sb)))
    for sched in SCHEDS:
        note(f"grouped mxfp4 {sched}")
        pg.pgemm_run_grouped(config(), ops, dtype, sched)
        sync()
        for C, qa, sa, qb, sb, M, N, K in outs:
            assert C.guards_intact()
            if M:
                check(C, *mx.gemm_mxfp4(qa, sa, qb, sb), K, dtype, (M, N, K, sched))
                C.view.zero_()


def test_unaligned_output():
    """C that starts on an odd element, rows of odd length."""
    for M, N in [(1, 63), (20, 131), (140, 77)]:
        K = 256
        qa, sa = operand(M, K, 5)
        qb, sb = operand(N, K, 6)
        Cref, Abs = mx.gemm_mxfp4(qa, sa, qb, sb)
        for dtype, t in (("mxfp4_out_bf16", torch.bfloat16), ("mxfp4_out_f32", torch.float32)):
            buf = torch.full((M * N + 3,), -3.0, dtype=t, device="cuda:0")
            A, B, SA, SB = dev_u8(qa), dev_u8(qb), dev_u8(sa), dev_u8(sb)
            note(f"unaligned C {M}x{N} {dtype}")
            pg.pgemm_run(config(), A, B, buf[1:-2], M, N, K, dtype, "grouped", pg.make_args(a_scale=SA, b_scale=SB))
            sync()
            h = buf.double().cpu().numpy()
            assert h[0] == -3 and h[-1] == -3 and h[-2] == -3
            bound = (K / 128 * 2.0 ** -22) * Abs
            bound = bound + (np.abs(Cref) + bound) * (2.0 ** -8 if t == torch.bfloat16 else 0)
            assert np.all(np.abs(h[1:-2].reshape(M, N) - Cref) <= bound)


@pytest.mark.parametrize("M,N,K", [(1, 1000, 512), (24, 900, 384), (600, 700, 256)])
def test_witness_every_tile_once(M, N, K):
    qa, sa = operand(M, K, 1)
    qb, sb = operand(N, K, 2)
    cfg = config()
    A, B, SA, SB = dev_u8(qa), dev_u8(qb), dev_u8(sa), dev_u8(sb)
    C = Guarded(M * N, "bf16")
    for sched in SCHEDS:
        args = pg.make_args(a_scale=SA, b_scale=SB, debug_flags=_abi.DEBUG_WITNESS)
        pl = pg.plan_gemm(cfg, M, N, K, "mxfp4_out_bf16", sched, args)
        assert pl["kernel"] == "fp4"
        cfg.witness_enable(pl["tiles"], pl["grid"])
        note(f"witness mxfp4 {M}x{N}x{K} {sched} {pl}")
        pg.pgemm_run(cfg, A, B, C.view, M, N, K, "mxfp4_out_bf16", sched, args)
        w = cfg.witness_read(pl["tiles"], pl["grid"])
        assert np.all(w["visits"] == 1), sched
        assert int(w["n_tiles"].sum()) == pl["tiles"]


def test_graph_replays():
    M, N, K = 48, 640, 512
    qb, sb = operand(N, K, 2)
    A = torch.zeros((M, K // 2), dtype=torch.uint8, device="cuda:0")
    SA = torch.zeros((K // 128, M, 4), dtype=torch.uint8, device="cuda:0")
    B, SB = dev_u8(qb), dev_u8(sb)
    C = torch.zeros((M, N), device="cuda:0")
    args = pg.make_args(a_scale=SA, b_scale=SB)
    call = lambda: pg.pgemm_run(config(), A, B, C, M, N, K, "mxfp4_out_f32", "work_stealing", args)  # noqa: E731
    call()
    sync()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for seed in range(3):
        qa, sa = operand(M, K, 60 + seed)
        A.copy_(torch.from_numpy(qa))
        SA.copy_(torch.from_numpy(sa))
        call()
        sync("eager")
        want = C.clone()
        C.zero_()
        sync("cleared")
        g.replay()
        sync("replay")
        assert torch.equal(C, want)


def test_refusals():
    cfg, L = config(), _abi.lib()
    M, N, K = 32, 48, 256
    A, B = (torch.zeros(n * K // 2 + 64, dtype=torch.uint8, device="cuda:0") for n in (M, N))
    SA, SB = (torch.zeros(n * K // 32 + 64, dtype=torch.uint8, device="cuda:0") for n in (M, N))
    C = torch.full((M * N,), 7.0, device="cuda:0")
    a, b, c = A.data_ptr(), B.data_ptr(), C.data_ptr()

    def call(A=a, B=b, C=c, m=M, n=N, k=K, d=4, s=0, sa=SA.data_ptr(), sb=SB.data_ptr(), tile=None):
        args = pg.make_args(tile=tile, a_scale=sa, b_scale=sb)
        return L.pgemm_run(cfg.handle, A, B, C, m, n, k, d, s, ctypes.byref(args), None)

    I, V = _abi.ERR_INVALID, _abi.ERR_UNSUPPORTED  # noqa: E741
    for bad in (dict(A=None), dict(B=None), dict(C=None), dict(k=192), dict(k=0), dict(m=0), dict(sa=None),
                dict(sb=None), dict(C=a), dict(C=SA.data_ptr(), m=1, n=8), dict(m=1 << 20), dict(n=1 << 20),
                dict(s=9)):
        assert call(**bad) == I, bad
    assert L.pgemm_run(cfg.handle, a, b, c, M, N, K, 4, 0, None, None) == I
    for bad in (dict(A=a + 8), dict(B=b + 4), dict(C=c + 2), dict(sa=SA.data_ptr() + 2), dict(sb=SB.data_ptr() + 1),
                dict(tile=(96, 96, 128)), dict(tile=(256, 256, 64))):
        assert call(**bad) == V, bad
    sync()
    assert torch.all(C == 7.0)
