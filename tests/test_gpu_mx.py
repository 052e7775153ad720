"""MXFP4 quantisation and dequantisation on the GPU against the 64-bit oracle:
every step is exact (power-of-two scaling, one rounding), so codes, scale
bytes and values are compared for equality."""
import ctypes

import numpy as np
import pytest
import torch

import tile_scheduling_persistent_amd as pg
from oracle import mx
from tile_scheduling_persistent_amd import _abi
from tests.gpu_util import config, dev_u8, note, sync

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAD = 256   # guard bytes on each side of an output


class Bytes:
    """Output of n bytes between guard bands of 0xA5."""

    def __init__(self, n):
        self.full = torch.full((n + 2 * PAD,), 0xA5, dtype=torch.uint8, device="cuda:0")
        self.view = self.full[PAD:PAD + n]

    def get(self):
        h = self.full.cpu().numpy()
        assert np.all(h[:PAD] == 0xA5) and np.all(h[len(h) - PAD:] == 0xA5), "guard bytes overwritten"
        return h[PAD:len(h) - PAD]


def make(rows, cols, kind, seed, special=False):
    """Values as the type holds them, in fp64, and the tensor."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[:, cols // 3:cols // 3 + 40] *= 2.0 ** -20
    # multiples of a quarter: ties of every kind
    x[rows // 2] = rng.integers(-28, 29, cols) / 4.0
    x[0, :min(cols, 64)] = -0.0
    if special:
        tiny, big = (2.0 ** -24, 6e4) if kind == "f16" else (2.0 ** -133, 3e38)
        x[rows // 3] = tiny * rng.integers(0, 9, cols)
        x[rows - 1] = big * rng.uniform(-1, 1, cols)
        x[rows // 4, cols // 2] = np.nan
        x[rows // 5, cols // 5] = np.inf
        x[rows // 6, cols - 1] = -np.inf
    t = torch.from_numpy(x.astype(np.float32)).to(TYPES[kind])
    return t.double().numpy(), t.to("cuda:0")


def quant(x, rows, cols, transpose, rule, **kw):
    lines, length = (cols, rows) if transpose else (rows, cols)
    nb = pg.mxfp4_bytes(lines, length)
    q, s = Bytes(nb["Q"]), Bytes(nb["scale"])
    note(f"pmx_quant_run {rows}x{cols} transpose={transpose} {rule} {x.dtype} stride={x.stride()}")
    pg.pmx_quant_run(config(), x, q.view, s.view, rows, cols, transpose=transpose, rule=rule, **kw)
    sync()
    kp = mx.padded(length)
    return q.get().reshape(lines, kp // 2), s.get().reshape(kp // 128, lines, 4)


SHAPES = [(1, 1), (1, 128), (3, 31), (2, 33), (7, 129), (16, 256), (33, 200), (64, 128), (65, 640), (130, 1000),
          (257, 96), (300, 2049)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rule", ["ceil", "floor"])
def test_quant_equals_the_oracle(kind, transpose, rule):
    for i, (rows, cols) in enumerate(SHAPES):
        v, x = make(rows, cols, kind, 10 + i)
        q, s = quant(x, rows, cols, transpose, rule)
        qr, sr = mx.quant_mxfp4(v, rule, transpose)
        assert np.array_equal(s, sr), (rows, cols)
        assert np.array_equal(q, qr), (rows, cols)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
def test_quant_special_values(kind, transpose):
    for rows, cols in [(40, 300), (129, 64)]:
        v, x = make(rows, cols, kind, 5, special=True)
        for rule in ("ceil", "floor"):
            q, s = quant(x, rows, cols, transpose, rule)
            qr, sr = mx.quant_mxfp4(v, rule, transpose)
            assert np.array_equal(s, sr) and np.array_equal(q, qr), (rows, cols, rule)


@pytest.mark.parametrize("transpose", [False, True])
def test_quant_strided_and_unaligned_rows(transpose):
    for rows, cols, ld, off in [(37, 256, 264, 0), (37, 256, 257, 0), (37, 250, 264, 8), (64, 256, 256, 3),
                                (70, 128, 300, 1)]:
        for kind in ("bf16", "f32"):
            v, x = make(rows, cols, kind, 77)
            big = torch.full((off + rows * ld,), float("nan"), dtype=TYPES[kind], device="cuda:0")
            view = big[off:].as_strided((rows, cols), (ld, 1), big.storage_offset() + off)
            view.copy_(x)
            q, s = quant(view, rows, cols, transpose, "ceil")
            qr, sr = mx.quant_mxfp4(v, "ceil", transpose)
            assert np.array_equal(s, sr) and np.array_equal(q, qr), (rows, cols, ld, off, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_dequant_equals_the_oracle(kind):
    for rows, cols, ld in [(1, 1, 1), (3, 31, 31), (5, 128, 128), (33, 200, 208), (65, 1000, 1001), (130, 256, 264)]:
        rng = np.random.default_rng(rows)
        kp = mx.padded(cols)
        q = rng.integers(0, 256, (rows, kp // 2), np.uint8)
        s = rng.integers(100 if kind != "f16" else 113, 140, (kp // 128, rows, 4)).astype(np.uint8)
        s.reshape(-1)[::17] = 255
        if kind != "f16":
            s.reshape(-1)[5::19] = 0
            s.reshape(-1)[7::23] = 254
        y = torch.full((rows, ld), -7.0, dtype=TYPES[kind], device="cuda:0")
        Q, S = torch.from_numpy(q).to("cuda:0"), torch.from_numpy(s).to("cuda:0")
        note(f"pmx_dequant_run {rows}x{cols} ld={ld} {kind}")
        pg.pmx_dequant_run(config(), Q, S, y[:, :cols], rows, cols)
        sync()
        want = torch.from_numpy(mx.dequant_mxfp4(q, s, cols)).to(TYPES[kind])
        got = y.cpu()
        assert torch.equal(torch.nan_to_num(got[:, :cols].float(), nan=1e9), torch.nan_to_num(want.float(), nan=1e9))
        assert torch.equal(torch.signbit(got[:, :cols][want == 0]), torch.signbit(want[want == 0]))
        assert torch.all(got[:, cols:] == -7.0)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_dequant_every_code_and_scale(kind):
    """All sixteen codes under all 256 scale bytes: subnormal results rounded,
    results past the range infinite, byte 255 NaN."""
    q = np.zeros((256, 64), np.uint8)
    q[:, :16] = 0x11 * np.arange(16)
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)[None]
    y = torch.zeros((256, 32), dtype=TYPES[kind], device="cuda:0")
    note(f"pmx_dequant_run every code {kind}")
    pg.pmx_dequant_run(config(), dev_u8(q), dev_u8(s), y, 256, 32)
    sync()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(mx.dequant_mxfp4(q, s, 32)).to(TYPES[kind])
    got = y.cpu()
    assert torch.isnan(got[255]).all() and not torch.isnan(got[:255]).any()
    bits = torch.int32 if kind == "f32" else torch.int16
    assert torch.equal(got[:255].view(bits), want[:255].view(bits))


def test_no_rows_is_a_call_that_does_nothing():
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda:0")
    e = torch.zeros(0, dtype=torch.uint8, device="cuda:0")
    pg.pmx_quant_run(config(), x, e, e, 0, 64)
    pg.pmx_dequant_run(config(), e, e, x, 0, 64)
    sync()


def test_other_stream_and_graph_replays():
    """On a stream of the caller's, and captured: each replay after new data
    and eager work in between equals the eager result."""
    rows, cols = 200, 640
    nb = pg.mxfp4_bytes(rows, cols)
    _, x = make(rows, cols, "bf16", 1)
    q = torch.zeros(nb["Q"], dtype=torch.uint8, device="cuda:0")
    s = torch.zeros(nb["scale"], dtype=torch.uint8, device="cuda:0")
    y = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda:0")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        pg.pmx_quant_run(config(), x, q, s, rows, cols)
        st.synchronize()
        with torch.cuda.graph(g, stream=st):
            pg.pmx_quant_run(config(), x, q, s, rows, cols)
            pg.pmx_dequant_run(config(), q, s, y, rows, cols)
    for seed in range(3):
        v, fresh = make(rows, cols, "bf16", 40 + seed)
        x.copy_(fresh)
        q.zero_()
        sync("eager copies")
        g.replay()
        sync("replay")
        qr, sr = mx.quant_mxfp4(v)
        assert np.array_equal(q.cpu().numpy().reshape(qr.shape), qr)
        assert np.array_equal(s.cpu().numpy().reshape(sr.shape), sr)
        assert np.array_equal(y.double().cpu().numpy(), mx.dequant_mxfp4(qr, sr, cols))


def test_refusals():
    L, h = _abi.lib(), config().handle
    x = torch.zeros(64 * 128, dtype=torch.float32, device="cuda:0")
    q = torch.full((64 * 64,), 7, dtype=torch.uint8, device="cuda:0")
    s = torch.full((64 * 4,), 7, dtype=torch.uint8, device="cuda:0")
    a, b, c = x.data_ptr(), q.data_ptr(), s.data_ptr()

    def run(X=a, t=0, rows=64, cols=128, ld=128, tr=0, rule=0, Q=b, S=c):
        return L.pmx_quant_run(h, X, t, rows, cols, ld, tr, rule, Q, S, None)

    I, U = _abi.ERR_INVALID, _abi.ERR_UNSUPPORTED  # noqa: E741
    big = 1 << 40
    for bad in (dict(X=None), dict(Q=None), dict(S=None), dict(t=3), dict(t=-1), dict(rows=-1), dict(cols=0),
                dict(ld=127), dict(tr=2), dict(rule=2), dict(rows=big), dict(ld=big), dict(X=a + 2),
                dict(rows=1 << 22), dict(Q=a), dict(S=b), dict(X=(ctypes.c_char * 64)())):
        assert run(**bad) == I, bad
    assert run(rows=32, Q=b + 2) == U and run(rows=32, S=c + 1) == U

    def back(Q=b, S=c, rows=64, cols=128, Y=a, t=0, ld=128):
        return L.pmx_dequant_run(h, Q, S, rows, cols, Y, t, ld, None)

    for bad in (dict(Q=None), dict(S=None), dict(Y=None), dict(t=3), dict(rows=-1), dict(cols=0), dict(ld=100),
                dict(rows=1 << 22), dict(Y=b), dict(Y=a + 2)):
        assert back(**bad) == I, bad
    assert back(rows=32, Q=b + 1) == U
    sync()
    assert torch.all(q == 7) and torch.all(s == 7)
