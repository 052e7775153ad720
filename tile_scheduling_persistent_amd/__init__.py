"""Persistent tiled GEMM and persistent 2-D add with tile schedulers, and the
operators that make the block-scaled GEMMs' operands (MXFP4 and e4m3
quantisation, RMS norm with a quantised output), and layers of experts in e4m3
(tokens sorted to experts and back, their products, gated activation, gradients),
for AMD Instinct MI355X (gfx950).

A thin Python binding over the C ABI of libpgemm.so (include/pgemm.h): the
functions keep the C names, marshal torch device tensors (or raw device
pointers) and the current HIP stream, and raise PgemmError on a non-zero
status.  Every step of the hot path runs in the library's HIP kernels;
PyTorch only provides device memory and streams.
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _abi
from ._abi import PgemmError, status_str  # noqa: F401

SCHEDULERS = {
    "blocked": _abi.SCHED_BLOCKED,
    "interleaved": _abi.SCHED_INTERLEAVED,
    "grouped": _abi.SCHED_GROUPED,
    "work_stealing": _abi.SCHED_WORK_STEALING,
    "blocked_grouped": _abi.SCHED_BLOCKED_GROUPED,
    "stream_k": _abi.SCHED_STREAM_K,
    "work_stealing_xcc": _abi.SCHED_WORK_STEALING_XCC,
}
DTYPES = {
    "bf16_out_f32": _abi.BF16_OUT_F32,
    "bf16_out_bf16": _abi.BF16_OUT_BF16,
    "fp8_b128_out_bf16": _abi.FP8E4M3_B128_OUT_BF16,
    "mxfp4_out_bf16": _abi.MXFP4_OUT_BF16,
    "mxfp4_out_f32": _abi.MXFP4_OUT_F32,
}
SCALE_RULES = {"ceil": _abi.PMX_SCALE_CEIL, "floor": _abi.PMX_SCALE_FLOOR}
RMS_OUTPUTS = {"same": _abi.PRMS_OUT_SAME, "fp8_b128": _abi.PRMS_OUT_FP8_B128, "mxfp4": _abi.PRMS_OUT_MXFP4}

__all__ = ["Config", "pgemm_run", "pgemm_run_noalloc", "pgemm_run_grouped", "padd_run", "padd_run_multi", "plan_gemm", "plan_add", "SCHEDULERS",
           "pmx_quant_run", "pmx_dequant_run", "prms_run", "prms_grad_run", "mxfp4_bytes", "SCALE_RULES",
           "pmoe_sort_run", "pmoe_gather_run", "pmoe_combine_run", "pmoe_combine_grad_run", "pfp8_quant_run",
           "pfp8_quant_weights_run", "pgemm_run_experts", "pgemm_run_experts_wgrad", "pglu_run", "pglu_grad_run",
           "fp8_bytes", "fp8_weight_bytes", "RMS_OUTPUTS", "DTYPES", "PgemmError", "status_str", "make_args"]


def _check(where, code):
    if code != _abi.OK:
        raise PgemmError(where, code)


_DTYPES_OF = {}


def _torch_dtypes(names):
    t = _DTYPES_OF.get(names)
    if t is None:
        import torch
        t = _DTYPES_OF[names] = tuple(getattr(torch, n) for n in names if hasattr(torch, n))
    return t


# Element types the calls accept: operands per pgemm_dtype, outputs, adds.
_OPERAND = {_abi.BF16_OUT_F32: ("bfloat16",), _abi.BF16_OUT_BF16: ("bfloat16",),
            _abi.FP8E4M3_B128_OUT_BF16: ("uint8", "float8_e4m3fn"),
            _abi.MXFP4_OUT_BF16: ("uint8", "float4_e2m1fn_x2"), _abi.MXFP4_OUT_F32: ("uint8", "float4_e2m1fn_x2")}
_OUTPUT = {_abi.BF16_OUT_F32: ("float32",), _abi.BF16_OUT_BF16: ("bfloat16",),
           _abi.FP8E4M3_B128_OUT_BF16: ("bfloat16",),
           _abi.MXFP4_OUT_BF16: ("bfloat16",), _abi.MXFP4_OUT_F32: ("float32",)}
_SCALE = ("uint8", "float8_e8m0fnu")
_F32 = ("float32",)
_FP4 = ("uint8", "float4_e2m1fn_x2")


def gemm_bytes(M: int, N: int, K: int, dtype) -> dict:
    """Bytes each buffer of a GEMM call spans: A [M][K], B [K][N], C [M][N]
    and (block-scaled fp8) the scales [K/128][M] and [K/128][N]; MXFP4:
    A [M][K/2], B [N][K/2] and the scales [K/128][M][4] and [K/128][N][4]."""
    d = _dtype(dtype)
    if d in (_abi.MXFP4_OUT_BF16, _abi.MXFP4_OUT_F32):
        return {"A": M * (K // 2), "B": N * (K // 2), "C": M * N * (2 if d == _abi.MXFP4_OUT_BF16 else 4),
                "a_scale": (K // 128) * M * 4, "b_scale": (K // 128) * N * 4}
    esz = 1 if d == _abi.FP8E4M3_B128_OUT_BF16 else 2
    csz = 4 if d == _abi.BF16_OUT_F32 else 2
    out = {"A": M * K * esz, "B": K * N * esz, "C": M * N * csz}
    if d == _abi.FP8E4M3_B128_OUT_BF16:
        out["a_scale"] = (K // 128) * M
        out["b_scale"] = (K // 128) * N
    return out


# torch is imported by the first call that needs it; a short call would spend
# as long on import statements as on its checks.
_TENSOR = None
_RAW_STREAM = None


def _tensor_type():
    global _TENSOR, _RAW_STREAM
    import torch
    _RAW_STREAM = torch._C._cuda_getCurrentRawStream
    _TENSOR = torch.Tensor
    return _TENSOR


def _check_tensor(x, what, dtypes=None, nbytes=None):
    """Layout, element type and extent of a tensor argument (host-side checks,
    before any device is involved).  Raw int pointers pass unchecked: the
    library itself checks that every range lies inside one device allocation."""
    if isinstance(x, int):
        return
    if not isinstance(x, _TENSOR or _tensor_type()):
        raise TypeError(f"{what}: expected a torch tensor or an int device pointer")
    if not x.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous (row-major)")
    if dtypes is not None and nbytes != 0:  # an empty buffer is never accessed
        allowed = _torch_dtypes(dtypes)
        if x.dtype not in allowed:
            raise ValueError(f"{what}: dtype {x.dtype} not in {allowed}")
    if nbytes is not None and x.nbytes < nbytes:
        raise ValueError(f"{what}: tensor holds {x.nbytes} bytes, "
                         f"the call reads or writes {nbytes}")


def _dev(x, what):
    """Device pointer of a checked tensor argument (or a raw int pointer)."""
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"{what}: tensor must live on the GPU")
    return x.data_ptr()


def _ptr(x, what, dtypes=None, nbytes=None):
    """Device pointer of a torch tensor (contiguous, on a GPU, of an allowed
    dtype, at least nbytes long) or a raw int pointer."""
    if (type(x) is _TENSOR and x.is_cuda and x.is_contiguous() and (nbytes is None or x.nbytes >= nbytes)
            and (dtypes is None or x.dtype in _torch_dtypes(dtypes))):
        return x.data_ptr()
    # what the short form does not take: named errors, raw pointers, empty buffers
    _check_tensor(x, what, dtypes, nbytes)
    return _dev(x, what)


def _stream(stream, device=None):
    """Raw HIP stream handle: `stream` itself (an int or a torch stream), else
    torch's current stream on `device` (the config's device)."""
    if stream is None:
        if device is not None:
            if _RAW_STREAM is None:
                _tensor_type()
            return _RAW_STREAM(device)
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _sched(s):
    return SCHEDULERS[s] if isinstance(s, str) else int(s)


def _dtype(d):
    return DTYPES[d] if isinstance(d, str) else int(d)


ORDERS = {"default": _abi.ORDER_DEFAULT, "dispatch": _abi.ORDER_DISPATCH, "xcd_major": _abi.ORDER_XCD_MAJOR}
PIPELINES = {"default": _abi.PIPELINE_DEFAULT, "four_wave": _abi.PIPELINE_FOUR_WAVE,
             "pingpong": _abi.PIPELINE_PINGPONG}


def make_args(tile=None, group_size=0, grid=0, claim_chunk=0, a_scale=None, b_scale=None,
              debug_flags=0, straggler_program=-1, straggler_ns=0, pipeline="default",
              program_order="default"):
    a = _abi.pgemm_args()
    # a new structure holds zeros; a field costs as much to set as a check
    if tile is not None:
        a.tile_m, a.tile_n, a.tile_k = (tuple(tile) + (0,))[:3]
    if group_size:
        a.group_size = group_size
    if grid:
        a.grid = grid
    if claim_chunk:
        a.claim_chunk = claim_chunk
    if a_scale is not None:
        a.a_scale = _ptr(a_scale, "a_scale", _SCALE)
    if b_scale is not None:
        a.b_scale = _ptr(b_scale, "b_scale", _SCALE)
    a._scales = (a_scale, b_scale)  # checked against M, N, K when the call is made
    if debug_flags:
        a.debug_flags = debug_flags
    a.straggler_program = straggler_program
    if straggler_ns:
        a.straggler_ns = straggler_ns
    a.pipeline = PIPELINES[pipeline] if isinstance(pipeline, str) else int(pipeline)
    a.program_order = ORDERS[program_order] if isinstance(program_order, str) else int(program_order)
    return a


class Config:
    """pgemm_config: device facts plus the reusable per-XCD counters."""

    def __init__(self, device: int = 0, max_xcds: int = 0):
        h = ctypes.c_void_p()
        _check("pgemm_config_create", _abi.lib().pgemm_config_create(int(device), int(max_xcds),
                                                                      ctypes.byref(h)))
        self.handle = h
        self.device = int(device)
        info = _abi.pgemm_info()
        _check("pgemm_config_query", _abi.lib().pgemm_config_query(h, ctypes.byref(info)))
        self.info = {
            "num_cus": info.num_cus, "num_xcds": info.num_xcds,
            "counter_capacity": info.counter_capacity, "wall_clock_khz": info.wall_clock_khz,
            "clock_khz": info.clock_khz, "lds_bytes_per_cu": info.lds_bytes_per_cu,
            "arch": info.arch.decode(),
        }

    def close(self):
        if self.handle is not None:
            _abi.lib().pgemm_config_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def witness_enable(self, max_tiles: int, max_programs: int):
        _check("pgemm_witness_enable",
               _abi.lib().pgemm_witness_enable(self.handle, int(max_tiles), int(max_programs)))

    def witness_read(self, tiles: int, programs: int, stream=None):
        out = {
            "visits": np.zeros(tiles, np.int32), "owner": np.zeros(tiles, np.int32),
            "order": np.zeros(tiles, np.int32), "t_start": np.zeros(programs, np.int64),
            "t_end": np.zeros(programs, np.int64), "hw_id": np.zeros(programs, np.int32),
            "n_tiles": np.zeros(programs, np.int32),
            "counters": np.zeros(self.info["counter_capacity"], np.int32),
            "cycles": np.zeros(programs, np.int64),
            "claims": np.zeros((programs, _abi.MAX_STEAL_COUNTERS), np.int32),
        }
        w = _abi.pgemm_witness()
        for k in ("visits", "owner", "order", "t_start", "t_end", "hw_id", "n_tiles", "counters",
                  "cycles", "claims"):
            setattr(w, k, out[k].ctypes.data)
        w.tiles = tiles
        w.programs = programs
        _check("pgemm_witness_read",
               _abi.lib().pgemm_witness_read(self.handle, ctypes.byref(w), _stream(stream, self.device)))
        return out


def pgemm_run(cfg: Config, A, B, C, M: int, N: int, K: int, dtype, sched, args=None,
              stream=None):
    """C[M][N] = A[M][K] . B[K][N] on the GPU (asynchronous on `stream`)."""
    code = _abi.lib().pgemm_run(cfg.handle, *_gemm_ptrs(A, B, C, M, N, K, dtype, args),
                                int(M), int(N), int(K), _dtype(dtype), _sched(sched),
                                ctypes.byref(args) if args is not None else None, _stream(stream, cfg.device))
    _check("pgemm_run", code)


def pgemm_run_noalloc(cfg: Config, A, B, C, M: int, N: int, K: int, dtype, sched, args=None,
                      stream=None):
    """pgemm_run without any device allocation: the work-stealing counters and
    the stream-K partial sums come from the library's static per-device
    scratch (calls on one GPU must not overlap)."""
    code = _abi.lib().pgemm_run_noalloc(cfg.handle, *_gemm_ptrs(A, B, C, M, N, K, dtype, args),
                                        int(M), int(N), int(K), _dtype(dtype), _sched(sched),
                                        ctypes.byref(args) if args is not None else None,
                                        _stream(stream, cfg.device))
    _check("pgemm_run_noalloc", code)


def _gemm_ptrs(A, B, C, M, N, K, dtype, args, where=""):
    """Device pointers of a GEMM's A, B, C after every host-side check of
    all its buffers (element types, extents, the scales passed in args)."""
    d = _dtype(dtype)
    nb = gemm_bytes(int(M), int(N), int(K), d) if d in _OPERAND else {}
    if args is not None and "a_scale" in nb:
        for name, t in zip(("a_scale", "b_scale"), getattr(args, "_scales", (None, None))):
            if t is not None:
                _check_tensor(t, name + where, _SCALE, nb[name])
    ops, outs = _OPERAND.get(d), _OUTPUT.get(d)
    _check_tensor(A, "A" + where, ops, nb.get("A"))
    _check_tensor(B, "B" + where, ops, nb.get("B"))
    _check_tensor(C, "C" + where, outs, nb.get("C"))
    return _dev(A, "A" + where), _dev(B, "B" + where), _dev(C, "C" + where)


def _plan_dict(pl) -> dict:
    return {"grid": pl.grid, "occupancy": pl.occupancy, "tiles": pl.tiles,
            "tile": (pl.tile_m, pl.tile_n, pl.tile_k), "threads": pl.threads,
            "lds_bytes": pl.lds_bytes, "kernel": _abi.KERNEL_NAMES.get(pl.kernel, str(pl.kernel)),
            "xcd_major": bool(pl.xcd_major)}


def plan_gemm(cfg: Config, M: int, N: int, K: int, dtype, sched, args=None, A=None, B=None,
              C=None) -> dict:
    """The launch pgemm_run would make (grid, occupancy, tiles, kernel, ...)."""
    pl = _abi.pgemm_plan()
    code = _abi.lib().pgemm_plan_gemm(
        cfg.handle, A.data_ptr() if A is not None else None, B.data_ptr() if B is not None else None,
        C.data_ptr() if C is not None else None, int(M), int(N), int(K), _dtype(dtype),
        _sched(sched), ctypes.byref(args) if args is not None else None, ctypes.byref(pl))
    _check("pgemm_plan_gemm", code)
    return _plan_dict(pl)


def plan_add(cfg: Config, rows: int, cols: int, tile_rows: int, tile_cols: int, sched, args=None,
             X=None, Y=None, C=None) -> dict:
    """The launch padd_run would make."""
    pl = _abi.pgemm_plan()
    code = _abi.lib().pgemm_plan_add(
        cfg.handle, X.data_ptr() if X is not None else None, Y.data_ptr() if Y is not None else None,
        C.data_ptr() if C is not None else None, int(rows), int(cols), int(tile_rows),
        int(tile_cols), _sched(sched), ctypes.byref(args) if args is not None else None,
        ctypes.byref(pl))
    _check("pgemm_plan_add", code)
    return _plan_dict(pl)


def padd_run(cfg: Config, X, Y, C, rows: int, cols: int, tile_rows: int, tile_cols: int, sched,
             args=None, stream=None):
    """C = X + Y (fp32) over tile_rows x tile_cols tiles (asynchronous on `stream`)."""
    nb = int(rows) * int(cols) * 4
    code = _abi.lib().padd_run(cfg.handle, _ptr(X, "X", _F32, nb), _ptr(Y, "Y", _F32, nb),
                               _ptr(C, "C", _F32, nb),
                               int(rows), int(cols), int(tile_rows), int(tile_cols), _sched(sched),
                               ctypes.byref(args) if args is not None else None, _stream(stream, cfg.device))
    _check("padd_run", code)


def padd_run_multi(cfg: Config, problems, tile_rows: int, tile_cols: int, sched, args=None,
                   stream=None):
    """Several adds C_g = X_g + Y_g (fp32) in one persistent launch; `problems`
    is a sequence of (X, Y, C, rows, cols)."""
    n = len(problems)
    arr = (_abi.padd_problem * max(n, 1))()
    for g, (X, Y, C, rows, cols) in enumerate(problems):
        nb = int(rows) * int(cols) * 4
        arr[g].X = _ptr(X, f"X[{g}]", _F32, nb)
        arr[g].Y = _ptr(Y, f"Y[{g}]", _F32, nb)
        arr[g].C = _ptr(C, f"C[{g}]", _F32, nb)
        arr[g].rows = int(rows)
        arr[g].cols = int(cols)
    code = _abi.lib().padd_run_multi(cfg.handle, arr, n, int(tile_rows), int(tile_cols), _sched(sched),
                                     ctypes.byref(args) if args is not None else None, _stream(stream, cfg.device))
    _check("padd_run_multi", code)


def pgemm_run_grouped(cfg: Config, problems, dtype, sched, args=None, stream=None):
    """Several GEMMs C_g = A_g . B_g in one persistent launch; `problems` is a
    sequence of (A, B, C, M, N, K), or (A, B, C, M, N, K, a_scale, b_scale)
    for block-scaled fp8 and MXFP4."""
    n = len(problems)
    arr = (_abi.pgemm_problem * max(n, 1))()
    for g, pr in enumerate(problems):
        A, B, C, M, N, K = pr[:6]
        arr[g].A, arr[g].B, arr[g].C = _gemm_ptrs(A, B, C, M, N, K, dtype, None, f"[{g}]")
        arr[g].M, arr[g].N, arr[g].K = int(M), int(N), int(K)
        if len(pr) == 8:
            nb = gemm_bytes(int(M), int(N), int(K), dtype)
            if "a_scale" not in nb:  # the scales of an unscaled type are ignored
                nb = {"a_scale": 0, "b_scale": 0}
            arr[g].a_scale = _ptr(pr[6], f"a_scale[{g}]", _SCALE, nb["a_scale"])
            arr[g].b_scale = _ptr(pr[7], f"b_scale[{g}]", _SCALE, nb["b_scale"])
    code = _abi.lib().pgemm_run_grouped(cfg.handle, arr, n, _dtype(dtype), _sched(sched),
                                        ctypes.byref(args) if args is not None else None,
                                        _stream(stream, cfg.device))
    _check("pgemm_run_grouped", code)


def mxfp4_bytes(rows: int, cols: int) -> dict:
    """Bytes of an MXFP4 operand of a [rows][cols] matrix: codes Q [rows][Kp/2]
    and scale [Kp/128][rows][4], Kp = cols rounded up to 128."""
    kp = -(-cols // 128) * 128
    return {"Q": rows * (kp // 2), "scale": (kp // 128) * rows * 4}


_ELEM = {}


def _elem(x, what, given=None):
    """PMX_* element type of a tensor argument (raw pointers: `given`)."""
    t = _ELEM.get(getattr(x, "dtype", None))
    if t is not None:
        return t
    if isinstance(x, int):
        if given is None:
            raise ValueError(f"{what}: a raw pointer needs its element type")
        return int(given)
    if not _ELEM:
        import torch
        _ELEM.update({torch.float32: _abi.PMX_F32, torch.bfloat16: _abi.PMX_BF16, torch.float16: _abi.PMX_F16})
    t = _ELEM.get(getattr(x, "dtype", None))
    if t is None:
        raise ValueError(f"{what}: expected a float32, bfloat16 or float16 tensor")
    return t


def _matrix(x, what, rows, cols, ld=None):
    """(device pointer, row stride) of a [rows][cols] matrix: a 2-D tensor with
    dense rows, a contiguous tensor of at least rows * cols elements, or a raw
    pointer with its row stride `ld`."""
    if ld is None and type(x) is _TENSOR and x.is_cuda and x.shape == (rows, cols):
        step = x.stride()
        if step[1] == 1 or cols == 1:
            return x.data_ptr(), step[0] if rows > 1 else cols
    if isinstance(x, int):
        return x, int(cols if ld is None else ld)
    if not isinstance(x, _TENSOR or _tensor_type()):
        raise TypeError(f"{what}: expected a torch tensor or an int device pointer")
    if ld is None and x.shape == (rows, cols) and (x.stride(1) == 1 or cols == 1):
        return _dev(x, what), int(x.stride(0)) if rows > 1 else cols
    ld = cols if ld is None else int(ld)
    need = ((rows - 1) * ld + cols if rows else 0) * x.element_size()
    _check_tensor(x, what, None, need)
    return _dev(x, what), ld


def pmx_quant_run(cfg: Config, X, Q, scale, rows: int, cols: int, transpose=False, rule="ceil", ldx=None,
                  x_type=None, stream=None):
    """MXFP4 codes Q and scale bytes of X [rows][cols] (float32, bfloat16 or
    float16), blocks of 32 along the columns, or with `transpose` along the
    rows (the operand of X^T), asynchronous on `stream`.  rule: "ceil" (no value
    saturates) or "floor" (OCP MX)."""
    rows, cols = int(rows), int(cols)
    t = _elem(X, "X", x_type)
    nb = mxfp4_bytes(cols, rows) if transpose else mxfp4_bytes(rows, cols)
    x, ld = _matrix(X, "X", rows, cols, ldx)
    code = _abi.lib().pmx_quant_run(cfg.handle, x, t, rows, cols, ld, int(bool(transpose)),
                                    SCALE_RULES[rule] if isinstance(rule, str) else int(rule),
                                    _ptr(Q, "Q", _FP4, nb["Q"]), _ptr(scale, "scale", _SCALE, nb["scale"]),
                                    _stream(stream, cfg.device))
    _check("pmx_quant_run", code)


def pmx_dequant_run(cfg: Config, Q, scale, Y, rows: int, cols: int, ldy=None, y_type=None, stream=None):
    """Y [rows][cols] (float32, bfloat16 or float16) = the values of an MXFP4
    operand (asynchronous on `stream`)."""
    rows, cols = int(rows), int(cols)
    t = _elem(Y, "Y", y_type)
    nb = mxfp4_bytes(rows, cols)
    y, ld = _matrix(Y, "Y", rows, cols, ldy)
    code = _abi.lib().pmx_dequant_run(cfg.handle, _ptr(Q, "Q", _FP4, nb["Q"]),
                                      _ptr(scale, "scale", _SCALE, nb["scale"]), rows, cols, y, t, ld,
                                      _stream(stream, cfg.device))
    _check("pmx_dequant_run", code)


def prms_run(cfg: Config, X, W, Y, rows: int, cols: int, eps: float = 1e-6, R=None, H=None, out="same",
             y_scale=None, rstd=None, stream=None):
    """h = X + R (into H; without R, h = X), Y = h / sqrt(mean(h^2) + eps) * W
    by rows (asynchronous on `stream`).  out: "same" (Y of X's type), "fp8_b128"
    (Y e4m3 [rows][Kp], y_scale [Kp/128][rows]: the A operand of a block-scaled
    fp8 GEMM) or "mxfp4" (Y codes [rows][Kp/2], y_scale [Kp/128][rows][4]), Kp =
    cols rounded up to 128.  rstd (float32 [rows]) takes the rows' factors for
    prms_grad_run.  H may be R (or X), Y (out="same") may be X.  The matrices and
    W are tensors (their types are the call's types)."""
    rows, cols = int(rows), int(cols)
    o = RMS_OUTPUTS[out] if isinstance(out, str) else int(out)
    xt, wt = _elem(X, "X"), _elem(W, "W")
    x, ldx = _matrix(X, "X", rows, cols)
    r = h = s = t = None
    rt, ldr, ldh, ldy = xt, cols, cols, cols
    if R is not None:
        rt = _elem(R, "R")
        r, ldr = _matrix(R, "R", rows, cols)
    if H is not None:
        if _elem(H, "H") != rt:
            raise ValueError("H: must have the type of R")
        h, ldh = _matrix(H, "H", rows, cols)
    if o == _abi.PRMS_OUT_SAME:
        if _elem(Y, "Y") != xt:
            raise ValueError("Y: must have the type of X")
        y, ldy = _matrix(Y, "Y", rows, cols)
    else:
        kp = -(-cols // 128) * 128
        if o == _abi.PRMS_OUT_FP8_B128:
            y = _ptr(Y, "Y", ("uint8", "float8_e4m3fn"), rows * kp)
            nb = kp // 128 * rows
        else:
            y = _ptr(Y, "Y", _FP4, rows * kp // 2)
            nb = kp // 128 * rows * 4
        if y_scale is None:
            raise ValueError("y_scale: a quantised output needs its scales")
        s = _ptr(y_scale, "y_scale", _SCALE, nb)
    if rstd is not None:
        t = _ptr(rstd, "rstd", _F32, rows * 4)
    code = _abi.lib().prms_run(cfg.handle, x, xt, ldx, r, rt, ldr, _ptr(W, "W", None, cols * (4 if wt == 0 else 2)), wt,
                               float(eps), rows, cols, h, ldh, o, y, ldy, s, t, _stream(stream, cfg.device))
    _check("prms_run", code)


def prms_grad_run(cfg: Config, dY, H, W, rstd, dX, dW, rows: int, cols: int, dH=None, stream=None):
    """Gradients of prms_run (asynchronous on `stream`): dX [rows][cols] of H's
    type (the gradient of X and of R), dW float32 [cols] (None: not wanted).  H:
    the forward's h; dH: the gradient that reaches h past the norm (None: none).
    Calls with dW share the config's buffer of partial sums: on several streams
    each waits for the one before (the first on a second stream synchronises the
    device); captured ones of one config must not be replayed at the same time."""
    rows, cols = int(rows), int(cols)
    yt, ht, wt = _elem(dY, "dY"), _elem(H, "H"), _elem(W, "W")
    if _elem(dX, "dX") != ht or (dH is not None and _elem(dH, "dH") != ht):
        raise ValueError("dX, dH: must have the type of H")
    dy, ldy = _matrix(dY, "dY", rows, cols)
    h, ldh = _matrix(H, "H", rows, cols)
    dx, ldx = _matrix(dX, "dX", rows, cols)
    dh, ldd = _matrix(dH, "dH", rows, cols) if dH is not None else (None, cols)
    code = _abi.lib().prms_grad_run(cfg.handle, dy, yt, ldy, h, ht, ldh, dh, ldd,
                                    _ptr(W, "W", None, cols * (4 if wt == 0 else 2)), wt,
                                    _ptr(rstd, "rstd", _F32, rows * 4), rows, cols, dx, ldx,
                                    _ptr(dW, "dW", _F32, cols * 4) if dW is not None else None,
                                    _stream(stream, cfg.device))
    _check("prms_grad_run", code)


# ------------------------------------------------------------- layers of experts

_I32 = ("int32",)
_FP8 = ("uint8", "float8_e4m3fn")


def fp8_bytes(rows: int, cols: int) -> dict:
    """Bytes of an e4m3 operand of a [rows][cols] matrix: Q [rows][Kp] and scale
    [Kp/128][rows], Kp = cols rounded up to 128."""
    kp = -(-cols // 128) * 128
    return {"Q": rows * kp, "scale": kp // 128 * rows}


def fp8_weight_bytes(experts: int, rows: int, cols: int) -> dict:
    """Bytes of e4m3 weights [experts][rows][cols]: Q [experts][rows][Kp], scale
    [experts][Rp/128][Kp/128], and the transposed Qt [experts][cols][Rp], scale_t
    [experts][Kp/128][Rp/128]."""
    rp, kp = -(-rows // 128) * 128, -(-cols // 128) * 128
    s = experts * (rp // 128) * (kp // 128)
    return {"Q": experts * rows * kp, "scale": s, "Qt": experts * cols * rp, "scale_t": s}


def _opt(x, what, dtypes, nbytes):
    return None if x is None else _ptr(x, what, dtypes, nbytes)


def _out_of(out):
    return RMS_OUTPUTS[out] if isinstance(out, str) else int(out)


def _rows_out(out, Y, what, x_type, scale, rows, cols):
    """(pointer, row stride, scale pointer) of an output under `out`."""
    if out == _abi.PRMS_OUT_FP8_B128:
        nb = fp8_bytes(rows, cols)
        if scale is None:
            raise ValueError(f"{what}: a quantised output needs its scales")
        return _ptr(Y, what, _FP8, nb["Q"]), cols, _ptr(scale, what + " scale", _SCALE, nb["scale"])
    if out == _abi.PRMS_OUT_SAME and not isinstance(Y, int) and _elem(Y, what) != x_type:
        raise ValueError(f"{what}: must have the input's type")
    y, ld = _matrix(Y, what, rows, cols)
    return y, ld, None


def pmoe_sort_run(cfg: Config, ids, place, order, offsets, tokens: int, topk: int, experts: int, ids_type=None,
                  stream=None):
    """Slots (token, choice) sorted by expert (asynchronous on `stream`): ids
    [tokens][topk] int32 or int64 (outside [0, experts): no row) to place [tokens][topk]
    (a slot's row or -1), order [tokens * topk] (a row's slot, -1 behind the last)
    and offsets [experts + 1], all int32.  Rows of an expert keep their slots' order."""
    tokens, topk, experts = int(tokens), int(topk), int(experts)
    if ids_type is None:
        ids_type = _abi.PMOE_I64 if str(getattr(ids, "dtype", "")) == "torch.int64" else _abi.PMOE_I32
    slots = tokens * topk
    code = _abi.lib().pmoe_sort_run(
        cfg.handle, _ptr(ids, "ids", ("int64",) if ids_type == _abi.PMOE_I64 else _I32, slots * (8 if ids_type else 4)),
        ids_type, tokens, topk, experts, _ptr(place, "place", _I32, slots * 4), _ptr(order, "order", _I32, slots * 4),
        _ptr(offsets, "offsets", _I32, (experts + 1) * 4), _stream(stream, cfg.device))
    _check("pmoe_sort_run", code)


def pmoe_gather_run(cfg: Config, X, order, Y, tokens: int, topk: int, cols: int, out="same", y_scale=None, stream=None):
    """Y[r] = X[order[r] / topk] for the tokens * topk rows (asynchronous on
    `stream`): X [tokens][cols], Y of X's type or (out="fp8_b128") e4m3 with y_scale.
    Rows without a slot are left as they were."""
    tokens, topk, cols = int(tokens), int(topk), int(cols)
    o, t, slots = _out_of(out), _elem(X, "X"), int(tokens) * int(topk)
    x, ldx = _matrix(X, "X", tokens, cols)
    y, ldy, s = _rows_out(o, Y, "Y", t, y_scale, slots, cols)
    code = _abi.lib().pmoe_gather_run(cfg.handle, x, t, ldx, _ptr(order, "order", _I32, slots * 4), tokens, topk, cols, o,
                                      y, ldy, s, _stream(stream, cfg.device))
    _check("pmoe_gather_run", code)


def pmoe_combine_run(cfg: Config, X, place, Y, tokens: int, topk: int, cols: int, weights=None, R=None, stream=None):
    """Y[t] = R[t] + sum over j of weights[t][j] * X[place[t][j]] (asynchronous on
    `stream`): X [tokens * topk][cols], weights float32 (None: ones), R (None: none)
    and Y [tokens][cols] of X's type or float32.  Y may be R."""
    tokens, topk, cols = int(tokens), int(topk), int(cols)
    t, yt, slots = _elem(X, "X"), _elem(Y, "Y"), int(tokens) * int(topk)
    x, ldx = _matrix(X, "X", slots, cols)
    y, ldy = _matrix(Y, "Y", tokens, cols)
    r, ldr = None, cols
    if R is not None:
        if _elem(R, "R") != yt:
            raise ValueError("R: must have the type of Y")
        r, ldr = _matrix(R, "R", tokens, cols)
    code = _abi.lib().pmoe_combine_run(cfg.handle, x, t, ldx, _ptr(place, "place", _I32, slots * 4),
                                       _opt(weights, "weights", _F32, slots * 4), r, ldr, y, yt, ldy, tokens, topk, cols,
                                       _stream(stream, cfg.device))
    _check("pmoe_combine_run", code)


def pmoe_combine_grad_run(cfg: Config, dY, X, place, order, dX, tokens: int, topk: int, cols: int, weights=None, dW=None,
                          out="same", dx_scale=None, stream=None):
    """Gradients of pmoe_combine_run (asynchronous on `stream`): dX[r] = weights *
    dY[token] by rows, of dY's type or (out="fp8_b128") e4m3 with dx_scale, and dW
    float32 [tokens][topk] (None: not wanted, X may be None).  Rows without a slot are
    left as they were."""
    tokens, topk, cols = int(tokens), int(topk), int(cols)
    o, t, slots = _out_of(out), _elem(dY, "dY"), int(tokens) * int(topk)
    d, ldy = _matrix(dY, "dY", tokens, cols)
    x, ldx = None, cols
    if dW is not None:
        if _elem(X, "X") != t:
            raise ValueError("X: must have the type of dY")
        x, ldx = _matrix(X, "X", slots, cols)
    dx, lddx, s = _rows_out(o, dX, "dX", t, dx_scale, slots, cols)
    code = _abi.lib().pmoe_combine_grad_run(
        cfg.handle, d, t, ldy, x, ldx, _ptr(place, "place", _I32, slots * 4), _ptr(order, "order", _I32, slots * 4),
        _opt(weights, "weights", _F32, slots * 4), tokens, topk, cols, o, dx, lddx, s, _opt(dW, "dW", _F32, slots * 4),
        _stream(stream, cfg.device))
    _check("pmoe_combine_grad_run", code)


def pfp8_quant_run(cfg: Config, X, Q, scale, rows: int, cols: int, ldx=None, x_type=None, stream=None):
    """e4m3 operand Q [rows][Kp] of X [rows][cols] (float32, bfloat16 or float16),
    scale [Kp/128][rows] (asynchronous on `stream`)."""
    rows, cols = int(rows), int(cols)
    t, nb = _elem(X, "X", x_type), fp8_bytes(rows, cols)
    x, ld = _matrix(X, "X", rows, cols, ldx)
    code = _abi.lib().pfp8_quant_run(cfg.handle, x, t, rows, cols, ld, _ptr(Q, "Q", _FP8, nb["Q"]),
                                     _ptr(scale, "scale", _SCALE, nb["scale"]), _stream(stream, cfg.device))
    _check("pfp8_quant_run", code)


def pfp8_quant_weights_run(cfg: Config, W, Q, scale, experts: int, rows: int, cols: int, Qt=None, scale_t=None,
                           w_type=None, stream=None):
    """e4m3 weights Q [experts][rows][Kp] of W [experts][rows][cols] with one scale
    per block of 128 x 128, scale [experts][Rp/128][Kp/128], and with Qt
    [experts][cols][Rp] and scale_t [experts][Kp/128][Rp/128] the transposed weights
    (asynchronous on `stream`)."""
    experts, rows, cols = int(experts), int(rows), int(cols)
    t, nb = _elem(W, "W", w_type), fp8_weight_bytes(experts, rows, cols)
    code = _abi.lib().pfp8_quant_weights_run(
        cfg.handle, _ptr(W, "W", None, experts * rows * cols * (4 if t == 0 else 2)), t, experts, rows, cols,
        _ptr(Q, "Q", _FP8, nb["Q"]), _ptr(scale, "scale", _SCALE, nb["scale"]), _opt(Qt, "Qt", _FP8, nb["Qt"]),
        _opt(scale_t, "scale_t", _SCALE, nb["scale_t"]), _stream(stream, cfg.device))
    _check("pfp8_quant_weights_run", code)


def pgemm_run_experts(cfg: Config, A, B, C, rows: int, N: int, K: int, a_scale, b_scale, experts: int = 1, offsets=None,
                      c_type=None, stream=None):
    """C[r] = A[r] . B[e]^T, e the expert of row r by the device's offsets
    (asynchronous on `stream`): A e4m3 [rows][K] with a_scale [K/128][rows], B e4m3
    weights [experts][N][K] with b_scale, C [rows][N] bfloat16 or float32.  Rows of no
    expert are left as they were."""
    rows, N, K, experts = int(rows), int(N), int(K), int(experts)
    t = _elem(C, "C", c_type)
    nb = fp8_weight_bytes(experts, N, K)
    code = _abi.lib().pgemm_run_experts(
        cfg.handle, _ptr(A, "A", _FP8, rows * K), _ptr(a_scale, "a_scale", _SCALE, K // 128 * rows),
        _ptr(B, "B", _FP8, nb["Q"]), _ptr(b_scale, "b_scale", _SCALE, nb["scale"]),
        _ptr(C, "C", None, rows * N * (4 if t == 0 else 2)), t, rows, N, K, experts,
        _opt(offsets, "offsets", _I32, (experts + 1) * 4), _stream(stream, cfg.device))
    _check("pgemm_run_experts", code)


def pgemm_run_experts_wgrad(cfg: Config, D, A, dB, rows: int, N: int, K: int, a_scale, d_scale=None, experts: int = 1,
                            offsets=None, base=None, stream=None):
    """dB[e] = base[e] + sum over the rows r of expert e of D[r]^T A[r] (asynchronous
    on `stream`): D [rows][N] bfloat16, or e4m3 with d_scale; A e4m3 [rows][Kp] with
    a_scale; base (None: zeros) and dB [experts][N][K] bfloat16 or float32.  base may
    be dB."""
    rows, N, K, experts = int(rows), int(N), int(K), int(experts)
    if d_scale is not None:
        nb = fp8_bytes(rows, N)
        d, ldd, dt = _ptr(D, "D", _FP8, nb["Q"]), N, _abi.PMX_FP8_B128
        ds = _ptr(d_scale, "d_scale", _SCALE, nb["scale"])
    else:
        dt, ds = _elem(D, "D"), None
        d, ldd = _matrix(D, "D", rows, N)
    bt, nb = _elem(dB, "dB"), fp8_bytes(rows, K)
    size = experts * N * K * (4 if bt == 0 else 2)
    if base is not None and _elem(base, "base") != bt:
        raise ValueError("base: must have the type of dB")
    code = _abi.lib().pgemm_run_experts_wgrad(
        cfg.handle, d, dt, ldd, ds, _ptr(A, "A", _FP8, nb["Q"]), _ptr(a_scale, "a_scale", _SCALE, nb["scale"]),
        _opt(base, "base", None, size), _ptr(dB, "dB", None, size), bt, rows, N, K, experts,
        _opt(offsets, "offsets", _I32, (experts + 1) * 4), _stream(stream, cfg.device))
    _check("pgemm_run_experts_wgrad", code)


def pglu_run(cfg: Config, X, Y, rows: int, cols: int, out="same", y_scale=None, kept=None, kept_scale=None, valid=None,
             stream=None):
    """Y = silu(g) * u of X = [g | u] [rows][2 * cols] (asynchronous on `stream`), of
    X's type or (out="fp8_b128") e4m3 with y_scale.  kept [rows][2][Kp] and kept_scale
    [2][Kp/128][rows] take g and u in e4m3 for pglu_grad_run.  valid (int32 [1], on the
    device): rows at or past it are left as they were."""
    rows, cols = int(rows), int(cols)
    o, t = _out_of(out), _elem(X, "X")
    x, ldx = _matrix(X, "X", rows, 2 * cols)
    y, ldy, s = _rows_out(o, Y, "Y", t, y_scale, rows, cols)
    nb = fp8_bytes(rows, -(-cols // 128) * 256)
    code = _abi.lib().pglu_run(cfg.handle, x, t, ldx, rows, cols, _opt(valid, "valid", _I32, 4), o, y, ldy, s,
                               _opt(kept, "kept", _FP8, nb["Q"]), _opt(kept_scale, "kept_scale", _SCALE, nb["scale"]),
                               _stream(stream, cfg.device))
    _check("pglu_run", code)


def pglu_grad_run(cfg: Config, dY, X, dX, rows: int, cols: int, x_scale=None, out="same", dx_scale=None, valid=None,
                  stream=None):
    """Gradient of pglu_run (asynchronous on `stream`): dY [rows][cols]; X the
    forward's X of dY's type, or what it kept with x_scale = kept_scale; dX = [dg | du]
    [rows][2 * cols] of dY's type or (out="fp8_b128", cols a multiple of 128) e4m3 with
    dx_scale."""
    rows, cols = int(rows), int(cols)
    o, t = _out_of(out), _elem(dY, "dY")
    d, ldy = _matrix(dY, "dY", rows, cols)
    if x_scale is not None:
        nb = fp8_bytes(rows, -(-cols // 128) * 256)
        x, ldx, xs = _ptr(X, "X", _FP8, nb["Q"]), 2 * cols, _ptr(x_scale, "x_scale", _SCALE, nb["scale"])
    else:
        if _elem(X, "X") != t:
            raise ValueError("X: must have the type of dY")
        x, ldx = _matrix(X, "X", rows, 2 * cols)
        xs = None
    dx, lddx, s = _rows_out(o, dX, "dX", t, dx_scale, rows, 2 * cols)
    code = _abi.lib().pglu_grad_run(cfg.handle, d, t, ldy, x, ldx, xs, rows, cols, _opt(valid, "valid", _I32, 4), o, dx,
                                    lddx, s, _stream(stream, cfg.device))
    _check("pglu_grad_run", code)
