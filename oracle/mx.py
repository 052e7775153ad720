"""MXFP4 operands, their product, and the RMS norm that makes operands, in 64
bits from the definitions (loops over blocks' values, searched tables).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

* e2m1 (OCP Microscaling Formats v1.0): S.EE.M, bias 1: magnitudes 0, 0.5, 1,
  1.5, 2, 3, 4, 6.  A scale byte b stands for 2**(b - 127), 255 for NaN.
* An MXFP4 operand of a [rows][K] matrix: codes [rows][Kp/2] (Kp = K rounded up
  to 128, even k in the low nibble), scales [Kp/128][rows][4].
* Scale exponent of a block with largest magnitude amax: "ceil" the smallest e
  with amax <= top * 2**e, "floor" floor(log2(amax)) - emax; clamped to
  [-127, 127].  Zero blocks: byte 0.  Blocks with an infinity or NaN: byte 255
  and zero codes.
"""
from __future__ import annotations

import numpy as np

from .codecs import E4M3_TABLE, e8m0_to_f64

E2M1_MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_TABLE = np.concatenate([E2M1_MAGNITUDES, -E2M1_MAGNITUDES])
E4M3_MAGNITUDES = E4M3_TABLE[:127]          # codes 0 .. 126, ascending to 448


def padded(n: int) -> int:
    return -(-n // 128) * 128


def nearest_code(t: np.ndarray, magnitudes: np.ndarray) -> np.ndarray:
    """Index of the magnitude nearest to |t|, the even index at a tie, the last
    past the end."""
    a = np.minimum(np.abs(t), magnitudes[-1])
    hi = np.clip(np.searchsorted(magnitudes, a), 1, len(magnitudes) - 1)
    lo = hi - 1
    dl, dh = a - magnitudes[lo], magnitudes[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def scale_exponent(amax: np.ndarray, top: float, emax: int, rule: str) -> np.ndarray:
    """Scale exponents (int) of blocks with finite largest magnitudes."""
    amax = np.asarray(amax, np.float64)
    _, e = np.frexp(np.where(amax > 0, amax, 1.0))   # amax = f * 2**e, f in [0.5, 1)
    e = e.astype(np.int64) - 1 - emax
    if rule == "ceil":
        e = e + (amax > top * np.ldexp(1.0, e))
    return np.where(amax > 0, np.clip(e, -127, 127), -127)


def blocks(x: np.ndarray, size: int, magnitudes: np.ndarray, emax: int, rule: str):
    """x [rows][K] (fp64) in blocks of `size` along K: codes (index + sign, as
    (index, negative)) [rows][Kp] and scale bytes [rows][Kp/size]."""
    rows, k = x.shape
    full = np.zeros((rows, padded(k)))
    full[:, :k] = x
    b = full.reshape(rows, -1, size)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = scale_exponent(np.abs(b).max(-1), magnitudes[-1], emax, rule)
    idx = nearest_code(np.ldexp(b, -e[..., None]), magnitudes)
    neg = np.signbit(b)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return idx.reshape(rows, -1), neg.reshape(rows, -1), byte


def quant_mxfp4(x: np.ndarray, rule: str = "ceil", transpose: bool = False):
    """(codes [lines][Kp/2], scales [Kp/128][lines][4]) of x or of its transpose."""
    x = np.asarray(x, np.float64)
    x = x.T if transpose else x
    idx, neg, byte = blocks(x, 32, E2M1_MAGNITUDES, 2, rule)
    code = (idx + 8 * neg).astype(np.uint8)
    rows = x.shape[0]
    return code[:, 0::2] | (code[:, 1::2] << 4), np.ascontiguousarray(byte.reshape(rows, -1, 4).transpose(1, 0, 2))


def dequant_mxfp4(q: np.ndarray, scale: np.ndarray, cols: int) -> np.ndarray:
    """Values [rows][cols] of codes and scales."""
    rows = q.shape[0]
    v = np.empty((rows, q.shape[1] * 2))
    v[:, 0::2] = E2M1_TABLE[q & 15]
    v[:, 1::2] = E2M1_TABLE[q >> 4]
    s = e8m0_to_f64(scale.transpose(1, 0, 2).reshape(rows, -1))
    with np.errstate(invalid="ignore"):
        return (v.reshape(rows, -1, 32) * s[..., None]).reshape(rows, -1)[:, :cols]


def gemm_mxfp4(qa, sa, qb, sb):
    """(C, Abs): sum over k of a * b and of |a| * |b|, [M][N]."""
    a, b = dequant_mxfp4(qa, sa, qa.shape[1] * 2), dequant_mxfp4(qb, sb, qb.shape[1] * 2)
    with np.errstate(invalid="ignore"):
        return a @ b.T, np.abs(a) @ np.abs(b).T


def rms(h: np.ndarray, w: np.ndarray, eps: float):
    """(y, rstd) of h [rows][cols] as stored, fp64."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def quant_e4m3(y: np.ndarray):
    """(bytes [rows][Kp], scales [Kp/128][rows]) under the ceil rule."""
    idx, neg, byte = blocks(y, 128, E4M3_MAGNITUDES, 8, "ceil")
    return (idx + 128 * neg).astype(np.uint8), np.ascontiguousarray(byte.T)


def rms_grad(dy, h, w, rstd, dh=None):
    """(dx, dw, |dx| terms, |dw| terms) in fp64; the last two are the sums of
    magnitudes that the rounding errors scale with: sum |g h| per row and sum
    |dy h rstd| per column."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    r = np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    c = (g * h).sum(1, keepdims=True)
    dx = r * g - h * r ** 3 * c / h.shape[1]
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h * r).sum(0), np.abs(g * h).sum(1, keepdims=True), np.abs(dy * h * r).sum(0)
