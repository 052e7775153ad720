"""A residual layer in MXFP4, forward and backward, through the library's entry
points:

    h = x + r                      the residual stream, stored
    y = rms_norm(h) * w            quantised to MXFP4 in the same pass
    c = y . W^T                    4-bit product, bf16

The weight matrix W [out][in] is laid out once, blocks along `in` for the
forward product and along `out` for the gradient's.  Training quantises the
incoming gradient along both of its directions: dy = dc . W contracts over the
outputs, dW = dc^T . y over the tokens.  A single new token takes the same
calls with one row.

    python examples/mxfp4_layer.py          # on an MI355X: errors and times
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import tile_scheduling_persistent_amd as pg  # noqa: E402


def up(n: int) -> int:
    return -(-n // 128) * 128


class Operand:
    """Buffers of an MXFP4 operand of a [rows][cols] matrix."""

    def __init__(self, rows: int, cols: int, device):
        nb = pg.mxfp4_bytes(rows, cols)
        self.rows, self.cols, self.k = rows, cols, up(cols)
        self.q = torch.empty(nb["Q"], dtype=torch.uint8, device=device)
        self.scale = torch.empty(nb["scale"], dtype=torch.uint8, device=device)

    def fill(self, cfg, x, transpose=False):
        pg.pmx_quant_run(cfg, x, self.q, self.scale, *x.shape, transpose=transpose)
        return self


def product(cfg, a: Operand, b: Operand, out) -> torch.Tensor:
    """out [a.rows][b.rows] = a . b^T over their common columns."""
    dtype = "mxfp4_out_f32" if out.dtype == torch.float32 else "mxfp4_out_bf16"
    pg.pgemm_run(cfg, a.q, b.q, out, a.rows, b.rows, a.k, dtype, "grouped",
                 pg.make_args(a_scale=a.scale, b_scale=b.scale))
    return out


class ResidualLinear:
    """The layer for up to `tokens` rows at a time; W [out][in] and w [in] in bf16."""

    def __init__(self, cfg, W: torch.Tensor, w: torch.Tensor, tokens: int, eps: float = 1e-6):
        self.cfg, self.w, self.eps = cfg, w, eps
        self.n_out, self.n_in = W.shape
        dev = self.dev = W.device
        self.W = Operand(self.n_out, self.n_in, dev).fill(cfg, W)
        self.Wt = Operand(self.n_in, self.n_out, dev).fill(cfg, W, transpose=True)
        self.h = torch.empty((tokens, self.n_in), dtype=torch.bfloat16, device=dev)
        self.rstd = torch.empty(tokens, device=dev)

    def forward(self, x: torch.Tensor, r: torch.Tensor):
        """(c, h) for x and the residual stream r, [tokens][in] bf16; keeps h and
        the rows' factors for backward."""
        t = x.shape[0]
        y = Operand(t, self.n_in, self.dev)
        h, rstd = self.h[:t], self.rstd[:t]
        pg.prms_run(self.cfg, x, self.w, y.q, t, self.n_in, eps=self.eps, R=r, H=h, out="mxfp4", y_scale=y.scale,
                    rstd=rstd)
        return product(self.cfg, y, self.W, torch.empty((t, self.n_out), dtype=torch.bfloat16, device=self.dev)), h

    def backward(self, dc: torch.Tensor, dh: torch.Tensor):
        """Gradients for the last forward: dc [tokens][out] of c and dh
        [tokens][in] of h, both bf16.  Returns (dx, dw, dW); dx is r's too."""
        cfg, t = self.cfg, dc.shape[0]
        h, rstd = self.h[:t], self.rstd[:t]
        dy = torch.empty((t, self.n_in), dtype=torch.bfloat16, device=self.dev)
        product(cfg, Operand(t, self.n_out, self.dev).fill(cfg, dc), self.Wt, dy)
        dx, dw = torch.empty_like(h), torch.empty(self.n_in, device=self.dev)
        pg.prms_grad_run(cfg, dy, h, self.w, rstd, dx, dw, t, self.n_in, dH=dh)
        # the normed rows again, along the tokens this time
        y = torch.empty_like(h)
        pg.prms_run(cfg, h, self.w, y, t, self.n_in, eps=self.eps)
        dW = torch.empty((self.n_out, self.n_in), device=self.dev)
        product(cfg, Operand(self.n_out, t, self.dev).fill(cfg, dc, transpose=True),
                Operand(self.n_in, t, self.dev).fill(cfg, y, transpose=True), dW)
        return dx, dw, dW


def main() -> None:
    cfg = pg.Config(0)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).bfloat16()

    tokens, n_in, n_out = 4096, 4096, 8192
    W, w = normal(n_out, n_in, scale=n_in ** -0.5), 1 + normal(n_in, scale=0.1)
    layer = ResidualLinear(cfg, W, w, tokens)
    x, r, dc, dh = normal(tokens, n_in), normal(tokens, n_in), normal(tokens, n_out), normal(tokens, n_in)
    c, h = layer.forward(x, r)
    dx, dw, dW = layer.backward(dc, dh)

    hf = h.float()
    n = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + layer.eps)
    y = n * w.float()

    def error(a, b):
        return ((a.float() - b).norm() / b.norm()).item()

    print(f"c   {error(c, y @ W.float().t()):.3f}   relative error against unquantised operands")
    print(f"dW  {error(dW, dc.float().t() @ y):.3f}")

    def time_us(f, reps=20):
        f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(reps):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / reps * 1e3

    print(f"forward {tokens} tokens {time_us(lambda: layer.forward(x, r)):.0f} us, "
          f"backward {time_us(lambda: layer.backward(dc, dh)):.0f} us, "
          f"one token {time_us(lambda: layer.forward(x[:1], r[:1])):.0f} us")


if __name__ == "__main__":
    main()
