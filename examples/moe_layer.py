"""A layer of experts in e4m3, forward and backward, through the library's entry
points:

    rows of A = the tokens' rows, sorted by expert, in e4m3
    G = A . W13[e]^T                   gate and up, bf16
    B = silu(gate) * up                in e4m3, G kept in e4m3
    Y = B . W2[e]^T
    y[t] = x[t] + sum_j w[t, j] * Y[row of (t, j)]

The weights are quantised once per step, in both orientations: the forward
products read W [out][in], the gradients' products the transposed blocks.  What the
backward needs of the forward is kept in 8 bits: A, G and B; the weight gradients
read A and B as they are.  The host never waits for the router's counts.

    python examples/moe_layer.py          # on an MI355X: errors and times
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


class Rows:
    """An e4m3 operand of a [rows][cols] matrix."""

    def __init__(self, rows: int, cols: int, device):
        nb = pg.fp8_bytes(rows, cols)
        self.rows, self.cols = rows, cols
        self.q = torch.empty(nb["Q"], dtype=torch.uint8, device=device)
        self.scale = torch.empty(nb["scale"], dtype=torch.uint8, device=device)


class Weights:
    """e4m3 weights [experts][out][in] in both orientations."""

    def __init__(self, cfg, w: torch.Tensor):
        self.experts, self.n_out, self.n_in = w.shape
        nb = pg.fp8_weight_bytes(*w.shape)
        self.q, self.scale, self.qt, self.scale_t = (torch.empty(nb[k], dtype=torch.uint8, device=w.device)
                                                     for k in ("Q", "scale", "Qt", "scale_t"))
        pg.pfp8_quant_weights_run(cfg, w, self.q, self.scale, *w.shape, Qt=self.qt, scale_t=self.scale_t)


class Experts:
    """The layer; W13 [experts][2 * inner][hidden] and W2 [experts][hidden][inner] in
    bf16, inner a multiple of 128."""

    def __init__(self, cfg, W13: torch.Tensor, W2: torch.Tensor):
        self.cfg, self.dev = cfg, W13.device
        self.experts, self.hidden, self.inner = W2.shape
        self.W13, self.W2 = Weights(cfg, W13), Weights(cfg, W2)

    def new(self, *shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=self.dev)

    def product(self, a: Rows, q, scale, n: int) -> torch.Tensor:
        c = self.new(a.rows, n)
        pg.pgemm_run_experts(self.cfg, a.q, q, c, a.rows, n, up(a.cols), a.scale, scale, experts=self.experts,
                             offsets=self.offsets)
        return c

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        """y [tokens][hidden] for tokens x (bf16), their experts ids [tokens][topk] (-1:
        none) and weights (fp32); keeps what backward needs."""
        cfg, (tokens, topk) = self.cfg, ids.shape
        slots, h, f = tokens * topk, self.hidden, self.inner
        self.weights, self.shape = weights, (tokens, topk)
        self.place, self.order = self.new(tokens, topk, dtype=torch.int32), self.new(slots, dtype=torch.int32)
        self.offsets = self.new(self.experts + 1, dtype=torch.int32)
        pg.pmoe_sort_run(cfg, ids, self.place, self.order, self.offsets, tokens, topk, self.experts)
        self.used = self.offsets[-1:]
        self.A, self.B, self.G = Rows(slots, h, self.dev), Rows(slots, f, self.dev), Rows(slots, 2 * f, self.dev)
        pg.pmoe_gather_run(cfg, x, self.order, self.A.q, tokens, topk, h, out="fp8_b128", y_scale=self.A.scale)
        g = self.product(self.A, self.W13.q, self.W13.scale, 2 * f)
        pg.pglu_run(cfg, g, self.B.q, slots, f, out="fp8_b128", y_scale=self.B.scale, kept=self.G.q,
                    kept_scale=self.G.scale, valid=self.used)
        self.Y = self.product(self.B, self.W2.q, self.W2.scale, h)
        y = torch.empty_like(x)
        pg.pmoe_combine_run(cfg, self.Y, self.place, y, tokens, topk, h, weights=weights, R=x)
        return y

    def backward(self, dy: torch.Tensor):
        """(dx, dweights, dW13, dW2) for the last forward and the gradient dy of y."""
        cfg, (tokens, topk), h, f = self.cfg, self.shape, self.hidden, self.inner
        slots = tokens * topk
        dY, dG = Rows(slots, h, self.dev), Rows(slots, 2 * f, self.dev)
        dw = self.new(tokens, topk, dtype=torch.float32)
        pg.pmoe_combine_grad_run(cfg, dy, self.Y, self.place, self.order, dY.q, tokens, topk, h, weights=self.weights,
                                 dW=dw, out="fp8_b128", dx_scale=dY.scale)
        dB = self.product(dY, self.W2.qt, self.W2.scale_t, f)
        pg.pglu_grad_run(cfg, dB, self.G.q, dG.q, slots, f, x_scale=self.G.scale, out="fp8_b128", dx_scale=dG.scale,
                         valid=self.used)
        dA = self.product(dG, self.W13.qt, self.W13.scale_t, h)
        dx = torch.empty_like(dy)
        pg.pmoe_combine_run(cfg, dA, self.place, dx, tokens, topk, h, R=dy)
        grads = []
        for d, a, w in ((dG, self.A, self.W13), (dY, self.B, self.W2)):
            grad = self.new(self.experts, w.n_out, w.n_in, dtype=torch.float32)
            pg.pgemm_run_experts_wgrad(cfg, d.q, a.q, grad, slots, w.n_out, w.n_in, a.scale, d_scale=d.scale,
                                       experts=self.experts, offsets=self.offsets)
            grads.append(grad)
        return (dx, dw, *grads)


def main() -> None:
    cfg = pg.Config(0)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).bfloat16()

    tokens, topk, experts, hidden, inner = 4096, 4, 16, 2048, 1024
    W13 = normal(experts, 2 * inner, hidden, scale=hidden ** -0.5)
    W2 = normal(experts, hidden, inner, scale=inner ** -0.5)
    layer = Experts(cfg, W13, W2)
    x, dy = normal(tokens, hidden), normal(tokens, hidden)
    top = torch.randn((tokens, experts), generator=g, device=dev).topk(topk, 1)
    ids, weights = top.indices, torch.softmax(top.values, 1)
    y = layer.forward(x, ids, weights)
    dx, dw, dW13, dW2 = layer.backward(dy)

    leaves = [t.float().requires_grad_() for t in (x, weights, W13, W2)]
    xf, wf, a, b = leaves
    parts = []
    for j in range(topk):
        out = torch.zeros_like(xf)
        for e in range(experts):
            at = (ids[:, j] == e).nonzero().view(-1)
            gate, up_ = (xf[at] @ a[e].t()).split(inner, 1)
            out = out.index_add(0, at, (torch.nn.functional.silu(gate) * up_) @ b[e].t() * wf[at, j:j + 1])
        parts.append(out)
    want = xf + sum(parts)
    grads = torch.autograd.grad(want, leaves, dy.float())

    def error(p, q):
        return ((p.float() - q).norm() / q.norm()).item()

    print(f"relative errors against unquantised operands: y {error(y - x, want.detach() - xf.detach()):.3f}, "
          f"dx {error(dx - dy, grads[0] - dy.float()):.3f}, dweights {error(dw, grads[1]):.3f}, "
          f"dW13 {error(dW13, grads[2]):.3f}, dW2 {error(dW2, grads[3]):.3f}")

    def time_us(f, reps=20):
        f()
        s, t = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s.record()
        for _ in range(reps):
            f()
        t.record()
        torch.cuda.synchronize()
        return s.elapsed_time(t) / reps * 1e3

    print(f"forward {tokens} tokens {time_us(lambda: layer.forward(x, ids, weights)):.0f} us, "
          f"backward {time_us(lambda: layer.backward(dy)):.0f} us, "
          f"one token {time_us(lambda: layer.forward(x[:1], ids[:1], weights[:1])):.0f} us")


if __name__ == "__main__":
    main()
