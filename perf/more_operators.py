"""Cases of the library's operators for layers of experts in 8 bits, each with
its plain form.

  dispatch  slots (token, choice) sorted by the expert they go to, and the tokens'
            rows in that order, as they are or in e4m3
  combine   the experts' rows back at their tokens, weighted and summed
  combine_grad  its gradients with respect to the rows and the weights
  quant     a matrix to e4m3 with a scale for each 128 columns of a row, or weights
            to e4m3 with a scale for each 128 x 128 block, both ways round
  product   C[r] = A[r] . B_e^T on such operands, e the expert that row r is of
  wgrad     dB_e = sum over the rows of e of dC[r]^T A[r], from 8-bit rows
  glu       silu(g) * u with g and u kept in e4m3, and its gradient from those

Storage.  e4m3 of a [rows][K] matrix: bytes [rows][Kp], Kp = K rounded up to 128,
e8m0 scales [Kp / 128][rows].  Weights [experts][N][K]: bytes [experts][N][Kp],
scales [experts][Np / 128][Kp / 128].  Padding holds zeros; a block of zeros has
scale byte 0.  A scale's exponent is the smallest under which the block's largest
magnitude is representable.  Rows are sorted by expert; expert e has the rows
offsets[e] .. offsets[e + 1].
"""
import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def up(n, m=128):
    return -(-n // m) * m


# ----------------------------------------------------------------- the cases


def listed():
    return [
        # a decoding batch before the experts' first product: latency
        dict(name="dispatch 64x8 of 64, 4096 e4m3", op="dispatch", x="bf16", tokens=64, topk=8, experts=64, cols=4096,
             out="e4m3", away=False),
        # a long prompt or a training batch
        dict(name="dispatch 8192x8 of 64, 4096 e4m3", op="dispatch", x="bf16", tokens=8192, topk=8, experts=64,
             cols=4096, out="e4m3", away=False),
        # the same batch's way back, with the residual stream
        dict(name="combine 8192x8, 4096 bf16", op="combine", x="bf16", y="bf16", tokens=8192, topk=8, experts=64,
             cols=4096, residual=True, away=False),
        # training with half of the experts on other devices, columns that end inside a group of 128
        dict(name="combine_grad 5000x2, 7000 bf16", op="combine_grad", x="bf16", tokens=5000, topk=2, experts=8,
             cols=7000, out="same", away=True),
        # the weights of sixteen experts after an optimizer step, for the product and its gradient
        dict(name="quant weights 16x4096x4096", op="quant", x="bf16", form="weights", experts=16, rows=4096, cols=4096),
        # an fp32 gradient as the next product's operand, odd sizes
        dict(name="quant rows 5000x7000 f32", op="quant", x="f32", form="rows", experts=1, rows=5000, cols=7000),
        # sixteen new tokens, eight experts each: the weights stream once
        dict(name="product 128 of 64, 4096x4096", op="product", rows=128, experts=64, n=4096, k=4096, out="bf16"),
        # a long prompt or a training batch
        dict(name="product 65536 of 64, 4096x4096", op="product", rows=65536, experts=64, n=4096, k=4096, out="bf16"),
        # training: the weight gradient of sixteen experts, fp32
        dict(name="wgrad 32768 of 16, 4096x2048", op="wgrad", d="bf16", rows=32768, experts=16, n=4096, k=2048,
             out="f32", add=False),
        # a gradient kept in 8 bits, added to the one of the batch before, odd sizes
        dict(name="wgrad 5000 of 8, 1000x1408", op="wgrad", d="e4m3", rows=5000, experts=8, n=1000, k=1408, out="f32",
             add=True),
        # training: forward and backward of the activation between an expert's products
        dict(name="glu 32768x2048 e4m3", op="glu", x="bf16", rows=32768, cols=2048, out="e4m3", dout="e4m3"),
        # a short batch, odd sizes, nothing quantised but what is kept
        dict(name="glu 300x1000 f16", op="glu", x="f16", rows=300, cols=1000, out="same", dout="same"),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return min(hi, max(lo, up(v, step)))

    op = rng.choice(("dispatch", "combine", "combine_grad", "quant", "product", "product", "wgrad", "glu"))
    x = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op in ("dispatch", "combine", "combine_grad"):
        experts = size(4, 256)
        topk = rng.choice([t for t in (1, 2, 4, 6, 8) if t <= experts])
        cols = size(128, 8192)
        tokens = size(1, max(1, min(16384, 8192 * 8 * 4096 // (topk * cols) // (2 if x == "f32" else 1))))
        c = dict(op=op, x=x, tokens=tokens, topk=topk, experts=experts, cols=cols, away=rng.random() < 0.3)
        if op == "combine":
            return dict(c, y=rng.choice((x, x, "f32")), residual=rng.random() < 0.5)
        return dict(c, out=rng.choice(("same", "e4m3")))
    if op == "quant":
        form = rng.choice(("rows", "weights"))
        experts = size(1, 16) if form == "weights" else 1
        rows, cols = size(1 if form == "rows" else 64, 8192), size(64, 8192)
        return dict(op=op, x=x, form=form, experts=min(experts, max(1, 16 * 4096 * 4096 // (rows * cols))), rows=rows,
                    cols=cols)
    if op == "glu":
        cols = size(64, 8192)
        rows = size(1, max(1, 32768 * 2048 // cols // (2 if x == "f32" else 1)))
        return dict(op=op, x=x, rows=rows, cols=cols, out=rng.choice(("same", "e4m3")),
                    dout=rng.choice(("same", "e4m3")) if cols % 128 == 0 else "same")
    experts = rng.choice((1, 4, 8, 16, 32, 64))
    if op == "product":
        n, k = size(128, 8192), size(128, 8192, 128)
        experts = min(experts, max(1, 64 * 4096 * 4096 // (n * k)))
        return dict(op=op, rows=size(1, max(1, min(65536, 65536 * 4096 * 4096 // (n * k)))), experts=experts, n=n, k=k,
                    out=rng.choice(("bf16", "bf16", "f32")))
    n, k = size(128, 4096), size(128, 4096)
    experts = min(experts, max(1, 16 * 4096 * 2048 // (n * k)))
    return dict(op=op, d=rng.choice(("bf16", "e4m3")), rows=size(1, max(1, min(32768, 32768 * 4096 * 2048 // (n * k)))),
                experts=experts, n=up(n, 8), k=k, out=rng.choice(("f32", "f32", "bf16")), add=rng.random() < 0.3)


def touched(case):
    """Experts that are expected to have rows."""
    e = case["experts"]
    return e * (1.0 - (1.0 - 1.0 / e) ** case["rows"])


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        slots = case["tokens"] * case["topk"]
        one, rows = case["tokens"] * case["cols"], slots * case["cols"] * (0.5 if case["away"] else 1.0)
        e = SIZE[case["x"]]
        if op == "combine":
            y = SIZE[case["y"]]
            return {"bytes": rows * e + one * y * (2 if case["residual"] else 1) + slots * 8, "flops": 2.0 * rows}
        out = rows * ((1 + 1 / 128) if case["out"] == "e4m3" else e)
        if op == "dispatch":
            return {"bytes": one * e + out + slots * 12, "flops": 2.0 * rows}
        return {"bytes": one * e + rows * e + out + slots * 16, "flops": 3.0 * rows}
    if op == "quant":
        t = case["experts"] * case["rows"] * case["cols"]
        return {"bytes": t * (SIZE[case["x"]] + (2 if case["form"] == "weights" else 1 + 1 / 128)), "flops": 3.0 * t}
    if op == "glu":
        t, e = case["rows"] * case["cols"], SIZE[case["x"]]
        y = 1 + 1 / 128 if case["out"] == "e4m3" else e
        dx = 2 + 2 / 128 if case["dout"] == "e4m3" else 2 * e
        return {"bytes": t * (2 * e + y + 2 * (2 + 2 / 128) + e + dx), "flops": 20.0 * t}
    r, n, k = case["rows"], case["n"], case["k"]
    if op == "product":
        return {"bytes": r * k * (1 + 1 / 128) + touched(case) * n * k + r * n * SIZE[case["out"]], "flops": 2.0 * r * n * k}
    d = 2 if case["d"] == "bf16" else 1 + 1 / 128
    out = case["experts"] * n * k * SIZE[case["out"]] * (2 if case["add"] else 1)
    return {"bytes": r * (n * d + k * (1 + 1 / 128)) + out, "flops": 2.0 * r * n * k}


# ---------------------------------------------------------------- the inputs


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def acts(rows, cols):  # hidden states: tokens of different size, a few strong channels
        v = normal(rows, cols) * torch.exp(0.5 * normal(rows, 1))
        return v * torch.where(torch.rand((1, cols), generator=g, device=dev) < 0.01, 12.0, 1.0)

    def empty(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype, device=dev)

    s = dict(case)
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        tokens, topk, experts, cols, x = case["tokens"], case["topk"], case["experts"], case["cols"], TYPES[case["x"]]
        # a router's choices: distinct experts per token, some of them preferred; of twice as many experts
        # where half of them are on other devices
        e = 2 * experts if case["away"] else experts
        logits = normal(tokens, e) + 0.5 * normal(1, e)
        top = logits.topk(topk, dim=1)
        s["IDS"] = torch.where(top.indices < experts, top.indices, -1).to(torch.int32).contiguous()
        slots = tokens * topk
        s.update(PLACE=empty(tokens, topk, dtype=torch.int32), ORDER=empty(slots, dtype=torch.int32),
                 OFFSETS=empty(experts + 1, dtype=torch.int32))
        if op == "dispatch":
            s["X"] = acts(tokens, cols).to(x)
        else:  # the sort's results are in hand
            s["PLACE"], s["ORDER"], s["OFFSETS"] = plain_sort(s["IDS"], experts)
            s["X"] = acts(slots, cols).to(x)
            s["WEIGHTS"] = torch.softmax(top.values, 1)
        if op == "combine":
            s["R"] = acts(tokens, cols).to(TYPES[case["y"]]) if case["residual"] else None
            s["Y"] = empty(tokens, cols, dtype=TYPES[case["y"]])
            return s
        if op == "combine_grad":
            s["DY"], s["DWEIGHTS"] = (1e-2 * normal(tokens, cols)).to(x), empty(tokens, topk, dtype=torch.float32)
        s["SCALE"] = empty(up(cols) // 128, slots)
        s["Y"] = empty(slots, up(cols)) if case["out"] == "e4m3" else empty(slots, cols, dtype=x)
        return s
    if op == "quant":
        experts, rows, cols, x = case["experts"], case["rows"], case["cols"], TYPES[case["x"]]
        if case["form"] == "rows":
            s.update(X=(1e-3 * acts(rows, cols)).to(x), Q=empty(rows, up(cols)), SCALE=empty(up(cols) // 128, rows))
        else:
            s.update(X=(normal(experts, rows, cols) / math.sqrt(cols)).to(x), Q=empty(experts, rows, up(cols)),
                     SCALE=empty(experts, up(rows) // 128, up(cols) // 128), QT=empty(experts, cols, up(rows)),
                     SCALET=empty(experts, up(cols) // 128, up(rows) // 128))
        return s
    if op == "glu":
        rows, cols, x = case["rows"], case["cols"], TYPES[case["x"]]
        s.update(X=(0.3 * acts(rows, 2 * cols)).to(x), DY=(1e-2 * normal(rows, cols)).to(x),
                 KEPT=empty(rows, 2 * up(cols)), KSCALE=empty(2 * up(cols) // 128, rows))
        s["Y"] = empty(rows, up(cols)) if case["out"] == "e4m3" else empty(rows, cols, dtype=x)
        s["YSCALE"] = empty(up(cols) // 128, rows)
        s["DX"] = empty(rows, 2 * cols) if case["dout"] == "e4m3" else empty(rows, 2 * cols, dtype=x)
        s["DSCALE"] = empty(2 * cols // 128, rows)
        return s
    rows, n, k, experts = case["rows"], case["n"], case["k"], case["experts"]
    share = torch.softmax(0.5 * normal(experts), 0)
    count = torch.bincount(torch.multinomial(share, rows, replacement=True, generator=g), minlength=experts)
    s["OFFSETS"] = torch.cat((count.new_zeros(1), count.cumsum(0))).to(torch.int32)
    s["sizes"] = count.tolist()  # the plain form's: it goes expert by expert
    q, e = plain_e4m3(acts(rows, k))
    s["A"], s["SA"] = store8(q, e)
    if op == "product":
        b = [plain_weights(normal(n, k) / math.sqrt(k)) for _ in range(experts)]
        s["B"] = torch.stack([q.to(torch.float8_e4m3fn).view(torch.uint8) for q, _ in b])
        s["SB"] = torch.stack([(e + 127).to(torch.uint8) for _, e in b])
        s["C"] = empty(rows, n, dtype=TYPES[case["out"]])
        return s
    d = 1e-2 * normal(rows, n)
    s["D"], s["SD"] = (d.bfloat16(), None) if case["d"] == "bf16" else store8(*plain_e4m3(d))
    s["BEFORE"] = normal(experts, n, k).to(TYPES[case["out"]]) if case["add"] else None
    s["DB"] = empty(experts, n, k, dtype=TYPES[case["out"]])
    return s


# ----------------------------------------------------------- the plain forms


def exponent(amax):
    """The exponents of e4m3 blocks with these largest magnitudes."""
    frac, e = torch.frexp(amax)  # amax = frac * 2^e, frac in [0.5, 1); the largest e4m3 is 0.875 * 2^9
    return torch.where(amax > 0, e - 9 + (frac > 0.875).int(), -127).clamp(-127, 127)


def pow2(e):
    """2^e in fp32, -127 < e < 128, by the exponent's bits (a power function may be off by a step)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def units(x, e):
    """x * 2^-e: e at its least only where x is zero or next to it."""
    return x * pow2(-e.clamp(min=-126))


def round_e4m3(v):
    """|v| <= 448 to the nearest e4m3 value, ties to the even code."""
    step = pow2(torch.frexp(v.abs())[1].clamp(min=-5) - 4)
    return torch.copysign(torch.round(v.abs() / step) * step, v)


def plain_e4m3(x):
    """x [rows][cols] as e4m3 values in units of their scale [rows][Kp] and scale
    exponents [rows][Kp / 128]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, up(cols) - cols)).view(rows, -1, 128)
    e = exponent(x.abs().amax(-1))
    return round_e4m3(units(x, e[..., None])).view(rows, -1), e


def plain_weights(w):
    """w [N][K] as e4m3 values [N][Kp] and exponents [Np / 128][Kp / 128]."""
    n, k = w.shape
    w = torch.nn.functional.pad(w.float(), (0, up(k) - k, 0, up(n) - n)).view(up(n) // 128, 128, up(k) // 128, 128)
    e = exponent(w.abs().amax((1, 3)))
    return round_e4m3(units(w, e[:, None, :, None])).view(up(n), up(k))[:n], e


def store8(q, e):
    return q.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8).t().contiguous()


def values8(codes, scale):
    """The values [rows][Kp] of e4m3 bytes and scale bytes [Kp / 128][rows]."""
    v = codes.view(torch.float8_e4m3fn).float().view(len(codes), -1, 128)
    return (v * pow2((scale.t().int() - 127).clamp(min=-126))[..., None]).view(len(codes), -1)


def weight_values8(codes, scale):
    """The values [N][Kp] of one expert's bytes and scale bytes [Np / 128][Kp / 128]."""
    n, k = codes.shape
    e = (scale.int() - 127).clamp(min=-126).repeat_interleave(128, 0)[:n]
    return (codes.view(torch.float8_e4m3fn).float().view(n, -1, 128) * pow2(e)[..., None]).view(n, k)


def two(v, e):
    """Values in units of their scale and the scales, as they are stored."""
    return v.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def rows_out(out, y, x_type):
    """y [rows][cols] fp32 in the output's form."""
    if out == "same":
        return {"y": y.to(TYPES[x_type])}
    v, e = two(*plain_e4m3(y))
    return {"y": v, "scale": e.view(torch.uint8).t().contiguous().view(torch.float8_e8m0fnu)}


def plain_sort(ids, experts):
    """(place, order, offsets) of the slots' experts."""
    flat = torch.where((ids >= 0) & (ids < experts), ids, experts).view(-1).long()
    slots = flat.numel()
    at = torch.arange(slots, device=ids.device)
    order = torch.sort(flat, stable=True).indices
    count = torch.zeros(experts + 1, dtype=torch.long, device=ids.device).scatter_add(0, flat, torch.ones_like(flat))
    offsets = torch.cat((count.new_zeros(1), count[:experts].cumsum(0)))
    place = torch.empty_like(order)
    place[order] = at
    place = torch.where(flat < experts, place, -1).view(ids.shape)
    order = torch.where(at < offsets[-1], order, -1)
    return place.to(torch.int32), order.to(torch.int32), offsets.to(torch.int32)


def plain_dispatch(s):
    place, order, offsets = plain_sort(s["IDS"], s["experts"])
    y = s["X"].float()[order.clamp(min=0).long() // s["topk"]] * (order >= 0)[:, None]
    return {"place": place, "order": order, "offsets": offsets, **rows_out(s["out"], y, s["x"])}


def plain_combine(s):
    place = s["PLACE"].long()
    w = torch.where(place >= 0, s["WEIGHTS"], 0.0)
    y = (s["X"][place.clamp(min=0)].float() * w[..., None]).sum(1)
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(TYPES[s["y"]])


def plain_combine_grad(s):
    place, slot = s["PLACE"].long(), s["ORDER"].clamp(min=0).long()
    dy = s["DY"].float()
    w = torch.where(s["ORDER"] >= 0, s["WEIGHTS"].view(-1)[slot], 0.0)
    dx = dy[slot // s["topk"]] * w[:, None] + 0.0  # no negative zeros where there is no row
    dw = (s["X"][place.clamp(min=0)].float() * dy[:, None]).sum(-1)
    return {"dweights": torch.where(place >= 0, dw, 0.0), **rows_out(s["out"], dx, s["x"])}


def plain_quant(s):
    if s["form"] == "rows":
        return rows_out("e4m3", s["X"].float(), s["x"])
    both = [two(*plain_weights(w)) + two(*plain_weights(w.t())) for w in s["X"]]
    parts = [torch.stack([x.view(torch.uint8) for x in t]).view(t[0].dtype) for t in zip(*both)]
    return dict(zip(("q", "scale", "qt", "scalet"), parts))


def plain_product(s):
    parts = s["sizes"]
    a = values8(s["A"], s["SA"]).split(parts)
    return torch.cat([a[i] @ weight_values8(s["B"][i], s["SB"][i]).t() for i, p in enumerate(parts) if p]).to(TYPES[s["out"]])


def plain_wgrad(s):
    d = s["D"].float() if s["SD"] is None else values8(s["D"], s["SD"])[:, :s["n"]]
    a = values8(s["A"], s["SA"])[:, :s["k"]]
    db = torch.stack([x.t() @ y for x, y in zip(d.split(s["sizes"]), a.split(s["sizes"]))])
    if s["BEFORE"] is not None:
        db = db + s["BEFORE"].float()
    return db.to(TYPES[s["out"]])


def plain_glu(s):
    cols = s["cols"]
    g, u = s["X"].float().split(cols, 1)
    y = rows_out(s["out"], g / (1 + torch.exp(-g)) * u, s["x"])
    (qg, eg), (qu, eu) = plain_e4m3(g), plain_e4m3(u)
    kept, scale = store8(torch.cat((qg, qu), 1), torch.cat((eg, eu), 1))
    g, u = (t[:, :cols] for t in values8(kept, scale).split(up(cols), 1))
    dy, sig = s["DY"].float(), 1 / (1 + torch.exp(-g))
    dx = rows_out(s["dout"], torch.cat((dy * u * sig * (1 + g * (1 - sig)), dy * g * sig), 1), s["x"])
    return {"y": y, "kept": kept.view(torch.float8_e4m3fn), "kscale": scale.view(torch.float8_e8m0fnu), "dx": dx}


PLAIN = {"dispatch": plain_dispatch, "combine": plain_combine, "combine_grad": plain_combine_grad, "quant": plain_quant,
         "product": plain_product, "wgrad": plain_wgrad, "glu": plain_glu}


# ----------------------------------------------------- the library's operators


@functools.lru_cache(None)
def library():
    import tile_scheduling_persistent_amd as pg
    return pg, pg.Config(torch.cuda.current_device())


def form(s, out, y, scale):
    """The output's arguments, and how it comes back."""
    if s[out] == "same":
        return dict(out="same"), {"y": s[y]}
    return dict(out="fp8_b128"), {"y": s[y].view(torch.float8_e4m3fn), "scale": s[scale].view(torch.float8_e8m0fnu)}


def own_dispatch(s):
    pg, cfg = library()
    tokens, topk = s["tokens"], s["topk"]
    pg.pmoe_sort_run(cfg, s["IDS"], s["PLACE"], s["ORDER"], s["OFFSETS"], tokens, topk, s["experts"])
    kw, back = form(s, "out", "Y", "SCALE")
    pg.pmoe_gather_run(cfg, s["X"], s["ORDER"], s["Y"], tokens, topk, s["cols"], y_scale=s["SCALE"], **kw)
    return {"place": s["PLACE"], "order": s["ORDER"], "offsets": s["OFFSETS"], **back}


def own_combine(s):
    pg, cfg = library()
    pg.pmoe_combine_run(cfg, s["X"], s["PLACE"], s["Y"], s["tokens"], s["topk"], s["cols"], weights=s["WEIGHTS"], R=s["R"])
    return s["Y"]


def own_combine_grad(s):
    pg, cfg = library()
    kw, back = form(s, "out", "Y", "SCALE")
    pg.pmoe_combine_grad_run(cfg, s["DY"], s["X"], s["PLACE"], s["ORDER"], s["Y"], s["tokens"], s["topk"], s["cols"],
                             weights=s["WEIGHTS"], dW=s["DWEIGHTS"], dx_scale=s["SCALE"], **kw)
    return {"dweights": s["DWEIGHTS"], **back}


def own_quant(s):
    pg, cfg = library()
    if s["form"] == "rows":
        pg.pfp8_quant_run(cfg, s["X"], s["Q"], s["SCALE"], s["rows"], s["cols"])
        return {"y": s["Q"].view(torch.float8_e4m3fn), "scale": s["SCALE"].view(torch.float8_e8m0fnu)}
    pg.pfp8_quant_weights_run(cfg, s["X"], s["Q"], s["SCALE"], s["experts"], s["rows"], s["cols"], Qt=s["QT"],
                              scale_t=s["SCALET"])
    return {"q": s["Q"].view(torch.float8_e4m3fn), "scale": s["SCALE"].view(torch.float8_e8m0fnu),
            "qt": s["QT"].view(torch.float8_e4m3fn), "scalet": s["SCALET"].view(torch.float8_e8m0fnu)}


def own_product(s):
    pg, cfg = library()
    pg.pgemm_run_experts(cfg, s["A"], s["B"], s["C"], s["rows"], s["n"], s["k"], s["SA"], s["SB"], experts=s["experts"],
                         offsets=s["OFFSETS"])
    return s["C"]


def own_wgrad(s):
    pg, cfg = library()
    pg.pgemm_run_experts_wgrad(cfg, s["D"], s["A"], s["DB"], s["rows"], s["n"], s["k"], s["SA"], d_scale=s["SD"],
                               experts=s["experts"], offsets=s["OFFSETS"], base=s["BEFORE"])
    return s["DB"]


def own_glu(s):
    pg, cfg = library()
    kw, y = form(s, "out", "Y", "YSCALE")
    pg.pglu_run(cfg, s["X"], s["Y"], s["rows"], s["cols"], y_scale=s["YSCALE"], kept=s["KEPT"], kept_scale=s["KSCALE"], **kw)
    kw, dx = form(s, "dout", "DX", "DSCALE")
    pg.pglu_grad_run(cfg, s["DY"], s["KEPT"], s["DX"], s["rows"], s["cols"], x_scale=s["KSCALE"], dx_scale=s["DSCALE"], **kw)
    return {"y": y, "kept": s["KEPT"].view(torch.float8_e4m3fn), "kscale": s["KSCALE"].view(torch.float8_e8m0fnu),
            "dx": dx}


OWN = {"dispatch": own_dispatch, "combine": own_combine, "combine_grad": own_combine_grad, "quant": own_quant,
       "product": own_product, "wgrad": own_wgrad, "glu": own_glu}


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------- the definitions, in 64 bits

E4M3 = [m / 512 for m in range(8)] + [2.0 ** e * (1 + m / 8) for e in range(-6, 9) for m in range(8)][:-1]


def nearest(t):
    """The e4m3 value nearest to t (at a tie the one of even code)."""
    table = torch.tensor(E4M3, dtype=torch.float64, device=t.device)
    mid = (table[1:] + table[:-1]) / 2
    odd = torch.arange(len(mid), device=t.device) % 2 == 1
    # the half-way point belongs to the even neighbour: the upper one where the lower's index is odd
    border = torch.where(odd, mid, torch.nextafter(mid, torch.full_like(mid, math.inf)))
    return torch.copysign(table[torch.bucketize(t.abs(), border, right=True)], t)


def power(e):
    """2^e in fp64, to the bit."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def scale_of(top):
    """The smallest power of two under which `top` is at most 448, by search."""
    e = torch.floor(torch.log2(top.clamp(min=1e-300))).clamp(min=-900) - 10
    for _ in range(4):
        e = e + (top > 448.0 * power(e))
    return power(e.clamp(-127, 127))


def rows64(t):
    """(values in units of their scale [rows][Kp], scales [Kp / 128][rows]) of t [rows][cols]."""
    rows, cols = t.shape
    full = torch.zeros((rows, up(cols)), dtype=torch.float64, device=t.device)
    full[:, :cols] = t
    full = full.view(rows, -1, 128)
    e = scale_of(full.abs().max(-1).values)
    return nearest(full / e[..., None]).reshape(rows, -1), e.t().contiguous()


def blocks64(w):
    n, k = w.shape
    full = torch.zeros((up(n), up(k)), dtype=torch.float64, device=w.device)
    full[:n, :k] = w
    e = scale_of(torch.nn.functional.max_pool2d(full.abs()[None], 128)[0])
    return nearest(full / e.repeat_interleave(128, 0).repeat_interleave(128, 1))[:n].contiguous(), e


def numbers(codes):
    """e4m3 bytes as fp64, by the format's fields."""
    b = codes.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m / 512, power(e - 7) * (1 + m / 8))
    return torch.where(b >= 128, -v, v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def out(how, y):
        if how == "same":
            return {"y": y}
        v, e = rows64(y)
        return {"y": v, "scale": e}

    if op in ("dispatch", "combine", "combine_grad"):
        ids = s["IDS"].view(-1)
        rows = torch.cat([torch.nonzero(ids == e).view(-1) for e in range(case["experts"])])  # slots, by expert
        token, n = rows // case["topk"], len(rows)
        if op == "dispatch":
            y = torch.zeros((len(ids), case["cols"]), dtype=torch.float64, device=ids.device)
            y[:n] = s["X"].double()[token]
            return {"place": None, "order": None, "offsets": None, **out(case["out"], y)}
        w = s["WEIGHTS"].double().view(-1)[rows].unsqueeze(1)
        x = s["X"].double()[:n]
        if op == "combine":
            y = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device=ids.device)
            y.index_add_(0, token, x * w)
            return y if s["R"] is None else y + s["R"].double()
        dx = torch.zeros((len(ids), case["cols"]), dtype=torch.float64, device=ids.device)
        dy = s["DY"].double()[token]
        dx[:n] = dy * w
        dw = torch.zeros(len(ids), dtype=torch.float64, device=ids.device)
        dw[rows] = (dy * x).sum(1)
        return {"dweights": dw.view(case["tokens"], -1), **out(case["out"], dx)}
    if op == "quant":
        if case["form"] == "rows":
            return out("e4m3", s["X"].double())
        a, b = [blocks64(w.double()) for w in s["X"]], [blocks64(w.double().t()) for w in s["X"]]
        return {"q": torch.stack([v for v, _ in a]), "scale": torch.stack([e for _, e in a]),
                "qt": torch.stack([v for v, _ in b]), "scalet": torch.stack([e for _, e in b])}
    if op == "glu":
        x = s["X"].double()
        g, u = x[:, :case["cols"]], x[:, case["cols"]:]
        y = out(case["out"], g * torch.sigmoid(g) * u)
        (vg, eg), (vu, eu) = rows64(g), rows64(u)

        def back(v, e):
            return (v.view(len(v), -1, 128) * e.t().unsqueeze(2)).view(len(v), -1)[:, :case["cols"]]
        a, b, dy = back(vg, eg), back(vu, eu), s["DY"].double()
        t = torch.sigmoid(a)
        dx = torch.cat((dy * b * (t + a * t * (1 - t)), dy * a * t), 1)
        return {"y": y, "kept": torch.cat((vg, vu), 1), "kscale": torch.cat((eg, eu)), "dx": out(case["dout"], dx)}
    ends = s["OFFSETS"].tolist()

    def spread(codes, scale):
        return numbers(codes) * power(scale.long() - 127).t().repeat_interleave(128, 1)

    a = spread(s["A"], s["SA"])
    if op == "product":
        c = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=a.device)
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                sb = power(s["SB"][e].long() - 127).repeat_interleave(128, 0)[:case["n"]].repeat_interleave(128, 1)
                c[lo:hi] = a[lo:hi] @ (numbers(s["B"][e]) * sb).t().contiguous()
        return c
    d = s["D"].double() if s["SD"] is None else spread(s["D"], s["SD"])
    d, a = d[:, :case["n"]], a[:, :case["k"]]
    db = torch.stack([d[lo:hi].t().contiguous() @ a[lo:hi].contiguous() for lo, hi in zip(ends, ends[1:])])
    return db if s["BEFORE"] is None else db + s["BEFORE"].double()
