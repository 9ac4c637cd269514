"""Measured cases of the 8-bit linear layer's operators: the root-mean-square
norm with the residual's addition and an 8-bit output, its backward pass, the
8-bit activation checkpoint (save and restore), the 8-bit integer matrix
product, and the two gradient products that read 8-bit rows.

`run` computes a case in its plain form (elementary torch operations in 32
bits), or, with `own` set, through this library's entry points; `exact` gives
the same outputs from the definitions in 64 bits.

The 8-bit form of a row v: scale = 2^e with the smallest e >= -126 for which
max|v| <= 127 * 2^e, q = round-half-to-even(v / scale).  8-bit rows are
returned as the values q * scale.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one generated token through a hidden-3584 model's norm: latency
        {"name": "norm 1 token", "op": "norm", "rows": 1, "cols": 3584, "dtype": "bf16", "residual": True, "q8": False},
        # the norm ahead of a layer's projections in training, 8192 tokens a
        # step: its 8-bit rows are the product's operand and the checkpoint
        {"name": "norm 8192 tokens, 8 bits", "op": "norm", "rows": 8192, "cols": 3584, "dtype": "bf16", "residual": True, "q8": True},
        # the same norm's backward pass, the residual stream's gradient added
        {"name": "norm backward", "op": "norm_back", "rows": 8192, "cols": 3584, "dtype": "bf16", "h8": False, "dh": True},
        # ragged batch and odd width, the norm's input kept in 8 bits
        {"name": "norm backward, 8-bit input", "op": "norm_back", "rows": 2047, "cols": 4095, "dtype": "bf16", "h8": True, "dh": False},
        # an MLP's hidden activations saved in 8 bits and restored
        {"name": "checkpoint 4096x18944", "op": "checkpoint", "rows": 4096, "cols": 18944, "dtype": "bf16"},
        # a key projection's fp32 master weights put in 8 bits for a step
        {"name": "checkpoint 512x3584 f32", "op": "checkpoint", "rows": 512, "cols": 3584, "dtype": "f32"},
        # one generated token through the gate projection: reads the weights
        {"name": "product 1 token", "op": "product", "t": 1, "n": 18944, "k": 3584, "dtype": "bf16"},
        # a training step's gate projection
        {"name": "product 4096 tokens", "op": "product", "t": 4096, "n": 18944, "k": 3584, "dtype": "bf16"},
        # a short odd sequence through a narrow projection, odd inner width
        {"name": "input gradient 77x1023", "op": "grad_input", "t": 77, "n": 512, "k": 1023, "dtype": "f32"},
        # the gate projection's input gradient
        {"name": "input gradient 4096 tokens", "op": "grad_input", "t": 4096, "n": 18944, "k": 3584, "dtype": "bf16"},
        # a key projection's weight gradient: few outputs, a long sum
        {"name": "weight gradient 512x3584", "op": "grad_weight", "t": 8192, "n": 512, "k": 3584, "dtype": "bf16"},
        # the gate projection's weight gradient, fp32 for the optimizer
        {"name": "weight gradient 18944x3584", "op": "grad_weight", "t": 4096, "n": 18944, "k": 3584, "dtype": "f32"},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm; half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "norm_back", "checkpoint", "product", "grad_input", "grad_weight"])
    while True:
        if op in ("norm", "norm_back", "checkpoint"):
            case = {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 33, 20480), "dtype": rng.choice(["bf16", "bf16", "f32"])}
            if case["rows"] * case["cols"] > 8192 * 3584:
                continue
            if op == "norm":
                case.update(residual=rng.random() < 0.7, q8=rng.random() < 0.6)
            elif op == "norm_back":
                case.update(h8=rng.random() < 0.4, dh=rng.random() < 0.6)
            return case
        case = {"op": op, "t": _size(rng, 1, 8192), "n": _size(rng, 33, 18944), "k": _size(rng, 33, 18944), "dtype": rng.choice(["bf16", "f32"])}
        if case["t"] * case["n"] * case["k"] <= 4096 * 18944 * 3584:
            return case


def _to8(v):
    """The 8-bit form of fp32 rows: (q as fp32, scale), by exponents."""
    top = v.abs().amax(dim=1, keepdim=True)
    m, e = torch.frexp(top)
    e = torch.clamp(torch.where(m <= 127 / 128, e - 7, e - 6), min=-126)
    e = torch.where(top > 0, e, torch.full_like(e, -126))
    scale = torch.ldexp(torch.ones_like(top), e)
    return torch.round(v / scale), scale


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _acts(g, rows, cols):
    """Activations: unit normal, channels of unlike size, a few large ones."""
    channel = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    channel = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 12 * channel, channel)
    return torch.randn(rows, cols, generator=g, device="cuda") * channel


def _rows8(v):
    q, scale = _to8(v)
    return q.to(torch.int8), scale[:, 0].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "case": case, "dtype": dt}
    if op in ("norm", "norm_back", "checkpoint"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _acts(g, rows, cols).to(dt)
        s["w"] = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
        if op == "norm":
            s["residual"] = torch.randn(rows, cols, generator=g, device="cuda").to(dt) if case["residual"] else None
        if op == "norm_back":
            s["dy"] = (1e-3 * torch.randn(rows, cols, generator=g, device="cuda")).to(dt)
            s["dh"] = (1e-3 * torch.randn(rows, cols, generator=g, device="cuda")).to(dt) if case["dh"] else None
            h = s["x"].float()
            s["rstd"] = torch.rsqrt(h.square().mean(dim=1) + EPS)
            if case["h8"]:
                s["h"], s["hscale"] = _rows8(h)
                del s["x"]
            else:
                s["h"] = s.pop("x")
        return s
    t, n, k = case["t"], case["n"], case["k"]
    if op in ("product", "grad_weight"):
        s["xq"], s["xs"] = _rows8(_acts(g, t, k))
    if op in ("product", "grad_input"):
        s["wq"], s["ws"] = _rows8(0.02 * torch.randn(n, k, generator=g, device="cuda"))
    if op != "product":
        s["dy"] = (1e-3 * torch.randn(t, n, generator=g, device="cuda")).to(torch.bfloat16)
    return s


def _run_own(s):
    from matrix_aware_optimizer_muon_amd import linear8 as l8

    op = s["op"]
    if op == "norm":
        y, h, rstd = l8.rmsnorm(s["x"], s["w"], residual=s["residual"], eps=EPS, q8=s["case"]["q8"])
        if s["case"]["q8"]:
            return {"y": l8.dequantize(y, s["dtype"]), "scale": y.scale, "h": h, "rstd": rstd}
        return {"y": y, "h": h, "rstd": rstd}
    if op == "norm_back":
        h = l8.Q8(s["h"], s["hscale"]) if s["case"]["h8"] else s["h"]
        dx, dw = l8.rmsnorm_backward(s["dy"], h, s["rstd"], s["w"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "checkpoint":
        kept = l8.quantize(s["x"])
        return {"x": l8.dequantize(kept, s["dtype"]), "scale": kept.scale}
    if op == "product":
        return l8.matmul(l8.Q8(s["xq"], s["xs"]), l8.Q8(s["wq"], s["ws"]), dtype=s["dtype"])
    if op == "grad_input":
        return l8.grad_input(s["dy"], l8.Q8(s["wq"], s["ws"]), dtype=s["dtype"])
    return l8.grad_weight(s["dy"], l8.Q8(s["xq"], s["xs"]), dtype=s["dtype"])


def run(s):
    if own:
        return _run_own(s)
    op, dt = s["op"], s["dtype"]
    if op == "norm":
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(dim=1) + EPS)
        y = hf * rstd[:, None] * s["w"]
        if s["case"]["q8"]:
            q, scale = _to8(y)
            return {"y": (q * scale).to(dt), "scale": scale[:, 0], "h": h, "rstd": rstd}
        return {"y": y.to(dt), "h": h, "rstd": rstd}
    if op == "norm_back":
        h = s["h"].float()
        if s["case"]["h8"]:
            h = h * s["hscale"][:, None]
        hat = h * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["w"]
        dx = s["rstd"][:, None] * (g - hat * (g * hat).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dw": (dy * hat).sum(dim=0)}
    if op == "checkpoint":
        q, scale = _to8(s["x"].float())
        return {"x": (q * scale).to(dt), "scale": scale[:, 0]}
    if op == "product":
        acc = s["xq"].float() @ s["wq"].float().t()
        return (acc * s["xs"][:, None] * s["ws"]).to(dt)
    if op == "grad_input":
        return (s["dy"].float() @ (s["wq"].float() * s["ws"][:, None])).to(dt)
    return (s["dy"].float().t() @ (s["xq"].float() * s["xs"][:, None])).to(dt)


def _near8(v):
    """The 8-bit form of fp64 rows, by looking the bound up in a table."""
    exps = torch.arange(-126, 128, device=v.device)
    bounds = torch.ldexp(torch.full((254,), 127.0, dtype=torch.float64, device=v.device), exps)
    at = torch.searchsorted(bounds, v.abs().amax(dim=1))
    step = torch.ldexp(torch.ones(v.shape[0], dtype=torch.float64, device=v.device), exps[at])
    return torch.round(v / step[:, None]) * step[:, None], step


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(dt).double()  # the stream is kept in its type
        root = ((h * h).sum(1) / case["cols"] + EPS).sqrt()
        y = h / root[:, None] * s["w"].double()
        if case["q8"]:
            y, step = _near8(y)
            return {"y": y, "scale": step, "h": h, "rstd": 1 / root}
        return {"y": y, "h": h, "rstd": 1 / root}
    if op == "norm_back":
        h = s["h"].double() * (s["hscale"].double()[:, None] if case["h8"] else 1.0)
        r, dy = s["rstd"].double()[:, None], s["dy"].double()
        a = dy * s["w"].double()
        along = (a * h).sum(1, keepdim=True) / case["cols"]
        dx = a * r - h * along * r ** 3
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("td,td->d", dy, h * r)}
    if op == "checkpoint":
        x, step = _near8(s["x"].double())
        return {"x": x, "scale": step}
    if op == "product":
        return torch.mm(s["xq"].double() * s["xs"].double()[:, None], (s["wq"].double() * s["ws"].double()[:, None]).t().contiguous())
    if op == "grad_input":
        return torch.mm(s["dy"].double(), s["wq"].double() * s["ws"].double()[:, None])
    return torch.mm(s["dy"].double().t().contiguous(), s["xq"].double() * s["xs"].double()[:, None])


def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_back", "checkpoint"):
        rows, cols = case["rows"], case["cols"]
        if op == "norm":  # x and the residual read, h and y written
            per = 4 * size if case["residual"] else 2 * size
            return {"bytes": rows * cols * per + 4 * cols + 4 * rows, "flops": 6 * rows * cols}
        if op == "norm_back":  # dy, h and dh read, dx written
            per = 2 * size + (1 if case["h8"] else size) + (size if case["dh"] else 0)
            return {"bytes": rows * cols * per + 8 * cols + 4 * rows, "flops": 10 * rows * cols}
        return {"bytes": 2 * size * rows * cols + 4 * rows, "flops": 4 * rows * cols}
    t, n, k = case["t"], case["n"], case["k"]
    moved = {"product": t * k + n * k + size * t * n + 4 * (t + n),
             "grad_input": 2 * t * n + n * k + size * t * k + 4 * n,
             "grad_weight": 2 * t * n + t * k + size * n * k + 4 * t}[op]
    return {"bytes": moved, "flops": 2 * t * n * k}
