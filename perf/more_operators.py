"""Measured cases of the 8-bit floating-point layer's operators and of gradient
clipping: rows and weights put in 8-bit floating point with a scale for each
block of 128, the product of the two with its two gradient products, the same
three grouped by expert with ragged sizes, and the global gradient norm over
many tensors with clipping.

`run` computes a case in its plain form (elementary torch operations), or, with
`own` set, through this library's entry points; `exact` gives the same outputs
from the definitions in 64 bits.

The 8-bit form of a block v (128 consecutive values of a row, or 128 x 128
values of a weight matrix): scale = 2^e with the smallest e >= -126 for which
max|v| <= 448 * 2^e, q = v / scale rounded to e4m3 (nearest, ties to even).
Scales are held as their exponent e + 127 (e8m0).  8-bit values are returned
as the values q * scale that they stand for, scales as their exponents.
"""
import math
import random

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LAYER = [(3584, 3584), (512, 3584), (512, 3584), (3584, 3584), (18944, 3584), (18944, 3584), (3584, 18944)]


def listed():
    return [
        # one generated token's activations on their way into a projection: latency
        {"name": "rows 1 token", "op": "rows", "rows": 1, "cols": 3584, "dtype": "bf16"},
        # a gate projection's fp32 master weights put in 8 bits for a step
        {"name": "weights 18944x3584", "op": "weights", "rows": 18944, "cols": 3584, "dtype": "f32"},
        # one generated token through the gate projection: reads the weights
        {"name": "product 1 token", "op": "product", "t": 1, "n": 18944, "k": 3584, "dtype": "bf16"},
        # a training step's gate projection
        {"name": "product 4096 tokens", "op": "product", "t": 4096, "n": 18944, "k": 3584, "dtype": "bf16"},
        # a short odd sequence through a projection of odd widths, fp32 out
        {"name": "input gradient 333x1023", "op": "grad_input", "t": 333, "n": 1000, "k": 1023, "dtype": "f32"},
        # a square projection's weight gradient, fp32 for the optimizer
        {"name": "weight gradient 3584x3584", "op": "grad_weight", "t": 8192, "n": 3584, "k": 3584, "dtype": "f32"},
        # two generated tokens, eight experts each of 64: reads 14 experts' weights
        {"name": "experts 16 rows", "op": "experts", "rows": 16, "idle": 0, "experts": 64, "active": 14, "n": 1408, "k": 2048, "dtype": "bf16"},
        # a training step's first expert projections, 4096 tokens to eight experts each
        {"name": "experts 32768 rows", "op": "experts", "rows": 32768, "idle": 0, "experts": 64, "active": 64, "n": 2816, "k": 2048, "dtype": "bf16"},
        # their input gradient, in a buffer with rows to spare behind the last expert's
        {"name": "experts input gradient", "op": "experts_input", "rows": 16640, "idle": 1000, "experts": 64, "active": 61, "n": 1408, "k": 2048, "dtype": "bf16"},
        # their weight gradients, fp32 for the optimizer; some experts got no token
        {"name": "experts weight gradient", "op": "experts_weight", "rows": 16384, "idle": 0, "experts": 64, "active": 61, "n": 1408, "k": 2048, "dtype": "f32"},
        # the gains of a few norms: latency
        {"name": "clip 8 small", "op": "clip", "shapes": "vectors 8 3584", "dtype": "f32", "std": 1e-3},
        # the gradients of four layers' projections ahead of the optimizer's step
        {"name": "clip 4 layers", "op": "clip", "shapes": "layers 4", "dtype": "f32", "std": 1e-3},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm; half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["rows", "weights", "product", "grad_input", "grad_weight", "experts", "experts", "experts_input", "experts_weight", "clip"])
    while True:
        if op in ("rows", "weights"):
            case = {"op": op, "rows": _size(rng, 1, 32768), "cols": _size(rng, 33, 20480), "dtype": rng.choice(["bf16", "f32"])}
            if case["rows"] * case["cols"] <= 18944 * 3584:
                return case
        elif op == "clip":  # matrices and vectors of a seeded choice
            case = {"op": op, "shapes": "mixed %d %d" % (_size(rng, 1, 200), rng.randrange(1 << 20)), "dtype": rng.choice(["bf16", "f32"]), "std": rng.choice([1e-5, 1e-3])}
            if sum(a * b for a, b in _shapes(case)) <= 4 * 233046016:
                return case
        elif op in ("product", "grad_input", "grad_weight"):
            case = {"op": op, "t": _size(rng, 1, 8192), "n": _size(rng, 33, 18944), "k": _size(rng, 33, 18944), "dtype": rng.choice(["bf16", "f32"])}
            if case["t"] * case["n"] * case["k"] <= 4096 * 18944 * 3584:
                return case
        else:
            rows, experts = _size(rng, 1, 32768), _size(rng, 2, 256)
            active = max(1, min(experts, rows) - (rng.randrange(1 + min(experts, rows) // 4) if rng.random() < 0.5 else 0))
            idle = rng.randrange(1 + (rows - active) // 8) if rng.random() < 0.5 else 0
            case = {"op": op, "rows": rows, "idle": idle, "experts": experts, "active": active, "n": _size(rng, 64, 4096), "k": _size(rng, 64, 4096), "dtype": rng.choice(["bf16", "f32"])}
            size = case["n"] * case["k"]
            if rows * size <= 32768 * 2816 * 2048 and experts * size <= 64 * 2816 * 2048:
                return case


def _shapes(case):
    """The (rows, columns) of a clip case's tensors."""
    kind, *v = case["shapes"].split()
    if kind == "layers":
        return LAYER * int(v[0])
    if kind == "mixed":
        r = random.Random(int(v[1]))
        top = math.exp(r.uniform(math.log(64), math.log(8192)))
        return [(1 if r.random() < 0.3 else _size(r, 1, top), _size(r, 1, top)) for _ in range(int(v[0]))]
    return [(1, int(v[1]))] * int(v[0])


def _exponents(top):
    """e + 127 of a block's scale, from its largest magnitude in fp32."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return (torch.where(top > 0, e, torch.full_like(e, -126)).clamp(min=-126) + 127).to(torch.uint8)


def _power(b):
    """2^(b - 127) from its bits (1 <= b <= 254)."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _wide(s, rows, cols, square):
    """Scales spread over the elements they belong to."""
    s = s.repeat_interleave(BLOCK, dim=-1)[..., :cols]
    return s.repeat_interleave(BLOCK, dim=-2)[..., :rows, :] if square else s


def _to8(v, square):
    """(q as e4m3, exponents) of fp32 (..., rows, cols)."""
    rows, cols = v.shape[-2:]
    pad = torch.nn.functional.pad(v.abs(), (0, -cols % BLOCK, 0, -rows % BLOCK if square else 0))
    top = pad.unflatten(-1, (-1, BLOCK)).amax(dim=-1)
    if square:
        top = top.unflatten(-2, (-1, BLOCK)).amax(dim=-2)
    b = _exponents(top)
    return (v / _wide(_power(b), rows, cols, square)).to(torch.float8_e4m3fn), b


def _plain(q, b, square):
    """The fp32 values that 8-bit ones stand for."""
    return q.float() * _wide(_power(b), q.shape[-2], q.shape[-1], square)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 23)
    return g


def _acts(g, rows, cols):
    """Activations: unit normal, channels of unlike size, a few large ones."""
    channel = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    channel = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 12 * channel, channel)
    return torch.randn(rows, cols, generator=g, device="cuda") * channel


def _held(v, square):
    """8-bit rows as a program keeps them: each starts at a multiple of 16 bytes."""
    q, b = _to8(v, square)
    cols = q.shape[-1]
    room = torch.zeros(*q.shape[:-1], (cols + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    room[..., :cols] = q.view(torch.uint8)
    return room.view(torch.float8_e4m3fn)[..., :cols], b


def _sizes(case, seed):
    """Rows of each expert: some get none, some many."""
    r = random.Random(seed * 31 + 5)
    busy = sorted(r.sample(range(case["experts"]), case["active"]))
    share = [math.exp(0.7 * r.gauss(0, 1)) for _ in busy]
    left = case["rows"] - case["idle"] - case["active"]
    at = [0] + [int(left * sum(share[:i + 1]) / sum(share)) for i in range(len(share) - 1)] + [left]
    sizes = [0] * case["experts"]
    for i, e in enumerate(busy):
        sizes[e] = 1 + at[i + 1] - at[i]
    return sizes


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "case": case, "dtype": dt}
    if op == "rows":
        s["x"] = _acts(g, case["rows"], case["cols"]).to(dt)
    elif op == "weights":
        s["x"] = (0.02 * torch.randn(case["rows"], case["cols"], generator=g, device="cuda")).to(dt)
    elif op == "clip":
        shapes = _shapes(case)
        flat = torch.randn(sum(a * b for a, b in shapes), generator=g, device="cuda").mul_(case["std"]).to(dt)
        # gradients and the optimizer's inputs, each in one bucket
        s["out"] = torch.zeros_like(flat)
        for name, bucket in (("grads", flat), ("outs", s["out"])):
            s[name] = [v.view(a, b) if a > 1 else v for v, (a, b) in zip(bucket.split([a * b for a, b in shapes]), shapes)]
    else:
        n, k = case["n"], case["k"]
        many = op.startswith("experts")
        t = case["rows"] if many else case["t"]
        s["sizes"] = _sizes(case, seed) if many else [t]
        if many:
            s["ends"] = torch.tensor(s["sizes"], device="cuda").cumsum(0).to(torch.int32)
        kind = s["kind"] = op if not many else {"experts": "product", "experts_input": "grad_input", "experts_weight": "grad_weight"}[op]
        if kind != "grad_input":
            s["x"] = _held(_acts(g, t, k), False)
        if kind != "grad_weight":
            shape = (case["experts"], n, k) if many else (n, k)
            s["w"] = _held(0.02 * torch.randn(*shape, generator=g, device="cuda"), True)
        if kind != "product":
            s["dy"] = (1e-3 * torch.randn(t, n, generator=g, device="cuda")).to(torch.bfloat16)
    return s


def _run_own(s):
    from matrix_aware_optimizer_muon_amd import clip
    from matrix_aware_optimizer_muon_amd import float8 as f8

    def f8_of(v):
        return f8.F8(v[0], v[1].view(torch.float8_e8m0fnu))

    op, dt = s["op"], s["dtype"]
    if op in ("rows", "weights"):
        kept = f8.quantize(s["x"]) if op == "rows" else f8.quantize_weight(s["x"])
        return {"x": f8.dequantize(kept, dt), "scale": kept.scale.view(torch.uint8)}
    if op == "clip":
        return {"norm": clip.clip_grad_norm(s["grads"], 1.0, out=s["outs"]), "grads": s["out"]}
    ends = s.get("ends")
    if s["kind"] == "product":
        return f8.matmul(f8_of(s["x"]), f8_of(s["w"]), ends=ends, dtype=dt)
    if s["kind"] == "grad_input":
        return f8.grad_input(s["dy"], f8_of(s["w"]), ends=ends, dtype=dt)
    return f8.grad_weight(s["dy"], f8_of(s["x"]), ends=ends, dtype=dt)


def run(s):
    if own:
        return _run_own(s)
    op, dt = s["op"], s["dtype"]
    if op in ("rows", "weights"):
        q, b = _to8(s["x"].float(), op == "weights")
        return {"x": _plain(q, b, op == "weights").to(dt), "scale": b}
    if op == "clip":
        # (a long sum of squares: 64 bits)
        norm = torch.stack([v.double().square().sum() for v in s["grads"]]).sum().sqrt()
        by = torch.where(norm > 1.0, 1.0 / norm, torch.ones_like(norm)).float()
        s["out"].copy_(torch.cat([(v.float() * by).reshape(-1) for v in s["grads"]]))
        return {"norm": norm.float(), "grads": s["out"]}
    many, sizes = "ends" in s, s["sizes"]
    if s["kind"] == "grad_weight":
        x, dy = _plain(*s["x"], False), s["dy"].float()
        parts = [b.t() @ a for a, b in zip(x[:sum(sizes)].split(sizes), dy[:sum(sizes)].split(sizes))]
        return (torch.stack(parts) if many else parts[0]).to(dt)
    w = _plain(*s["w"], True)
    w = w if many else w[None]
    if s["kind"] == "product":
        x = _plain(*s["x"], False)
        parts = [a @ m.t() for a, m in zip(x[:sum(sizes)].split(sizes), w)]
    else:
        x = s["dy"].float()
        parts = [a @ m for a, m in zip(x[:sum(sizes)].split(sizes), w)]
    # (rows behind the last expert's belong to none: zero)
    return torch.nn.functional.pad(torch.cat(parts), (0, 0, 0, x.shape[0] - sum(sizes))).to(dt)


def _powers(lo, hi):
    """2^lo to 2^hi in 64 bits (a pow on the GPU is not exact)."""
    return torch.tensor([math.ldexp(1.0, e) for e in range(lo, hi + 1)], dtype=torch.float64, device="cuda")


def _exact8(v, square):
    """The values that the 8-bit form of fp64 (rows, cols) stands for, and the
    exponents, block by block of columns, by searching the bounds."""
    scales, steps = _powers(-126, 121), _powers(-9, 5)
    bounds = 448.0 * scales
    out, kept = torch.empty_like(v), []
    for c in range(0, v.shape[1], BLOCK):
        part = v[:, c:c + BLOCK]
        top = part.abs().amax(dim=1)
        if square:
            whole = torch.zeros(-(-len(top) // BLOCK) * BLOCK, dtype=torch.float64, device=v.device)
            whole[:len(top)] = top
            top = whole.view(-1, BLOCK).amax(dim=1)
        at = torch.searchsorted(bounds, top)
        kept.append(at + 1)
        scale = scales[at].repeat_interleave(BLOCK)[:v.shape[0], None] if square else scales[at][:, None]
        u = part / scale
        # e4m3's spacing: 2^-9 under 2^-6, else an eighth of the power below
        step = steps[torch.frexp(u.abs().clamp(min=2.0 ** -6))[1].long() - 4 + 9]
        out[:, c:c + BLOCK] = torch.round(u / step) * step * scale
    return out, torch.stack(kept, dim=1)


def _double(held, square):
    q, b = held
    scale = _powers(-127, 127)[b.long()]
    scale = scale[..., torch.arange(q.shape[-1], device=q.device) // BLOCK]
    if square:
        scale = scale[..., torch.arange(q.shape[-2], device=q.device) // BLOCK, :]
    return q.double() * scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rows", "weights"):
        x, e = _exact8(s["x"].double(), op == "weights")
        return {"x": x, "scale": e}
    if op == "clip":
        total = sum(float(torch.linalg.vecdot(v.double().reshape(-1), v.double().reshape(-1))) for v in s["grads"])
        norm = math.sqrt(total)
        by = min(1.0, 1.0 / norm) if norm else 1.0
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": torch.cat([v.double().reshape(-1) for v in s["grads"]]) * by}
    many = "ends" in s
    x = s["dy"].double() if s["kind"] == "grad_input" else _double(s["x"], False)
    if s["kind"] == "grad_weight":
        dy, at, parts = s["dy"].double(), 0, []
        for size in s["sizes"]:
            parts.append(torch.mm(dy[at:at + size].t().contiguous(), x[at:at + size]))
            at += size
        return torch.stack(parts) if many else parts[0]
    w = _double(s["w"], True)
    w = w if many else w[None]
    y, at = torch.zeros(x.shape[0], w.shape[1 if s["kind"] == "product" else 2], dtype=torch.float64, device="cuda"), 0
    for m, size in zip(w, s["sizes"]):
        y[at:at + size] = torch.mm(x[at:at + size], m.t().contiguous() if s["kind"] == "product" else m)
        at += size
    return y


def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("rows", "weights"):  # read, and the restored values written
        cells = case["rows"] * case["cols"]
        return {"bytes": 2 * size * cells + cells // BLOCK, "flops": 3 * cells}
    if op == "clip":  # each gradient read, its clipped form written
        cells = sum(a * b for a, b in _shapes(case))
        return {"bytes": 2 * size * cells, "flops": 3 * cells}
    n, k = case["n"], case["k"]
    if op.startswith("experts"):
        t, read, held = case["rows"] - case["idle"], case["active"], case["experts"]
    else:
        t, read, held = case["t"], 1, 1
    kind = op if op in ("product", "grad_input", "grad_weight") else {"experts": "product", "experts_input": "grad_input", "experts_weight": "grad_weight"}[op]
    moved = {"product": t * k + read * n * k + size * t * n,
             "grad_input": 2 * t * n + read * n * k + size * t * k,
             "grad_weight": 2 * t * n + t * k + size * held * n * k}[kind]
    return {"bytes": moved, "flops": 2 * t * n * k}
