"""ctypes view of include/muon_float8.h, plain forms and exact data for the tests."""
import ctypes

import numpy as np
import torch

from matrix_aware_optimizer_muon_amd import float8 as f8
from matrix_aware_optimizer_muon_amd._lib import load

EXPORTED = ("muon_f8_quantize", "muon_f8_dequantize", "muon_f8_workspace", "muon_f8_matmul", "muon_f8_grad_input",
            "muon_f8_grad_weight")
MATMUL, GRAD_INPUT, GRAD_WEIGHT = 0, 1, 2
CODE = {torch.float32: 0, torch.bfloat16: 1}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def abi():
    lib = load()
    P, I, L, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "muon_f8_quantize": [P, L, L, I, L, L, L, I, P, L, L, P, P],
        "muon_f8_dequantize": [P, L, L, P, L, L, L, I, P, L, L, I, P],
        "muon_f8_workspace": [I, P, L, I, L, L, L, L, I, P],
        "muon_f8_matmul": [P, L, P, P, L, L, P, P, L, L, L, L, P, L, I, P, S, P],
        "muon_f8_grad_input": [P, L, P, L, L, P, P, L, L, L, L, P, L, I, P, S, P],
        "muon_f8_grad_weight": [P, L, P, L, P, P, L, L, L, L, P, L, L, I, I, P, S, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    return lib


CHOICE = ("kind", "few", "tile", "groups", "pack", "direct", "split", "splits")


def choice(product, a, lda, grouped, experts, t, n, k, bf16):
    """How a product runs (csrc/float8.h)."""
    f = load().muon_f8_choice
    f.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int] + [ctypes.c_int64] * 4 + [ctypes.c_int, ctypes.c_void_p]
    f.restype = None
    out = (ctypes.c_int64 * len(CHOICE))()
    f(product, a, lda, int(grouped), experts, t, n, k, int(bf16), out)
    return dict(zip(CHOICE, out))


def workspace(product, a, lda, grouped, experts, t, n, k, dtype=1):
    z = ctypes.c_size_t()
    assert abi().muon_f8_workspace(product, a, lda, int(grouped), experts, t, n, k, dtype, ctypes.addressof(z)) == 0
    return z.value


def blocks(n):
    return (n + 127) // 128


def spread(e, shape, square):
    """Scale exponents (e + 127, int) over the elements they belong to, as fp64 powers."""
    rows, cols = shape[-2:]
    e = e.repeat_interleave(128, dim=-1)[..., :cols]
    if square:
        e = e.repeat_interleave(128, dim=-2)[..., :rows, :]
    return powers(-127, 128, e.device)[e.long()]


def powers(lo, hi, device):
    """2^lo to 2^hi in 64 bits (torch's pow and ldexp on the GPU are not exact); 2^128 stands for NaN."""
    v = np.ldexp(1.0, np.arange(lo, hi + 1))
    v[np.arange(lo, hi + 1) == 128] = np.nan
    return torch.from_numpy(v).to(device)


def values(x, square):
    """The fp64 values an F8 stands for."""
    return x.q.double() * spread(x.scale.view(torch.uint8), x.q.shape, square)


def held(q, e, gap=0x7F):
    """An F8 of e4m3 values q (as floats) and scale bytes e, its rows at
    multiples of 16 bytes, the gaps filled with NaN."""
    cols = q.shape[-1]
    room = torch.full((*q.shape[:-1], (cols + 15) // 16 * 16), gap, dtype=torch.uint8, device=q.device)
    room[..., :cols] = q.to(E4M3).view(torch.uint8)
    return f8.F8(room.view(E4M3)[..., :cols], e.to(torch.uint8).view(E8M0))


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def exact8(shape, seed, square, device="cuda"):
    """An F8 of small whole numbers times 1/2, 1 or 2: products of two of them
    (of at most 9 * 4, in steps of 1/4) add up exactly in fp32."""
    g = gen(seed, device)
    q = torch.randint(-3, 4, shape, generator=g, device=device).float()
    s = list(shape)
    s[-1] = blocks(s[-1])
    if square:
        s[-2] = blocks(s[-2])
    e = torch.randint(126, 129, s, generator=g, device=device)
    return held(q, e)


def exact_grad(shape, seed, device="cuda"):
    return torch.randint(-3, 4, shape, generator=gen(seed, device), device=device).to(torch.bfloat16)
