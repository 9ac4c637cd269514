"""Host-side checks of gradient clipping's C ABI and torch entry points, no GPU
needed: exports, refusals before any device memory is touched (the pointers here
are not device memory), and workspace sizes."""
import ctypes
import os
import re

import pytest
import torch

from matrix_aware_optimizer_muon_amd import _lib as L
from matrix_aware_optimizer_muon_amd import clip

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "muon_clip.h")
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
P = 1 << 20
EXPORTED = {"muon_clip_workspace", "muon_grad_norm", "muon_clip_grads"}


def abi():
    lib = L.load()
    V, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    for name, args in {"muon_clip_workspace": [I, V, V, V], "muon_grad_norm": [I, V, V, V, V, V, S, V],
                       "muon_clip_grads": [I, V, V, V, V, V, F, V, V, S, V]}.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    return lib


def arrays(g, n, types):
    return (ctypes.c_void_p * len(g))(*g), (ctypes.c_int64 * len(n))(*n), (ctypes.c_int * len(types))(*types)


def call(g=(P, 2 * P), n=(100, 200), types=(0, 1), out=None, otypes=None, max_norm=1.0, norm=8 * P, ws=16 * P, wsb=1 << 20,
         num=None):
    out, otypes = out or g, otypes or types
    a, b, c = arrays(g, n, types)
    d, _, e = arrays(out, n, otypes)
    return abi().muon_clip_grads(len(n) if num is None else num, a, b, c, d, e, max_norm, norm, ws, wsb, None)


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M))
    assert names == EXPORTED
    lib = L.load()
    for n in names:
        assert hasattr(lib, n)


@pytest.mark.parametrize("kw, want", [
    ({"num": -1}, INVALID), ({"n": (-1, 5)}, INVALID), ({"types": (0, 2)}, INVALID), ({"otypes": (0, 7)}, INVALID),
    ({"n": (5, (1 << 40) + 1)}, UNSUPPORTED), ({"n": (1 << 40, 1)}, UNSUPPORTED), ({"g": (0, P)}, INVALID),
    ({"g": (P + 2, 2 * P)}, INVALID), ({"g": (P, 2 * P + 1)}, INVALID), ({"norm": 0}, INVALID), ({"norm": P + 2}, INVALID),
    ({"max_norm": -1.0}, INVALID), ({"max_norm": float("nan")}, INVALID), ({"out": (P, 0)}, INVALID),
    ({"out": (P, 2 * P), "otypes": (1, 1)}, INVALID),                         # in place with another type
    ({"g": (P, P + 396)}, INVALID), ({"g": (P, P), "types": (0, 0)}, INVALID),      # what is written overlaps
    ({"out": (4 * P, 4 * P + 396)}, INVALID), ({"out": (2 * P + 396, 4 * P)}, INVALID),
    ({"g": (P, P), "types": (0, 0), "out": (P, 4 * P)}, INVALID),
    ({"norm": P + 8}, INVALID), ({"wsb": 8}, SMALL), ({"ws": 0}, INVALID), ({"ws": P + 8}, INVALID)])
def test_refusals(kw, want):
    assert call(**kw) == want


def test_norm_refusals():
    a, b, c = arrays((P,), (100,), (0,))
    f = abi().muon_grad_norm
    assert f(1, a, b, c, 0, P, 1 << 20, None) == INVALID
    assert f(1, a, b, c, P, P, 0, None) == SMALL
    assert f(1, None, b, c, P, P, 1 << 20, None) == INVALID
    assert f(1, a, None, c, P, P, 1 << 20, None) == INVALID


@pytest.mark.parametrize("n", [(1,), (0,), (2048,), (2049,), (1 << 30, 5, 0), (3, 4, 5, 1 << 22)])
def test_workspaces(n):
    _, b, c = arrays((P,) * len(n), n, (0,) * len(n))
    z = ctypes.c_size_t()
    assert abi().muon_clip_workspace(len(n), b, c, ctypes.addressof(z)) == OK
    # a partial sum for each workgroup
    assert z.value % 8 == 0 and sum(v > 0 for v in n) <= z.value // 8 <= 4096 + len(n)
    assert abi().muon_clip_workspace(len(n), b, c, None) == INVALID


def test_entry_points_refuse():
    g = torch.zeros(4, 6)
    for call_, match in [
            (lambda: clip.grad_norm([]), "at least one"), (lambda: clip.grad_norm(3), "sequence"),
            (lambda: clip.grad_norm([None]), "must be a tensor"), (lambda: clip.grad_norm([g.double()]), "fp32 or bf16"),
            (lambda: clip.grad_norm([g[:, :3]]), "dense"), (lambda: clip.grad_norm([g[:1].expand(4, 6)]), "dense"),
            (lambda: clip.grad_norm([g]), "CUDA"), (lambda: clip.clip_grad_norm([g], 1.0), "CUDA")]:
        with pytest.raises(ValueError, match=match):
            call_()
