"""Host-side checks of the 8-bit floating-point layer's C ABI and torch entry
points, no GPU needed: exports, refusals before any device memory is touched
(the pointers here are not device memory), empty calls, and workspace sizes."""
import os
import re

import pytest
import torch

from float8_common import E4M3, E8M0, EXPORTED, abi, workspace
from matrix_aware_optimizer_muon_amd import _lib as L
from matrix_aware_optimizer_muon_amd import float8 as f8

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "muon_float8.h")
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
FAR = 1 << 60  # a distance whose multiples pass 64 bits
P = 1 << 20  # a non-null, 256-byte aligned address that is never read


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M))
    assert names == set(EXPORTED)
    lib = L.load()
    for n in names:
        assert hasattr(lib, n)


@pytest.mark.parametrize("kw, want", [
    ({"rows": 0, "x": 0, "q": 0}, OK), ({"cols": 0, "x": 0}, OK), ({"count": 0, "x": 0}, OK), ({"rows": -1}, INVALID),
    ({"cols": -1}, INVALID), ({"count": -1}, INVALID), ({"dtype": 5}, INVALID), ({"block": 64}, INVALID),
    ({"block": 0}, INVALID), ({"rows": (1 << 24) + 1}, UNSUPPORTED), ({"cols": (1 << 24) + 1}, UNSUPPORTED),
    ({"x": 0}, INVALID), ({"x": P + 1}, INVALID), ({"ldx": 63}, INVALID), ({"q": 0}, INVALID), ({"q": P + 8}, INVALID),
    ({"ldq": 72}, INVALID), ({"ldq": 48}, INVALID), ({"scale": 0}, INVALID), ({"count": 2, "sq": 200, "sx": 400}, INVALID),
    ({"count": 2, "sq": 264, "sx": 400}, INVALID), ({"ldx": FAR}, UNSUPPORTED), ({"ldq": FAR}, UNSUPPORTED),
    ({"count": 2, "sq": FAR, "sx": 400}, UNSUPPORTED), ({"count": 2, "sq": 256, "sx": FAR}, UNSUPPORTED)])
def test_form_refusals(kw, want):
    a = dict(x=P, ldx=64, sx=0, dtype=1, count=1, rows=4, cols=64, block=1, q=P, ldq=64, sq=0, scale=P)
    a.update(kw)
    f = abi()
    assert f.muon_f8_quantize(a["x"], a["ldx"], a["sx"], a["dtype"], a["count"], a["rows"], a["cols"], a["block"], a["q"],
                              a["ldq"], a["sq"], a["scale"], None) == want
    if not (a["count"] == 2 and a["sq"] == 200):
        assert f.muon_f8_dequantize(a["q"], a["ldq"], a["sq"], a["scale"], a["count"], a["rows"], a["cols"], a["block"],
                                    a["x"], a["ldx"], a["sx"], a["dtype"], None) == want


def product(kind, t=40, n=48, k=64, a=P, lda=None, sa=P, b=P, ldb=None, bs=None, sb=P, ends=0, experts=1, out=P, ldo=None,
            os_=None, dtype=0, ws=P, wsb=1 << 30):
    f = abi()
    lda = lda if lda is not None else (k + 15) // 16 * 16 if kind == 0 else n
    ldb = ldb if ldb is not None else (k + 15) // 16 * 16
    bs = bs if bs is not None else n * ldb
    ldo = ldo if ldo is not None else (n if kind == 0 else k)
    os_ = os_ if os_ is not None else n * ldo
    if kind == 0:
        return f.muon_f8_matmul(a, lda, sa, b, ldb, bs, sb, ends, experts, t, n, k, out, ldo, dtype, ws, wsb, None)
    if kind == 1:
        return f.muon_f8_grad_input(a, lda, b, ldb, bs, sb, ends, experts, t, n, k, out, ldo, dtype, ws, wsb, None)
    return f.muon_f8_grad_weight(a, lda, b, ldb, sb, ends, experts, t, n, k, out, ldo, os_, dtype, 0, ws, wsb, None)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("kw, want", [
    ({"t": -1}, INVALID), ({"n": -1}, INVALID), ({"k": -1}, INVALID), ({"t": (1 << 24) + 1}, UNSUPPORTED),
    ({"n": (1 << 24) + 1}, UNSUPPORTED), ({"k": (1 << 24) + 1}, UNSUPPORTED), ({"dtype": 2}, INVALID), ({"a": 0}, INVALID),
    ({"a": P + 1}, INVALID), ({"b": 0}, INVALID), ({"b": P + 8}, INVALID), ({"ldb": 72}, INVALID), ({"ldb": 48}, INVALID),
    ({"lda": 20}, INVALID), ({"out": 0}, INVALID), ({"out": P + 2}, INVALID), ({"ldo": 20}, INVALID), ({"sb": 0}, INVALID),
    ({"experts": 0}, INVALID), ({"experts": 2}, INVALID), ({"ends": P, "experts": 1025}, UNSUPPORTED),
    ({"ends": P + 2, "experts": 2}, INVALID), ({"lda": FAR}, UNSUPPORTED), ({"ldb": FAR}, UNSUPPORTED),
    ({"ldo": FAR}, UNSUPPORTED), ({"ends": P, "experts": 2, "bs": FAR, "os_": FAR}, UNSUPPORTED)])
def test_product_refusals(kind, kw, want):
    assert product(kind, **kw) == want


def test_product_refusals_by_kind():
    assert product(0, lda=72) == INVALID                     # 8-bit rows off 16 bytes
    assert product(0, sa=0) == INVALID
    for kind in (0, 1, 2):                                   # 8-bit rows that 32 bits do not reach
        assert product(kind, ldb=(1 << 23) + 16) == UNSUPPORTED
    assert product(0, lda=(1 << 23) + 16) == UNSUPPORTED
    for kind in (1, 2):
        assert product(kind, n=(1 << 23) + 8) == UNSUPPORTED
    for kind in (0, 1):                                      # the experts' weights overlap, or lie off 16 bytes
        assert product(kind, ends=P, experts=2, bs=48 * 64 - 16) == INVALID
        assert product(kind, ends=P, experts=2, bs=48 * 64 + 8) == INVALID
    assert product(2, ends=P, experts=2, os_=48 * 64 - 1) == INVALID
    for kind in (1, 2):                                      # rows that are laid out again
        for kw in ({"n": 49}, {"a": P + 2}, {"lda": 50}):
            assert product(kind, wsb=16, **kw) == SMALL
            assert product(kind, ws=0, **kw) == INVALID
            assert product(kind, ws=P + 16, **kw) == INVALID


def test_products_without_outputs_do_nothing():
    for kind in (0, 1):
        assert product(kind, t=0, a=0, out=0, b=0) == OK
        assert product(kind, t=0, a=0, out=0, b=0, ends=P, experts=7) == OK
    assert product(0, n=0, b=0, out=0) == OK
    assert product(1, k=0, b=0, out=0, ldb=0) == OK
    assert product(2, n=0, a=0, out=0, lda=0) == OK and product(2, k=0, b=0, out=0, ldb=0) == OK


def test_workspaces():
    assert workspace(0, P, 64, False, 1, 40, 48, 64) == 0
    assert workspace(1, P, 48, False, 1, 40, 48, 64) == 0
    for kind in (1, 2):
        assert workspace(kind, P, 49, False, 1, 4000, 49, 64) >= 4000 * 112
    f = abi()
    assert f.muon_f8_workspace(0, P, 64, 0, 1, 40, 48, 64, 1, None) == INVALID
    assert f.muon_f8_workspace(3, P, 64, 0, 1, 40, 48, 64, 1, P) == INVALID
    assert f.muon_f8_workspace(0, P, 64, 0, 2, 40, 48, 64, 1, P) == INVALID
    assert f.muon_f8_workspace(1, P, FAR, 0, 1, 40, 48, 64, 1, P) == UNSUPPORTED


def f8_of(shape, square=False, cols=None):
    s = list(shape)
    s[-1] = (s[-1] + 127) // 128
    if square:
        s[-2] = (s[-2] + 127) // 128
    return f8.F8(torch.zeros(shape, dtype=torch.uint8).view(E4M3), torch.zeros(s, dtype=torch.uint8).view(E8M0))


def test_entry_points_refuse():
    """The checks come ahead of the device's: CPU tensors reach them."""
    x, w, dy = f8_of((8, 64)), f8_of((48, 64), True), torch.zeros(8, 48, dtype=torch.bfloat16)
    for call, match in [
            (lambda: f8.quantize(torch.zeros(3, 4, dtype=torch.float16)), "fp32 or bf16"),
            (lambda: f8.quantize(torch.zeros(())), "at least one dimension"),
            (lambda: f8.quantize(torch.zeros(4, 4).t()), "unit stride"),
            (lambda: f8.quantize("x"), "must be a tensor"),
            (lambda: f8.quantize(torch.zeros(3, 4)), "CUDA"),
            (lambda: f8.quantize_weight(torch.zeros(4)), "two or three"),
            (lambda: f8.quantize_weight(torch.zeros(2, 4, 4).transpose(1, 2)), "unit stride"),
            (lambda: f8.quantize_weight(torch.zeros(2, 4)), "CUDA"),
            (lambda: f8.dequantize(x, torch.float16), "fp32 or bf16"),
            (lambda: f8.dequantize(x), "CUDA"),
            (lambda: f8.matmul(tuple(x), w), "must be an F8"),
            (lambda: f8.matmul(f8.F8(x.q.view(torch.int8), x.scale), w), "float8_e4m3fn"),
            (lambda: f8.matmul(f8.F8(x.q, x.scale.float()), w), "float8_e8m0fnu"),
            (lambda: f8.matmul(f8.F8(x.q, x.scale[:4]), w), "each 128 values of a row"),
            (lambda: f8.matmul(f8.F8(x.q[:, 1:], x.scale), w), "multiples of 16 bytes"),
            (lambda: f8.matmul(f8_of((8, 40)), w), "multiples of 16 bytes"),
            (lambda: f8.matmul(x, w, dtype=torch.float16), "fp32 or bf16"),
            (lambda: f8.matmul(x, w), "CUDA"),
            (lambda: f8.grad_input(dy.float(), w), "dy must be bf16"),
            (lambda: f8.grad_input(dy, w), "CUDA"),
            (lambda: f8.grad_weight(dy, f8_of((9, 64))), "same number of rows"),
            (lambda: f8.grad_weight(dy, x), "CUDA")]:
        with pytest.raises(ValueError, match=match):
            call()


def test_a_last_row_without_room_is_refused():
    room = torch.zeros(7 * 48 + 40, dtype=torch.uint8)
    q = room.view(E4M3).as_strided((8, 40), (48, 1))
    scale = torch.zeros(8, 1, dtype=torch.uint8).view(E8M0)
    with pytest.raises(ValueError, match="room for 16 bytes"):
        f8.matmul(f8.F8(q, scale), f8_of((48, 64), True))
