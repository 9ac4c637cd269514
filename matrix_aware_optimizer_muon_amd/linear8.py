"""Torch-facing entry points of the 8-bit linear layer
(include/muon_linear8.h): the operators from a residual stream to the weight
gradient that a Muon step takes, with activations and weights kept in 8 bits.

    y, h, rstd = rmsnorm(x, weight, residual=r, q8=True)   # y: Q8
    out = matmul(y, w8)                                    # w8 = quantize(W)
    dx  = grad_input(dout, w8)
    dW  = grad_weight(dout, y)                             # y is the checkpoint
    dh, dweight = rmsnorm_backward(dx, h, rstd, weight, dh=dstream)

An 8-bit tensor is a `Q8`: int8 rows and one power-of-two fp32 scale per row
(value = q * scale).  Tensors are CUDA tensors with unit stride in the last
dimension; 2-D ones may have any row stride, others are taken as rows of their
last dimension and must be contiguous.  Work is enqueued on the current
stream of the tensors' device; results and workspaces come from torch's
allocator.  Argument errors raise ValueError here, or MuonError from the C ABI.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import NamedTuple, Optional, Tuple, Union

import torch

from ._lib import MUON_BF16, MUON_F32, MUON_OK, MuonError, load

__all__ = ["Q8", "quantize", "dequantize", "rmsnorm", "rmsnorm_backward", "matmul", "grad_input",
           "grad_weight"]

EXPORTED = ("muon_rmsnorm_forward", "muon_rmsnorm_backward_workspace", "muon_rmsnorm_backward",
            "muon_q8_quantize", "muon_q8_dequantize", "muon_q8_workspace", "muon_q8_matmul",
            "muon_q8_grad_input", "muon_q8_grad_weight")
MATMUL, GRAD_INPUT, GRAD_WEIGHT = 0, 1, 2

_DTYPE = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}


class Q8(NamedTuple):
    """8-bit rows: `q` int8 (..., n), `scale` fp32 with q's leading shape."""
    q: torch.Tensor
    scale: torch.Tensor


_fn = None


def _abi():
    global _fn
    if _fn is None:
        lib = load()
        P, I, L, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        sig = {
            "muon_rmsnorm_forward": [P, L, P, L, P, I, L, L, F, P, L, P, L, P, L, P, P, P],
            "muon_rmsnorm_backward_workspace": [L, L, P],
            "muon_rmsnorm_backward": [P, L, P, L, P, P, P, P, L, I, L, L, P, L, P, P, S, P],
            "muon_q8_quantize": [P, L, I, L, L, P, L, P, P],
            "muon_q8_dequantize": [P, L, P, L, L, P, L, I, P],
            "muon_q8_workspace": [I, P, L, P, L, L, L, L, P],
            "muon_q8_matmul": [P, L, P, P, L, P, L, L, L, P, L, I, P, S, P],
            "muon_q8_grad_input": [P, L, P, L, P, L, L, L, P, L, I, P, S, P],
            "muon_q8_grad_weight": [P, L, P, L, P, L, L, L, P, L, I, I, P, S, P],
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        _fn = lib
    return _fn


def _check(status: int, where: str):
    if status != MUON_OK:
        raise MuonError(status, where)


def _rows(t: torch.Tensor, what: str) -> Tuple[int, int, int]:
    """(rows, columns, row distance) of a tensor taken as rows of its last
    dimension."""
    d = t.dim()
    if d == 2:
        r, c = t.shape
        sr, sc = t.stride()
        if sc != 1 and c > 1 and r > 0:
            raise ValueError(f"{what} must have unit stride in its last dimension")
        if r > 1 and sr < c:
            raise ValueError(f"{what} must have rows that do not overlap")
        return r, c, max(sr, c)
    if d == 0:
        raise ValueError(f"{what} must have at least one dimension")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous (or 2-D with any row stride)")
    c = t.shape[-1]
    return t.shape[:-1].numel(), c, c


def _device(*ts: Optional[torch.Tensor]) -> torch.device:
    dev = ts[0].device
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors")
            if t.device != dev:
                raise ValueError("tensors must be on one device")
    return dev


def _typed(t: torch.Tensor, what: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be fp32 or bf16")
    return code


def _vector(t: torch.Tensor, n: int, what: str):
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous fp32 with {n} elements")


def _q8(t: Q8, what: str) -> Tuple[int, int, int]:
    if not isinstance(t, Q8):
        raise ValueError(f"{what} must be a Q8")
    if t.q.dtype != torch.int8:
        raise ValueError(f"{what}.q must be int8")
    r, c, ld = _rows(t.q, what + ".q")
    _vector(t.scale, r, what + ".scale")
    return r, c, ld


class _on:
    """The device made current if it is not, and its current stream."""

    def __init__(self, dev: torch.device):
        self.dev = dev

    def __enter__(self):
        i = self.dev.index
        self.prev = torch.cuda.current_device()
        if self.prev != i:
            torch.cuda.set_device(i)
        return torch.cuda.current_stream(i).cuda_stream

    def __exit__(self, *exc):
        if self.prev != self.dev.index:
            torch.cuda.set_device(self.prev)


def quantize(x: torch.Tensor) -> Q8:
    """The 8-bit form of x's rows (muon_q8_quantize)."""
    dev = _device(x)
    code = _typed(x, "x")
    r, c, ld = _rows(x, "x")
    q = torch.empty(x.shape, dtype=torch.int8, device=dev)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    with _on(dev) as s:
        _check(_abi().muon_q8_quantize(x.data_ptr(), ld, code, r, c, q.data_ptr(), c, scale.data_ptr(), s),
               "muon_q8_quantize")
    return Q8(q, scale)


def dequantize(x: Q8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values x stands for (muon_q8_dequantize)."""
    r, c, ld = _q8(x, "x")
    dev = _device(x.q, x.scale)
    out = torch.empty(x.q.shape, dtype=dtype, device=dev)
    code = _typed(out, "dtype")
    with _on(dev) as s:
        _check(_abi().muon_q8_dequantize(x.q.data_ptr(), ld, x.scale.data_ptr(), r, c, out.data_ptr(), c,
                                         code, s), "muon_q8_dequantize")
    return out


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
            eps: float = 1e-6, q8: bool = False
            ) -> Tuple[Union[torch.Tensor, Q8], torch.Tensor, torch.Tensor]:
    """(y, h, rstd): h = x + residual (x itself without one), rstd =
    1 / sqrt(mean(h^2) + eps), y = h * rstd * weight, in 8 bits if q8
    (muon_rmsnorm_forward)."""
    dev = _device(x, weight, residual)
    code = _typed(x, "x")
    r, c, ld = _rows(x, "x")
    _vector(weight, c, "weight")
    h, hp, rp, ldr = x, 0, 0, 0
    if residual is not None:
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("residual must have x's shape and type")
        ldr = _rows(residual, "residual")[2]
        h = torch.empty(x.shape, dtype=x.dtype, device=dev)
        hp, rp = h.data_ptr(), residual.data_ptr()
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    if q8:
        y = Q8(torch.empty(x.shape, dtype=torch.int8, device=dev),
               torch.empty(x.shape[:-1], dtype=torch.float32, device=dev))
        yp, qp, sp = 0, y.q.data_ptr(), y.scale.data_ptr()
    else:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        yp, qp, sp = y.data_ptr(), 0, 0
    with _on(dev) as s:
        _check(_abi().muon_rmsnorm_forward(x.data_ptr(), ld, rp, ldr, weight.data_ptr(), code, r, c, eps, hp,
                                           c, yp, c, qp, c, sp, rstd.data_ptr(), s), "muon_rmsnorm_forward")
    return y, h, rstd


@lru_cache(maxsize=4096)
def _back_workspace(r: int, c: int) -> int:
    n = ctypes.c_size_t()
    _check(_abi().muon_rmsnorm_backward_workspace(r, c, ctypes.addressof(n)), "muon_rmsnorm_backward_workspace")
    return n.value


def rmsnorm_backward(dy: torch.Tensor, h: Union[torch.Tensor, Q8], rstd: torch.Tensor,
                     weight: torch.Tensor, dh: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of rmsnorm, from its h (or a Q8 of it) and rstd; dh is the
    gradient that reaches h through the residual stream.  dx is the gradient
    of both x and the residual (muon_rmsnorm_backward)."""
    code = _typed(dy, "dy")
    r, c, ld = _rows(dy, "dy")
    if isinstance(h, Q8):
        rh, ch, ldh = _q8(h, "h")
        ht, hs = h
        if rh != r or ch != c:
            raise ValueError("h must have dy's shape")
    else:
        ht, hs = h, None
        if h.shape != dy.shape or h.dtype != dy.dtype:
            raise ValueError("h must have dy's shape and type")
        ldh = _rows(h, "h")[2]
    dev = _device(dy, ht, hs, rstd, weight, dh)
    _vector(rstd, r, "rstd")
    _vector(weight, c, "weight")
    lddh = 0
    if dh is not None:
        if dh.shape != dy.shape or dh.dtype != dy.dtype:
            raise ValueError("dh must have dy's shape and type")
        lddh = _rows(dh, "dh")[2]
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dev)
    dw = torch.empty(c, dtype=torch.float32, device=dev)
    need = _back_workspace(r, c)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    with _on(dev) as s:
        _check(_abi().muon_rmsnorm_backward(
            dy.data_ptr(), ld, ht.data_ptr(), ldh, hs.data_ptr() if hs is not None else 0, rstd.data_ptr(),
            weight.data_ptr(), dh.data_ptr() if dh is not None else 0, lddh, code, r, c, dx.data_ptr(), c,
            dw.data_ptr(), ws.data_ptr() if need else 0, need, s), "muon_rmsnorm_backward")
    return dx, dw


@lru_cache(maxsize=4096)
def _product_workspace(kind: int, a: int, lda: int, b: int, ldb: int, t: int, n: int, k: int) -> int:
    z = ctypes.c_size_t()  # a and b: the addresses modulo 16, all that counts
    _check(_abi().muon_q8_workspace(kind, a, lda, b, ldb, t, n, k, ctypes.addressof(z)), "muon_q8_workspace")
    return z.value


def _product(kind, name, a, lda, a_scale, b, ldb, b_scale, t, n, k, out, ldo, code, accumulate):
    ap, bp = a.data_ptr(), b.data_ptr()
    need = _product_workspace(kind, ap % 16, lda, bp % 16, ldb, t, n, k)
    dev = out.device
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    wp = ws.data_ptr() if need else 0
    fn = _abi()
    with _on(dev) as s:
        if kind == MATMUL:
            st = fn.muon_q8_matmul(ap, lda, a_scale.data_ptr(), bp, ldb, b_scale.data_ptr(), t, n, k,
                                   out.data_ptr(), ldo, code, wp, need, s)
        elif kind == GRAD_INPUT:
            st = fn.muon_q8_grad_input(ap, lda, bp, ldb, b_scale.data_ptr(), t, n, k, out.data_ptr(), ldo,
                                       code, wp, need, s)
        else:
            st = fn.muon_q8_grad_weight(ap, lda, bp, ldb, b_scale.data_ptr(), t, n, k, out.data_ptr(), ldo,
                                        code, int(accumulate), wp, need, s)
    _check(st, name)
    return out


def matmul(x: Q8, w: Q8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y = x w^T for x (..., k) and weights w (n, k), as `dtype`: exact
    integer sums, scaled per row of x and of w (muon_q8_matmul)."""
    t, k, ldx = _q8(x, "x")
    n, kw, ldw = _q8(w, "w")
    if kw != k or w.q.dim() != 2:
        raise ValueError("w must be (n, k) with x's last dimension k")
    dev = _device(x.q, x.scale, w.q, w.scale)
    out = torch.empty(x.q.shape[:-1] + (n,), dtype=dtype, device=dev)
    return _product(MATMUL, "muon_q8_matmul", x.q, ldx, x.scale, w.q, ldw, w.scale, t, n, k, out, n,
                    _typed(out, "dtype"), False)


def grad_input(dy: torch.Tensor, w: Q8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """dx = dy w for bf16 dy (..., n) and weights w (n, k), as `dtype`
    (muon_q8_grad_input)."""
    n, k, ldw = _q8(w, "w")
    t, nd, ld = _rows(dy, "dy")
    if dy.dtype != torch.bfloat16:
        raise ValueError("dy must be bf16")
    if nd != n or w.q.dim() != 2:
        raise ValueError("w must be (n, k) with dy's last dimension n")
    dev = _device(dy, w.q, w.scale)
    out = torch.empty(dy.shape[:-1] + (k,), dtype=dtype, device=dev)
    return _product(GRAD_INPUT, "muon_q8_grad_input", dy, ld, None, w.q, ldw, w.scale, t, n, k, out, k,
                    _typed(out, "dtype"), False)


def grad_weight(dy: torch.Tensor, x: Q8, dtype: torch.dtype = torch.float32,
                out: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """dW = dy^T x (n, k) for bf16 dy (..., n) and the checkpoint x (..., k), as
    `dtype` or into `out`; accumulate adds to what out holds
    (muon_q8_grad_weight)."""
    t, k, ldx = _q8(x, "x")
    td, n, ld = _rows(dy, "dy")
    if dy.dtype != torch.bfloat16:
        raise ValueError("dy must be bf16")
    if td != t:
        raise ValueError("dy and x must have the same number of rows")
    dev = _device(dy, x.q, x.scale, out)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((n, k), dtype=dtype, device=dev)
    elif out.shape != (n, k):
        raise ValueError("out must be (n, k)")
    ldo = _rows(out, "out")[2]
    return _product(GRAD_WEIGHT, "muon_q8_grad_weight", dy, ld, None, x.q, ldx, x.scale, t, n, k, out, ldo,
                    _typed(out, "out"), accumulate)
