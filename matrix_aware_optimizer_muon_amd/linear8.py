"""Torch-facing entry points of the 8-bit linear layer
(include/muon_linear8.h): the operators from a residual stream to the weight
gradient that a Muon step takes, with activations and weights kept in 8 bits.

    y, h, rstd = rmsnorm(x, weight, residual=r, q8=True)   # y: Q8
    out = matmul(y, w8)                                    # w8 = quantize(W)
    dn  = grad_input(dout, w8)
    dW  = grad_weight(dout, y)                             # y is the checkpoint
    dx, dweight = rmsnorm_backward(dn, h, rstd, weight, dh=dstream)

An 8-bit tensor is a `Q8`: int8 rows and one power-of-two fp32 scale per row
(value = q * scale).  Tensors are CUDA tensors with unit stride in the last
dimension; 2-D ones may have any row stride, others are taken as rows of their
last dimension and must be contiguous.  Forward and backward are calls of
their own: nothing is recorded for autograd.  Where an input of a forward call
requires a gradient, the results do too, and torch's backward pass through them
raises; a torch.autograd.Function around the calls gives them a gradient.  A
forward-mode tangent raises NotImplementedError.  Work is enqueued on the current
stream of the tensors' device; results and workspaces come from torch's allocator.
Argument errors raise ValueError, or MuonError from the C ABI.

The functions only forward to the compiled binding (csrc/linear8_torch.cpp),
which checks, allocates and calls libmuon.so; there is no fallback.
"""
from __future__ import annotations

import os
from typing import NamedTuple, Optional, Tuple, Union

import torch

from ._lib import MuonError, load

__all__ = ["Q8", "quantize", "dequantize", "rmsnorm", "rmsnorm_backward", "matmul", "grad_input",
           "grad_weight"]


class Q8(NamedTuple):
    """8-bit rows: `q` int8 (..., n), `scale` fp32 with q's leading shape."""
    q: torch.Tensor
    scale: torch.Tensor


load()  # libmuon.so, which the binding links to
if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_linear8.so")):
    raise ImportError("_linear8.so is not built; run __graft_entry__.build() first")
from . import _linear8  # noqa: E402

_linear8.set_classes(Q8, MuonError)


def quantize(x: torch.Tensor) -> Q8:
    """The 8-bit form of x's rows (muon_q8_quantize)."""
    return _linear8.quantize(x)


def dequantize(x: Q8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values x stands for (muon_q8_dequantize)."""
    return _linear8.dequantize(x, dtype)


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
            eps: float = 1e-6, q8: bool = False
            ) -> Tuple[Union[torch.Tensor, Q8], torch.Tensor, torch.Tensor]:
    """(y, h, rstd): h = x + residual (x itself without one), rstd =
    1 / sqrt(mean(h^2) + eps), y = h * rstd * weight, in 8 bits if q8
    (muon_rmsnorm_forward)."""
    return _linear8.rmsnorm(x, weight, residual, eps, q8)


def rmsnorm_backward(dy: torch.Tensor, h: Union[torch.Tensor, Q8], rstd: torch.Tensor,
                     weight: torch.Tensor, dh: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of rmsnorm, from its h (or a Q8 of it) and rstd; dh is the
    gradient that reaches h through the residual stream.  dx is the gradient
    of both x and the residual (muon_rmsnorm_backward)."""
    return _linear8.rmsnorm_backward(dy, h, rstd, weight, dh)


def matmul(x: Q8, w: Q8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y = x w^T for x (..., k) and weights w (n, k), as `dtype`: exact
    integer sums, scaled per row of x and of w (muon_q8_matmul)."""
    return _linear8.matmul(x, w, dtype)


def grad_input(dy: torch.Tensor, w: Q8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """dx = dy w for bf16 dy (..., n) and weights w (n, k), as `dtype`
    (muon_q8_grad_input)."""
    return _linear8.grad_input(dy, w, dtype)


def grad_weight(dy: torch.Tensor, x: Q8, dtype: torch.dtype = torch.float32,
                out: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """dW = dy^T x (n, k) for bf16 dy (..., n) and the checkpoint x (..., k), as
    `dtype` or into `out`; accumulate adds to what out holds
    (muon_q8_grad_weight)."""
    return _linear8.grad_weight(dy, x, dtype, out, accumulate)
