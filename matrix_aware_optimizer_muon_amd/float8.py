"""Torch-facing entry points of the 8-bit floating-point layer
(include/muon_float8.h): rows and weights in e4m3 with a power-of-two scale for
each block of 128, the product of the two, the gradient products that lead to a
Muon step, and the same three grouped by expert with ragged sizes.

    w8 = quantize_weight(W)                      # (n, k) or (experts, n, k)
    x8 = quantize(x)                             # (..., k)
    y  = matmul(x8, w8)
    dx = grad_input(dy, w8)
    dW = grad_weight(dy, x8)                     # the G of a Muon step

    # rows sorted by expert, expert e's up to ends[e] (int32 on the device)
    ends = torch.bincount(expert, minlength=E).cumsum(0).to(torch.int32)
    y  = matmul(x8, w8, ends=ends)               # w8 of (E, n, k)
    dx = grad_input(dy, w8, ends=ends)
    dW = grad_weight(dy, x8, ends=ends)          # (E, n, k)

An 8-bit tensor is an `F8`: float8_e4m3fn values and float8_e8m0fnu scales
(value = q * scale), of which a row has one for each 128 columns and a weight
matrix one for each 128 x 128.  Rows of q start at multiples of 16 bytes: where
the last dimension is no multiple of 16, `quantize` leaves a gap behind each row,
and a `.contiguous()` copy of it is refused.  Products that do not run on the 8-bit
matrix cores take q * scale as bf16, as `dequantize` gives it: scales under 2^-124
lose what lies under 2^-133, and values from 2^128 on are infinite.

Grouped: nothing is copied to the host, so a call can be captured into a graph
and replayed with other ends.  Experts without rows are allowed.  Rows from the
last end on belong to no expert: they are not read and come out as zeros; the
weight gradient of an expert without rows is zero.

Tensors are CUDA tensors with unit stride in the last dimension; dy is bf16, 2-D
with any row stride or contiguous.  Forward and backward are calls of their own:
nothing is recorded for autograd.  Where an input of a forward call requires a
gradient, the result does too, and torch's backward pass through it raises; a
torch.autograd.Function around the calls gives them a gradient.  A forward-mode
tangent raises NotImplementedError.  Work is enqueued on the current stream of the
tensors' device; results and workspaces come from torch's allocator.  Argument
errors raise ValueError, or MuonError from the C ABI.

The functions only forward to the compiled binding (csrc/float8_torch.cpp),
which checks, allocates and calls libmuon.so; there is no fallback.
"""
from __future__ import annotations

import os
from typing import NamedTuple, Optional

import torch

from ._lib import MuonError, load

__all__ = ["F8", "quantize", "quantize_weight", "dequantize", "matmul", "grad_input", "grad_weight"]


class F8(NamedTuple):
    """8-bit values: `q` float8_e4m3fn (..., n, k), `scale` float8_e8m0fnu of
    shape (..., n, ceil(k / 128)) for rows or (..., ceil(n / 128), ceil(k / 128))
    for weights."""
    q: torch.Tensor
    scale: torch.Tensor


load()  # libmuon.so, which the binding links to
if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_float8.so")):
    raise ImportError("_float8.so is not built; run __graft_entry__.build() first")
from . import _float8  # noqa: E402

_float8.set_classes(F8, MuonError)


def quantize(x: torch.Tensor) -> F8:
    """The 8-bit form of x's rows, a scale for each 128 values (muon_f8_quantize)."""
    return _float8.quantize(x)


def quantize_weight(w: torch.Tensor) -> F8:
    """The 8-bit form of a matrix (n, k) or of (experts, n, k), a scale for each
    128 x 128 values (muon_f8_quantize)."""
    return _float8.quantize_weight(w)


def dequantize(x: F8, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values x stands for, rows or weights (muon_f8_dequantize)."""
    return _float8.dequantize(x, dtype)


def matmul(x: F8, w: F8, ends: Optional[torch.Tensor] = None,
           dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y = x w^T for rows x (..., k) and weights w (n, k), as `dtype`; with ends,
    w is (experts, n, k) (muon_f8_matmul).  fp32 results are fp32 sums of exact
    products; bf16 ones may come from the 8-bit matrix cores, whose sums inside
    eight products lie up to 2^-10 of their magnitudes off, 2^-16 of the
    result's root mean square for normally distributed operands, 2^-15 where
    some columns of x are far larger than others."""
    return _float8.matmul(x, w, ends, dtype)


def grad_input(dy: torch.Tensor, w: F8, ends: Optional[torch.Tensor] = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """dx = dy w for bf16 dy (..., n) and weights w (n, k), as `dtype`; with ends,
    w is (experts, n, k) (muon_f8_grad_input)."""
    return _float8.grad_input(dy, w, ends, dtype)


def grad_weight(dy: torch.Tensor, x: F8, ends: Optional[torch.Tensor] = None,
                dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                accumulate: bool = False) -> torch.Tensor:
    """dW = dy^T x (n, k) for bf16 dy (..., n) and rows x (..., k), as `dtype` or
    into `out`, which must not require a gradient (but under no_grad); with ends,
    (experts, n, k).  accumulate adds to what out holds (muon_f8_grad_weight)."""
    return _float8.grad_weight(dy, x, ends, dtype, out, accumulate)
