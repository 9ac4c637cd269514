"""Torch-facing entry points of gradient clipping (include/muon_clip.h): the
global norm over many tensors, and their scaling to a largest norm.

    norm = grad_norm(grads)
    norm = clip_grad_norm(grads, 1.0)            # in place
    norm = clip_grad_norm(grads, 1.0, out=outs)  # grads stay as they are

`MuonMI355X.step(..., max_norm=1.0)` clips ahead of the step.

norm = sqrt(sum of all squares), a 0-dim fp32 tensor on the device; no call waits
for the GPU.  Where norm > max_norm each gradient is multiplied by max_norm /
norm (in fp32, rounded to the output's type).  Sums and the norm behind the factor
are held in 64 bits, in a fixed order: finite gradients are clipped right where
the norm is infinite in fp32.  An infinite gradient makes finite ones 0 and
infinite ones NaN, a NaN one all NaN.

Gradients are fp32 or bf16 CUDA tensors of one device, dense (without gaps, in
any order of dimensions).  Outputs have their gradient's shape and strides and
either type.  No tensor that is written may share memory with another of the
call (the same gradient twice included).  Work is enqueued on the current stream
of the tensors' device.  Argument errors raise ValueError, or MuonError from the
C ABI; a forward-mode tangent raises NotImplementedError.
"""
from __future__ import annotations

import os
from typing import Optional, Sequence

import torch

from ._lib import MuonError, load

__all__ = ["grad_norm", "clip_grad_norm"]

load()  # libmuon.so, which the binding links to
if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_clip.so")):
    raise ImportError("_clip.so is not built; run __graft_entry__.build() first")
from . import _clip  # noqa: E402

_clip.set_classes(MuonError)


def grad_norm(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """The global norm of the gradients (muon_grad_norm)."""
    return _clip.grad_norm(grads)


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scales the gradients to a global norm of at most max_norm (a number that
    fp32 holds, or infinity), in place or into `out`, and returns the norm they
    had (muon_clip_grads)."""
    return _clip.clip_grad_norm(grads, max_norm, out)
