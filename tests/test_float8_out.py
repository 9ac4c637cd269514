"""The output that grad_weight is given, no GPU needed: the check comes ahead of
the device's, so CPU tensors reach it."""
import pytest
import torch

from float8_common import E4M3, E8M0
from matrix_aware_optimizer_muon_amd import float8 as f8


def arguments():
    x = f8.F8(torch.zeros(8, 64, dtype=torch.uint8).view(E4M3), torch.zeros(8, 1, dtype=torch.uint8).view(E8M0))
    return torch.zeros(8, 48, dtype=torch.bfloat16), x


@pytest.mark.parametrize("accumulate", [False, True])
def test_an_output_that_requires_a_gradient_is_refused(accumulate):
    dy, x = arguments()
    leaf = torch.zeros(48, 64, requires_grad=True)
    for out in (leaf, leaf * 1):
        with pytest.raises(ValueError, match="must not require a gradient"):
            f8.grad_weight(dy, x, out=out, accumulate=accumulate)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # (past that check)
        f8.grad_weight(dy, x, out=leaf, accumulate=accumulate)
    with pytest.raises(ValueError, match="CUDA"):
        f8.grad_weight(dy, x, out=leaf.detach(), accumulate=accumulate)
