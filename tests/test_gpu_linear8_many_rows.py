"""Row kernels on more rows than one launch has threads for: a launch takes
fewer than 2^32 threads, and up to 64 columns a row takes eight of them."""
import pytest
import torch

from matrix_aware_optimizer_muon_amd import linear8 as l8

pytestmark = pytest.mark.gpu

ROWS = (1 << 29) + 4099  # 2^32 threads and some


def alternating(first, second, dtype):
    """One column of ROWS rows: `first`, `second`, `first`, ..."""
    x = torch.full((ROWS, 1), first, dtype=dtype, device="cuda")
    x[1::2] = second
    return x


def holds(t, first, second):
    """(torch's comparisons index within 2^32 themselves: in parts)"""
    step = 1 << 27
    for i in range(0, ROWS, step):
        part = t[i:i + step]
        if not bool((part[0::2] == first).all()) or not bool((part[1::2] == second).all()):
            return False
    return True


def test_quantize_and_back():
    x = alternating(1.0, -254.0, torch.bfloat16)
    got = l8.quantize(x)
    torch.cuda.synchronize()
    assert holds(got.scale, 2.0 ** -6, 2.0) and holds(got.q, 64, -127)
    back = l8.dequantize(got)
    assert holds(back, 1.0, -254.0)


def test_norm():
    x = alternating(1.0, -3.0, torch.bfloat16)
    w = torch.full((1,), 2.0, device="cuda")
    y, h, rstd = l8.rmsnorm(x, w, residual=x, eps=0.0)
    torch.cuda.synchronize()
    assert holds(h, 2.0, -6.0) and holds(y, 2.0, -2.0)
    assert holds(rstd, 0.5, float(torch.tensor(1 / 6)))
    del y, h
    y, _, _ = l8.rmsnorm(x, w, eps=0.0, q8=True)
    assert holds(y.scale, 2.0 ** -5, 2.0 ** -5) and holds(y.q, 64, -64)
