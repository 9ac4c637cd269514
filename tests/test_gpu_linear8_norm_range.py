"""The norm of rows whose rstd lies outside fp32's normal numbers: y is an
ordinary value there, in rows of the type as in 8 bits."""
import numpy as np
import pytest
import torch

from matrix_aware_optimizer_muon_amd import linear8 as l8

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


# rms from the smallest subnormal of the type on; from 2^-128 to 2^126 rstd is
# normal, beyond it is infinite or subnormal
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [2.0 ** -130, 1e-39, 2.0 ** -127, 1e-37, 1.0, 2.0 ** 125, 1.1e38, 2e38])
@pytest.mark.parametrize("cols", [1, 64, 3000, 8192, 20000])
def test_typed_rows(cols, rms, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    h = (1 + 0.5 * torch.rand(6, cols, generator=g, device="cuda"))  # at most 1.5
    h = (h.double() * rms * torch.sign(torch.randn(6, cols, generator=g, device="cuda"))).to(dtype)
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    y, _, rstd = l8.rmsnorm(h, w, eps=0.0)
    h64 = h.double()
    want_r = 1 / torch.sqrt((h64 * h64).mean(dim=1))
    want = h64 * want_r[:, None] * w.double()
    # rstd and two products rounded in fp32, then the type's own rounding
    bound = want.abs() * (3 * U * 1.001 + (HALF[dtype] * 1.001 if dtype == torch.bfloat16 else 0))
    assert bool(((y.double() - want).abs() <= bound).all())
    assert torch.equal(rstd, want_r.to(torch.float32)) or bool(
        ((rstd.double() - want_r).abs() <= want_r * U * 1.001 + 2.0 ** -149).all())


def test_rows_that_have_no_norm():
    w = torch.ones(40, device="cuda")
    h = torch.randn(4, 40, device="cuda")
    h[1] = 0  # 0 / 0 with eps = 0
    h[3, 5] = float("nan")
    y, _, rstd = l8.rmsnorm(h, w, eps=0.0)
    assert y.isnan().all(dim=1).tolist() == [False, True, False, True]
    assert rstd.isinf().tolist() == [False, True, False, False] and bool(rstd[3].isnan())
    assert np.isfinite(y[0].cpu().numpy()).all()
