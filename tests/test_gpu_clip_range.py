"""Clipping by factors under fp32's normal numbers, against 64-bit formulas.  The
factor and the product are rounded once each to 24 bits, 2^-24 of the value (the
norm behind the factor is held in 64 bits), a bf16 output once more by half its
step, 2^-8 of the value, and what lies under the type's normal numbers by half the
smallest subnormal at each of the two roundings."""
import pytest
import torch

from matrix_aware_optimizer_muon_amd.clip import clip_grad_norm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


# a norm past fp32's range; a factor that fp32 holds with a few bits, or not at all
@pytest.mark.parametrize("scale, max_norm", [(1e38, 1.0), (1e37, 1.0), (1e37, 1e-3), (1e20, 1e-22), (1e25, 1e-20),
                                             (1e38, 1e-37), (1e30, 2.0 ** -149)])
@pytest.mark.parametrize("n", [3000, 100000])  # one launch, and two
@pytest.mark.parametrize("dtype", [F32, BF])
def test_factors_under_the_normal_numbers(scale, max_norm, n, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    g = ((2 * torch.rand(n, generator=gen, device="cuda") - 1) * scale).to(dtype)
    norm = float(g.double().norm())
    by = float(torch.tensor(max_norm, dtype=F32)) / norm
    assert by < 2.0 ** -120
    want = g.double() * by
    for out in (torch.empty_like(g), torch.empty_like(g, dtype=BF if dtype == F32 else F32), g):
        clip_grad_norm([g], max_norm, out=None if out is g else [out])
        half, least = (2.0 ** -8, 2.0 ** -133) if out.dtype == BF else (0.0, 2.0 ** -149)
        d = (out.double() - want).abs()
        assert bool((d <= want.abs() * (2.001 * U + half * 1.001) + least).all())


def test_the_last_factor_of_one_product_and_the_first_of_two():
    """max_norm / norm on both sides of 2^-126: powers of two, exact."""
    for e in (-125, -126, -127, -140):
        g = torch.zeros(5000, device="cuda")
        g[17] = 2.0 ** 100
        out = torch.empty_like(g)
        clip_grad_norm([g], 2.0 ** (100 + e), out=[out])
        assert float(out[17]) == 2.0 ** (100 + e) and int(out.count_nonzero()) == 1


def test_infinite_gradients_beside_a_norm_past_the_range():
    g = torch.full((4000,), 3e38, device="cuda")
    assert float(clip_grad_norm([g], 1.0)) == float("inf")
    # 1 / sqrt(4000), by three roundings
    assert bool(((g.double() * 4000 ** 0.5 - 1).abs() <= 3 * U).all())
    g[5] = float("inf")
    clip_grad_norm([g], 1.0)
    assert bool(g[5].isnan()) and int(g.count_nonzero()) == 1
