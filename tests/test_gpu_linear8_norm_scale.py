"""The 8-bit norm's scale comes from the row's largest |y| = |h rstd weight|,
wherever |h weight| lies: below fp32's smallest values, above its largest, and
next to the borders 127 * 2^e."""
import numpy as np
import pytest
import torch

from matrix_aware_optimizer_muon_amd import linear8 as l8

pytestmark = pytest.mark.gpu


def formula(h, w, eps):
    """y of each row in 64 bits, and its 8-bit form (q, scale)."""
    h = h.cpu().double()
    y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + float(np.float32(eps))) * w.cpu().double()
    steps = torch.from_numpy(np.ldexp(1.0, np.arange(-126, 128)))
    step = steps[torch.searchsorted(127.0 * steps, y.abs().amax(dim=1))]
    return y, torch.round(y / step[:, None]), step


def check(h, w, eps):
    """Scales equal; q equal but within 1e-9 of a rounding border."""
    got, _, _ = l8.rmsnorm(h, w, eps=eps, q8=True)
    y, q, step = formula(h, w, eps)
    assert torch.equal(got.scale.cpu().double(), step)
    t = y / step[:, None]
    border = ((t - torch.floor(t)) - 0.5).abs() < 1e-9
    assert bool(((got.q.cpu().double() == q) | border).all())
    assert int(got.q.int().abs().max()) <= 127


# |h w| from below fp32's smallest value (2^-149 = 1.4e-45), over its subnormal
# range, to above its largest (3.4e38)
@pytest.mark.parametrize("hs, ws", [(1e-25, 6e-21), (1e-30, 1e-20), (1e-22, 1e-22), (1e-25, 1e-17), (1e-12, 1e-30),
                                    (1e30, 1e10), (2e37, 30.0)])
@pytest.mark.parametrize("cols", [1, 7, 64, 700, 2049, 3584, 18945])
def test_products_outside_fp32(cols, hs, ws):
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    h = hs * torch.randn(5, cols, generator=g, device="cuda")
    w = ws * (1 + 0.1 * torch.randn(cols, generator=g, device="cuda"))
    check(h, w, 0.0)


def test_one_large_value_beside_products_that_vanish():
    h = torch.full((3, 300), 1e-30, device="cuda")
    h[1, 299] = -3e-30
    w = torch.full((300,), 1e-20, device="cuda")
    w[299] = 2e-20
    check(h, w, 0.0)
    check(h, w, 1e-38)


@pytest.mark.parametrize("to, scale", [(200.0, 2.0), (0.0, 1.0)])
def test_next_to_a_border(to, scale):
    # one column, eps = 0: y = +-weight, here fp32's neighbours of 127
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.randn(4096, 1, generator=g, device="cuda")
    w = torch.nextafter(torch.tensor([127.0]), torch.tensor([to])).cuda()
    got, _, _ = l8.rmsnorm(h, w, eps=0.0, q8=True)
    assert bool((got.scale == scale).all())
    assert torch.equal(got.q.float(), torch.sign(h) * round(127 / scale + (0.1 if to > 127 else 0)))


def test_rows_that_are_not_finite():
    h = torch.randn(9, 520, device="cuda")
    w = 1 + 0.1 * torch.randn(520, device="cuda")
    want = l8.rmsnorm(h, w, q8=True)[0]
    h[1, 3], h[4, 519], h[7, 0] = float("nan"), float("inf"), float("-inf")
    h[5] = 0
    got = l8.rmsnorm(h, w, q8=True)[0]
    bad = torch.zeros(9, dtype=torch.bool, device="cuda")
    bad[[1, 4, 7]] = True
    assert torch.equal(got.scale.isnan(), bad) and not got.q[bad].any() and not got.q[5].any()
    ok = ~bad
    ok[5] = False
    assert torch.equal(got.q[ok], want.q[ok]) and torch.equal(got.scale[ok], want.scale[ok])
    for v in ("nan", "inf", "-inf"):  # a weight that is not finite takes every row
        ww = w.clone()
        ww[519] = float(v)
        got = l8.rmsnorm(h[:1], ww, q8=True)[0]
        assert bool(got.scale.isnan().all()) and not got.q.any()
    # eps = 0 and a row of zeros: 0 / 0
    assert bool(l8.rmsnorm(torch.zeros(2, 9, device="cuda"), w[:9].contiguous(), eps=0.0, q8=True)[0].scale.isnan().all())
    # a row whose largest |y| passes fp32's range has no scale; one that does not has
    big = torch.tensor([[1.0, 0.0]], device="cuda")  # y = (sqrt(2) w, 0)
    for v, finite in ((2.5e38, False), (2.4e38, True)):
        got = l8.rmsnorm(big, torch.tensor([v, 1.0], device="cuda"), eps=0.0, q8=True)[0]
        assert bool(got.scale.isfinite()) == finite
