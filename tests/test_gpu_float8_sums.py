"""The sums of the forward product in every form that it takes
(tests/float8_forms.py) against 64 bits.

fp32 results, and few rows: exact products, at most one rounding of 2^-24 per
addition.  bf16 results of the tiles: of eight products each is cut 13 bits under
the largest one's power of two, which is itself not cut, so a group's seven others
are off by less than 7 * 2^-13 of the largest: under 2^-10 of the magnitudes' sum.

For normal values the cuts are far smaller: an e4m3 product has 8 significant
bits, so only those 7 powers of two and more under the largest lose any.  Summed
up in 64 bits for cuts towards zero this is 2^-15.58 of the result's root mean
square, at any length, and moves 1.6 % of the results to another bf16 number.
Results near zero show it, whose rounding to bf16 is smaller."""
import pytest
import torch

from float8_common import MATMUL, blocks, gen, held, values
from float8_forms import SIZES, form
from matrix_aware_optimizer_muon_amd import float8 as f8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FORWARD = [s for s in SIZES if s[0] == MATMUL]


def spread8(shape, seed, square):
    """Any e4m3 numbers, all exponents alike, under scales of 2^-3 to 2^3."""
    g = gen(seed)
    b = torch.randint(0, 256, shape, generator=g, device="cuda")
    b = torch.where(b % 128 == 127, b - 1, b).to(torch.uint8)
    s = list(shape)
    s[-1] = blocks(s[-1])
    if square:
        s[-2] = blocks(s[-2])
    return held(b.view(torch.float8_e4m3fn).float(), torch.randint(124, 131, s, generator=g, device="cuda"))


def split_rows(experts, t):
    E = max(experts, 1)
    sizes = [t // E + (i < t % E) for i in range(E)]
    if experts > 1:  # uneven: the first expert's rows are the second's
        sizes[1] += sizes[0]
        sizes[0] = 0
    return sizes


def product(size, x, w):
    """The library's result, the exact one, and the sums of the magnitudes."""
    _, bf16, experts, t, n, k = size
    assert form(*size, a=x.q.data_ptr()) == form(*size)
    sizes = split_rows(experts, t)
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32) if experts else None
    flat = w if experts else f8.F8(w.q[0], w.scale[0])
    dtype = torch.bfloat16 if bf16 else torch.float32
    got = f8.matmul(x, flat, ends=ends, dtype=dtype)
    again = f8.matmul(x, flat, ends=ends, dtype=dtype)
    assert torch.equal(got, again)  # the same bits on every run
    xv, wv = values(x, False), values(w, True)
    parts = [(xv[a - s:a] @ m.t().contiguous(), xv[a - s:a].abs() @ m.abs().t().contiguous())
             for s, a, m in zip(sizes, torch.tensor(sizes).cumsum(0).tolist(), wv)]
    return got.double(), torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def fine(size, got, y, sums):
    _, bf16, _, _, _, k = size
    if not bf16:
        return (got - y).abs() <= k * U * sums
    cut = 0.0 if form(*size)[0] == "few" else 2.0 ** -10
    return (got - y).abs() <= (cut + k * U) * sums * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()


@pytest.mark.parametrize("size", FORWARD, ids=lambda s: "-".join(map(str, s)))
def test_values_far_apart(size):
    _, _, experts, t, n, k = size
    x, w = spread8((t, k), t, False), spread8((max(experts, 1), n, k), n, True)
    assert bool(fine(size, *product(size, x, w)).all())


@pytest.mark.parametrize("size", FORWARD, ids=lambda s: "-".join(map(str, s)))
def test_normal_values(size):
    _, bf16, experts, t, n, k = size
    x = f8.quantize(torch.randn(t, k, generator=gen(t), device="cuda"))
    w = f8.quantize_weight(torch.randn(max(experts, 1), n, k, generator=gen(n), device="cuda") * 0.02)
    got, y, sums = product(size, x, w)
    assert bool(fine(size, got, y, sums).all())
    if not bf16:
        return
    # 1.6 % and 2^-15.58 of the model, and room for what a sample of them varies by
    assert float((got != y.to(torch.bfloat16).double()).double().mean()) <= 0.02
    rms = y.square().mean().sqrt()
    near = y.abs() <= rms * 2.0 ** -9
    if int(near.sum()) >= 400:
        assert float((got - y)[near].square().mean().sqrt() / rms) <= 2.0 ** -15.4


@pytest.mark.parametrize("every, at", [(8, 0), (8, 3), (8, 7), (16, 5), (32, 0), (64, 9), (4, 1), (2, 0)])
def test_one_large_product_among_small_ones(every, at):
    """Small products 14 powers of two under the large ones, which cut the most."""
    t, n, k = 64, 128, 1024
    q = torch.full((n, k), 7 * 2.0 ** -9, device="cuda")  # 1.75 * 2^-7
    q[:, at::every] = 128.0
    x = held(torch.ones(t, k, device="cuda"), torch.full((t, 8), 127, device="cuda"))
    w = held(q, torch.full((1, 8), 127, device="cuda"))
    assert form(MATMUL, 1, 0, t, n, k)[0] == 0
    want = q[0].double().sum()
    got = f8.matmul(x, w).double()
    assert bool(((got - want).abs() <= (2.0 ** -10 + k * U) * want * (1 + 2.0 ** -8) + 2.0 ** -8 * want).all())
    # alternating signs: the large ones cancel, and what is left shows the cut itself
    sign = torch.ones(k, device="cuda")
    sign[at::2 * every] = -1.0
    w = held(q * sign, torch.full((1, 8), 127, device="cuda"))
    y, sums = (q[0] * sign).double().sum(), q[0].double().sum()
    got = f8.matmul(x, w).double()
    assert bool(((got - y).abs() <= (2.0 ** -10 + k * U) * sums * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()).all())
    assert torch.equal(f8.matmul(x, w, dtype=torch.float32).double(), y.expand(t, n))  # exact products, fp32 sums
