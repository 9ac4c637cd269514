"""The ends of the 8-bit floating-point layer's range on the GPU: every e4m3 value
under the smallest and the largest scales, one value a row, so that each result is
one product and has to be equal.  The 8-bit matrix cores take a value and its
scale apart; everything else takes value * scale as bf16 holds it: multiples of
2^-133 (nearest, ties to even), infinite from 2^128 on."""
import pytest
import torch

from float8_common import MATMUL, choice, exact8, held, values
from matrix_aware_optimizer_muon_amd import float8 as f8

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LOW, HIGH = (0, 1, 2, 3, 4), (246, 247, 248, 252, 253, 254)
# (bytes of the other operand's scales, so that results are normal numbers)
CASES = [(b, 219) for b in LOW] + [(b, 20) for b in HIGH]


def each_value(k, byte, square=False):
    """254 rows of k, a row for each e4m3 value that is a number, at a place of its own."""
    b = torch.tensor([v for v in range(256) if v & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    q = torch.zeros(254, k, device="cuda")
    q[torch.arange(254), torch.arange(254) * 7 % k] = b.view(torch.float8_e4m3fn).float()
    return held(q, torch.full((2 if square else 254, (k + 127) // 128), byte, device="cuda"))


def other(shape, byte, square):
    w = exact8(shape, 2, square)
    return f8.F8(w.q, torch.full_like(w.scale.view(torch.uint8), byte).view(w.scale.dtype))


def as_bf16(x, square):
    """The operand as bf16 holds it (converted on the CPU)."""
    return values(x, square).cpu().float().to(BF).double().cuda()


def same(got, want):
    want = want.to(got.dtype)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0, posinf=1e30, neginf=-1e30), want.nan_to_num(0.0, posinf=1e30, neginf=-1e30))


@pytest.mark.parametrize("byte, at", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_products(byte, at, dtype):
    n, k = 130, 256
    x, w = each_value(k, byte), other((n, k), at, True)
    wv = values(w, True).t().contiguous()
    assert choice(MATMUL, 1 << 20, k, False, 1, 254, n, k, dtype == BF)["few"] == 0
    whole = values(x, False) if dtype == BF else as_bf16(x, False)
    same(f8.matmul(x, w, dtype=dtype), whole @ wv)
    few = f8.F8(x.q[:16], x.scale[:16]), f8.F8(x.q[120:136], x.scale[120:136])
    for part, r in zip(few, (slice(0, 16), slice(120, 136))):
        assert choice(MATMUL, 1 << 20, k, False, 1, 16, n, k, dtype == BF)["few"] > 0
        same(f8.matmul(part, w, dtype=dtype), as_bf16(x, False)[r] @ wv)


@pytest.mark.parametrize("byte, at", CASES)
def test_gradients(byte, at):
    # a row of dy for each weight row, and whole numbers for the weight gradient
    k, n = 256, 254
    w = each_value(k, byte, square=True)
    dy = (torch.eye(n, device="cuda") * 3 * 2.0 ** (at - 127)).to(BF)
    same(f8.grad_input(dy, w, dtype=F32), dy.double() @ as_bf16(w, True))
    x = each_value(k, byte)
    same(f8.grad_weight(dy, x), dy.double().t().contiguous() @ as_bf16(x, False))


@pytest.mark.parametrize("byte", [3, 120, 247])
def test_scales_that_hold_every_value(byte):
    """From 2^-124 to 2^119 bf16 holds every value: nothing is rounded."""
    x = each_value(256, byte)
    assert torch.equal(as_bf16(x, False), values(x, False)) == (byte <= 246)
    assert byte <= 246 or float(values(x, False).abs().max()) == 448 * 2.0 ** 120


def test_what_quantize_makes_of_the_smallest_blocks():
    """A block of at most 448 * 2^-125 gets a scale under which bf16 does not hold
    all of its values."""
    x = torch.zeros(2, 128, device="cuda")
    x[0, 0], x[1, 0] = 448 * 2.0 ** -125, 449 * 2.0 ** -125
    x[:, 1] = 2.0 ** -134
    assert f8.quantize(x).scale.view(torch.uint8)[:, 0].tolist() == [2, 3]
