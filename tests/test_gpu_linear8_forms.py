"""Every form of the tile kernels on sums that fp32 (and int32) hold exactly
whatever their order: the results have to be equal to the last bit.

Gradients: |dy| <= 2, |q| <= 15, scales 1, 2 or 4, so a sum of 20000 products
stays under 2^22.  Integer product: any q, power-of-two scales; the int32 sum
is rounded to fp32 once.  Outside the operands lie NaN (dy, scales) and -128
(q), outside the output and the workspace guards."""
import pytest
import torch

from linear8_common import GRAD_WEIGHT, MATMUL, product
from linear8_forms import FORMS, PAD, choice

pytestmark = pytest.mark.gpu

GUARD = 12345.0


def inside(values, fill):
    """The values in a matrix whose rows are PAD further apart, with a row
    below, all filled with `fill`."""
    r, c = values.shape
    big = torch.full((r + 1, c + PAD), fill, dtype=values.dtype, device="cuda")
    big[:r, :c] = values
    return big[:r, :c]


def scales(rows, powers, gen):
    s = torch.full((rows + 64,), float("nan"), device="cuda")
    table = torch.tensor([2.0 ** p for p in powers], device="cuda")
    s[:rows] = table[torch.randint(0, len(powers), (rows,), generator=gen, device="cuda")]
    return s[:rows]


def ints(shape, top, dtype, gen):
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(dtype)


def run(form, size, dtype, accumulate=False):
    t, n, k = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(t + n + k)
    if form.product == MATMUL:
        a, a_s = ints((t, k), 127, torch.int8, gen), scales(t, (-9, -5, 0), gen)
        b, b_s = ints((n, k), 127, torch.int8, gen), scales(n, (-3, 1, 4), gen)
        want = (a.double() @ b.double().t().contiguous()).float() * a_s[:, None] * b_s
        a, b = inside(a, -128), inside(b, -128)
    else:
        rows = t if form.product == GRAD_WEIGHT else n
        a, a_s = ints((t, n), 2, torch.bfloat16, gen), None
        b, b_s = ints((rows, k), 15, torch.int8, gen), scales(rows, (0, 1, 2), gen)
        left = a.double().t().contiguous() if form.product == GRAD_WEIGHT else a.double()
        want = (left @ (b.double() * b_s.double()[:, None])).float()
        assert float(want.abs().max()) < 2 ** 23
        a, b = inside(a, float("nan")), inside(b, -128)
    big = torch.full((want.shape[0] + 2, want.shape[1] + 5), GUARD, dtype=dtype, device="cuda")
    out = big[1:-1, 3:-2]
    if accumulate:
        base = ints(want.shape, 200, torch.float32, gen)  # exact in bf16
        out.copy_(base)
        want = want + base
    product(form.product, a, a_s, b, b_s, out, accumulate)
    assert torch.equal(out, want.to(dtype))
    g = torch.tensor(GUARD, dtype=dtype).item()
    assert bool((big[0] == g).all()) and bool((big[-1] == g).all())
    assert bool((big[:, :3] == g).all()) and bool((big[:, -2:] == g).all())


def name(form):
    return "-".join(str(int(v) if isinstance(v, bool) else v) for v in form)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form, size", FORMS.items(), ids=[name(f) for f in FORMS])
def test_form(form, size, dtype):
    assert choice(form.product, *size)[0] == form
    run(form, size, dtype)


WEIGHT = {f: s for f, s in FORMS.items() if f.product == GRAD_WEIGHT}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form, size", WEIGHT.items(), ids=[name(f) for f in WEIGHT])
def test_form_accumulates(form, size, dtype):
    run(form, size, dtype, accumulate=True)
