"""Weight gradients added to what an output holds, in every form that they take
(tests/float8_forms.py): tiles of one workgroup, split ones, grouped ones.  Whole
numbers, so results have to be equal."""
import pytest
import torch

from float8_common import GRAD_WEIGHT, exact8, exact_grad, gen, values
from float8_forms import SIZES, form
from matrix_aware_optimizer_muon_amd import float8 as f8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [s for s in SIZES if s[0] == GRAD_WEIGHT], ids=lambda s: "-".join(map(str, s)))
def test_accumulate(size):
    _, bf16, experts, t, n, k = size
    E, dtype = max(experts, 1), torch.bfloat16 if bf16 else torch.float32
    dy, x = exact_grad((t, n), t), exact8((t, k), n, False)
    assert form(*size, a=dy.data_ptr()) == form(*size)
    sizes = [t // E + (i < t % E) for i in range(E)]
    if experts > 1:  # uneven: the first expert's rows are the second's
        sizes[1] += sizes[0]
        sizes[0] = 0
    # within rows of a larger matrix, each place a number of its own
    held = torch.randint(-40, 41, (E, n, k + 5), generator=gen(k), device="cuda").to(dtype)
    want, at = held[..., 3:k + 3].double(), 0
    for e, rows in enumerate(sizes):
        want[e] += dy[at:at + rows].double().t().contiguous() @ values(f8.F8(x.q[at:at + rows], x.scale[at:at + rows]), False)
        at += rows
    around = held.clone()
    out = held[..., 3:k + 3] if experts else held[0, :, 3:k + 3]
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32) if experts else None
    assert f8.grad_weight(dy, x, ends=ends, out=out, accumulate=True) is out
    assert torch.equal(held[..., 3:k + 3], want.to(dtype))
    assert torch.equal(held[..., :3], around[..., :3]) and torch.equal(held[..., k + 3:], around[..., k + 3:])
