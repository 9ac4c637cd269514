"""The forward operators record nothing for autograd, and say so: a backward
pass through one of their results raises instead of leaving gradients out."""
import pytest
import torch

from matrix_aware_optimizer_muon_amd import linear8 as l8

pytestmark = pytest.mark.gpu


def leaf(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype).requires_grad_()


def forwards():
    """(name, result) of each forward operator, one input requiring a gradient."""
    x, w, g = leaf(5, 48), leaf(7, 48), leaf(48)
    plain = x.detach()
    q, wq = l8.quantize(plain), l8.quantize(w)
    yield "quantize", l8.dequantize(wq, torch.float32)
    yield "quantize", l8.quantize(x).scale
    yield "dequantize", l8.dequantize(l8.Q8(q.q, q.scale.clone().requires_grad_()), torch.float32)
    yield "matmul", l8.matmul(q, wq, torch.float32)
    yield "matmul", l8.matmul(l8.quantize(x), l8.quantize(w.detach()), torch.float32)
    yield "rmsnorm", l8.rmsnorm(x, g.detach())[0]
    yield "rmsnorm", l8.rmsnorm(plain, g)[0]
    yield "rmsnorm", l8.rmsnorm(plain, g.detach(), residual=x)[1]
    yield "rmsnorm", l8.rmsnorm(x, g.detach())[2]
    yield "rmsnorm", l8.rmsnorm(plain, g, q8=True)[0].scale
    yield "rmsnorm", l8.matmul(l8.rmsnorm(plain, g, q8=True)[0], q, torch.float32)
    # through a layer into torch's own operators and out again
    yield "matmul", torch.relu(l8.matmul(l8.quantize(x), q)).float().square()


def test_a_backward_pass_through_an_operator_raises():
    seen = set()
    for name, out in forwards():
        assert out.requires_grad
        with pytest.raises(RuntimeError, match=r"derivative for linear8\.\w+ is not implemented"):
            out.sum().backward()
        seen.add(name)
    assert seen == {"quantize", "dequantize", "matmul", "rmsnorm"}


def test_results_are_the_same_and_plain_where_nothing_requires_a_gradient():
    x, g = leaf(6, 40), leaf(40)
    y, h, rstd = l8.rmsnorm(x, g, residual=x)
    with torch.no_grad():
        want = l8.rmsnorm(x, g, residual=x)
        q = l8.quantize(x)
        out = l8.matmul(q, q)
    for a, b in zip((y, h, rstd), want):
        assert torch.equal(a, b) and not b.requires_grad and b.grad_fn is None
    assert not out.requires_grad and not q.scale.requires_grad
    assert not any(t.requires_grad for t in l8.rmsnorm(x.detach(), g.detach()))
    with torch.inference_mode():
        assert torch.equal(l8.matmul(l8.quantize(x), l8.quantize(x)), out)


def test_inside_a_function_of_ones_own():
    """The way to give them a gradient: the calls of the backward pass in a
    torch.autograd.Function, whose forward runs without recording."""
    class Linear8(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            x8, w8 = l8.quantize(x), l8.quantize(w)
            ctx.save_for_backward(*x8, *w8)
            return l8.matmul(x8, w8)

        @staticmethod
        def backward(ctx, dy):
            xq, xs, wq, ws = ctx.saved_tensors
            return l8.grad_input(dy, l8.Q8(wq, ws), torch.float32), l8.grad_weight(dy, l8.Q8(xq, xs))

    x, w = leaf(20, 48), leaf(32, 48)
    dy = torch.randn(20, 32, device="cuda").bfloat16()
    Linear8.apply(x, w).backward(dy)
    x8, w8 = l8.quantize(x.detach()), l8.quantize(w.detach())
    assert torch.equal(x.grad, l8.grad_input(dy, w8, torch.float32)) and torch.equal(w.grad, l8.grad_weight(dy, x8))


def test_the_backward_operators_give_constants():
    # their results are gradients: no graph grows along a loop that adds them up
    x, w = leaf(20, 48), leaf(32, 48)
    x8, w8 = l8.quantize(x), l8.quantize(w)
    dy = leaf(20, 32, dtype=torch.bfloat16)
    assert not l8.grad_input(dy, w8).requires_grad and not l8.grad_weight(dy, x8).requires_grad
    y, h, rstd = l8.rmsnorm(x, leaf(48))
    assert not any(t.requires_grad for t in l8.rmsnorm_backward(y, h, rstd, leaf(48)))


@pytest.mark.parametrize("accumulate", [False, True])
def test_writing_into_out_counts_as_a_write(accumulate):
    x = l8.quantize(torch.randn(20, 48, device="cuda"))
    dy = torch.randn(20, 32, device="cuda").bfloat16()
    out = torch.ones(32, 48, device="cuda")
    factor = leaf(32, 48)
    loss = (factor * out).sum()  # keeps out for factor's gradient
    before = out._version
    assert l8.grad_weight(dy, x, out=out, accumulate=accumulate) is out
    assert out._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # such tensors have no version
        fresh = torch.zeros(32, 48, device="cuda")
        assert torch.equal(l8.grad_weight(dy, x, out=fresh), l8.grad_weight(dy, x))
