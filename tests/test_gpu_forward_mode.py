"""Forward-mode derivatives are not implemented: a tensor with a tangent raises
in every operator of the 8-bit layers and of clipping, instead of losing it."""
import pytest
import torch
import torch.autograd.forward_ad as fw

from matrix_aware_optimizer_muon_amd import clip
from matrix_aware_optimizer_muon_amd import float8 as f8
from matrix_aware_optimizer_muon_amd import linear8 as l8

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def calls():
    """name, a call of one tensor that makes a tangent, that tensor"""
    x, w = torch.randn(6, 64, device="cuda"), torch.randn(32, 64, device="cuda")
    dy, out, gain = torch.randn(6, 32, device="cuda").to(BF), torch.empty(32, 64, device="cuda"), torch.ones(64, device="cuda")
    x8, w8, xq, wq = f8.quantize(x), f8.quantize_weight(w), l8.quantize(x), l8.quantize(w)
    h, rstd = l8.rmsnorm(x, gain)[0], l8.rmsnorm(x, gain)[2]
    return [
        ("float8.quantize", f8.quantize, x), ("float8.quantize_weight", f8.quantize_weight, w),
        ("float8.grad_input", lambda v: f8.grad_input(v, w8), dy), ("float8.grad_weight", lambda v: f8.grad_weight(v, x8), dy),
        ("float8.grad_weight", lambda v: f8.grad_weight(dy, x8, out=v), out),
        ("clip.grad_norm", lambda v: clip.grad_norm([w, v]), x), ("clip.clip_grad_norm", lambda v: clip.clip_grad_norm([w, v], 1.0), x),
        ("clip.clip_grad_norm", lambda v: clip.clip_grad_norm([w], 1.0, out=[v]), out),
        ("linear8.quantize", l8.quantize, x), ("linear8.rmsnorm", lambda v: l8.rmsnorm(v, gain), x),
        ("linear8.rmsnorm", lambda v: l8.rmsnorm(x, v), gain), ("linear8.rmsnorm", lambda v: l8.rmsnorm(x, gain, v), x),
        ("linear8.dequantize", lambda v: l8.dequantize(l8.Q8(xq.q, v)), xq.scale),
        ("linear8.matmul", lambda v: l8.matmul(l8.Q8(xq.q, v), wq), xq.scale),
        ("linear8.rmsnorm_backward", lambda v: l8.rmsnorm_backward(v, h, rstd, gain), x),
        ("linear8.grad_input", lambda v: l8.grad_input(v, wq), dy), ("linear8.grad_weight", lambda v: l8.grad_weight(v, xq), dy),
    ]


@pytest.mark.parametrize("at", range(17))
def test_a_tangent_raises(at):
    assert len(calls()) == 17
    name, call, v = calls()[at]
    call(v)
    keep = v.clone()
    with fw.dual_level():
        dual = fw.make_dual(v, torch.ones_like(v))
        with pytest.raises(NotImplementedError, match=f"forward-mode derivative for {name} is not implemented"):
            call(dual)
        assert torch.equal(v, keep)  # (what writes has not)
        call(fw.unpack_dual(dual).primal)


def test_inside_a_function_with_a_jvp():
    """A torch.autograd.Function that brings its own jvp may call them."""
    class Rounded(torch.autograd.Function):
        @staticmethod
        def forward(x):
            return f8.dequantize(f8.quantize(x), torch.float32)

        @staticmethod
        def setup_context(ctx, inputs, output):
            pass

        @staticmethod
        def jvp(ctx, dx):
            return dx.clone()

    x = torch.randn(3, 40, device="cuda")
    with fw.dual_level():
        out = fw.unpack_dual(Rounded.apply(fw.make_dual(x, torch.full_like(x, 2.0))))
        assert torch.equal(out.primal, f8.dequantize(f8.quantize(x), torch.float32)) and bool((out.tangent == 2).all())
