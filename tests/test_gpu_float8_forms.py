"""Every form of the 8-bit floating-point layer's products on the GPU, on small
whole numbers (tests/test_gpu_float8.py), so results have to be equal; the
workspace is of exactly the asked size between guard bytes."""
import pytest
import torch

from float8_common import CODE, E8M0, GRAD_INPUT, GRAD_WEIGHT, MATMUL, abi, exact8, exact_grad, values, workspace
from float8_forms import SIZES, form
from matrix_aware_optimizer_muon_amd import float8 as f8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_form(size):
    product, bf16, experts, t, n, k = size
    E, dtype = max(experts, 1), torch.bfloat16 if bf16 else torch.float32
    fwd, dw = product == MATMUL, product == GRAD_WEIGHT
    a = exact8((t, k), t, False) if fwd else exact_grad((t, n), t)
    aq = a.q if fwd else a
    lda = aq.stride(0) if t > 1 else (k + 15) // 16 * 16 if fwd else n
    assert form(*size, a=aq.data_ptr()) == form(*size)
    b = exact8((t, k), n, False) if dw else exact8((E, n, k), n, True)
    av, bv = values(a, False) if fwd else a.double(), values(b, not dw)
    ldb, bs = b.q.stride(-2), (b.q.stride(0) if not dw else 0)
    sizes = [t // E + (i < t % E) for i in range(E)]
    if experts > 1:  # uneven: the first expert's rows are the second's
        sizes[1] += sizes[0]
        sizes[0] = 0
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)
    out = torch.full((E, n, k) if dw else (t, n if fwd else k), 7.0, device="cuda", dtype=dtype)
    want = torch.zeros_like(out, dtype=torch.float64)
    at = 0
    for e, rows in enumerate(sizes):
        r = slice(at, at + rows)
        if dw:
            want[e] = av[r].t().contiguous() @ bv[r]
        else:
            want[r] = av[r] @ (bv[e].t().contiguous() if fwd else bv[e])
        at += rows
    need = workspace(product, aq.data_ptr(), lda, experts > 0, E, t, n, k, CODE[dtype])
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    s, f, g = torch.cuda.current_stream().cuda_stream, abi(), ends.data_ptr() if experts else 0
    tail = (CODE[dtype], ws.data_ptr() + 256, need, s)
    if fwd:
        st = f.muon_f8_matmul(aq.data_ptr(), lda, a.scale.data_ptr(), b.q.data_ptr(), ldb, bs, b.scale.data_ptr(), g, E, t, n, k,
                              out.data_ptr(), n, *tail)
    elif product == GRAD_INPUT:
        st = f.muon_f8_grad_input(aq.data_ptr(), lda, b.q.data_ptr(), ldb, bs, b.scale.data_ptr(), g, E, t, n, k,
                                  out.data_ptr(), k, *tail)
    else:
        st = f.muon_f8_grad_weight(aq.data_ptr(), lda, b.q.data_ptr(), ldb, b.scale.data_ptr(), g, E, t, n, k, out.data_ptr(), k,
                                   n * k, CODE[dtype], 0, ws.data_ptr() + 256, need, s)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want.to(dtype))
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + need:] == 0xA5).all())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("t", [8, 30, 200])
def test_scales_far_apart(t, bf16):
    """2^-126 times 2^125: exact, whichever way the scales go in."""
    n, k, dtype = 130, 300, torch.bfloat16 if bf16 else torch.float32
    x, w = exact8((t, k), 1, False), exact8((n, k), 2, True)
    low = f8.F8(x.q, (x.scale.view(torch.uint8) - 125).view(E8M0))
    high = f8.F8(w.q, (w.scale.view(torch.uint8) + 124).view(E8M0))
    want = values(x, False) @ values(w, True).t() / 2
    assert torch.equal(f8.matmul(low, high, dtype=dtype), want.to(dtype))
    dy = exact_grad((t, n), 3)
    assert torch.equal(f8.grad_input((dy.double() * 2.0 ** -120).bfloat16(), high, dtype=dtype),
                       (dy.double() @ values(w, True) * 16).to(dtype))
    assert torch.equal(f8.grad_weight((dy.double() * 2.0 ** 120).bfloat16(), low, dtype=dtype),
                       (dy.double().t() @ values(x, False) / 32).to(dtype))


def test_rows_of_a_gradient_far_apart():
    """More than 2^24 bytes apart, and more than 2^32 in all: laid out again."""
    t, n, k, ld = 300, 64, 96, (1 << 23) + 8
    far = torch.empty(t * ld, dtype=torch.bfloat16, device="cuda").as_strided((t, n), (ld, 1))
    dy, w, x = exact_grad((t, n), 1), exact8((n, k), 2, True), exact8((t, k), 3, False)
    far.copy_(dy)
    assert torch.equal(f8.grad_input(far, w), f8.grad_input(dy, w))
    assert torch.equal(f8.grad_weight(far, x), f8.grad_weight(dy, x))


def test_8_bit_rows_far_apart():
    t, n, k, ld = 260, 300, 200, 1 << 23
    x, w, dy = exact8((t, k), 1, False), exact8((n, k), 2, True), exact_grad((t, n), 3)
    q = torch.empty(t * ld, dtype=torch.uint8, device="cuda").as_strided((t, k), (ld, 1))
    q.copy_(x.q.view(torch.uint8))
    far = f8.F8(q.view(x.q.dtype), x.scale)
    assert torch.equal(f8.matmul(far, w), f8.matmul(x, w))
    assert torch.equal(f8.grad_weight(dy, far), f8.grad_weight(dy, x))


def test_more_matrices_than_a_launch_has_workgroups():
    """2^24 workgroups and more: the call is cut in parts."""
    x = torch.randn(1000, 1030, device="cuda").bfloat16()
    many = 1 << 21
    w = x.repeat(many // 1000 + 1, 1)[:many].view(many, 1, 1030)
    got = f8.quantize_weight(w)
    want = f8.quantize(x)
    assert got.scale.shape == (many, 1, 9)
    for at in (0, 1000, many // 1000 * 1000 - 1000):
        assert torch.equal(got.q[at:at + 1000, 0].view(torch.uint8), want.q.view(torch.uint8))
        assert torch.equal(got.scale[at:at + 1000, 0].view(torch.uint8), want.scale.view(torch.uint8))
    last = many % 1000
    assert torch.equal(got.q[-last:, 0].view(torch.uint8), want.q[:last].view(torch.uint8))


def test_a_backward_pass_through_an_operator_raises():
    x, w = torch.randn(5, 48, device="cuda").requires_grad_(), torch.randn(7, 48, device="cuda").requires_grad_()
    plain = f8.quantize(x.detach())
    for out in (f8.quantize(x).scale.float(), f8.dequantize(f8.quantize(x)), f8.dequantize(f8.quantize_weight(w)),
                f8.matmul(plain, f8.quantize_weight(w)), f8.matmul(f8.quantize(x), f8.quantize_weight(w.detach())).relu()):
        assert out.requires_grad
        with pytest.raises(RuntimeError, match=r"derivative for float8\.\w+ is not implemented"):
            out.float().sum().backward()
    with torch.no_grad():
        assert not f8.matmul(f8.quantize(x), f8.quantize_weight(w)).requires_grad


def test_inside_a_function_of_ones_own():
    """The calls of the backward pass in a torch.autograd.Function, grouped."""
    class Experts8(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, ends):
            x8, w8 = f8.quantize(x), f8.quantize_weight(w)
            ctx.save_for_backward(*x8, *w8, ends)
            return f8.matmul(x8, w8, ends=ends)

        @staticmethod
        def backward(ctx, dy):
            xq, xs, wq, ws, ends = ctx.saved_tensors
            return (f8.grad_input(dy, f8.F8(wq, ws), ends, torch.float32), f8.grad_weight(dy, f8.F8(xq, xs), ends), None)

    x, w = torch.randn(20, 50, device="cuda").requires_grad_(), torch.randn(3, 32, 50, device="cuda").requires_grad_()
    ends = torch.tensor([7, 7, 18], dtype=torch.int32, device="cuda")
    dy = torch.randn(20, 32, device="cuda").bfloat16()
    Experts8.apply(x, w, ends).backward(dy)
    xv, wv = values(f8.quantize(x.detach()), False), values(f8.quantize_weight(w.detach()), True)
    d = dy.double()
    dx, dw = torch.zeros(20, 50, device="cuda", dtype=torch.float64), torch.zeros(3, 32, 50, device="cuda", dtype=torch.float64)
    for e, (a, b) in enumerate(((0, 7), (7, 7), (7, 18))):
        dx[a:b], dw[e] = d[a:b] @ wv[e], d[a:b].t() @ xv[a:b]
    # sums of 32 and of at most 11 products, one rounding each at most
    assert bool(((x.grad.double() - dx).abs() <= 33 * 2.0 ** -24 * (d.abs().sum(1, keepdim=True) * wv.abs().max())).all())
    assert bool(((w.grad.double() - dw).abs() <= 12 * 2.0 ** -24 * 11 * d.abs().max() * xv.abs().max()).all())
