"""Outputs in the place of inputs, where include/muon_linear8.h allows it: h for
x or the residual, y for x, dx for dy or dh.  Bit for bit what separate outputs
hold; widths on either side of what one wave, one workgroup and the registers
hold, ragged ends (read from columns that other lanes store) among them."""
import pytest
import torch

from linear8_common import CODE, abi, back_workspace

pytestmark = pytest.mark.gpu

WIDTHS = [1, 7, 9, 64, 515, 1023, 2049, 3584, 4097, 8193, 16384, 16385, 18945, 32767]
ROWS = 300


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def norm(x, res, w, h, y, q, scale, rstd):
    rows, cols = x.shape
    p = lambda t: t.data_ptr() if t is not None else 0
    st = abi().muon_rmsnorm_forward(p(x), cols, p(res), cols, p(w), CODE[x.dtype], rows, cols, 1e-6, p(h), cols,
                                    p(y), cols, p(q), cols, p(scale), p(rstd),
                                    torch.cuda.current_stream().cuda_stream)
    assert st == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("eight", [False, True])
def test_norm(cols, dtype, eight):
    x, r = rand((ROWS, cols), 1, dtype), rand((ROWS, cols), 2, dtype)
    w = 1 + 0.1 * rand((cols,), 3, torch.float32)

    def call(x, res, h, y=None):
        q = torch.empty(ROWS, cols, dtype=torch.int8, device="cuda") if eight else None
        scale = torch.empty(ROWS, device="cuda") if eight else None
        if not eight and y is None:
            y = torch.empty_like(x)
        rstd = torch.empty(ROWS, device="cuda")
        norm(x, res, w, h, None if eight else y, q, scale, rstd)
        torch.cuda.synchronize()
        return [q, scale, rstd] if eight else [y, rstd]

    h = torch.empty_like(x)
    want = call(x, r, h)
    for at_x in (True, False):  # h over x, over the residual
        a, b = x.clone(), r.clone()
        got = call(a, b, a if at_x else b)
        assert torch.equal(a if at_x else b, h) and torch.equal(b if at_x else a, r if at_x else x)
        assert all(torch.equal(u, v) for u, v in zip(got, want))
    if not eight:
        a, h2 = x.clone(), torch.empty_like(x)  # y over x, with and without a residual
        got = call(a, r, h2, y=a)
        assert torch.equal(h2, h) and all(torch.equal(u, v) for u, v in zip(got, want))
        a, b = x.clone(), r.clone()  # both
        got = call(a, b, b, y=a)
        assert torch.equal(b, h) and all(torch.equal(u, v) for u, v in zip(got, want))
        want = call(x, None, None)
        a = x.clone()
        assert all(torch.equal(u, v) for u, v in zip(call(a, None, None, y=a), want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("h8", [False, True])
def test_norm_backward(cols, dtype, h8):
    dy, dh = rand((ROWS, cols), 1, dtype, 1e-2), rand((ROWS, cols), 2, dtype, 1e-2)
    w = 1 + 0.1 * rand((cols,), 3, torch.float32)
    h = torch.randint(-127, 128, (ROWS, cols), device="cuda", dtype=torch.int8) if h8 else rand((ROWS, cols), 4, dtype)
    scale = torch.full((ROWS,), 2.0 ** -5, device="cuda") if h8 else None
    rstd = 0.5 + torch.rand(ROWS, device="cuda")
    need = back_workspace(ROWS, cols)

    def call(dy, dh, dx):
        ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        dw = torch.empty(cols, device="cuda")
        st = abi().muon_rmsnorm_backward(dy.data_ptr(), cols, h.data_ptr(), cols, scale.data_ptr() if h8 else 0,
                                         rstd.data_ptr(), w.data_ptr(), dh.data_ptr() if dh is not None else 0, cols,
                                         CODE[dtype], ROWS, cols, dx.data_ptr(), cols, dw.data_ptr(), ws.data_ptr(),
                                         need, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        return dw

    dx = torch.empty_like(dy)
    dw = call(dy, dh, dx)
    a = dy.clone()
    assert torch.equal(call(a, dh, a), dw) and torch.equal(a, dx)
    a = dh.clone()
    assert torch.equal(call(dy, a, a), dw) and torch.equal(a, dx)
    dw = call(dy, None, dx)
    a = dy.clone()
    assert torch.equal(call(a, None, a), dw) and torch.equal(a, dx)
