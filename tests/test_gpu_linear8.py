"""The 8-bit linear layer's operators on the GPU against plain 64-bit
formulas.  Tolerances count roundings: half a step relative to the value is
2^-8 in bf16 and 2^-24 in fp32."""
import numpy as np
import pytest
import torch

from matrix_aware_optimizer_muon_amd import linear8 as l8
from linear8_common import GRAD_INPUT, GRAD_WEIGHT, MATMUL, abi, product

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
GUARD = 12345.0


def rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, off, extra):
    """t's values in a view with a larger row distance and a shifted start."""
    r, c = t.shape
    big = torch.full((r, c + off + extra), 7, dtype=t.dtype, device=t.device)
    big[:, off:off + c] = t
    return big[:, off:off + c]


def rows8(v):
    """The 8-bit form in 64 bits: (q, scale)."""
    top = v.abs().amax(dim=1)
    steps = torch.from_numpy(np.ldexp(1.0, np.arange(-126, 128))).to(v.device)  # (torch's pow is not exact)
    step = steps[torch.searchsorted(127.0 * steps, top)]
    return torch.round(v / step[:, None]), step


def within(got, ref, bound, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / bound.clamp_min(1e-300)).max()):.3g} of the bound")


def same8(got, want_q, want_scale, v):
    """Equal 8-bit rows, but for values within 1e-9 of a rounding border."""
    assert torch.equal(got.scale.double(), want_scale)
    t = v / want_scale[:, None]
    border = ((t - torch.floor(t)) - 0.5).abs() < 1e-9
    assert bool(((got.q.double() == want_q) | border).all())


WIDTHS = [1, 2, 7, 8, 9, 63, 512, 513, 1000, 1025, 2047, 2049, 3584, 4095, 4097, 8192, 8193, 18944, 32768]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_quantize_round_trip(cols, dtype):
    x = rand((5, cols), cols, dtype)
    x[3] *= 1e-30
    got = l8.quantize(x)
    q, s = rows8(x.double())
    same8(got, q, s, x.double())
    for out in (BF, F32):  # q * scale has at most 7 significant bits: exact in both
        assert torch.equal(l8.dequantize(got, out).double(), q * s[:, None])


def test_quantize_scale_borders():
    # 127 * 2^e itself keeps exponent e, the next value above takes e + 1
    x = torch.zeros(6, 4, device="cuda")
    x[0, 1] = 127.0
    x[1, 2] = -float(np.nextafter(np.float32(127.0), np.float32(200.0)))
    x[2, 0] = 2.0 ** -149
    x[4, 0] = 3.0e38
    x[5, :3] = torch.tensor([127.0, 0.5, 2.5])
    got = l8.quantize(x)
    assert got.scale.tolist() == [1.0, 2.0, 2.0 ** -126, 2.0 ** -126, 2.0 ** 121, 1.0]
    assert got.q[0].tolist() == [0, 127, 0, 0] and got.q[1].tolist() == [0, 0, -64, 0]
    assert got.q[3].tolist() == [0] * 4 and got.q[5].tolist() == [127, 0, 2, 0]  # ties to even
    assert torch.equal(l8.dequantize(got, F32)[3], x[3])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_non_finite_rows(dtype):
    x = rand((5, 700), 1, dtype)
    x[1, 699] = float("nan")
    x[3, 0] = float("-inf")
    got = l8.quantize(x)
    bad = torch.tensor([False, True, False, True, False])
    assert got.scale.isnan().cpu().equal(bad)
    assert not got.q[1].any() and not got.q[3].any()
    assert l8.dequantize(got, dtype).isnan().all(dim=1).cpu().equal(bad)
    clean = l8.quantize(x[::2])
    assert torch.equal(got.q[::2], clean.q) and torch.equal(got.scale[::2], clean.scale)


def norm_ref(x, r, w, eps, dtype):
    h = x.double() if r is None else (x.float() + r.float()).to(dtype).double()
    rstd = 1 / torch.sqrt((h * h).mean(dim=1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("res", [False, True])
def test_norm(cols, res, dtype):
    x = rand((7, cols), cols, dtype)
    r = strided(rand((7, cols), cols + 1, dtype), 1, 2) if res else None
    w = 1 + 0.1 * rand((cols,), 5)
    eps = 1e-6
    h64, rstd64, y64 = norm_ref(x, r, w, eps, dtype)
    y, h, rstd = l8.rmsnorm(x, w, residual=r, eps=eps)
    if res:
        within(h, x.double() + r.double(), (x.double() + r.double()).abs() * (HALF[dtype] + U) , "h")
    else:
        assert h is x
    h64 = h.double()
    rstd64 = 1 / torch.sqrt((h64 * h64).mean(dim=1) + float(np.float32(eps)))
    y64 = h64 * rstd64[:, None] * w.double()
    within(rstd, rstd64, rstd64 * U * 1.001, "rstd")
    # rstd and two products in fp32, then the type's own rounding
    within(y, y64, y64.abs() * (3 * U * 1.001 + (HALF[BF] * 1.001 if dtype == BF else 0)) + 1e-40, "y")
    y8, h2, rstd2 = l8.rmsnorm(x, w, residual=r, eps=eps, q8=True)
    assert torch.equal(h2, h) and torch.equal(rstd2, rstd)
    q, s = rows8(y64)
    same8(y8, q, s, y64)


def test_norm_shapes_strides_and_empty():
    x = rand((2, 3, 40), 1, BF)
    w = rand((40,), 2)
    y, h, rstd = l8.rmsnorm(x, w)
    assert y.shape == x.shape and rstd.shape == (2, 3)
    y8, _, _ = l8.rmsnorm(x, w, q8=True)
    assert y8.q.shape == x.shape and y8.scale.shape == (2, 3)
    xs = strided(x.reshape(6, 40), 3, 5)
    assert torch.equal(l8.rmsnorm(xs, w)[0], y.reshape(6, 40))
    y, h, rstd = l8.rmsnorm(x[:0], w)
    assert y.shape == (0, 3, 40) and rstd.shape == (0, 3)
    dx, dw = l8.rmsnorm_backward(x[:0], x[:0], rstd, w)
    assert dx.shape == (0, 3, 40) and not dw.any()


def test_norm_zero_and_non_finite_rows():
    x = rand((6, 300), 3)
    x[1] = 0
    x[2, 5] = float("inf")
    x[4, 299] = float("nan")
    w = torch.ones(300, device="cuda")
    y, _, rstd = l8.rmsnorm(x, w)
    assert not y[1].any() and bool(y[4].isnan().all()) and bool(y[2, 5].isnan())
    y8, _, _ = l8.rmsnorm(x, w, q8=True)
    assert y8.scale.isnan().tolist() == [False, False, True, False, True, False]
    assert not y8.q[1].any()
    clean = l8.rmsnorm(x[[0, 3, 5]], w, q8=True)[0]
    assert torch.equal(y8.q[[0, 3, 5]], clean.q)


def test_norm_writes_only_its_rows():
    rows, cols, ld = 9, 515, 530
    x = rand((rows, cols), 1, BF)
    w = rand((cols,), 2)
    f = abi()
    s = torch.cuda.current_stream().cuda_stream
    y = torch.full((rows + 2, ld), GUARD, dtype=BF, device="cuda")
    h = torch.full((rows + 2, ld), GUARD, dtype=BF, device="cuda")
    q = torch.full((rows + 2, ld), 99, dtype=torch.int8, device="cuda")
    vec = torch.full((3, rows + 2), GUARD, device="cuda")
    for yp, qp in ((y, None), (None, q)):
        st = f.muon_rmsnorm_forward(x.data_ptr(), cols, x.data_ptr(), cols, w.data_ptr(), 1, rows, cols, 1e-6,
                                    h[1].data_ptr(), ld, yp[1].data_ptr() if yp is not None else 0, ld,
                                    qp[1].data_ptr() if qp is not None else 0, ld,
                                    vec[0, 1:].data_ptr() if qp is not None else 0, vec[1, 1:].data_ptr(), s)
        assert st == 0
    torch.cuda.synchronize()
    for b, g in ((y, y[0, 0].item()), (h, h[0, 0].item()), (q, 99)):
        assert (b[0] == g).all() and (b[-1] == g).all() and (b[1:-1, cols:] == g).all()
        assert (b[1:-1, :cols] != g).any(dim=1).all()
    assert (vec[:2, 0] == GUARD).all() and (vec[:2, -1] == GUARD).all()


def back_ref(dy, h, rstd, w, dh):
    n = h * rstd[:, None]
    g = dy * w
    mean = (g * n).mean(dim=1, keepdim=True)
    dx = rstd[:, None] * (g - n * mean) + (dh if dh is not None else 0.0)
    # roundings: n, g, the dot (per lane 8 NC <= 32 terms, 6 + 4 levels), the
    # two fused terms; each relative to its term's magnitude
    mag = rstd[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(dim=1, keepdim=True) * 50)
    mag = 4 * mag + (dh.abs() if dh is not None else 0.0)
    return dx, (dy * n).sum(dim=0), mag, (dy * n).abs().sum(dim=0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 3584), (3, 9), (5, 512), (40, 513), (33, 2048), (700, 100),
                                        (5000, 64), (1500, 3584), (17, 4097), (9, 8193), (600, 8192), (4, 18944),
                                        (3, 32768)])
@pytest.mark.parametrize("h8, with_dh", [(False, True), (True, False), (True, True), (False, False)])
def test_norm_backward(rows, cols, dtype, h8, with_dh):
    h = rand((rows, cols), 1, dtype, 3.0)
    dy = strided(rand((rows, cols), 2, dtype, 1e-2), 1, 0)
    dh = strided(rand((rows, cols), 3, dtype, 1e-2), 0, 3) if with_dh else None
    w = 1 + 0.1 * rand((cols,), 4)
    rstd = torch.rsqrt(h.float().square().mean(dim=1) + 1e-6)
    hk = l8.quantize(h) if h8 else h
    h64 = l8.dequantize(hk, F32).double() if h8 else h.double()
    dx, dw = l8.rmsnorm_backward(dy, hk, rstd, w, dh=dh)
    rx, rw, mag, magw = back_ref(dy.double(), h64, rstd.double(), w.double(),
                                 dh.double() if dh is not None else None)
    within(dx, rx, 2 * U * mag + (HALF[BF] * 1.001 if dtype == BF else 0) * rx.abs() + 1e-30, "dx")
    within(dw, rw, (min(rows, 64) + rows / 512 + 20) * U * magw + 1e-30, "dweight")
    again = l8.rmsnorm_backward(dy, hk, rstd, w, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_norm_backward_against_differences():
    x = rand((3, 50), 1)
    w = 1 + 0.1 * rand((50,), 2)
    c = rand((3, 50), 3)
    _, h, rstd = l8.rmsnorm(x, w, eps=1e-3)
    dx, dw = l8.rmsnorm_backward(c, h, rstd, w)

    def loss(xv, wv):
        return (norm_ref(xv, None, wv, float(np.float32(1e-3)), F32)[2] * c.double()).sum()

    step = 1e-6
    for i, j in ((0, 0), (1, 17), (2, 49)):
        d = torch.zeros(3, 50, dtype=torch.float64, device="cuda")
        d[i, j] = step
        num = (loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())) / (2 * step)
        assert abs(float(num) - float(dx[i, j])) < 1e-5
        d = torch.zeros(50, dtype=torch.float64, device="cuda")
        d[j] = step
        num = (loss(x.double(), w.double() + d) - loss(x.double(), w.double() - d)) / (2 * step)
        assert abs(float(num) - float(dw[j])) < 1e-5


def test_norm_backward_non_finite_row_stays_in_its_row():
    h = rand((4, 200), 1)
    dy = rand((4, 200), 2)
    dy[2, 7] = float("nan")
    w = torch.ones(200, device="cuda")
    rstd = torch.rsqrt(h.square().mean(dim=1))
    dx, dw = l8.rmsnorm_backward(dy, h, rstd, w)
    assert dx.isnan().any(dim=1).tolist() == [False, False, True, False]
    assert dw.isnan().nonzero().flatten().tolist() == [7]


# products -----------------------------------------------------------------

def q8rand(rows, cols, seed, scales="pow2"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(-127, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    if scales == "pow2":
        table = torch.from_numpy(np.ldexp(np.float32(1.0), np.arange(-9, -3))).cuda()
        s = table[torch.randint(0, 6, (rows,), generator=g, device="cuda")]
    else:
        s = torch.rand(rows, generator=g, device="cuda") * 0.02 + 0.001
    return l8.Q8(q, s)


def guarded(rows, cols, dtype):
    big = torch.full((rows + 2, cols + 5), GUARD, dtype=dtype, device="cuda")
    return big, big[1:-1, 3:3 + cols]


def check_guard(big, cols):
    torch.cuda.synchronize()
    g = torch.tensor(GUARD, dtype=big.dtype)
    assert (big[0] == g.item()).all() and (big[-1] == g.item()).all()
    assert (big[:, :3] == g.item()).all() and (big[:, 3 + cols:] == g.item()).all()


def dense(x):
    return x.q.double() * x.scale.double()[:, None]


def check_matmul(t, n, k, dtype, x=None, w=None, scales="pow2"):
    x = x if x is not None else q8rand(t, k, 1, scales)
    w = w if w is not None else q8rand(n, k, 2, scales)
    big, out = guarded(t, n, dtype)
    product(MATMUL, x.q, x.scale, w.q, w.scale, out)
    ref = dense(x) @ dense(w).t().contiguous()
    within(out, ref, ref.abs() * (3 * U * 1.001 + (HALF[BF] * 1.001 if dtype == BF else 0)) + 1e-30, "y")
    check_guard(big, n)
    return x, w, out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n, k", [(1, 1), (2, 5), (15, 16), (16, 63), (17, 64), (100, 65), (33, 255), (48, 257),
                                  (1000, 1024), (37, 3584), (8201, 100)])
def test_matmul_few_rows(t, n, k, dtype):
    check_matmul(t, n, k, dtype)


@pytest.mark.parametrize("t, n, k", [(1, 40, 8192), (16, 40, 8193), (2, 3, 30001), (32, 50, 4096), (17, 50, 4100),
                                     (32, 4097, 4095), (5, 16383, 70), (16, 16385, 130), (31, 70, 20000)])
def test_matmul_few_rows_either_side_of_their_rules(t, n, k):
    check_matmul(t, n, k, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t, n, k", [(65, 1, 16), (100, 8, 33), (128, 128, 64), (129, 127, 80), (300, 130, 512),
                                     (257, 400, 1), (96, 64, 48), (95, 513, 100), (72, 260, 4096), (130, 130, 8191),
                                     (81, 70, 15), (70, 3, 7), (4000, 3500, 80), (3900, 3585, 97)])
def test_matmul_tiles(t, n, k, dtype):
    check_matmul(t, n, k, dtype)


@pytest.mark.parametrize("t", [3, 50, 100])
def test_matmul_scales_strides_and_extremes(t):
    check_matmul(t, 70, 200, F32, scales="any")
    x, w = q8rand(t, 160, 3), q8rand(66, 160, 4)
    a = check_matmul(t, 66, 160, F32, x=x, w=w)[2].clone()
    for off, extra in ((0, 16), (16, 0), (1, 2)):
        xs, wsx = l8.Q8(strided(x.q, off, extra), x.scale), l8.Q8(strided(w.q, off, extra), w.scale)
        assert torch.equal(check_matmul(t, 66, 160, F32, x=xs, w=wsx)[2], a)
    k = 131071  # the longest sum, every product 128 * 128
    big = l8.Q8(torch.full((t, k), -128, dtype=torch.int8, device="cuda"), torch.ones(t, device="cuda"))
    y = l8.matmul(big, l8.Q8(big.q[:2], big.scale[:2]), dtype=F32)
    assert bool((y == float(np.float32(131071 * 16384))).all())


def test_matmul_empty_and_non_finite_rows():
    x, w = q8rand(80, 64, 1), q8rand(50, 64, 2)
    e = l8.Q8(x.q[:, :0].contiguous(), x.scale)
    assert not l8.matmul(e, l8.Q8(w.q[:, :0].contiguous(), w.scale)).any()
    assert not l8.matmul(l8.Q8(e.q[:3], e.scale[:3]), l8.Q8(w.q[:, :0].contiguous(), w.scale)).any()
    assert l8.matmul(l8.Q8(x.q[:0], x.scale[:0]), w).shape == (0, 50)
    clean = l8.matmul(x, w)
    xs, wsc = x.scale.clone(), w.scale.clone()
    xs[7] = float("nan")
    wsc[3] = float("nan")
    y = l8.matmul(l8.Q8(x.q, xs), l8.Q8(w.q, wsc))
    bad = y.isnan()
    want = torch.zeros_like(bad)
    want[7] = True
    want[:, 3] = True
    assert torch.equal(bad, want) and torch.equal(y[~bad], clean[~bad])
    x3 = l8.Q8(x.q.reshape(4, 20, 64), x.scale.reshape(4, 20))
    assert torch.equal(l8.matmul(x3, w), clean.reshape(4, 20, 50))


def check_grad(kind, t, n, k, dtype, dy=None, other=None, scales="pow2", accumulate=False):
    dy = dy if dy is not None else rand((t, n), 5, BF, 1e-2)
    rows = n if kind == GRAD_INPUT else t
    other = other if other is not None else q8rand(rows, k, 6, scales)
    orow = t if kind == GRAD_INPUT else n
    big, out = guarded(orow, k, dtype)
    base = torch.zeros(orow, k, dtype=torch.float64, device="cuda")
    if accumulate:
        out.copy_(rand((orow, k), 9, dtype))
        base = out.double()
    ref0 = (dy.double() if kind == GRAD_INPUT else dy.double().t().contiguous())
    product(kind, dy, None, other.q, other.scale, out, accumulate)
    ref = ref0 @ dense(other)
    mag = ref0.abs() @ dense(other).abs()
    kd = n if kind == GRAD_INPUT else t
    # products are exact for power-of-two scales; every fp32 addition may be
    # off by a whole step (2^-23) of a partial sum
    bound = (kd + 40) * 2 * U * mag + 1e-30
    if scales != "pow2":
        bound = bound + HALF[BF] * mag
    bound = bound + (HALF[BF] * 1.001 if dtype == BF else U) * (ref + base).abs()
    within(out, ref + base, bound, "gradient")
    check_guard(big, k)
    return out


GRADS = [(1, 1, 1), (1, 300, 7), (7, 33, 64), (32, 32, 128), (33, 31, 129), (64, 128, 8), (100, 136, 256),
         (129, 257, 100), (77, 512, 1023), (500, 96, 130), (2048, 130, 264), (3000, 40, 65), (48, 3500, 4000),
         (35, 4001, 3585), (3900, 96, 3600), (4001, 33, 3585)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t, n, k", GRADS)
@pytest.mark.parametrize("kind", [GRAD_INPUT, GRAD_WEIGHT])
def test_gradient_products(kind, t, n, k, dtype):
    check_grad(kind, t, n, k, dtype)


@pytest.mark.parametrize("kind", [GRAD_INPUT, GRAD_WEIGHT])
def test_gradient_products_scales_and_strides(kind):
    t, n, k = 90, 72, 80
    check_grad(kind, t, n, k, F32, scales="any")
    dy, o = rand((t, n), 5, BF), q8rand(n if kind == GRAD_INPUT else t, k, 6)
    a = check_grad(kind, t, n, k, F32, dy=dy, other=o).clone()
    for off, extra in ((0, 8), (8, 0), (1, 2)):
        b = check_grad(kind, t, n, k, F32, dy=strided(dy, off, extra),
                       other=l8.Q8(strided(o.q, off, extra), o.scale))
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t, n, k", [(50, 70, 33), (1500, 130, 264), (0, 20, 30), (40, 3500, 4000)])
def test_weight_gradient_accumulates(t, n, k, dtype):
    check_grad(GRAD_WEIGHT, t, n, k, dtype, accumulate=True)


def test_gradient_products_empty():
    assert not l8.grad_weight(rand((0, 20), 1, BF), q8rand(0, 30, 1)).any()
    assert not l8.grad_input(rand((5, 0), 1, BF), q8rand(0, 30, 1)).any()
    assert l8.grad_weight(rand((5, 0), 1, BF), q8rand(5, 30, 1)).shape == (0, 30)
    assert l8.grad_input(rand((5, 6), 1, BF), q8rand(6, 0, 1)).shape == (5, 0)


@pytest.mark.parametrize("t, n, k", [(40, 48, 64), (45, 51, 65), (1000, 130, 40)])
def test_gradient_products_keep_non_finite_values_in_their_place(t, n, k):
    dy, x, w = rand((t, n), 5, BF), q8rand(t, k, 6), q8rand(n, k, 7)
    x.q[x.q == 0] = 1
    w.q[w.q == 0] = 1
    ci, cw = l8.grad_input(dy, w, F32), l8.grad_weight(dy, x, F32)
    dy[t - 1, n - 1] = float("inf")  # next to every ragged edge
    di, dw = l8.grad_input(dy, w, F32), l8.grad_weight(dy, x, F32)
    assert bool(di[t - 1].isinf().all()) and bool(dw[n - 1].isinf().all())
    assert torch.equal(di[:t - 1], ci[:t - 1]) and torch.equal(dw[:n - 1], cw[:n - 1])


def test_gradient_products_against_differences():
    t, n, k = 9, 40, 33
    x, w, c = q8rand(t, k, 1), q8rand(n, k, 2), rand((t, n), 3, BF)
    di, dw = l8.grad_input(c, w, F32), l8.grad_weight(c, x, F32)
    xd, wd, cd = dense(x), dense(w), c.double()

    def loss(xv, wv):
        return float((xv @ wv.t().contiguous() * cd).sum())

    # the loss is linear in each operand: a difference of any width is exact but
    # for the 64-bit sums
    for i, j, m in ((0, 0, 0), (4, 17, 20), (8, 39, 32)):
        d = torch.zeros_like(xd)
        d[i, m] = 1.0
        num = (loss(xd + d, wd) - loss(xd - d, wd)) / 2
        assert abs(num - float(di[i, m])) <= (n + 40) * 2 * U * float(cd[i].abs() @ wd[:, m].abs()) + 1e-9
        d = torch.zeros_like(wd)
        d[j, m] = 1.0
        num = (loss(xd, wd + d) - loss(xd, wd - d)) / 2
        assert abs(num - float(dw[j, m])) <= (t + 40) * 2 * U * float(cd[:, j].abs() @ xd[:, m].abs()) + 1e-9


def run_all(x, r, w, wq, dout):
    y, h, rstd = l8.rmsnorm(x, w, residual=r, q8=True)
    out = l8.matmul(y, wq)
    dn = l8.grad_input(dout, wq)
    dW = l8.grad_weight(dout, y)
    kept = l8.quantize(h)
    dx, dweight = l8.rmsnorm_backward(dn, kept, rstd, w, dh=r)
    return [y.q, y.scale, h, rstd, out, dn, dW, dx, dweight, l8.dequantize(kept)]


def layer(t, k, n):
    return (rand((t, k), 1, BF), rand((t, k), 2, BF), 1 + 0.1 * rand((k,), 3), l8.quantize(rand((n, k), 4)),
            rand((t, n), 5, BF, 1e-2))


@pytest.mark.parametrize("t, k, n", [(5, 256, 100), (700, 264, 130), (333, 515, 77)])
def test_other_streams_and_repeats(t, k, n):
    a = layer(t, k, n)
    want = run_all(*a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [run_all(*a) for _ in range(3)]
    side.synchronize()
    for g in got:
        for u, v in zip(g, want):
            assert torch.equal(u, v)


@pytest.mark.parametrize("t, k, n", [(5, 256, 100), (1500, 264, 130), (333, 515, 77)])
def test_graph_replays(t, k, n):
    a = layer(t, k, n)
    want = run_all(*a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run_all(*a)
    for i in range(4):
        a[0].copy_(rand((t, k), 10 + i, BF))
        a[4].copy_(rand((t, n), 20 + i, BF, 1e-2))
        g.replay()
        torch.cuda.synchronize()
        want = run_all(*a)
        for u, v in zip(out, want):
            assert torch.equal(u, v)


def test_offsets_past_32_bits():
    # row distances that put the last rows past 2^31 and 2^32 bytes
    rows, cols, ld = 3, 40, (1 << 31) - 56
    big = torch.zeros(rows * ld, dtype=torch.int8, device="cuda")
    q = big.as_strided((rows, cols), (ld, 1))
    src = q8rand(rows, cols, 3)
    q.copy_(src.q)
    x = l8.Q8(q, src.scale)
    assert torch.equal(l8.dequantize(x, F32), l8.dequantize(src, F32))
    w = q8rand(20, cols, 4)
    assert torch.equal(l8.matmul(x, w), l8.matmul(src, w))
    assert torch.equal(l8.matmul(w, x), l8.matmul(w, src))
    dy = rand((rows, 24), 5, BF)
    assert torch.equal(l8.grad_weight(dy, x), l8.grad_weight(dy, src))
    assert torch.equal(l8.grad_input(rand((30, rows), 6, BF), x), l8.grad_input(rand((30, rows), 6, BF), src))
    del big, q, x
    many = 1 << 17  # 2^17 rows of 2^14 + 8 columns: element offsets past 2^31
    v = torch.zeros(many, 16392, dtype=BF, device="cuda")
    v[-1] = rand((16392,), 7, BF)
    got = l8.quantize(v)
    want = l8.quantize(v[-1:])
    assert torch.equal(got.q[-1:], want.q) and torch.equal(got.scale[-1:], want.scale)
    assert not got.q[-2].any()
