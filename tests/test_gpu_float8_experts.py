"""Products grouped by expert on the GPU against one plain product per expert,
on small whole numbers (tests/test_gpu_float8.py), so results have to be equal."""
import pytest
import torch

from float8_common import E8M0, exact8, exact_grad, values
from matrix_aware_optimizer_muon_amd import float8 as f8

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def ends_of(sizes):
    return torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)


def plain(sizes, t, x, w, dy):
    """(y, dx, dw) in 64 bits; rows behind the last expert's are zero."""
    E, n, k = w.shape
    y, dx = torch.zeros(t, n, device="cuda").double(), torch.zeros(t, k, device="cuda").double()
    dw = torch.zeros(E, n, k, device="cuda").double()
    at = 0
    for e, s in enumerate(sizes):
        r = slice(at, at + s)
        y[r], dx[r] = x[r] @ w[e].t(), dy[r] @ w[e]
        dw[e] = dy[r].t().contiguous() @ x[r]
        at += s
    return y, dx, dw


# rows per expert; rows behind them; widths
CASES = [([1], 0, 1, 1), ([0, 1], 0, 16, 128), ([3, 0, 2], 4, 40, 100), ([0, 0, 0], 5, 33, 70), ([16, 1, 15, 0, 17], 0, 130, 257),
         ([50, 33, 100], 20, 64, 128), ([200, 0, 1, 127, 129, 128], 7, 129, 300), ([0, 300, 0], 0, 256, 512),
         ([1] * 70, 3, 48, 64), ([5, 0] * 65 + [40], 1, 20, 150), ([2000, 3], 100, 70, 90), ([640, 600, 700, 513], 90, 300, 260),
         ([0] * 1023 + [9], 0, 24, 40)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes, idle, n, k", CASES)
def test_experts_exact(sizes, idle, n, k, dtype):
    t, E = sum(sizes) + idle, len(sizes)
    x, w, dy = exact8((t, k), t, False), exact8((E, n, k), n, True), exact_grad((t, n), k)
    y, dx, dw = plain(sizes, t, values(x, False), values(w, True), dy.double())
    ends = ends_of(sizes)
    assert torch.equal(f8.matmul(x, w, ends=ends, dtype=dtype), y.to(dtype))
    assert torch.equal(f8.grad_input(dy, w, ends=ends, dtype=dtype), dx.to(dtype))
    assert torch.equal(f8.grad_weight(dy, x, ends=ends, dtype=dtype), dw.to(dtype))
    out = torch.full((E, n, k), 4.0, device="cuda", dtype=dtype)
    f8.grad_weight(dy, x, ends=ends, out=out, accumulate=True)
    assert torch.equal(out, (dw + 4).to(dtype))


def test_one_expert_is_the_dense_product():
    x, w, dy = exact8((300, 200), 1, False), exact8((1, 150, 200), 2, True), exact_grad((300, 150), 3)
    one, ends = f8.F8(w.q[0], w.scale[0]), ends_of([300])
    assert torch.equal(f8.matmul(x, w, ends=ends), f8.matmul(x, one))
    assert torch.equal(f8.grad_input(dy, w, ends=ends), f8.grad_input(dy, one))
    assert torch.equal(f8.grad_weight(dy, x, ends=ends)[0], f8.grad_weight(dy, x))


@pytest.mark.parametrize("t", [20, 400])
def test_rows_of_no_expert_are_not_read(t):
    n, k, E = 100, 200, 3
    sizes = [t // 4, 0, t // 4]
    used = sum(sizes)
    x, w, dy = exact8((t, k), 1, False), exact8((E, n, k), 2, True), exact_grad((t, n), 3)
    want = [f8.matmul(x, w, ends=ends_of(sizes)), f8.grad_input(dy, w, ends=ends_of(sizes)),
            f8.grad_weight(dy, x, ends=ends_of(sizes))]
    x.q.view(torch.uint8)[used:] = 0x7F
    x.scale.view(torch.uint8)[used:] = 255
    dy[used:] = float("nan")
    # the weights of the expert without rows are not read either
    w.q.view(torch.uint8)[1] = 0x7F
    w.scale.view(torch.uint8)[1] = 255
    got = [f8.matmul(x, w, ends=ends_of(sizes)), f8.grad_input(dy, w, ends=ends_of(sizes)),
           f8.grad_weight(dy, x, ends=ends_of(sizes))]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_ends_out_of_range_or_falling():
    """Such ends name no rows outside the batch: values outside count as its
    borders, falling ones as no rows."""
    t, n, k = 200, 64, 96
    x, w, dy = exact8((t, k), 1, False), exact8((4, n, k), 2, True), exact_grad((t, n), 3)
    for ends, like in (([-5, 100, 300, 2 ** 31 - 1], [0, 100, 200, 200]), ([100, 100, 150, 500], [100, 100, 150, 200])):
        a, b = (torch.tensor(v, dtype=torch.int64).to(torch.int32).cuda() for v in (ends, like))
        assert torch.equal(f8.matmul(x, w, ends=a), f8.matmul(x, w, ends=b))
        assert torch.equal(f8.grad_input(dy, w, ends=a), f8.grad_input(dy, w, ends=b))
        assert torch.equal(f8.grad_weight(dy, x, ends=a), f8.grad_weight(dy, x, ends=b))
    fall = torch.tensor([150, 20, 60, 200], dtype=torch.int32, device="cuda")
    dw = f8.grad_weight(dy, x, ends=fall)
    assert not dw[1].any()
    assert torch.equal(dw[2], f8.grad_weight(dy[20:60], f8.F8(x.q[20:60], x.scale[20:60])))
    f8.matmul(x, w, ends=fall)
    f8.grad_input(dy, w, ends=fall)
    torch.cuda.synchronize()


@pytest.mark.parametrize("t", [24, 500])
def test_captured_and_replayed_with_other_ends(t):
    n, k, E = 130, 144, 5
    x, w, dy = exact8((t, k), 1, False), exact8((E, n, k), 2, True), exact_grad((t, n), 3)
    ends = ends_of([t // E] * E)
    run = lambda: (f8.matmul(x, w, ends=ends), f8.grad_input(dy, w, ends=ends), f8.grad_weight(dy, x, ends=ends),  # noqa: E731
                   f8.matmul(x, w, ends=ends, dtype=F32))
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for sizes in ([t // E] * E, [0, t, 0, 0, 0], [1, 0, 2, 0, 3], [0] * E, [t // 3, 1, t // 3, 0, 2]):
        ends.copy_(ends_of(sizes))
        for o in out:
            o.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run()):
            assert torch.equal(a, b)


def test_a_training_step_of_experts():
    """Routing, the experts' forward and backward, clipping and the optimizer's
    step together, as they are used."""
    from matrix_aware_optimizer_muon_amd.clip import clip_grad_norm
    from matrix_aware_optimizer_muon_amd.optim import MuonMI355X
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tokens, hidden, ffn, E = 96, 128, 192, 4
    W = torch.randn(E, ffn, hidden, generator=g, device="cuda") * 0.1
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(BF)
    expert = torch.randint(0, E - 1, (tokens,), generator=g, device="cuda")  # the last one gets none
    order = expert.argsort(stable=True)
    ends = torch.bincount(expert, minlength=E).cumsum(0).to(torch.int32)
    w8, x8 = f8.quantize_weight(W), f8.quantize(x[order])
    y = f8.matmul(x8, w8, ends=ends)
    dy = (y.float() * 1e-2).to(BF)
    dW, dx = f8.grad_weight(dy, x8, ends=ends), f8.grad_input(dy, w8, ends=ends)
    xv, wv = values(x8, False), values(w8, True)
    at, want = 0, torch.zeros_like(W).double()
    for e, end in enumerate(ends.tolist()):
        want[e] = dy[at:end].double().t().contiguous() @ xv[at:end]
        back, size = dy[at:end].double() @ wv[e], dy[at:end].double().abs() @ wv[e].abs()
        # fp32 sums of exact products, rounded once to bf16
        assert bool(((dx[at:end].double() - back).abs() <= 2.0 ** -8 * back.abs() + ffn * 2.0 ** -23 * size).all())
        at = end
    norm = float(want.norm())
    assert norm > 0.1
    params = [W[e].clone() for e in range(E)]
    opt = MuonMI355X(params)
    grads = list(dW.unbind(0))
    got = clip_grad_norm(grads, 0.1)
    assert abs(float(got) - norm) <= 1e-5 * norm
    assert abs(float(dW.double().norm()) - 0.1) <= 1e-6
    opt.step(grads, 0.02, 0.0)
    other = [W[e].clone() for e in range(E)]
    same = MuonMI355X(other)
    back = same.step(list(f8.grad_weight(dy, x8, ends=ends).unbind(0)), 0.02, 0.0, max_norm=0.1)
    assert float(back) == float(got)
    for a, b in zip(params, other):
        assert torch.equal(a, b)
    assert all(torch.isfinite(p).all() for p in params)
    assert torch.equal(params[E - 1], W[E - 1])  # no gradient, no momentum
