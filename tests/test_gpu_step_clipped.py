"""MuonMI355X.step(max_norm=) as a call: what it refuses leaves the gradients, the
parameters and the step count as they were."""
import pytest
import torch

from matrix_aware_optimizer_muon_amd import MuonError
from matrix_aware_optimizer_muon_amd.optim import MuonMI355X

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("lr, wd, max_norm, out, error", [
    (NAN, 0.0, 1.0, None, MuonError), (0.02, INF, 1.0, None, MuonError), (1e39, 0.0, 1.0, None, MuonError),
    ("x", 0.0, 1.0, None, TypeError), (0.02, 0.0, -1.0, None, ValueError), (0.02, 0.0, NAN, None, ValueError),
    (0.02, 0.0, 1.0, [3, 4], AttributeError)])
@pytest.mark.parametrize("refresh", [True, False])
def test_a_refused_step_writes_nothing(lr, wd, max_norm, out, error, refresh):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    params = [torch.randn(128, 256, generator=g, device="cuda") for _ in range(2)]
    grads = [torch.randn(128, 256, generator=g, device="cuda") for _ in range(2)]
    before = [t.clone() for t in params + grads]
    opt = MuonMI355X(params)
    with pytest.raises(error):
        opt.step(grads, lr, wd, refresh=refresh, out=out, max_norm=max_norm)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(params + grads, before)) and opt.t == 0
    norm = opt.step(grads, 0.02, 0.0, refresh=refresh, max_norm=1.0)
    # 64-bit sums, rounded to fp32 once
    want = sum(float(t.double().square().sum()) for t in before[2:]) ** 0.5
    assert abs(float(norm) - want) <= want * 1.001 * 2.0 ** -24 and opt.t == 1
