"""The largest norm that gradient clipping takes, no GPU needed: the checks come
ahead of the device's, so CPU tensors reach them."""
import pytest
import torch

from matrix_aware_optimizer_muon_amd.clip import clip_grad_norm


@pytest.mark.parametrize("max_norm, match", [(3.5e38, "fp32's range"), (1e39, "fp32's range"), (1e300, "fp32's range"),
                                             (-1.0, "negative"), (float("nan"), "negative")])
def test_refused(max_norm, match):
    with pytest.raises(ValueError, match=match):
        clip_grad_norm([torch.zeros(3)], max_norm)


@pytest.mark.parametrize("max_norm", [0, 3, 1e-300, 3.4028234663852886e38, float("inf")])
def test_taken(max_norm):
    with pytest.raises(ValueError, match="CUDA"):
        clip_grad_norm([torch.zeros(3)], max_norm)


def test_no_number():
    with pytest.raises(TypeError):
        clip_grad_norm([torch.zeros(3)], "1")
