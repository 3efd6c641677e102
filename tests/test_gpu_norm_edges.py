"""Layer norm on rows where rounding or overflow could show, at widths that are no power of two, on the GPU."""
import pytest
import torch

from causal import DT
from video_diffusion_linear_b200 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [2, 3, 6, 7, 12, 77, 130, 511, 1000, 1999, 5000, 12345])
def test_constant_rows(dtype, d):
    """A row of one value with few digits: its sum is exact in fp32, so the mean is that value, the centred row is zero
    and y is the bias, whatever the width."""
    vals = torch.tensor([3.0, 1000.0, -0.8125, 249.0, 1.0625, 65280.0])
    x = vals[:, None].expand(-1, d).to(DT[dtype]).contiguous().cuda()
    assert torch.equal(x[:, 0].float().cpu(), vals)
    b = torch.linspace(-2, 2, d).bfloat16().float().cuda()
    y, mean, _ = api.layer_norm_forward(x, None, b, eps=1e-6)
    assert torch.equal(mean.cpu(), vals)
    assert torch.equal(y.float(), b.expand(len(vals), d))
