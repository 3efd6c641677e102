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


@pytest.mark.parametrize("d", [2, 6, 130, 514])
def test_gradient_of_a_far_constant_row(d):
    """fp32, x = 2^112 throughout: (x - mean) rstd is zero, and dx is rstd (g - mean g).  What lies outside the row in
    its last vector must not enter, though 2^112 rstd there passes the fp32 range."""
    x = torch.full((5, d), 2.0 ** 112, device="cuda")
    g = torch.Generator("cuda").manual_seed(d)
    dy = torch.randn(5, d, generator=g, device="cuda")
    mean, rstd = torch.full((5,), 2.0 ** 112, device="cuda"), torch.full((5,), 2.0 ** 17, device="cuda")
    w = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    got = api.layer_norm_backward(x, dy, mean, rstd, w, bias=True)
    G = dy.double() * w.double()
    ref = 2.0 ** 17 * (G - G.mean(-1, keepdim=True))
    # the mean of g: 42 roundings of its terms' magnitudes; its product, the difference and the factor: 4
    bound = 2.0 ** 17 * 50 * 2.0 ** -24 * (G.abs() + G.abs().mean(-1, keepdim=True))
    assert bool(((got["dx"].double() - ref).abs() <= bound).all())
    assert not got["dweight"].any()
