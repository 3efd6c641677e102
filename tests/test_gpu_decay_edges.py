"""Decayed attention at the edges of its arguments, on the GPU: decays outside their range, optional outputs."""
import pytest
import torch

from causal import cuda, inputs
from video_diffusion_linear_b200 import api

pytestmark = pytest.mark.gpu

# dtype, d, T: one pass and several segments of both paths
PATHS = [("bf16", 128, 200), ("bf16", 128, 1700), ("f32", 128, 20), ("f32", 128, 420), ("f32", 16, 20), ("f32", 16, 420)]


@pytest.mark.parametrize("bad", [float("nan"), -0.5])
@pytest.mark.parametrize("dtype,d,T", PATHS)
def test_a_decay_that_is_no_decay_shows_in_every_result(dtype, d, T, bad):
    """A NaN or negative decay makes every result of its head NaN, in all three forms, and no other head's."""
    x = cuda(inputs(31, dtype, 2, T, 2, d))
    x["decay"] = torch.tensor([0.9, 0.8], device="cuda")
    broken = torch.tensor([bad, 0.8], device="cuda")
    lens = torch.tensor([T, 0], dtype=torch.int32, device="cuda")

    def call(decay):
        args = (x["q"], x["k"], x["v"], decay, x["state"])
        out, last = api.decay_forward(*args, lengths=lens)
        g = api.decay_backward(*args, dout=x["dout"], dfinal=x["dfinal"], lengths=lens)
        S = x["state"].clone()
        tok = api.decay_step(*(x[n][:, 0].contiguous() for n in "qkv"), decay, S)
        return dict(tokens=[out, g["dq"], g["dk"], g["dv"]], states=[last, g["dstate"]], step=[tok, S])

    want, got = call(x["decay"]), call(broken)
    for a, b in zip(want["tokens"], got["tokens"]):
        assert bool(torch.isnan(b[0, :, 0]).all()) and torch.equal(a[0, :, 1], b[0, :, 1])
    for a, b in zip(want["states"], got["states"]):
        assert bool(torch.isnan(b[0, 0]).all()) and torch.equal(a[0, 1], b[0, 1])
        assert torch.equal(a[1], b[1])                   # an empty sequence passes its state through
    for a, b in zip(want["step"], got["step"]):
        assert bool(torch.isnan(b[:, 0]).all()) and torch.equal(a[:, 1], b[:, 1])


@pytest.mark.parametrize("dtype,d,T", PATHS)
def test_optional_outputs_change_no_other(dtype, d, T):
    x = cuda(inputs(32, dtype, 2, T, 2, d))
    x["decay"] = torch.tensor([0.999, 0.9], device="cuda")
    args = (x["q"], x["k"], x["v"], x["decay"], x["state"])
    a, _ = api.decay_forward(*args)
    b, none = api.decay_forward(*args, want_state=False)
    assert none is None and torch.equal(a, b)
    full = api.decay_backward(*args, dout=x["dout"], dfinal=x["dfinal"])
    assert full["dstate"] is not None
    grads = {n: torch.empty_like(x["q"]) for n in ("dq", "dk", "dv")}
    api.decay_backward(*args, dout=x["dout"], dfinal=x["dfinal"], grads=grads)
    for n in grads:
        assert torch.equal(full[n], grads[n]), n
