"""The binding's own checks of the causal operators, beyond those of each tensor (CPU)."""
import types

import pytest
import torch

from video_diffusion_linear_b200 import _lib, api


@pytest.mark.parametrize("shape,par", [((2 ** 32 + 5,), (5,)), ((3, 2 ** 31), None), ((2 ** 32 + 3, 1), (2 ** 32 + 3, 1)), ((2 ** 32 + 3, 1), None)])
def test_layer_norm_refuses_sizes_that_wrap_in_an_int(shape, par):
    """A row of 2^32 + 5 elements is 8 GB of bf16; the library takes the width and the groups as 32-bit integers."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    w = None if par is None else torch.empty(par, device="meta")
    with pytest.raises(_lib.VdnError) as e:
        api._norm_shape(x, w)
    assert e.value.status == _lib.VDN_ERR_UNSUPPORTED


def test_layer_norm_sizes_in_range_pass():
    x = torch.empty(2 ** 20, 3, 2 ** 31 - 1, dtype=torch.bfloat16, device="meta")
    assert api._norm_shape(x, None)[:3] == (3 * 2 ** 20, 1, 2 ** 31 - 1)
    assert api._norm_shape(x, torch.empty(3, 2 ** 31 - 1, device="meta"))[:3] == (3 * 2 ** 20, 3, 2 ** 31 - 1)
    assert api._norm_shape(torch.empty(5, 0), None)[:3] == (0, 1, 0)


def test_a_stream_of_another_device_is_refused():
    """The default streams of all devices have the handle 0: such a call would run on the tensors' device unordered with
    the stream that was named."""
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        api._Call(torch.device("cuda", 0), stream)
