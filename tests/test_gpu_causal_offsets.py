"""The causal operators on tensors of more than 2^31 elements, on the GPU: the last rows equal the same rows alone."""
import pytest
import torch

from video_diffusion_linear_b200 import api

pytestmark = pytest.mark.gpu


def _needs(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB of device memory")


def _rms(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def test_gradients_past_int32():
    _needs(60)
    B, T, H, d = 9, 16384, 120, 128           # 2.26e9 elements per tensor
    g = torch.Generator("cuda").manual_seed(0)
    mk = lambda: torch.randn(1, T, H, d, generator=g, device="cuda").bfloat16()
    one = {n: mk() for n in ("q", "k", "v", "dout")}
    x = {n: torch.zeros(B, T, H, d, dtype=torch.bfloat16, device="cuda") for n in one}
    for n in x:
        x[n][-1:] = one[n]
    lam = torch.linspace(0.5, 1.0, H, device="cuda")
    lens = torch.tensor([1] * (B - 1) + [T], dtype=torch.int32, device="cuda")
    got = api.decay_backward(x["q"], x["k"], x["v"], lam, dout=x["dout"], lengths=lens)
    want = api.decay_backward(one["q"], one["k"], one["v"], lam, dout=one["dout"])
    for n in ("dq", "dk", "dv"):
        # splits into segments differ, so two bf16 roundings each: 2^-7 of the size
        assert _rms(got[n][-1:], want[n]) < 2.0 ** -7, n
        assert not got[n][:-1].any()          # one zero token each


def test_fp32_sequence_past_int32():
    _needs(60)
    B, T, H, d = 5, 4096, 1100, 128           # 2.88e9 elements per tensor
    g = torch.Generator("cuda").manual_seed(1)
    one = torch.randn(1, T, H, d, generator=g, device="cuda")
    x = torch.zeros(B, T, H, d, device="cuda")
    x[-1:] = one
    lam = torch.linspace(0.5, 0.99, H, device="cuda")
    lens = torch.tensor([0] * (B - 1) + [T], dtype=torch.int32, device="cuda")
    out, last = api.decay_forward(x, x, x, lam, lengths=lens)
    want, want_last = api.decay_forward(one, one, one, lam)
    assert torch.equal(out[-1:], want) and torch.equal(last[-1:], want_last)
    assert not out[:-1].any() and not last[:-1].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_states_past_int32(dtype):
    _needs(20)
    n, H, d = 5600, 24, 128                   # 2.2e9 elements of state
    g = torch.Generator("cuda").manual_seed(2)
    S = torch.zeros(n, H, d, d, device="cuda")
    S[-3:] = torch.randn(3, H, d, d, generator=g, device="cuda")
    small = S[-3:].clone()
    q, k, v = (torch.randn(3, H, d, generator=g, device="cuda").to(dtype) for _ in range(3))
    lam = torch.linspace(0.5, 1.0, H, device="cuda")
    out = api.decay_step(q, k, v, lam, S, slots=torch.tensor([n - 1, n - 3, n - 2], dtype=torch.int32, device="cuda"))
    want = api.decay_step(q, k, v, lam, small, slots=torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, want) and torch.equal(S[-3:], small) and not S[:-3].any()


@pytest.mark.parametrize("rows,groups,d", [(700001, 24, 128), (1100003, 1, 1999)])
def test_norm_past_int32(rows, groups, d):
    _needs(40)
    g = torch.Generator("cuda").manual_seed(3)
    tail = 5
    x, dy = (torch.ones(rows, groups, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, dy):
        t[-tail:] = torch.randn(tail, groups, d, generator=g, device="cuda").bfloat16()
        t[:tail] = torch.randn(tail, groups, d, generator=g, device="cuda").bfloat16()
    w, b = (torch.randn(groups, d, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = api.layer_norm_forward(x, w, b)
    got = api.layer_norm_backward(x, dy, mean, rstd, w, bias=True)
    keep = torch.cat([torch.arange(tail), torch.arange(rows - tail, rows)]).cuda()
    xs, dys = x[keep].contiguous(), dy[keep].contiguous()
    ys, ms, rs = api.layer_norm_forward(xs, w, b)
    want = api.layer_norm_backward(xs, dys, ms, rs, w, bias=True)
    if d % 8 == 0:
        assert torch.equal(y[keep], ys) and torch.equal(mean[keep], ms) and torch.equal(rstd[keep], rs)
        assert torch.equal(got["dx"][keep], want["dx"])
    else:
        # A row's elements are summed from the 16-byte boundary before it, and row r starts r d mod 8 elements behind
        # one: the same row at rows - tail and at tail is summed in another order.  Two orders' means differ by twice
        # 48 roundings of mean |x|, rstd by twice (32 roundings and the mean's against sigma, here below 48); y and dx,
        # whose fp32 values move by less than 2^-16 of the magnitudes that are added, may round to the next bf16.
        u = 2.0 ** -24
        assert bool(((mean[keep] - ms).abs() <= 96 * u * xs.float().abs().mean(-1)).all())
        assert bool(((rstd[keep] - rs).abs() <= 160 * u * rs).all())
        xh = ((xs.float() - ms[..., None]) * rs[..., None]).abs()
        mag = w.abs() * xh + b.abs()
        assert bool(((y[keep].float() - ys.float()).abs() <= 2.0 ** -7 * ys.float().abs() + 2.0 ** -16 * mag).all())
        G = (dys.float() * w).abs()
        mag = rs[..., None] * (G + G.mean(-1, keepdim=True) + xh * (G * xh).mean(-1, keepdim=True))
        dx = want["dx"].float()
        assert bool(((got["dx"][keep].float() - dx).abs() <= 2.0 ** -7 * dx.abs() + 2.0 ** -16 * mag).all())
    assert torch.equal(y[tail:-tail].amax(0), y[tail]) and torch.equal(y[tail:-tail].amin(0), y[tail])   # constant rows
    # the constant rows have x = mean: they add nothing to dweight, and one each to dbias (exact in fp32: powers of two
    # apart, below 2^24)
    err = (got["dweight"] - want["dweight"]).abs().max()
    assert float(err) <= 20 * 2.0 ** -24 * float(want["dweight"].abs().max()) * tail * 2
    assert float((got["dbias"] - want["dbias"] - (rows - 2 * tail)).abs().max()) <= 64 * 2.0 ** -24 * rows
