"""Calls of the causal operators that a program makes around the plain ones, on the GPU: several at once, captured in
fp32, a state carried in place over a split axis, streams that are named, and tensors of one axis."""
import pytest
import torch

from causal import cuda, inputs
from video_diffusion_linear_b200 import api

pytestmark = pytest.mark.gpu

PATHS = [("bf16", 128, 1700), ("f32", 128, 420), ("f32", 16, 420)]


@pytest.mark.parametrize("dtype,d,T", PATHS)
@pytest.mark.parametrize("ragged", [False, True])
def test_state_in_place_over_several_segments(dtype, d, T, ragged):
    x = cuda(inputs(41, dtype, 3, T, 2, d))
    lens = torch.tensor([T, 0, T // 3], dtype=torch.int32, device="cuda") if ragged else None
    args = (x["q"], x["k"], x["v"], x["decay"])
    assert api.decay_workspace_size(api._decay_shape(x["q"])) > 256        # split
    want, want_S = api.decay_forward(*args, x["state"], lengths=lens)
    S = x["state"].clone()
    got, got_S = api.decay_forward(*args, S, lengths=lens, state_out=S)
    assert got_S is S and torch.equal(got, want) and torch.equal(S, want_S)


@pytest.mark.parametrize("d,T", [(128, 420), (16, 420), (128, 20), (16, 20)])
def test_fp32_calls_at_once_and_captured(d, T):
    a, b = (cuda(inputs(s, "f32", 2, T, 3, d)) for s in (42, 43))
    def call(x, **kw):
        args = (x["q"], x["k"], x["v"], x["decay"], x["state"])
        o, S = api.decay_forward(*args, **kw)
        g = api.decay_backward(*args, dout=x["dout"], dfinal=x["dfinal"], **kw)
        return [o, S, *g.values()]
    want = [call(a), call(b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(x, stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(g, w))
    buf = {n: t.clone() for n, t in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = call(buf)
    for x, w in ((b, want[1]), (a, want[0])):
        for n in buf:
            buf[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(res, w))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_calls_at_once_on_named_streams(dtype):
    g = torch.Generator("cuda").manual_seed(44)
    data = [(torch.randn(9000, d, generator=g, device="cuda").to(dtype), torch.randn(9000, d, generator=g, device="cuda").to(dtype),
             torch.randn(d, generator=g, device="cuda")) for d in (128, 777, 777)]

    def call(x, dy, w, **kw):
        y, m, r = api.layer_norm_forward(x, w, **kw)
        return [y, m, r, *api.layer_norm_backward(x, dy, m, r, w, bias=True, **kw).values()]

    want = [call(*t) for t in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(*t, stream=s) for t, s in zip(data, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_a_single_axis(dtype):
    g = torch.Generator("cuda").manual_seed(45)
    x, dy = (torch.randn(100, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.randn(100, generator=g, device="cuda")
    y, m, r = api.layer_norm_forward(x, w)
    got = api.layer_norm_backward(x, dy, m, r, w, bias=True)
    y2, m2, r2 = api.layer_norm_forward(x[None], w)
    want = api.layer_norm_backward(x[None], dy[None], m2, r2, w, bias=True)
    assert m.shape == () and torch.equal(y, y2[0]) and torch.equal(m, m2[0]) and torch.equal(r, r2[0])
    assert torch.equal(got["dx"], want["dx"][0]) and torch.equal(got["dweight"], want["dweight"])
    assert torch.equal(got["dbias"], dy.float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured_steps_of_a_pool_with_rows_of_one_sequence(dtype):
    """A decoding loop in a graph: slots change between replays, several rows may step one sequence."""
    B, H, d, n = 6, 4, 128, 5
    g = torch.Generator("cuda").manual_seed(46)
    q, k, v = (torch.randn(B, H, d, generator=g, device="cuda").to(dtype) for _ in range(3))
    S = torch.randn(n, H, d, d, generator=g, device="cuda")
    lam = torch.linspace(0.5, 1.0, H, device="cuda")
    slots = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, T = torch.zeros_like(q), S.clone()
    api.decay_step(q, k, v, lam, T.clone(), slots=slots, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decay_step(q, k, v, lam, T, slots=slots, out=out)
    T.copy_(S)
    for rows in ([0, 1, 2, 3, 4, -1], [2, 2, 2, 5, 2, 0], [4, 3, 4, 3, 9, 4]):
        slots.copy_(torch.tensor(rows, dtype=torch.int32))
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        for b, s in enumerate(rows):                     # the same, row after row
            if not 0 <= s < n:
                assert bool((out[b] == -7.0).all())
                continue
            one = S[s:s + 1].clone()
            want = api.decay_step(q[b:b + 1], k[b:b + 1], v[b:b + 1], lam, one)
            S[s] = one[0]
            assert torch.equal(out[b:b + 1], want)
        assert torch.equal(T, S)
