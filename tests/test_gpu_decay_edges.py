"""Decayed attention at the edges of its arguments, on the GPU: decays outside their range, optional outputs, and
sequences that end at every place of a chunk."""
import pytest
import torch

from causal import cuda, inputs, live, scan_bound, within
from oracle import causal_oracle as C
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


@pytest.mark.parametrize("first", [0, 128, 896])
def test_sequences_that_end_at_every_place_of_a_chunk(first):
    """bf16: a sequence that ends inside a chunk before T leaves by another way than whole chunks."""
    B, T, H, d = 128, first + 131, 1, 128
    g = torch.Generator("cuda").manual_seed(first)
    x = {n: torch.randn(B, T, H, d, generator=g, device="cuda").bfloat16() for n in ("q", "k", "v", "dout")}
    x["q"], x["k"], x["v"], x["dout"] = (t[:1].expand(B, T, H, d).contiguous() for t in x.values())
    lam = torch.tensor([0.97], device="cuda")
    counts = [first + 1 + b for b in range(B)]
    lens = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = torch.full_like(x["q"], -77.0)
    api.decay_forward(x["q"], x["k"], x["v"], lam, lengths=lens, out=out)
    grads = {n: torch.full_like(x["q"], -77.0) for n in ("dq", "dk", "dv")}
    api.decay_backward(x["q"], x["k"], x["v"], lam, dout=x["dout"], lengths=lens, grads=grads)
    m = live(counts, T)
    ref, _ = C.decay_forward(x["q"][:1], x["k"][:1], x["v"][:1], lam)
    bound = scan_bound("bf16", ref, x["q"][:1], x["k"][:1], x["v"][:1], lam, None, [T], d ** -0.5)
    got = out.double().cpu().numpy()
    assert bool((got[~m] == -77.0).all())
    for b, n in enumerate(counts):
        within(got[b, :n], ref[0, :n], bound[0, :n], ("out", b))
    for b in (0, 1, 14, 15, 16, 62, 63, 64, 100, 126, 127):
        n = counts[b]
        one = [x[a][:1, :n] for a in ("q", "k", "v", "dout")]
        rg = C.decay_backward(one[0], one[1], one[2], lam, one[3])
        for what, (u, y, z), rev in (("dq", (3, 2, 1), False), ("dk", (2, 3, 0), True), ("dv", (1, 0, 3), True)):
            bd = scan_bound("bf16", rg[what], one[u], one[y], one[z], lam, None, [n], d ** -0.5, rev)
            have = grads[what].double().cpu().numpy()[b]
            assert bool((have[n:] == -77.0).all())
            within(have[:n], rg[what][0], bd[0], (what, b))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,d,T", [("bf16", 128, 300), ("bf16", 128, 1700), ("f32", 128, 300), ("f32", 16, 300)])
def test_what_an_infinite_token_reaches(dtype, d, T, value):
    """The results that an infinity or NaN in one token of an operand leaves alone keep their bits.  fp32: all before it
    (from the end: behind it).  bf16: the same, but for the operand whose terms the output sums (v; in the gradients k,
    q and dout): there the whole chunk of 128 tokens is reached."""
    t, chunk = 200, (128, 256)
    x = cuda(inputs(33, dtype, 2, T, 2, d))
    x["decay"] = torch.tensor([0.97, 0.9], device="cuda")

    def call(y):
        args = (y["q"], y["k"], y["v"], y["decay"], y["state"])
        out, last = api.decay_forward(*args)
        g = api.decay_backward(*args, dout=y["dout"], dfinal=y["dfinal"])
        return {"out": out, "state": last, **g}

    clean = call(x)
    # result: the operand read at the output's token, the two that are summed, the second of them into the output
    roles = {"out": ("q", "k", "v", False), "dq": ("dout", "v", "k", False), "dk": ("v", "dout", "q", True),
             "dv": ("k", "q", "dout", True)}
    for name in ("q", "k", "v", "dout"):
        y = {**x, name: x[name].clone()}
        y[name][0, t, 0, 3] = value
        got = call(y)
        for result, (own, key, term, reverse) in roles.items():
            reached = torch.zeros(T, dtype=torch.bool)
            if name == own:
                reached[t] = True
            if name in (key, term):
                reached[:t + 1] |= reverse
                reached[t:] |= not reverse
                if name == term and dtype == "bf16":
                    reached[chunk[0]:chunk[1]] = True
            reached = reached.cuda()
            assert torch.equal(got[result][0, ~reached, 0], clean[result][0, ~reached, 0]), (name, result)
            assert not bool(torch.isfinite(got[result][0, t, 0]).all()) or not bool(reached[t]), (name, result)
            assert torch.equal(got[result][1], clean[result][1]) and torch.equal(got[result][0, :, 1], clean[result][0, :, 1])
        for result, operands in (("state", "k v"), ("dstate", "q dout")):
            assert torch.equal(got[result][1], clean[result][1]) and torch.equal(got[result][0, 1], clean[result][0, 1])
            if name not in operands.split():
                assert torch.equal(got[result], clean[result]), (name, result)
