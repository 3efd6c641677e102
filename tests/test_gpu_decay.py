"""Linear attention with a decay per head on the GPU, against the float64 oracle: both paths, lengths from one
token over several segments, padded batches, states in and out, gradients, the single-token step, and the calls
a serving or training program makes around them (in place, other streams, graphs, refusals on the device)."""
import numpy as np
import pytest
import torch

from causal import cuda, inputs, live, scan_bound, state_bound, within
from oracle import causal_oracle as C
from video_diffusion_linear_b200 import api

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().double().cpu().numpy()


def _counts(lengths, B, T):
    return C.token_counts(lengths, B, T)


CASES = [  # dtype, d, B, T, H, state, lengths
    ("bf16", 128, 1, 1, 6, True, None),
    ("bf16", 128, 1, 1, 6, False, None),
    ("bf16", 128, 1, 2, 2, True, None),
    ("bf16", 128, 2, 127, 3, True, None),
    ("bf16", 128, 1, 128, 6, False, None),
    ("bf16", 128, 1, 129, 6, True, None),
    ("bf16", 128, 2, 300, 3, False, None),
    ("bf16", 128, 5, 200, 2, True, [200, 0, 1, 128, 137]),
    ("bf16", 128, 3, 90, 2, False, [-7, 1000, 33]),          # clamped to [0, T]
    ("bf16", 128, 1, 1030, 6, True, None),                    # five segments
    ("bf16", 128, 3, 1601, 2, True, [1601, 700, 0]),          # segments that a sequence does not reach
    ("bf16", 128, 1, 2048, 1, False, [1025]),
    ("f32", 128, 1, 1, 3, True, None),
    ("f32", 128, 2, 8, 3, False, None),
    ("f32", 128, 3, 77, 6, True, [77, 0, 9]),
    ("f32", 128, 1, 333, 6, True, None),                      # several segments
    ("f32", 16, 1, 1, 1, False, None),
    ("f32", 16, 1, 160, 2, False, None),
    ("f32", 16, 3, 403, 6, True, [403, 64, 0]),
    ("f32", 16, 5, 31, 7, True, None),
]
IDS = ["%s-d%d-B%d-T%d-H%d%s%s" % (c[0], c[1], c[2], c[3], c[4], "-state" if c[5] else "", "-ragged" if c[6] else "")
       for c in CASES]


def _behind(x, counts, names):
    """NaN and infinities in the rows behind each sequence, which no result may see."""
    for n in names:
        for b, c in enumerate(counts):
            x[n][b, c:] = float("nan")
            x[n][b, c + 1:] = float("inf")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_matches_oracle(case):
    dtype, d, B, T, H, with_state, lengths = case
    x = inputs(T + H, dtype, B, T, H, d, with_state)
    counts = _counts(lengths, B, T)
    _behind(x, counts, ("q", "k", "v"))
    dev = cuda(x)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = torch.full_like(dev["q"], -77.0)
    ws = torch.empty(api.decay_workspace_size(api._decay_shape(dev["q"])), dtype=torch.uint8, device="cuda")
    got, last = api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], lengths=lens, out=out,
                                  workspace=ws)
    assert got is out and api.workspace_status(ws) == 0
    ref, ref_last = C.decay_forward(x["q"], x["k"], x["v"], x["decay"], x["state"], lengths)
    m = live(counts, T)
    assert bool((got.float().cpu().numpy()[~m] == -77.0).all())     # rows behind a sequence stay
    scale = d ** -0.5
    bound = scan_bound(dtype, ref, x["q"], x["k"], x["v"], x["decay"], x["state"], counts, scale)
    within(_np(got)[m], ref[m], bound[m], "out")
    within(_np(last), ref_last, state_bound(dtype, x["k"], x["v"], x["decay"], x["state"], counts), "state")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_matches_oracle(case):
    dtype, d, B, T, H, with_state, lengths = case
    x = inputs(T + H + 100, dtype, B, T, H, d, with_state)
    counts = _counts(lengths, B, T)
    _behind(x, counts, ("q", "k", "v", "dout"))
    dev = cuda(x)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    grads = {n: torch.full_like(dev["q"], -77.0) for n in ("dq", "dk", "dv")}
    grads["dstate"] = torch.empty(B, H, d, d, device="cuda")
    ws = torch.empty(api.decay_workspace_size(api._decay_shape(dev["q"]), True), dtype=torch.uint8, device="cuda")
    g = api.decay_backward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], dout=dev["dout"],
                           dfinal=dev["dfinal"], lengths=lens, grads=grads, workspace=ws)
    assert api.workspace_status(ws) == 0
    ref = C.decay_backward(x["q"], x["k"], x["v"], x["decay"], x["dout"], x["state"], x["dfinal"], lengths)
    m, s, lam = live(counts, T), d ** -0.5, x["decay"]
    st = None if x["state"] is None else x["state"].transpose(-1, -2)
    end = x["dfinal"]
    end_t = None if end is None else end.transpose(-1, -2)
    bounds = {
        "dq": scan_bound(dtype, ref["dq"], x["dout"], x["v"], x["k"], lam, st, counts, s),
        # the state's gradient enters dk and dv without the scale: its bound is taken with init / scale
        "dk": scan_bound(dtype, ref["dk"], x["v"], x["dout"], x["q"], lam, None if end is None else end_t / s, counts, s, True),
        "dv": scan_bound(dtype, ref["dv"], x["k"], x["q"], x["dout"], lam, None if end is None else end / s, counts, s, True),
    }
    for n, b in bounds.items():
        assert bool((g[n].float().cpu().numpy()[~m] == -77.0).all()), n
        within(_np(g[n])[m], ref[n][m], b[m], n)
    within(_np(g["dstate"]), ref["dstate"], state_bound(dtype, x["q"], x["dout"], lam, end, counts, s, True), "dstate")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("f32", 16)])
def test_gradient_against_differences(dtype, d):
    """Directional differences of the oracle's forward against the kernels' gradients, as the loss would move."""
    B, T, H = 1, 140, 2
    x = inputs(9, dtype, B, T, H, d)
    x["decay"] = torch.tensor([0.97, 0.6])
    dev = cuda(x)
    g = api.decay_backward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], dout=dev["dout"], dfinal=dev["dfinal"])
    args = {n: C._f64(x[n]) for n in ("q", "k", "v", "state")}
    do, dS = C._f64(x["dout"]), C._f64(x["dfinal"])

    def loss(a):
        o, last = C.decay_forward(a["q"], a["k"], a["v"], x["decay"], a["state"])
        return (o * do).sum() + (last * dS).sum()

    rng = np.random.default_rng(0)
    for n in args:
        u = rng.normal(size=args[n].shape)
        e = 1e-4
        fd = (loss({**args, n: args[n] + e * u}) - loss({**args, n: args[n] - e * u})) / (2 * e)
        got = _np(g["d" + n])
        # each gradient entry is good to 2^-7 of the tensor's scale (bf16; twice its rounding) or 2^-14: independent
        # errors meet a normal direction, six standard deviations
        rms = np.sqrt((got ** 2).sum())
        assert abs((got * u).sum() - fd) <= 6 * (2.0 ** -7 if dtype == "bf16" else 2.0 ** -14) * rms, n


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("f32", 16)])
@pytest.mark.parametrize("B,H,slots", [(1, 1, None), (3, 5, None), (4, 24, [5, 0, -1, 2]), (5, 3, [3, 7, 3, 99, 3]),
                                       (130, 2, "many")])
def test_step_matches_oracle(dtype, d, B, H, slots):
    x = inputs(B + H, dtype, B, 1, H, d)
    n = B if slots is None else 8
    if slots == "many":          # every slot several times, rows far apart
        n, slots = 40, [(b * 7) % 43 for b in range(B)]
    S = torch.randn(n, H, d, d, generator=torch.Generator().manual_seed(1))
    q, k, v = (x[a][:, 0].contiguous() for a in "qkv")
    ref, ref_S = C.decay_step(q, k, v, x["decay"], S, slots)
    dev_S = S.cuda()
    out = torch.full_like(q, -77.0).cuda()
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    api.decay_step(q.cuda(), k.cuda(), v.cuda(), x["decay"].cuda(), dev_S, slots=sl, out=out)
    got = _np(out)
    rows = ~np.isnan(ref[:, 0, 0])
    assert bool((got[~rows] == -77.0).all())
    named = sorted({s for s in (range(B) if slots is None else slots) if 0 <= s < n})
    untouched = [s for s in range(n) if s not in named]
    assert torch.equal(dev_S.cpu()[untouched], S[untouched])
    # an entry of the state: a multiply-add per token; the output sums d products of it
    steps = max((list(slots).count(s) for s in named), default=1) if slots is not None else 1
    amp = np.abs(S.numpy()).max() + steps * np.abs(C._f64(v)).max() * np.abs(C._f64(k)).max()
    within(_np(dev_S), ref_S, np.full(ref_S.shape, 3 * steps * 2.0 ** -24 * amp), "state")
    qa = np.abs(C._f64(q)).sum(-1, keepdims=True)
    bound = np.broadcast_to((3 * steps + 12) * 2.0 ** -24 * amp * qa * d ** -0.5, ref.shape)
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(np.nan_to_num(ref))
    within(got[rows], ref[rows], bound[rows], "out")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 16)])
def test_prompt_then_steps_equals_the_longer_prompt(dtype, d):
    """A prompt, its state carried in place through a second piece, then single tokens: the whole sequence."""
    B, T, H = 2, 150, 3
    x = inputs(3, dtype, B, T, H, d, state=False)
    dev = cuda(x)
    ref, ref_last = C.decay_forward(x["q"], x["k"], x["v"], x["decay"])
    piece = lambda a, b: [dev[n][:, a:b].contiguous() for n in "qkv"]
    o1, S = api.decay_forward(*piece(0, 130), dev["decay"])
    o2, S2 = api.decay_forward(*piece(130, 147), dev["decay"], S, state_out=S)
    assert S2 is S
    rest = [api.decay_step(*(t[:, 0] for t in piece(t, t + 1)), dev["decay"], S)[:, None] for t in range(147, 150)]
    got = torch.cat([o1, o2, *rest], 1)
    bound = scan_bound(dtype, ref, x["q"], x["k"], x["v"], x["decay"], None, [T] * B, d ** -0.5)
    within(_np(got), ref, bound, "out")
    within(_np(S), ref_last, state_bound(dtype, x["k"], x["v"], x["decay"], None, [T] * B), "state")


@pytest.mark.parametrize("dtype,d,T", [("bf16", 128, 1100), ("f32", 128, 200), ("f32", 16, 200)])
def test_explicit_scale_and_repeated_runs(dtype, d, T):
    x = inputs(4, dtype, 1, T, 2, d)
    dev = cuda(x)
    a, Sa = api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], scale=0.25)
    b, Sb = api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], scale=0.25)
    assert torch.equal(a, b) and torch.equal(Sa, Sb)
    ref, _ = C.decay_forward(x["q"], x["k"], x["v"], x["decay"], x["state"], scale=0.25)
    within(_np(a), ref, scan_bound(dtype, ref, x["q"], x["k"], x["v"], x["decay"], x["state"], [T], 0.25))
    assert api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], want_state=False)[1] is None
    args = (dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"])
    g1 = api.decay_backward(*args, dout=dev["dout"], dfinal=dev["dfinal"], scale=0.25)
    g2 = api.decay_backward(*args, dout=dev["dout"], dfinal=dev["dfinal"], scale=0.25)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)
    g = api.decay_backward(*args[:4], dout=dev["dout"])
    assert g["dstate"] is None


def test_allocated_outputs_are_zero_behind_a_sequence():
    dev = cuda(inputs(5, "bf16", 2, 40, 2, 128))
    lens = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    out, last = api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], lengths=lens)
    assert not out[0, 3:].any() and not out[1].any() and torch.equal(last[1], dev["state"][1])
    g = api.decay_backward(dev["q"], dev["k"], dev["v"], dev["decay"], dev["state"], dout=dev["dout"], lengths=lens)
    assert not g["dk"][0, 3:].any() and not g["dv"][1].any() and not g["dstate"][1].any()
    o = api.decay_step(dev["q"][:, 0].contiguous(), dev["k"][:, 0].contiguous(), dev["v"][:, 0].contiguous(),
                       dev["decay"], dev["state"], slots=torch.tensor([-1, 0], dtype=torch.int32, device="cuda"))
    assert not o[0].any() and o[1].any()


@pytest.mark.parametrize("dtype,d,T", [("bf16", 128, 1700), ("f32", 128, 420), ("f32", 16, 420)])
def test_rows_behind_in_made_and_given_buffers(dtype, d, T):
    """Over several segments, of which the sequences reach none, one and all: zero where the call made the buffer,
    untouched where it was given, the workspace given or not."""
    x = cuda(inputs(12, dtype, 4, T, 2, d))
    counts = [0, 5, T - 3, T]
    lens = torch.tensor(counts, dtype=torch.int32, device="cuda")
    args = (x["q"], x["k"], x["v"], x["decay"], x["state"])
    m = live(counts, T)
    dirty = [torch.full((4, T, 2, d), -7.0, device="cuda").to(x["q"].dtype) for _ in range(8)]
    del dirty                                         # what empty buffers are made of
    made, _ = api.decay_forward(*args, lengths=lens)
    gmade = api.decay_backward(*args, dout=x["dout"], lengths=lens)
    given = torch.full_like(x["q"], -7.0)
    api.decay_forward(*args, lengths=lens, out=given)
    names = ("dq", "dk", "dv")
    ggiven = {n: torch.full_like(x["q"], -7.0) for n in names}
    ggiven["dstate"] = torch.empty_like(x["state"])   # as in gmade: a state that leaves is kept more exactly
    api.decay_backward(*args, dout=x["dout"], lengths=lens, grads=ggiven)
    assert torch.equal(gmade["dstate"], ggiven["dstate"])
    for a, b in [(made, given)] + [(gmade[n], ggiven[n]) for n in names]:
        a, b = a.float().cpu().numpy(), b.float().cpu().numpy()
        assert not a[~m].any() and bool((b[~m] == -7.0).all()) and bool((a[m] == b[m]).all())


def test_other_stream_and_two_calls_at_once():
    x = [cuda(inputs(s, "bf16", 1, 1500, 4, 128)) for s in (6, 7)]
    want = [api.decay_forward(d["q"], d["k"], d["v"], d["decay"], d["state"]) for d in x]
    want_g = [api.decay_backward(d["q"], d["k"], d["v"], d["decay"], d["state"], dout=d["dout"]) for d in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for rep in range(5):
        got = [api.decay_forward(d["q"], d["k"], d["v"], d["decay"], d["state"], stream=s) for d, s in zip(x, streams)]
        got_g = [api.decay_backward(d["q"], d["k"], d["v"], d["decay"], d["state"], dout=d["dout"], stream=s)
                 for d, s in zip(x, streams)]
        torch.cuda.synchronize()
        for (o, S), (wo, wS), g, wg in zip(got, want, got_g, want_g):
            assert torch.equal(o, wo) and torch.equal(S, wS) and all(torch.equal(g[n], wg[n]) for n in g)


def test_captured_and_replayed():
    """A prompt, its gradient and a step in one graph, replayed on new inputs in the same buffers."""
    a, b = (cuda(inputs(s, "bf16", 2, 1100, 3, 128)) for s in (8, 9))
    buf = {n: a[n].clone() for n in a}
    S = torch.zeros_like(a["state"])
    ws = torch.empty(api.decay_workspace_size(api._decay_shape(a["q"]), True), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([1100, 500], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(a["q"])
    grads = {n: torch.zeros_like(a["q"]) for n in ("dq", "dk", "dv")}
    tok = [buf[n][:, 0].contiguous() for n in "qkv"]

    def call():
        api.decay_forward(buf["q"], buf["k"], buf["v"], buf["decay"], buf["state"], lengths=lens, out=out, state_out=S,
                          workspace=ws)
        api.decay_backward(buf["q"], buf["k"], buf["v"], buf["decay"], buf["state"], dout=buf["dout"], lengths=lens,
                           grads=grads, workspace=ws)
        return api.decay_step(*tok, buf["decay"], S)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    for src, ln in ((b, [1100, 500]), (a, [1, 0]), (b, [640, 1100])):
        for n in buf:
            buf[n].copy_(src[n])
        lens.copy_(torch.tensor(ln, dtype=torch.int32))
        for t in [out, *grads.values()]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone(), S.clone(), o.clone(), *(grads[n].clone() for n in grads)]
        for t in [out, *grads.values()]:
            t.zero_()
        o2 = call()
        torch.cuda.synchronize()
        for u, w in zip(got, [out, S, o2, *(grads[n] for n in grads)]):
            assert torch.equal(u, w)


def test_offsets_past_int32():
    """Element offsets above 2^31: the last sequence of a large batch equals the same sequence alone."""
    B, T, H, d = 9, 16384, 120, 128           # 2.26e9 elements per tensor
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator("cuda").manual_seed(0)
    q = torch.zeros(B, T, H, d, dtype=torch.bfloat16, device="cuda")
    one = torch.randn(1, T, H, d, generator=g, device="cuda").bfloat16()
    q[-1:] = one
    lam = torch.linspace(0.5, 1.0, H, device="cuda")
    lens = torch.tensor([1] * (B - 1) + [T], dtype=torch.int32, device="cuda")
    out, last = api.decay_forward(q, q, q, lam, lengths=lens)
    o1, l1 = api.decay_forward(one, one, one, lam)
    # the splits into segments differ: the state to fp32 rounding, the output to bf16's
    assert torch.allclose(last[-1:], l1, rtol=1e-4, atol=1e-4 * float(l1.abs().max()))
    assert ((out[-1:].float() - o1.float()).norm() / o1.float().norm()) < 2.0 ** -7
    del out, o1, q


def test_library_refuses_short_workspace_and_noncontiguous():
    dev = cuda(inputs(10, "bf16", 1, 1200, 2, 128))
    with pytest.raises(Exception, match="workspace"):
        api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"],
                          workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        api.decay_forward(dev["q"].transpose(1, 2).contiguous().transpose(1, 2), dev["k"], dev["v"], dev["decay"])
    with pytest.raises(Exception, match="status 1"):
        api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], out=dev["v"])


def test_binding_refuses_mismatched_device_tensors():
    dev = cuda(inputs(11, "bf16", 2, 3, 2, 128))
    tok = [dev[n][:, 0].contiguous() for n in "qkv"]
    with pytest.raises(ValueError, match="state has shape"):
        api.decay_step(*tok, dev["decay"], torch.zeros(3, 2, 128, 128, device="cuda"))   # no slots: a state per row
    with pytest.raises(ValueError, match="state is required"):
        api.decay_step(*tok, dev["decay"], None)
    with pytest.raises(ValueError, match="lengths has dtype"):
        api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"], lengths=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="k has shape"):
        api.decay_backward(dev["q"], dev["k"][:, :2], dev["v"], dev["decay"], dout=dev["dout"])
    with pytest.raises(ValueError, match="decay is on cpu"):
        api.decay_forward(dev["q"], dev["k"], dev["v"], dev["decay"].cpu())
