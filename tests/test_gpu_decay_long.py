"""Decayed attention over many chunks on the GPU: every pipeline runs long past the point where its buffers and
barrier phases come round again (two tiles and the outputs from the fourth chunk on, the three stages of the own states
from the third), split and unsplit, forwards and from the end, with sequences that end in late chunks.  A few (batch,
head) pairs of each call are compared with the float64 oracle."""
import ctypes

import numpy as np
import pytest
import torch

from causal import DECAYS, DT, scan_bound, state_bound, within
from oracle import causal_oracle as C
from video_diffusion_linear_b200 import _lib, api

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().double().cpu().numpy()


def _segments(B, T, H, d, dtype):
    """(segments, chunks of 128 or tokens of each) of the call, from the states that its workspace holds."""
    shape = _lib.VdnShape(B, H, 1, T, d, 1, _lib.VDN_DTYPE[dtype])
    n = _lib.load().vdn_decay_workspace_size(ctypes.byref(shape)) - 256
    segments = max(1, n // (B * H * d * d * 4))
    units = -(-T // 128) if dtype == "bf16" else T
    return segments, -(-units // segments)


CASES = [  # dtype, d, B, T, H, lengths, (segments, at least so many chunks or tokens each), compared pairs
    ("bf16", 128, 4, 2048, 16, None, (2, 8), [(0, 0), (3, 15), (1, 5)]),
    ("bf16", 128, 4, 2048, 16, [2048, 1100, 641, 2047], (2, 8), [(0, 1), (1, 2), (2, 3), (3, 6)]),
    ("bf16", 128, 6, 1560, 24, [1560, 515, 640, 1559, 0, 1025], (1, 7), [(0, 0), (1, 1), (2, 2), (3, 8), (4, 3), (5, 6)]),
    ("bf16", 128, 2, 3000, 30, [2999, 1700], (2, 7), [(0, 2), (1, 6)]),
    ("bf16", 128, 2, 2300, 75, None, (1, 18), [(0, 0), (1, 74)]),        # more rows than SMs, one pass
    ("bf16", 128, 5, 8192, 30, [2000, 8192, 8192, 8192, 1153], (8, 8), [(0, 0), (4, 29)]),   # and split all the same
    ("f32", 128, 2, 2048, 75, [2048, 1500], (12, 100), [(0, 0), (1, 74)]),
    ("f32", 128, 3, 900, 50, None, (1, 900), [(0, 1), (2, 49)]),
    ("f32", 16, 8, 1000, 150, None, (1, 900), [(0, 1), (7, 147)]),
]
IDS = ["%s-d%d-B%d-T%d-H%d%s" % (c[0], c[1], c[2], c[3], c[4], "-ragged" if c[5] else "") for c in CASES]


def _draw(seed, dtype, d, B, T, H, state):
    g = torch.Generator("cuda").manual_seed(seed)
    mk = lambda: torch.randn(B, T, H, d, generator=g, device="cuda").to(DT[dtype])
    x = dict(q=mk(), k=mk(), v=mk(), dout=mk())
    x["decay"] = torch.tensor([DECAYS[h % len(DECAYS)] for h in range(H)], device="cuda")
    for n in ("state", "dfinal"):
        x[n] = torch.randn(B, H, d, d, generator=g, device="cuda") if state else None
    return x


def _pair(x, b, h):
    """The inputs of one (batch, head) pair, on the host."""
    return {n: None if t is None else t[h:h + 1].cpu() if n == "decay" else
            t[b:b + 1, h:h + 1].cpu() if n in ("state", "dfinal") else t[b:b + 1, :, h:h + 1].cpu() for n, t in x.items()}


@pytest.mark.parametrize("state", [False, True], ids=["", "state"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_many_chunks_forward_and_backward(case, state):
    dtype, d, B, T, H, lengths, (segments, least), pairs = case
    n_seg, per = _segments(B, T, H, d, dtype)
    assert n_seg == segments and per >= least            # else the case does not reach what it is here for
    x = _draw(T + H, dtype, d, B, T, H, state)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    counts = C.token_counts(lengths, B, T)
    for b, c in enumerate(counts):                       # nothing behind a sequence may be seen
        for n in ("q", "k", "v", "dout"):
            x[n][b, c:] = float("nan")
    args = (x["q"], x["k"], x["v"], x["decay"], x["state"])
    out = torch.full_like(x["q"], -77.0)
    ws = torch.empty(api.decay_workspace_size(api._decay_shape(x["q"]), True), dtype=torch.uint8, device="cuda")
    _, last = api.decay_forward(*args, lengths=lens, out=out, workspace=ws)
    assert api.workspace_status(ws) == 0
    grads = {n: torch.full_like(x["q"], -77.0) for n in ("dq", "dk", "dv")}
    grads["dstate"] = torch.empty(B, H, d, d, device="cuda")
    g = api.decay_backward(*args, dout=x["dout"], dfinal=x["dfinal"], lengths=lens, grads=grads, workspace=ws)
    assert api.workspace_status(ws) == 0
    for b, c in enumerate(counts):
        for t in (out, g["dq"], g["dk"], g["dv"]):
            assert bool((t[b, c:] == -77.0).all())
            assert bool(torch.isfinite(t[b, :c]).all())
    s = d ** -0.5
    for b, h in pairs:
        p, n = _pair(x, b, h), [counts[b]]
        one = lambda t: _np(t[b:b + 1, :n[0], h:h + 1])
        ref, ref_last = C.decay_forward(p["q"], p["k"], p["v"], p["decay"], p["state"], n)
        rg = C.decay_backward(p["q"], p["k"], p["v"], p["decay"], p["dout"], p["state"], p["dfinal"], n)
        lam, end = p["decay"], p["dfinal"]
        st = None if p["state"] is None else p["state"].transpose(-1, -2)
        end_t = None if end is None else end.transpose(-1, -2)
        bounds = [
            ("out", out, ref, scan_bound(dtype, ref, p["q"], p["k"], p["v"], lam, p["state"], n, s)),
            ("dq", g["dq"], rg["dq"], scan_bound(dtype, rg["dq"], p["dout"], p["v"], p["k"], lam, st, n, s)),
            # the state's gradient enters dk and dv without the scale
            ("dk", g["dk"], rg["dk"], scan_bound(dtype, rg["dk"], p["v"], p["dout"], p["q"], lam,
                                                 None if end is None else end_t / s, n, s, True)),
            ("dv", g["dv"], rg["dv"], scan_bound(dtype, rg["dv"], p["k"], p["q"], p["dout"], lam,
                                                 None if end is None else end / s, n, s, True)),
        ]
        for what, got, want, bound in bounds:
            if n[0]:
                within(one(got), want[:, :n[0]], bound[:, :n[0]], (what, b, h))
        within(_np(last[b:b + 1, h:h + 1]), ref_last, state_bound(dtype, p["k"], p["v"], lam, p["state"], n), ("state", b, h))
        within(_np(g["dstate"][b:b + 1, h:h + 1]), rg["dstate"],
               state_bound(dtype, p["q"], p["dout"], lam, end, n, s, True), ("dstate", b, h))
