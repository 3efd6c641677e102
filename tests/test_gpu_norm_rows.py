"""Layer norm where every team of threads walks several rows (the next row's loads, the alternating halves of the
sums' buffers, parameter gradients kept over the rows, teams that end at different steps), against the formulas in
64 bits."""
import pytest
import torch

from causal import DT
from video_diffusion_linear_b200 import _lib, api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _team(dtype, d):
    """Threads of a row: two (fp32: four) vectors of 16 bytes each, and one vector more where rows are shifted."""
    vec, nv = (8, 2) if dtype == "bf16" else (4, 4)
    vecs = d // vec + (2 if d % vec else 0)
    team = 1
    while team < 1024 and vecs > nv * team:
        team *= 2
    return team


def _within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(err).all()) and float((err - bound).max()) <= 1e-30, (what, float((err - bound).max()))


SHAPES = [  # rows, groups (0: parameters shared), d: teams of 1 to 1024 threads, whole vectors and shifted rows
    (2000003, 0, 16), (300007, 0, 77), (450001, 0, 128), (20001, 24, 128), (90000, 7, 33), (8003, 0, 300), (4032, 0, 1999),
    (5000, 0, 2048), (3000, 0, 4097), (2000, 0, 8192), (1500, 0, 8193), (1500, 0, 16383), (1200, 0, 16384),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,d", SHAPES)
def test_several_rows_per_team(dtype, rows, groups, d):
    g = torch.Generator("cuda").manual_seed(rows + d)
    n_groups = max(1, groups)
    shape, ps = (rows, n_groups, d), (n_groups, d)
    x = (torch.randn(shape, generator=g, device="cuda") + 0.5).to(DT[dtype])
    dy = torch.randn(shape, generator=g, device="cuda").to(DT[dtype])
    w = 1 + 0.3 * torch.randn(ps, generator=g, device="cuda")
    b = torch.randn(ps, generator=g, device="cuda")
    # the backward's blocks leave 2 x parts x groups x d partial sums: each must hold several rows for each team
    team = _team(dtype, d)
    parts = _lib.load().vdn_layer_norm_backward_workspace_size(rows * n_groups, n_groups, d, _lib.VDN_DTYPE[dtype]) // (
        8 * n_groups * d)
    assert rows >= 2.5 * parts * max(1, 256 // team)
    eps = 1e-3
    y, mean, rstd = api.layer_norm_forward(x, w, b, eps=eps)
    got = api.layer_norm_backward(x, dy, mean, rstd, w, bias=True)

    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    sums = {n: torch.zeros(ps, dtype=torch.float64, device="cuda") for n in ("w", "b", "w_mag", "b_mag", "w_err")}
    step = max(1, (1 << 24) // (n_groups * d))
    for i in range(0, rows, step):
        X, D, W = x[i:i + step].double(), dy[i:i + step].double(), w.double()
        m = X.mean(-1, keepdim=True)
        r = ((X - m).square().mean(-1, keepdim=True) + eps).rsqrt()
        xh = (X - m) * r
        # the mean: sums of at most 32 adds in a thread and a tree of 10; rstd: the centred squares' sum (half of its
        # error, and the mean's against sigma) and the root; the rest as the formulas are evaluated
        dm = 48 * U * X.abs().mean(-1, keepdim=True)
        dr = r * (32 * U + r * dm)
        _within(mean[i:i + step], m[..., 0], dm[..., 0], "mean")
        _within(rstd[i:i + step], r[..., 0], dr[..., 0], "rstd")
        dxh = r * (dm + 2 * U * X.abs()) + xh.abs() * (dr / r + 2 * U)
        ref = xh * W + b.double()
        _within(y[i:i + step], ref, W.abs() * dxh + 3 * U * ((W * xh).abs() + b.double().abs()) + half * ref.abs(), "y")
        G = D * W
        ref = r * (G - G.mean(-1, keepdim=True) - xh * (G * xh).mean(-1, keepdim=True))
        c1, c2 = G.abs().mean(-1, keepdim=True), (G * xh).abs().mean(-1, keepdim=True)
        bound = r * (50 * U * (G.abs() + c1 + xh.abs() * c2) + dxh * c2 + xh.abs() * (G.abs() * dxh).mean(-1, keepdim=True)) \
            + ref.abs() * (dr / r) + half * ref.abs()
        _within(got["dx"][i:i + step], ref, bound, "dx")
        for n, t in (("w", D * xh), ("b", D), ("w_mag", (D * xh).abs()), ("b_mag", D.abs()), ("w_err", D.abs() * dxh)):
            sums[n] += t.sum(0)
    # sums over the rows in fp32: no entry is added in more steps than there are rows
    _within(got["dweight"].reshape(ps), sums["w"], sums["w_err"] + (rows + 8) * U * sums["w_mag"], "dweight")
    _within(got["dbias"].reshape(ps), sums["b"], (rows + 8) * U * sums["b_mag"], "dbias")
