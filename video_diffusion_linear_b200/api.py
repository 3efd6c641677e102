"""Thin Python binding of libvdn (include/vdn.h).

Argument marshalling only: torch supplies device memory and the stream, every
step of the branch runs in the library's CUDA kernels.  Tensors must be CUDA
tensors in the layouts documented in vdn.h.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import VDN_DTYPE, VDN_IMPL, VDN_RULE, VdnDebugOut, VdnShape, check

_TORCH_DTYPE = {torch.float32: "f32", torch.bfloat16: "bf16"}


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libvdn must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _validate(specs, device) -> None:
    """Checks (name, tensor, shape, dtype, optional) specs before any pointer reaches the library:
    the kernels read each buffer with the element type and extent vdn.h fixes, so a tensor of
    another dtype, shape or device would be read out of its bounds."""
    if device.type != "cuda":
        raise ValueError(f"libvdn takes CUDA tensors, got a tensor on {device}")
    for name, t, shape, dtype, optional in specs:
        if t is None:
            if optional:
                continue
            raise ValueError(f"{name} is required")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _bytes(name, t, device) -> None:
    """A caller-owned byte buffer (workspace, saved state): a uint8 CUDA tensor on `device`, whose
    numel is the byte count the library is told."""
    if t is None:
        return
    if t.device != device or t.dtype != torch.uint8:
        raise ValueError(f"{name} must be a uint8 tensor on {device}, got {t.dtype} on {t.device}")


def _branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F, out=None):
    """Specs of the branch's inputs (vdn.h, vdn_branch_forward) for q of shape [B, F*S, H, d]."""
    B, N, H, d = q.shape
    f32 = torch.float32
    K = conv_k_w.shape[-1] if conv_k_w is not None else (conv_v_w.shape[-1] if conv_v_w is not None else 1)
    return [("q", q, (B, N, H, d), q.dtype, False), ("k", k, (B, N, H, d), q.dtype, False),
            ("v", v, (B, N, H, d), q.dtype, False), ("gate", gate, (B, N, H, d), q.dtype, False),
            ("beta", beta, (B, N, H), f32, False), ("alpha", alpha, (B, F, H, d), f32, False),
            ("rms_w", rms_w, (d,), f32, False), ("conv_k_w", conv_k_w, (H, d, K), f32, True),
            ("conv_v_w", conv_v_w, (H, d, K), f32, True), ("text_state", text_state, (H, d, d), f32, True),
            ("out", out, (B, N, H, d), q.dtype, True)]


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_shape(B, H, F, S, d, conv_width=3, dtype="bf16") -> VdnShape:
    if isinstance(dtype, torch.dtype):
        dtype = _TORCH_DTYPE[dtype]
    return VdnShape(B, H, F, S, d, conv_width, VDN_DTYPE[dtype])


def shape_from(q: torch.Tensor, F: int, conv_k_w=None) -> VdnShape:
    B, N, H, d = q.shape
    if N % F:
        raise ValueError(f"token count {N} is not a multiple of F={F}")
    K = 1 if conv_k_w is None else conv_k_w.shape[-1]
    return make_shape(B, H, F, N // F, d, K, q.dtype)


def workspace_size(shape: VdnShape, rule="vdn_solve", impl="auto") -> int:
    n = _lib.load().vdn_branch_workspace_size_impl(ctypes.byref(shape), VDN_RULE[rule], VDN_IMPL[impl])
    if n == 0:
        raise _lib.VdnError(_lib.VDN_ERR_INVALID_ARG, "vdn_branch_workspace_size")
    return n


def alloc_workspace(shape: VdnShape, rule="vdn_solve", impl="auto", device="cuda") -> torch.Tensor:
    return torch.empty(workspace_size(shape, rule, impl), dtype=torch.uint8, device=device)


def _forward_args(shape, q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, rule, c, chunk,
                  radius, workspace, out, stream):
    return (ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(gate), _ptr(rms_w),
            _ptr(conv_k_w), _ptr(conv_v_w), _ptr(text_state), VDN_RULE[rule], float(c), int(chunk), int(radius),
            _ptr(workspace), workspace.numel(), _ptr(out), _stream_ptr(stream))


def branch_forward(q, k, v, beta, alpha, gate, rms_w, conv_k_w=None, conv_v_w=None, text_state=None, *,
                   F: int, rule="vdn_solve", c=1.0, chunk=5, radius=1, out=None, workspace=None, stream=None):
    """vdn_branch_forward: the whole branch.  Returns `out` ([B, F*S, H, d], q's dtype)."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate(_branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F, out), q.device)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(shape, rule, "auto", q.device)
    _bytes("workspace", workspace, q.device)
    st = _lib.load().vdn_branch_forward(*_forward_args(shape, q, k, v, beta, alpha, gate, rms_w, conv_k_w,
                                                       conv_v_w, text_state, rule, c, chunk, radius, workspace,
                                                       out, stream))
    check(st, "vdn_branch_forward")
    return out


def window_softmax_forward(q_rope, k_rope, v, *, F: int, chunk=5, radius=1, scale=0.0, accumulate=False,
                           out=None, workspace=None, stream=None):
    """vdn_window_softmax_forward: the windowed softmax branch (out = or += its
    output).  Returns `out` ([B, F*S, H, d], q_rope's dtype)."""
    shape = shape_from(q_rope, F)
    _validate([(n, t, q_rope.shape, q_rope.dtype, n == "out") for n, t in
               (("q_rope", q_rope), ("k_rope", k_rope), ("v", v), ("out", out))], q_rope.device)
    if out is None:
        out = torch.zeros_like(q_rope) if accumulate else torch.empty_like(q_rope)
    if workspace is None:
        workspace = torch.empty(_lib.load().vdn_window_softmax_workspace_size(ctypes.byref(shape)),
                                dtype=torch.uint8, device=q_rope.device)
    _bytes("workspace", workspace, q_rope.device)
    st = _lib.load().vdn_window_softmax_forward(ctypes.byref(shape), _ptr(q_rope), _ptr(k_rope), _ptr(v), int(chunk),
                                                int(radius), float(scale), int(bool(accumulate)), _ptr(workspace),
                                                workspace.numel(), _ptr(out), _stream_ptr(stream))
    check(st, "vdn_window_softmax_forward")
    return out


def hybrid_forward(q_rope, k_rope, q, k, v, beta, alpha, gate, rms_w, conv_k_w=None, conv_v_w=None,
                   text_state=None, *, F: int, rule="vdn_solve", c=1.0, chunk=5, radius=1, scale=0.0, out=None,
                   workspace=None, stream=None):
    """vdn_hybrid_forward: windowed softmax branch + linear branch.  Returns `out`."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate(_branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F, out) +
              [("q_rope", q_rope, q.shape, q.dtype, False), ("k_rope", k_rope, q.shape, q.dtype, False)], q.device)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(shape, rule, "auto", q.device)
    _bytes("workspace", workspace, q.device)
    fa = _forward_args(shape, q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, rule, c, chunk,
                       radius, workspace, out, stream)
    st = _lib.load().vdn_hybrid_forward(fa[0], _ptr(q_rope), _ptr(k_rope), *fa[1:15], float(scale), *fa[15:])
    check(st, "vdn_hybrid_forward")
    return out


def launch_count(shape: VdnShape, impl="auto") -> int:
    return _lib.load().vdn_branch_launch_count(ctypes.byref(shape), VDN_IMPL[impl])


def branch_forward_timed(q, k, v, beta, alpha, gate, rms_w, conv_k_w=None, conv_v_w=None, text_state=None, *,
                         F: int, events, rule="vdn_solve", c=1.0, chunk=5, radius=1, out=None, workspace=None,
                         stream=None):
    """vdn_branch_forward_timed: like branch_forward, recording `events` (torch.cuda.Event
    objects with timing enabled, already recorded once so their handles exist) before the
    first kernel and after each kernel."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate(_branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F, out), q.device)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(shape, rule, "auto", q.device)
    _bytes("workspace", workspace, q.device)
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    st = _lib.load().vdn_branch_forward_timed(*_forward_args(shape, q, k, v, beta, alpha, gate, rms_w, conv_k_w,
                                                             conv_v_w, text_state, rule, c, chunk, radius,
                                                             workspace, out, stream), arr, len(events))
    check(st, "vdn_branch_forward_timed")
    return out


DEBUG_FIELDS = ("A", "B", "N", "P", "Q", "W")


def branch_forward_debug(q, k, v, beta, alpha, gate, rms_w, conv_k_w=None, conv_v_w=None, text_state=None, *,
                         F: int, rule="vdn_solve", c=1.0, chunk=5, radius=1, impl="auto", want=DEBUG_FIELDS,
                         out=None, workspace=None, stream=None):
    """vdn_branch_forward_debug: returns (out, {name: fp32 [B, H, F, d, d]}) for the requested intermediates."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate(_branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F, out), q.device)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(shape, rule, impl, q.device)
    _bytes("workspace", workspace, q.device)
    B, N, H, d = q.shape
    mats = {name: torch.full((B, H, F, d, d), float("nan"), dtype=torch.float32, device=q.device) for name in want}
    dbg = VdnDebugOut(VDN_IMPL[impl], *[mats[n].data_ptr() if n in mats else None for n in DEBUG_FIELDS])
    st = _lib.load().vdn_branch_forward_debug(*_forward_args(shape, q, k, v, beta, alpha, gate, rms_w, conv_k_w,
                                                             conv_v_w, text_state, rule, c, chunk, radius,
                                                             workspace, out, stream), ctypes.byref(dbg))
    check(st, "vdn_branch_forward_debug")
    return out, mats


def feature_prep(q, k, v, conv_k_w=None, conv_v_w=None, *, F: int, stream=None, out=None):
    """vdn_feature_prep: Step 1 alone.  Returns (q', k', v') in q's dtype (into `out`, a tuple
    of three tensors shaped like q, when given)."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate([s for s in _branch_specs(q, k, v, None, None, None, None, conv_k_w, conv_v_w, None, F)
               if s[0] in ("q", "k", "v", "conv_k_w", "conv_v_w")], q.device)
    if out is None:
        qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        qo, ko, vo = out
        _validate([("q_out", qo, q.shape, q.dtype, False), ("k_out", ko, q.shape, q.dtype, False),
                   ("v_out", vo, q.shape, q.dtype, False)], q.device)
    st = _lib.load().vdn_feature_prep(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(conv_k_w),
                                      _ptr(conv_v_w), _ptr(qo), _ptr(ko), _ptr(vo), _stream_ptr(stream))
    check(st, "vdn_feature_prep")
    return qo, ko, vo


def window_bounds(t: int, F: int, chunk: int = 5, radius: int = 1):
    lo, hi = ctypes.c_int(), ctypes.c_int()
    check(_lib.load().vdn_window_bounds(t, F, chunk, radius, ctypes.byref(lo), ctypes.byref(hi)),
          "vdn_window_bounds")
    return lo.value, hi.value


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    return _lib.load().vdn_workspace_status(_ptr(workspace), workspace.numel(), _stream_ptr(stream))


def to_device(inp: dict, device="cuda") -> dict:
    """Copies the host tensors of synth.make_inputs to the device (None stays None)."""
    return {k: (None if t is None else t.to(device)) for k, t in inp.items()}


def saved_size(shape: VdnShape) -> int:
    n = _lib.load().vdn_branch_saved_size(ctypes.byref(shape))
    if n == 0:
        raise _lib.VdnError(_lib.VDN_ERR_INVALID_ARG, "vdn_branch_saved_size")
    return n


def branch_forward_train(q, k, v, beta, alpha, gate, rms_w, conv_k_w=None, conv_v_w=None, text_state=None, *,
                         F: int, rule="vdn_solve", c=1.0, chunk=5, radius=1, out=None, saved=None, workspace=None,
                         stream=None):
    """vdn_branch_forward_train: the branch's output and the per-frame state its backward
    reads.  Returns (out, saved); pass `saved` to branch_backward(..., saved=saved)."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate(_branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F, out), q.device)
    if out is None:
        out = torch.empty_like(q)
    if saved is None:
        saved = torch.empty(saved_size(shape), dtype=torch.uint8, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(shape, rule, "auto", q.device)
    _bytes("saved", saved, q.device)
    _bytes("workspace", workspace, q.device)
    fa = _forward_args(shape, q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, rule, c, chunk,
                       radius, workspace, out, stream)
    st = _lib.load().vdn_branch_forward_train(*fa[:-1], _ptr(saved), saved.numel(), fa[-1])
    check(st, "vdn_branch_forward_train")
    return out, saved


def backward_workspace_size(shape: VdnShape, rule="vdn_solve", saved=False) -> int:
    if saved:
        n = _lib.load().vdn_branch_backward_saved_workspace_size(ctypes.byref(shape), VDN_RULE[rule])
        if n == 0:
            raise _lib.VdnError(_lib.VDN_ERR_INVALID_ARG, "vdn_branch_backward_saved_workspace_size")
        return n
    n = _lib.load().vdn_branch_backward_workspace_size(ctypes.byref(shape), VDN_RULE[rule])
    if n == 0:
        raise _lib.VdnError(_lib.VDN_ERR_INVALID_ARG, "vdn_branch_backward_workspace_size")
    return n


def branch_backward(q, k, v, beta, alpha, gate, rms_w, conv_k_w=None, conv_v_w=None, text_state=None, *, dout,
                    F: int, rule="vdn_solve", c=1.0, chunk=5, radius=1, grads=None, workspace=None, stream=None,
                    events=None, saved=None):
    """vdn_branch_backward: gradients of <dout, branch_forward(...)> with respect to every
    input.  Returns a dict dq, dk, dv, dgate (q's dtype), dbeta, dalpha, drms_w, and
    dconv_k_w, dconv_v_w, dtext_state (fp32; None where the input is None).  With
    `events` (8 torch.cuda.Event), vdn_branch_backward_timed records them between the
    forward recompute and each backward kernel.  With `saved` (from branch_forward_train),
    vdn_branch_backward_saved runs instead, without the forward recompute."""
    shape = shape_from(q, F, conv_k_w if conv_k_w is not None else conv_v_w)
    dev = q.device
    specs = _branch_specs(q, k, v, beta, alpha, gate, rms_w, conv_k_w, conv_v_w, text_state, F)
    _validate(specs + [("dout", dout, q.shape, q.dtype, False)], dev)
    if grads is None:
        f32 = dict(dtype=torch.float32, device=dev)
        grads = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
                 "dgate": torch.empty_like(gate), "dbeta": torch.empty(beta.shape, **f32),
                 "dalpha": torch.empty(alpha.shape, **f32), "drms_w": torch.empty(rms_w.shape, **f32),
                 "dconv_k_w": None if conv_k_w is None else torch.empty(conv_k_w.shape, **f32),
                 "dconv_v_w": None if conv_v_w is None else torch.empty(conv_v_w.shape, **f32),
                 "dtext_state": None if text_state is None else torch.empty(text_state.shape, **f32)}
    if workspace is None:
        workspace = torch.empty(backward_workspace_size(shape, rule, saved is not None), dtype=torch.uint8,
                                device=dev)
    _bytes("workspace", workspace, dev)
    _bytes("saved", saved, dev)
    # each gradient has its input's shape: q's dtype for the token tensors, fp32 for the rest
    _validate([("d" + n, grads.get("d" + n), shp, dt if n in ("q", "k", "v", "gate") else torch.float32, True)
               for n, _, shp, dt, _ in specs if n != "out"], dev)
    g = grads
    args = (ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(gate), _ptr(rms_w),
            _ptr(conv_k_w), _ptr(conv_v_w), _ptr(text_state), VDN_RULE[rule], float(c), int(chunk), int(radius),
            _ptr(dout), _ptr(workspace), workspace.numel(), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
            _ptr(g["dbeta"]), _ptr(g["dalpha"]), _ptr(g["dgate"]), _ptr(g["drms_w"]), _ptr(g["dconv_k_w"]),
            _ptr(g["dconv_v_w"]), _ptr(g["dtext_state"]), _stream_ptr(stream))
    if saved is not None:
        if events is not None:
            raise ValueError("events are recorded by the recomputing backward only")
        st = _lib.load().vdn_branch_backward_saved(*args[:16], _ptr(saved), saved.numel(), *args[16:])
    elif events is None:
        st = _lib.load().vdn_branch_backward(*args)
    else:
        arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
        st = _lib.load().vdn_branch_backward_timed(*args, arr, len(events))
    check(st, "vdn_branch_backward")
    return grads


def forward_inputs(dev: dict):
    """Positional tensor arguments of branch_forward from a synth-style dict."""
    return (dev["q"], dev["k"], dev["v"], dev["beta"], dev["alpha"], dev["gate"], dev["rms_w"],
            dev.get("conv_k_w"), dev.get("conv_v_w"), dev.get("text_state"))


# ----------------------------------------------------------------------------- frame sharding
def frame_range(F: int, world: int, rank: int, chunk: int = 5) -> tuple[int, int]:
    """vdn_frame_range: the frames [f0, f1) rank `rank` of `world` owns under frame sharding
    (whole chunks, split as evenly as possible)."""
    f0, f1 = ctypes.c_int(), ctypes.c_int()
    check(_lib.load().vdn_frame_range(F, world, rank, chunk, ctypes.byref(f0), ctypes.byref(f1)), "vdn_frame_range")
    return f0.value, f1.value


def frame_owner(F: int, world: int, frame: int, chunk: int = 5) -> int:
    r = ctypes.c_int()
    check(_lib.load().vdn_frame_owner(F, world, chunk, frame, ctypes.byref(r)), "vdn_frame_owner")
    return r.value


def frames_map_bytes(shape: VdnShape, F_total: int, world: int, rank: int, chunk: int = 5) -> int:
    n = _lib.load().vdn_frames_map_bytes(ctypes.byref(shape), F_total, world, rank, chunk)
    if n == 0:
        raise _lib.VdnError(_lib.VDN_ERR_INVALID_ARG, "vdn_frames_map_bytes")
    return n


def frames_workspace_size(shape: VdnShape, F_total: int, world: int, rank: int, rule="vdn_solve",
                          chunk: int = 5) -> int:
    n = _lib.load().vdn_frames_workspace_size(ctypes.byref(shape), F_total, world, rank, VDN_RULE[rule], chunk)
    if n == 0:
        raise _lib.VdnError(_lib.VDN_ERR_INVALID_ARG, "vdn_frames_workspace_size")
    return n


def frames_maps(k, v, beta, alpha, conv_k_w=None, conv_v_w=None, *, F_total: int, world: int, rank: int,
                rule="vdn_solve", c=1.0, chunk=5, workspace=None, maps=None, stream=None) -> torch.Tensor:
    """vdn_frames_maps, phase 1 of the frame-sharded branch: k, v, beta, alpha hold the rank's
    frames only.  Returns the rank's per-chunk affine maps (flat fp32, frames_map_bytes / 4)."""
    f0, f1 = frame_range(F_total, world, rank, chunk)
    shape = shape_from(k, f1 - f0, conv_k_w if conv_k_w is not None else conv_v_w)
    _validate([s for s in _branch_specs(k, k, v, beta, alpha, k, None, conv_k_w, conv_v_w, None, f1 - f0)
               if s[0] in ("k", "v", "beta", "alpha", "conv_k_w", "conv_v_w")], k.device)
    nb = frames_map_bytes(shape, F_total, world, rank, chunk)
    if maps is None:
        maps = torch.empty(nb // 4, dtype=torch.float32, device=k.device)
    if workspace is None:
        workspace = torch.empty(frames_workspace_size(shape, F_total, world, rank, rule, chunk), dtype=torch.uint8,
                                device=k.device)
    _validate([("maps", maps, (maps.numel(),), torch.float32, False)], k.device)
    _bytes("workspace", workspace, k.device)
    st = _lib.load().vdn_frames_maps(ctypes.byref(shape), F_total, world, rank, _ptr(k), _ptr(v), _ptr(beta),
                                     _ptr(alpha), _ptr(conv_k_w), _ptr(conv_v_w), VDN_RULE[rule], float(c),
                                     int(chunk), _ptr(workspace), workspace.numel(), _ptr(maps),
                                     maps.numel() * maps.element_size(), _stream_ptr(stream))
    check(st, "vdn_frames_maps")
    return maps


def frames_finish(q, alpha_all, gate, rms_w, text_state, maps_all, *, F_total: int, world: int, rank: int,
                  rule="vdn_solve", c=1.0, chunk=5, radius=1, out=None, workspace=None, stream=None):
    """vdn_frames_finish, phase 2: q and gate hold the rank's frames, alpha_all the whole clip's,
    maps_all every rank's maps in rank order.  Returns the branch output of the rank's frames."""
    f0, f1 = frame_range(F_total, world, rank, chunk)
    shape = shape_from(q, f1 - f0)
    B, N, H, d = q.shape
    f32 = torch.float32
    _validate([("q", q, q.shape, q.dtype, False), ("gate", gate, q.shape, q.dtype, False),
               ("out", out, q.shape, q.dtype, True), ("alpha_all", alpha_all, (B, F_total, H, d), f32, False),
               ("rms_w", rms_w, (d,), f32, False), ("text_state", text_state, (H, d, d), f32, True),
               ("maps_all", maps_all, (maps_all.numel(),), f32, False)], q.device)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.empty(frames_workspace_size(shape, F_total, world, rank, rule, chunk), dtype=torch.uint8,
                                device=q.device)
        workspace[:256].zero_()   # phase 2 keeps the device status word it is given
    _bytes("workspace", workspace, q.device)
    st = _lib.load().vdn_frames_finish(ctypes.byref(shape), F_total, world, rank, _ptr(q), _ptr(alpha_all),
                                       _ptr(gate), _ptr(rms_w), _ptr(text_state), VDN_RULE[rule], float(c),
                                       int(chunk), int(radius), _ptr(maps_all),
                                       maps_all.numel() * maps_all.element_size(), _ptr(workspace),
                                       workspace.numel(), _ptr(out), _stream_ptr(stream))
    check(st, "vdn_frames_finish")
    return out


# ----------------------------------------------------------------------------- causal linear attention
# These calls run once per token of a decoding loop, where the binding's own time counts: one check per tensor (none
# for a buffer made here), plain integers for pointers, and a device switch or a second stream only where one is
# asked for.
_F32, _I32 = torch.float32, torch.int32


def _arg(name, t, shape, dtype, device):
    """The address of a required tensor after its checks (_validate's, and contiguity)."""
    if t is None or t.shape != shape or t.dtype != dtype or t.device != device:
        _validate([(name, t, shape, dtype, False)], device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(name, t, shape, dtype, device):
    return None if t is None else _arg(name, t, shape, dtype, device)


def _work(t, device):
    _bytes("workspace", t, device)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr()


class _Call:
    """The device and the stream of one call: `with` makes the tensors' device current where it is not.
    Buffers that the call makes belong to the device's current stream; used() lets another stream use them:
    after the work queued on them so far (a fill), and without their memory being handed out again before that
    stream is done with them."""
    __slots__ = ("device", "given", "guard")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError(f"libvdn takes CUDA tensors, got a tensor on {device}")
        if stream is not None and stream.device != device:      # both devices' default streams have the handle 0
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self.device, self.given = device, stream
        self.guard = torch.cuda.device(device) if device.index != torch.cuda.current_device() else None

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def used(self, *buffers):
        """The stream's handle, once it may use the buffers made so far."""
        handle = torch._C._cuda_getCurrentRawStream(self.device.index)   # current_stream() makes an object first
        s = self.given
        if s is None or s.cuda_stream == handle:
            return handle
        s.wait_stream(torch.cuda.current_stream(self.device))
        for t in buffers:
            if t is not None:
                t.record_stream(s)
        return s.cuda_stream


def _dtype_id(x, name):
    d = _TORCH_DTYPE.get(x.dtype)
    if d is None:
        raise ValueError(f"{name} has dtype {x.dtype}, expected torch.float32 or torch.bfloat16")
    return VDN_DTYPE[d]


def _decay_shape(q: torch.Tensor) -> VdnShape:
    if q.dim() != 4:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [B, T, H, d]")
    B, T, H, d = q.shape
    return VdnShape(B, H, 1, T, d, 1, _dtype_id(q, "q"))


def decay_workspace_size(shape: VdnShape, backward=False) -> int:
    lib = _lib.load()
    n = (lib.vdn_decay_backward_workspace_size if backward else lib.vdn_decay_workspace_size)(ctypes.byref(shape))
    if n == 0:
        raise _lib.VdnError(_lib.VDN_ERR_UNSUPPORTED, "vdn_decay_workspace_size")
    return n


def decay_forward(q, k, v, decay, state=None, *, lengths=None, scale=0.0, want_state=True, out=None, state_out=None,
                  workspace=None, stream=None):
    """vdn_decay_forward: causal linear attention with a decay for each head over q, k, v [B, T, H, d], from
    `state` [B, H, d, d] (None: zero).  Returns (out, state after the last token); the state is None with
    want_state=False, and written to `state_out` (which may be `state`) when given.  `lengths` [B] int32:
    a padded batch; rows behind a sequence stay as they are in `out`, zero in an `out` made here."""
    shape, dev, tok, dt = _decay_shape(q), q.device, q.shape, q.dtype
    B, T, H, d = tok
    states = (B, H, d, d)
    with _Call(dev, stream) as call:
        pq, pk, pv = _arg("q", q, tok, dt, dev), _arg("k", k, tok, dt, dev), _arg("v", v, tok, dt, dev)
        pd, ps = _arg("decay", decay, (H,), _F32, dev), _opt("state", state, states, _F32, dev)
        pl = _opt("lengths", lengths, (B,), _I32, dev)
        clear = out is None and lengths is not None
        made = ()
        if out is None:
            out = torch.empty_like(q)
            po, made = out.data_ptr(), (out,)
        else:
            po = _arg("out", out, tok, dt, dev)
        if state_out is None and want_state:
            state_out = q.new_empty(states, dtype=_F32)
            pf, made = state_out.data_ptr(), made + (state_out,)
        else:
            pf = _opt("state_out", state_out, states, _F32, dev)
        if workspace is None:
            workspace = q.new_empty(decay_workspace_size(shape), dtype=torch.uint8)
            pw, made = workspace.data_ptr(), made + (workspace,)
        else:
            pw = _work(workspace, dev)
        st = _lib.load().vdn_decay_forward(ctypes.byref(shape), pq, pk, pv, pd, ps, pl, clear, scale, pw,
                                           workspace.numel(), po, pf, call.used(*made))
    check(st, "vdn_decay_forward")
    return out, state_out


def decay_backward(q, k, v, decay, state=None, *, dout, dfinal=None, lengths=None, scale=0.0, grads=None,
                   workspace=None, stream=None):
    """vdn_decay_backward: gradients of <dout, out> + <dfinal, final state> of decay_forward with respect to
    q, k, v and the state.  Returns a dict dq, dk, dv (q's dtype) and dstate (fp32; None where `state` is
    None).  `grads`, such a dict, gives the buffers; there dstate may be set without a state, too.  Rows behind
    a sequence of `lengths` stay as they are in `grads`, zero in buffers made here."""
    shape, dev, tok, dt = _decay_shape(q), q.device, q.shape, q.dtype
    B, T, H, d = tok
    states = (B, H, d, d)
    with _Call(dev, stream) as call:
        pq, pk, pv = _arg("q", q, tok, dt, dev), _arg("k", k, tok, dt, dev), _arg("v", v, tok, dt, dev)
        pd, ps = _arg("decay", decay, (H,), _F32, dev), _opt("state", state, states, _F32, dev)
        pl, pdo = _opt("lengths", lengths, (B,), _I32, dev), _arg("dout", dout, tok, dt, dev)
        pdf = _opt("dfinal", dfinal, states, _F32, dev)
        clear = grads is None and lengths is not None      # not what a caller's buffers hold behind a sequence
        made = ()
        if grads is None:
            grads = {"dq": torch.empty_like(q), "dk": torch.empty_like(q), "dv": torch.empty_like(q),
                     "dstate": None if state is None else q.new_empty(states, dtype=_F32)}
            made = tuple(grads.values())
        g = [_arg(n, grads.get(n), tok, dt, dev) for n in ("dq", "dk", "dv")]
        g.append(_opt("dstate", grads.get("dstate"), states, _F32, dev))
        if workspace is None:
            workspace = q.new_empty(decay_workspace_size(shape, True), dtype=torch.uint8)
            made += (workspace,)
        st = _lib.load().vdn_decay_backward(ctypes.byref(shape), pq, pk, pv, pd, ps, pl, clear, scale, pdo, pdf,
                                            _work(workspace, dev), workspace.numel(), *g, call.used(*made))
    check(st, "vdn_decay_backward")
    return grads


def decay_step(q, k, v, decay, state, *, slots=None, scale=0.0, out=None, stream=None):
    """vdn_decay_step: one token of each row, q, k, v [B, H, d]; `state` [slots, H, d, d] is updated in place.
    `slots` [B] int32 names each row's state (None: row b has state b); a row whose slot is negative or
    past the end holds no sequence and keeps its row of `out` (zero in an `out` made here).  Returns `out`."""
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [B, H, d]")
    row, dt, dev = q.shape, q.dtype, q.device
    B, H, d = row
    shape = VdnShape(B, H, 1, 1, d, 1, _dtype_id(q, "q"))
    n_slots = B if slots is None or state is None else state.shape[0]
    with _Call(dev, stream) as call:
        made = None
        if out is None:
            out = made = torch.empty_like(q) if slots is None else torch.zeros_like(q)
            po = out.data_ptr()
        else:
            po = _arg("out", out, row, dt, dev)
        st = _lib.load().vdn_decay_step(
            ctypes.byref(shape), _arg("q", q, row, dt, dev), _arg("k", k, row, dt, dev), _arg("v", v, row, dt, dev),
            _arg("decay", decay, (H,), _F32, dev), _arg("state", state, (n_slots, H, d, d), _F32, dev),
            _opt("slots", slots, (B,), _I32, dev), n_slots, scale, po, call.used(made))
    check(st, "vdn_decay_step")
    return out


# ----------------------------------------------------------------------------- layer norm
def _norm_shape(x: torch.Tensor, par):
    """(rows, groups, d, the parameters' shape, dtype id): parameters of shape [d] are shared by all rows, those of
    shape [groups, d] go with the second last axis of x."""
    if x.dim() < 1:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [..., d]")
    dt, d = _dtype_id(x, "x"), x.shape[-1]
    pshape = (d,) if par is None or par.dim() < 2 else tuple(x.shape[-2:])
    if max(x.shape[-2:]) > 0x7fffffff:      # the width or the groups would wrap in the library's int
        raise _lib.VdnError(_lib.VDN_ERR_UNSUPPORTED, f"layer norm of x with shape {tuple(x.shape)}")
    return x.numel() // max(1, d), 1 if len(pshape) == 1 else pshape[0], d, pshape, dt


def layer_norm_forward(x, weight=None, bias=None, *, eps=1e-6, out=None, mean=None, rstd=None, stream=None):
    """vdn_layer_norm_forward: layer norm over the last axis of x, weight and bias fp32, [d] or [groups, d]
    (groups: x's second last axis).  Returns (out, mean, rstd), the statistics fp32 in x's shape without
    its last axis, as layer_norm_backward takes them."""
    rows, groups, d, pshape, dt = _norm_shape(x, weight if weight is not None else bias)
    dev, rshape = x.device, x.shape[:-1]
    with _Call(dev, stream) as call:
        px = _arg("x", x, x.shape, x.dtype, dev)
        pw, pb = _opt("weight", weight, pshape, _F32, dev), _opt("bias", bias, pshape, _F32, dev)
        made = ()
        if out is None:
            out = torch.empty_like(x)
            po, made = out.data_ptr(), (out,)
        else:
            po = _arg("out", out, x.shape, x.dtype, dev)
        if mean is None:
            mean = x.new_empty(rshape, dtype=_F32)
            pm, made = mean.data_ptr(), made + (mean,)
        else:
            pm = _arg("mean", mean, rshape, _F32, dev)
        if rstd is None:
            rstd = x.new_empty(rshape, dtype=_F32)
            pr, made = rstd.data_ptr(), made + (rstd,)
        else:
            pr = _arg("rstd", rstd, rshape, _F32, dev)
        st = _lib.load().vdn_layer_norm_forward(px, pw, pb, rows, groups, d, dt, eps, po, pm, pr, call.used(*made))
    check(st, "vdn_layer_norm_forward")
    return out, mean, rstd


def layer_norm_backward(x, dy, mean, rstd, weight=None, *, bias=False, groups=None, grads=None, workspace=None,
                        stream=None):
    """vdn_layer_norm_backward: from the statistics of layer_norm_forward.  Returns a dict dx (x's dtype),
    dweight (fp32, weight's shape; None without a weight) and dbias (None unless `bias`; of weight's shape,
    else [d], or [groups, d] when `groups`, the size of x's second last axis, is given)."""
    rows, n_groups, d, pshape, dt = _norm_shape(x, weight)
    if weight is None and groups is not None:
        if x.dim() < 2 or x.shape[-2] != groups:
            raise ValueError(f"groups is {groups}, x has shape {tuple(x.shape)}")
        n_groups, pshape = groups, (groups, d)
    dev, rshape, xt = x.device, x.shape[:-1], x.dtype
    with _Call(dev, stream) as call:
        px, py = _arg("x", x, x.shape, xt, dev), _arg("dy", dy, x.shape, xt, dev)
        pm, pr = _arg("mean", mean, rshape, _F32, dev), _arg("rstd", rstd, rshape, _F32, dev)
        pw = _opt("weight", weight, pshape, _F32, dev)
        made = ()
        if grads is None:
            grads = {"dx": torch.empty_like(x),
                     "dweight": None if weight is None else x.new_empty(pshape, dtype=_F32),
                     "dbias": x.new_empty(pshape, dtype=_F32) if bias else None}
            made = tuple(grads.values())
        pdx = _arg("dx", grads.get("dx"), x.shape, xt, dev)
        pdw, pdb = _opt("dweight", grads.get("dweight"), pshape, _F32, dev), _opt("dbias", grads.get("dbias"), pshape, _F32, dev)
        lib = _lib.load()
        if workspace is None:
            workspace = x.new_empty(lib.vdn_layer_norm_backward_workspace_size(rows, n_groups, d, dt), dtype=torch.uint8)
            made += (workspace,)
        st = lib.vdn_layer_norm_backward(px, py, pm, pr, pw, rows, n_groups, d, dt, _work(workspace, dev),
                                         workspace.numel(), pdx, pdw, pdb, call.used(*made))
    check(st, "vdn_layer_norm_backward")
    return grads
