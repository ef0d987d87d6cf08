"""Binding of the operators around the KDA mixer (``include/kda.h``): the
gated linear recurrence with a vector state, the gated head norm, and the
norms around a block.  Argument marshalling only, like the package itself.

A call runs on the device of its tensors, on `stream` or else on that device's
current stream; what it allocates belongs to the stream it runs on.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import (KDA_EUNSUPPORTED, KdaError, _check, _dt, _f, _gate_dt,
               _i, _io_dtype, _need, _sig, _sz, _vp)

KDA_SCAN_CHUNK = 128  # tokens per chunk of kda_scan's chunk states
_ll = ctypes.c_longlong

_scan = _sig("kda_scan", _i,
             [_vp, _i, _vp, _vp, _i] + [_vp] * 5 + [_i] * 4 + [_vp, _sz, _vp])
_scan_bwd = _sig("kda_scan_backward", _i,
                 [_vp, _i, _vp, _vp, _i] + [_vp] * 9 + [_i] * 4 +
                 [_vp, _sz, _vp])
_scan_step = _sig("kda_scan_step", _i,
                  [_vp, _i, _vp, _vp, _i, _vp, _vp] + [_i] * 3 + [_vp])
_scan_ws = _sig("kda_scan_workspace_size", _sz, [_i] * 4)
_scan_bwd_ws = _sig("kda_scan_backward_workspace_size", _sz, [_i] * 4)
_gated = _sig("kda_gated_norm", _i,
              [_vp, _vp, _i, _vp, _i, _f, _vp, _ll, _i, _vp])
_gated_bwd = _sig("kda_gated_norm_backward", _i,
                  [_vp, _vp, _i, _vp, _i, _f] + [_vp] * 4 +
                  [_ll, _i, _vp, _sz, _vp])
_gated_ws = _sig("kda_gated_norm_backward_workspace_size", _sz, [_ll, _i])
_block = _sig("kda_block_norm", _i,
              [_vp, _i, _vp, _i, _vp, _i, _vp, _vp] + [_f] * 3 +
              [_vp, _vp, _i, _i, _vp])
_block_bwd = _sig("kda_block_norm_backward", _i,
                  [_vp, _i, _vp, _i, _vp, _i, _vp, _vp] + [_f] * 3 +
                  [_vp] * 7 + [_i, _i, _vp, _sz, _vp])
_block_ws = _sig("kda_block_norm_backward_workspace_size", _sz, [_i, _i])

_ACTS = {"sigmoid": 1, "silu": 2}


def _act(act, z):
    if act not in _ACTS:
        raise ValueError(f"act: {act!r}, expected one of {sorted(_ACTS)}")
    return 0 if z is None else _ACTS[act]


def _ptrs(dev, *ts):
    """Data pointers of tensors (or None) that all live on GPU `dev`."""
    out = []
    for t in ts:
        if t is None:
            out.append(None)
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        out.append(t.data_ptr())
    return out


def _on(dev, stream):
    """Context in which allocations and the launch go to `stream` (or to the
    current stream) of `dev`."""
    if not dev.type == "cuda":
        raise ValueError("tensors must live on the GPU")
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return contextlib.nullcontext()
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream on {stream.device}, tensors on {dev}")
    return torch.cuda.stream(stream)


def _cur(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _ws(workspace, need, dev, where):
    if need == 0:
        raise KdaError(KDA_EUNSUPPORTED, where)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8:
        raise ValueError(f"workspace: dtype {workspace.dtype}, expected "
                         "uint8")
    return workspace


def _scan_shapes(x, g, beta, lead_ndim):
    """Check x [*lead, D], g [*lead, D] or [*lead], beta [*lead] or None;
    returns (lead, D, io dtype, gate code)."""
    if x.dim() != lead_ndim + 1:
        raise ValueError(f"x has {x.dim()} dimensions, expected "
                         f"{lead_ndim + 1}")
    lead, D = tuple(x.shape[:-1]), x.shape[-1]
    io = _io_dtype(x, "x")
    gd = _io_dtype(g, "g")
    if g.dim() == lead_ndim + 1:
        _need(g, (*lead, D), gd, "g")
    else:
        _need(g, lead, gd, "g (per-head gate)")
    _need(beta, lead, gd, "beta (must have g's dtype)")
    return lead, D, io, _gate_dt(g, lead_ndim + 1)


def kda_scan_workspace_size(B, T, H, D) -> int:
    return int(_scan_ws(B, T, H, D))


def kda_scan_backward_workspace_size(B, T, H, D) -> int:
    return int(_scan_bwd_ws(B, T, H, D))


def kda_scan(x, g, beta=None, *, h0=None, lengths=None, y=None, h_out=None,
             want_state=True, chunk_states=False, workspace=None,
             stream=None):
    """h_t = exp(g_t) h_{t-1} + beta_t x_t over sequences, y = h.

    x [B,T,H,D]; g [B,T,H,D], or [B,T,H] for one log-decay per head; beta
    [B,T,H] in g's dtype or None (ones); h0 [B,H,D] fp32 or None (zeros);
    lengths [B] int32 on the GPU or None: tokens from lengths[b] on leave the
    state alone and give zeros.  chunk_states: True for a new
    [B,ceil(T/128),H,D] fp32 tensor of the state before each chunk of
    KDA_SCAN_CHUNK tokens (for kda_scan_backward), a tensor to fill, or False.
    h_out may be h0.  Returns (y [B,T,H,D], state after the last token
    [B,H,D] fp32 or None, chunk states or None)."""
    (B, T, H), D, io, gt = _scan_shapes(x, g, beta, 3)
    NC = -(-T // KDA_SCAN_CHUNK)
    f32 = torch.float32
    _need(h0, (B, H, D), f32, "h0")
    _need(h_out, (B, H, D), f32, "h_out")
    _need(lengths, (B,), torch.int32, "lengths")
    _need(y, (B, T, H, D), io, "y")
    cs = None
    if chunk_states is not False and chunk_states is not True:
        cs = chunk_states
        _need(cs, (B, NC, H, D), f32, "chunk_states")
    dev = x.device
    with _on(dev, stream):
        if y is None:
            y = torch.empty_like(x)
        if h_out is None and want_state:
            h_out = torch.empty((B, H, D), dtype=f32, device=dev)
        if chunk_states is True:
            cs = torch.empty((B, NC, H, D), dtype=f32, device=dev)
        ws = _ws(workspace, kda_scan_workspace_size(B, T, H, D), dev,
                 "kda_scan")
        px, pg, pb, ph, pl, py, po, pc, pw = _ptrs(
            dev, x, g, beta, h0, lengths, y, h_out, cs, ws)
        st = _scan(px, _dt(x), pg, pb, gt, ph, pl, py, po, pc, B, T, H, D, pw,
                   ws.numel(), _cur(dev))
    _check(st, "kda_scan")
    return y, h_out, cs


def kda_scan_backward(x, g, beta, dy, *, h0=None, dhT=None, lengths=None,
                      chunk_states=None, want_dh0=True, workspace=None,
                      stream=None):
    """Gradient of kda_scan for the loss sum(y*dy) + sum(h_out*dhT).
    chunk_states: those kda_scan returned for the same inputs, or None (they
    are recomputed).  Returns (dx, dg shaped like g, dbeta or None, dh0 or
    None)."""
    (B, T, H), D, io, gt = _scan_shapes(x, g, beta, 3)
    f32 = torch.float32
    _need(dy, (B, T, H, D), io, "dy (must have x's dtype)")
    _need(h0, (B, H, D), f32, "h0")
    _need(dhT, (B, H, D), f32, "dhT")
    _need(lengths, (B,), torch.int32, "lengths")
    _need(chunk_states, (B, -(-T // KDA_SCAN_CHUNK), H, D), f32,
          "chunk_states")
    dev = x.device
    with _on(dev, stream):
        dx, dg = torch.empty_like(x), torch.empty_like(g)
        dbeta = None if beta is None else torch.empty_like(beta)
        dh0 = (torch.empty((B, H, D), dtype=f32, device=dev) if want_dh0
               else None)
        ws = _ws(workspace, kda_scan_backward_workspace_size(B, T, H, D), dev,
                 "kda_scan_backward")
        px, pg, pb, *rest, pw = _ptrs(dev, x, g, beta, h0, lengths, dy, dhT,
                                      chunk_states, dx, dg, dbeta, dh0, ws)
        st = _scan_bwd(px, _dt(x), pg, pb, gt, *rest, B, T, H, D, pw,
                       ws.numel(), _cur(dev))
    _check(st, "kda_scan_backward")
    return dx, dg, dbeta, dh0


def kda_scan_step(x, g, beta, state, *, y=None, stream=None):
    """One token of kda_scan per sequence: x [N,H,D], g [N,H,D] or [N,H],
    beta [N,H] or None; `state` [N,H,D] fp32 is updated in place.  Returns
    y [N,H,D]."""
    (N, H), D, io, gt = _scan_shapes(x, g, beta, 2)
    _need(state, (N, H, D), torch.float32, "state")
    _need(y, (N, H, D), io, "y")
    dev = x.device
    with _on(dev, stream):
        if y is None:
            y = torch.empty_like(x)
        px, pg, pb, ps, py = _ptrs(dev, x, g, beta, state, y)
        st = _scan_step(px, _dt(x), pg, pb, gt, ps, py, N, H, D, _cur(dev))
    _check(st, "kda_scan_step")
    return y


def _gated_shapes(o, z, w):
    if o.dim() < 1:
        raise ValueError("o has no dimension")
    io, D = _io_dtype(o, "o"), o.shape[-1]
    _need(z, o.shape, io, "z (must have o's shape and dtype)")
    _need(w, (D,), torch.float32, "w")
    return io, D, o.numel() // max(D, 1)


def kda_gated_norm(o, z, w, *, act="sigmoid", eps=1e-6, y=None, stream=None):
    """RMS norm of a mixer's heads times a gate:
    y = o / sqrt(mean(o^2) + eps) * w * act(z) over the last dimension.
    o, z [..., D] (z None: no gate), w [D] fp32, act "sigmoid" or "silu"."""
    io, D, rows = _gated_shapes(o, z, w)
    _need(y, o.shape, io, "y")
    a, dev = _act(act, z), o.device
    with _on(dev, stream):
        if y is None:
            y = torch.empty_like(o)
        po, pz, pw, py = _ptrs(dev, o, z, w, y)
        st = _gated(po, pz, _dt(o), pw, a, eps, py, rows, D, _cur(dev))
    _check(st, "kda_gated_norm")
    return y


def kda_gated_norm_backward_workspace_size(rows, D) -> int:
    return int(_gated_ws(rows, D))


def kda_gated_norm_backward(o, z, w, dy, *, act="sigmoid", eps=1e-6,
                            workspace=None, stream=None):
    """Gradient of kda_gated_norm.  Returns (do, dz or None, dw [D] fp32)."""
    io, D, rows = _gated_shapes(o, z, w)
    _need(dy, o.shape, io, "dy (must have o's shape and dtype)")
    a, dev = _act(act, z), o.device
    with _on(dev, stream):
        do = torch.empty_like(o)
        dz = None if z is None else torch.empty_like(z)
        dw = torch.empty_like(w)
        ws = _ws(workspace, kda_gated_norm_backward_workspace_size(rows, D),
                 dev, "kda_gated_norm_backward")
        po, pz, pw, pd, p0, p1, p2, pk = _ptrs(dev, o, z, w, dy, do, dz, dw,
                                               ws)
        st = _gated_bwd(po, pz, _dt(o), pw, a, eps, pd, p0, p1, p2, rows, D,
                        pk, ws.numel(), _cur(dev))
    _check(st, "kda_gated_norm_backward")
    return do, dz, dw


def _block_shapes(y, r, z, w_post, w_pre, r_name):
    if y.dim() < 1:
        raise ValueError("y has no dimension")
    io, C = _io_dtype(y, "y"), y.shape[-1]
    _need(r, y.shape, _io_dtype(r, r_name), r_name)
    _need(z, y.shape, io, "z (must have y's shape and dtype)")
    _need(w_post, (C,), torch.float32, "w_post")
    _need(w_pre, (C,), torch.float32, "w_pre")
    return io, C, y.numel() // max(C, 1)


def kda_block_norm(y, r, *, w_post=None, z=None, w_pre=None, act="sigmoid",
                   res_scale=1.0, branch_scale=1.0, eps=1e-6, r_out=None,
                   x=None, stream=None):
    """Between two blocks, over rows of the last dimension C:
    r_out = res_scale r + branch_scale act(z) norm(y; w_post);
    x = norm(r_out; w_pre).
    y the block's output, r the residual stream (its own dtype), z a gate like
    y or None, w_post / w_pre [C] fp32 or None (no norm there; x is then
    None).  r_out may be r.  Returns (r_out, x)."""
    io, C, rows = _block_shapes(y, r, z, w_post, w_pre, "r")
    _need(r_out, y.shape, r.dtype, "r_out (must have r's dtype)")
    _need(x, y.shape, io, "x")
    if x is not None and w_pre is None:
        raise ValueError("x without w_pre")
    a, dev = _act(act, z), y.device
    with _on(dev, stream):
        if r_out is None:
            r_out = torch.empty_like(r)
        if x is None and w_pre is not None:
            x = torch.empty_like(y)
        py, pr, pz, p1, p2, po, px = _ptrs(dev, y, r, z, w_post, w_pre, r_out,
                                           x)
        st = _block(py, _dt(y), pr, _dt(r), pz, a, p1, p2, res_scale,
                    branch_scale, eps, po, px, rows, C, _cur(dev))
    _check(st, "kda_block_norm")
    return r_out, x


def kda_block_norm_backward_workspace_size(rows, C) -> int:
    return int(_block_ws(rows, C))


def kda_block_norm_backward(y, r_out, *, dx=None, dr_out=None, w_post=None,
                            z=None, w_pre=None, act="sigmoid", res_scale=1.0,
                            branch_scale=1.0, eps=1e-6, workspace=None,
                            stream=None):
    """Gradient of kda_block_norm from the stream r_out it left.  dx (given
    exactly when w_pre is) and dr_out (or None) are the gradients of its
    outputs.  Returns (dy, dr, dz or None, dw_post or None, dw_pre or
    None)."""
    io, C, rows = _block_shapes(y, r_out, z, w_post, w_pre, "r_out")
    _need(dx, y.shape, io, "dx (must have y's dtype)")
    _need(dr_out, y.shape, r_out.dtype, "dr_out (must have r_out's dtype)")
    if (dx is None) != (w_pre is None):
        raise ValueError("dx and w_pre go together")
    if dx is None and dr_out is None:
        raise ValueError("neither dx nor dr_out")
    a, dev = _act(act, z), y.device
    with _on(dev, stream):
        dy, dr = torch.empty_like(y), torch.empty_like(r_out)
        dz, d1, d2 = (None if t is None else torch.empty_like(t)
                      for t in (z, w_post, w_pre))
        ws = _ws(workspace, kda_block_norm_backward_workspace_size(rows, C),
                 dev, "kda_block_norm_backward")
        py, pr, pz, p1, p2, *rest, pk = _ptrs(
            dev, y, r_out, z, w_post, w_pre, dx, dr_out, dy, dr, dz, d1, d2,
            ws)
        st = _block_bwd(py, _dt(y), pr, _dt(r_out), pz, a, p1, p2, res_scale,
                        branch_scale, eps, *rest, rows, C, pk, ws.numel(),
                        _cur(dev))
    _check(st, "kda_block_norm_backward")
    return dy, dr, dz, d1, d2
