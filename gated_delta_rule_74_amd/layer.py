"""Binding of the operators around the KDA mixer (``include/kda.h``): the
gated linear recurrence with a vector state, the gated head norm, and the
norms around a block.  Argument marshalling only, like the package itself.

A call runs on the device of its tensors, on `stream` or else on that device's
current stream; what it allocates belongs to the stream it runs on.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (KDA_BF16, KDA_EUNSUPPORTED, KDA_F32, KDA_GATE_HEAD, KdaError,
               _check, _f, _i, _io_dtype, _need, _sig, _sz, _vp)

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
_CODE = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
_F32 = torch.float32
_INT_MAX = 2 ** 31 - 1
# the handle of a device's current stream without building a Stream object
# (2 us of a decode step's host time)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _act(act, z):
    if act not in _ACTS:
        raise ValueError(f"act: {act!r}, expected one of {sorted(_ACTS)}")
    return 0 if z is None else _ACTS[act]


def _must(t, shape, dtype, name):
    """_need, quick where all is well"""
    if t is not None and (t.shape != shape or t.dtype is not dtype):
        _need(t, shape, dtype, name)


def _int(n, name):
    """a size that the C interface takes as an int: anything above would be
    cut to its lower bits on the way"""
    if n > _INT_MAX:
        raise KdaError(KDA_EUNSUPPORTED, f"{name} = {n}")


def _size(f, *n):
    """The workspace size f(*n); 0 (unsupported) for sizes that the C interface
    would cut to their lower bits."""
    if any(c(v).value != v for c, v in zip(f.argtypes, n)):
        return 0
    return int(f(*n))


def _bad(t, dev):
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"tensors on cuda:{dev} and {t.device}")
    raise ValueError("tensors must be contiguous")


def _ptrs(dev, *ts):
    """Data pointers of tensors (or None) that all live on GPU number
    `dev`."""
    return [None if t is None else
            t.data_ptr() if t.get_device() == dev and t.is_contiguous() else
            _bad(t, dev) for t in ts]


def _elsewhere(t, stream):
    """None where a call on tensor t's device and the current stream can go
    ahead; else the context it has to be made in."""
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if stream is None:
        if t.get_device() == torch.cuda.current_device():
            return None
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream on {stream.device}, tensors on {t.device}")
    return torch.cuda.stream(stream)


def _state(like, shape, x):
    """A new state: like one that is there (1.2 us of host time, not 1.8) or
    None."""
    if like is not None:
        return torch.empty_like(like)
    return torch.empty(shape, dtype=_F32, device=x.device)


def _ws(workspace, need, t, where):
    if need == 0:
        raise KdaError(KDA_EUNSUPPORTED, where)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=t.device)
    if workspace.dtype != torch.uint8:
        raise ValueError(f"workspace: dtype {workspace.dtype}, expected "
                         "uint8")
    return workspace


def _scan_codes(x, g, beta, nd):
    """Check x [*lead, D], g [*lead, D] or [*lead], beta [*lead] or None, with
    nd leading dimensions; returns the dtype codes of x and of the gate."""
    xs = x.shape
    if len(xs) != nd + 1:
        raise ValueError(f"x has {len(xs)} dimensions, expected {nd + 1}")
    _int(max(xs), "size of x")
    io, gt = _CODE.get(x.dtype), _CODE.get(g.dtype)
    if io is None or gt is None:
        _io_dtype(x, "x")
        _io_dtype(g, "g")
    lead = xs[:-1]
    if g.shape != xs:
        if g.dim() == nd + 1:
            _need(g, xs, g.dtype, "g")
        _must(g, lead, g.dtype, "g (per-head gate)")
        gt |= KDA_GATE_HEAD
    _must(beta, lead, g.dtype, "beta (must have g's dtype)")
    return io, gt


@functools.lru_cache(maxsize=256)
def kda_scan_workspace_size(B, T, H, D) -> int:
    return _size(_scan_ws, B, T, H, D)


@functools.lru_cache(maxsize=256)
def kda_scan_backward_workspace_size(B, T, H, D) -> int:
    return _size(_scan_bwd_ws, B, T, H, D)


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
    io, gt = _scan_codes(x, g, beta, 3)
    B, T, H, D = x.shape
    _must(h0, (B, H, D), _F32, "h0")
    _must(h_out, (B, H, D), _F32, "h_out")
    _must(lengths, (B,), torch.int32, "lengths")
    _must(y, x.shape, x.dtype, "y")
    states = (B, -(-T // KDA_SCAN_CHUNK), H, D)
    if chunk_states is not False and chunk_states is not True:
        _must(chunk_states, states, _F32, "chunk_states")
    away = _elsewhere(x, stream)
    if away is not None:
        with away:
            return kda_scan(x, g, beta, h0=h0, lengths=lengths, y=y,
                            h_out=h_out, want_state=want_state,
                            chunk_states=chunk_states, workspace=workspace)
    if y is None:
        y = torch.empty_like(x)
    if h_out is None and want_state:
        h_out = _state(h0, (B, H, D), x)
    if chunk_states is True:
        chunk_states = torch.empty(states, dtype=_F32, device=x.device)
    elif chunk_states is False:
        chunk_states = None
    ws = _ws(workspace, kda_scan_workspace_size(B, T, H, D), x, "kda_scan")
    dev = x.get_device()
    px, pg, *rest, pw = _ptrs(dev, x, g, beta, h0, lengths, y, h_out,
                              chunk_states, ws)
    _check(_scan(px, io, pg, rest[0], gt, *rest[1:], B, T, H, D, pw,
                 ws.numel(), _raw_stream(dev)), "kda_scan")
    return y, h_out, chunk_states


def kda_scan_backward(x, g, beta, dy, *, h0=None, dhT=None, lengths=None,
                      chunk_states=None, want_dh0=True, workspace=None,
                      stream=None):
    """Gradient of kda_scan for the loss sum(y*dy) + sum(h_out*dhT).
    chunk_states: those kda_scan returned for the same inputs (h0 is then not
    read and may have been overwritten), or None (they are recomputed).
    Returns (dx, dg shaped like g, dbeta or None, dh0 or None)."""
    io, gt = _scan_codes(x, g, beta, 3)
    B, T, H, D = x.shape
    _must(dy, x.shape, x.dtype, "dy (must have x's dtype)")
    _must(h0, (B, H, D), _F32, "h0")
    _must(dhT, (B, H, D), _F32, "dhT")
    _must(lengths, (B,), torch.int32, "lengths")
    _must(chunk_states, (B, -(-T // KDA_SCAN_CHUNK), H, D), _F32,
          "chunk_states")
    away = _elsewhere(x, stream)
    if away is not None:
        with away:
            return kda_scan_backward(x, g, beta, dy, h0=h0, dhT=dhT,
                                     lengths=lengths,
                                     chunk_states=chunk_states,
                                     want_dh0=want_dh0, workspace=workspace)
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    dbeta = None if beta is None else torch.empty_like(beta)
    dh0 = _state(h0, (B, H, D), x) if want_dh0 else None
    ws = _ws(workspace, kda_scan_backward_workspace_size(B, T, H, D), x,
             "kda_scan_backward")
    dev = x.get_device()
    px, pg, pb, *rest, pw = _ptrs(dev, x, g, beta, h0, lengths, dy, dhT,
                                  chunk_states, dx, dg, dbeta, dh0, ws)
    _check(_scan_bwd(px, io, pg, pb, gt, *rest, B, T, H, D, pw, ws.numel(),
                     _raw_stream(dev)), "kda_scan_backward")
    return dx, dg, dbeta, dh0


def kda_scan_step(x, g, beta, state, *, y=None, stream=None):
    """One token of kda_scan per sequence: x [N,H,D], g [N,H,D] or [N,H],
    beta [N,H] or None; `state` [N,H,D] fp32 is updated in place.  Returns
    y [N,H,D]."""
    io, gt = _scan_codes(x, g, beta, 2)
    shape = x.shape
    _must(state, shape, _F32, "state")
    _must(y, shape, x.dtype, "y")
    away = _elsewhere(x, stream)
    if away is not None:
        with away:
            return kda_scan_step(x, g, beta, state, y=y)
    if y is None:
        y = torch.empty_like(x)
    dev = x.get_device()
    px, pg, pb, ps, py = _ptrs(dev, x, g, beta, state, y)
    _check(_scan_step(px, io, pg, pb, gt, ps, py, *shape, _raw_stream(dev)),
           "kda_scan_step")
    return y


def _gated_codes(o, z, w):
    """Check o, z [..., D] and w [D]; returns o's dtype code, D and rows."""
    if o.dim() < 1:
        raise ValueError("o has no dimension")
    io, D = _CODE.get(o.dtype), o.shape[-1]
    if io is None:
        _io_dtype(o, "o")
    _int(D, "width of o")
    _must(z, o.shape, o.dtype, "z (must have o's shape and dtype)")
    _must(w, (D,), _F32, "w")
    return io, D, o.numel() // max(D, 1)


def kda_gated_norm(o, z, w, *, act="sigmoid", eps=1e-6, y=None, stream=None):
    """RMS norm of a mixer's heads times a gate:
    y = o / sqrt(mean(o^2) + eps) * w * act(z) over the last dimension.
    o, z [..., D] (z None: no gate), w [D] fp32, act "sigmoid" or "silu"."""
    io, D, rows = _gated_codes(o, z, w)
    _must(y, o.shape, o.dtype, "y")
    a = _act(act, z)
    away = _elsewhere(o, stream)
    if away is not None:
        with away:
            return kda_gated_norm(o, z, w, act=act, eps=eps, y=y)
    if y is None:
        y = torch.empty_like(o)
    dev = o.get_device()
    po, pz, pw, py = _ptrs(dev, o, z, w, y)
    _check(_gated(po, pz, io, pw, a, eps, py, rows, D, _raw_stream(dev)),
           "kda_gated_norm")
    return y


@functools.lru_cache(maxsize=256)
def kda_gated_norm_backward_workspace_size(rows, D) -> int:
    return _size(_gated_ws, rows, D)


def kda_gated_norm_backward(o, z, w, dy, *, act="sigmoid", eps=1e-6,
                            workspace=None, stream=None):
    """Gradient of kda_gated_norm.  Returns (do, dz or None, dw [D] fp32)."""
    io, D, rows = _gated_codes(o, z, w)
    _must(dy, o.shape, o.dtype, "dy (must have o's shape and dtype)")
    a = _act(act, z)
    away = _elsewhere(o, stream)
    if away is not None:
        with away:
            return kda_gated_norm_backward(o, z, w, dy, act=act, eps=eps,
                                           workspace=workspace)
    do, dw = torch.empty_like(o), torch.empty_like(w)
    dz = None if z is None else torch.empty_like(z)
    ws = _ws(workspace, kda_gated_norm_backward_workspace_size(rows, D), o,
             "kda_gated_norm_backward")
    dev = o.get_device()
    po, pz, pw, *rest, pk = _ptrs(dev, o, z, w, dy, do, dz, dw, ws)
    _check(_gated_bwd(po, pz, io, pw, a, eps, *rest, rows, D, pk, ws.numel(),
                      _raw_stream(dev)), "kda_gated_norm_backward")
    return do, dz, dw


def _block_codes(y, r, z, w_post, w_pre, r_name):
    """Check a block's tensors; returns the dtype codes of the block and of
    the stream, C and the rows."""
    shape = y.shape
    if len(shape) < 1:
        raise ValueError("y has no dimension")
    io, rt, C = _CODE.get(y.dtype), _CODE.get(r.dtype), shape[-1]
    if io is None or rt is None:
        _io_dtype(y, "y")
        _io_dtype(r, r_name)
    _must(r, shape, r.dtype, r_name)
    _must(z, shape, y.dtype, "z (must have y's shape and dtype)")
    _must(w_post, (C,), _F32, "w_post")
    _must(w_pre, (C,), _F32, "w_pre")
    rows = y.numel() // max(C, 1)
    _int(max(rows, C), "rows or width of y")
    return io, rt, C, rows


def kda_block_norm(y, r, *, w_post=None, z=None, w_pre=None, act="sigmoid",
                   res_scale=1.0, branch_scale=1.0, eps=1e-6, r_out=None,
                   x=None, stream=None):
    """Between two blocks, over rows of the last dimension C:
    r_out = res_scale r + branch_scale act(z) norm(y; w_post);
    x = norm(r_out; w_pre).
    y the block's output, r the residual stream (its own dtype), z a gate like
    y or None, w_post / w_pre [C] fp32 or None (no norm there; x is then
    None).  r_out may be r.  Returns (r_out, x)."""
    io, rt, C, rows = _block_codes(y, r, z, w_post, w_pre, "r")
    _must(r_out, y.shape, r.dtype, "r_out (must have r's dtype)")
    _must(x, y.shape, y.dtype, "x")
    if x is not None and w_pre is None:
        raise ValueError("x without w_pre")
    a = _act(act, z)
    away = _elsewhere(y, stream)
    if away is not None:
        with away:
            return kda_block_norm(y, r, w_post=w_post, z=z, w_pre=w_pre,
                                  act=act, res_scale=res_scale,
                                  branch_scale=branch_scale, eps=eps,
                                  r_out=r_out, x=x)
    if r_out is None:
        r_out = torch.empty_like(r)
    if x is None and w_pre is not None:
        x = torch.empty_like(y)
    dev = y.get_device()
    py, pr, pz, p1, p2, po, px = _ptrs(dev, y, r, z, w_post, w_pre, r_out, x)
    _check(_block(py, io, pr, rt, pz, a, p1, p2, res_scale, branch_scale, eps,
                  po, px, rows, C, _raw_stream(dev)), "kda_block_norm")
    return r_out, x


@functools.lru_cache(maxsize=256)
def kda_block_norm_backward_workspace_size(rows, C) -> int:
    return _size(_block_ws, rows, C)


def kda_block_norm_backward(y, r_out, *, dx=None, dr_out=None, w_post=None,
                            z=None, w_pre=None, act="sigmoid", res_scale=1.0,
                            branch_scale=1.0, eps=1e-6, workspace=None,
                            stream=None):
    """Gradient of kda_block_norm from the stream r_out it left.  dx (given
    exactly when w_pre is) and dr_out (or None) are the gradients of its
    outputs.  Returns (dy, dr, dz or None, dw_post or None, dw_pre or
    None)."""
    io, rt, C, rows = _block_codes(y, r_out, z, w_post, w_pre, "r_out")
    _must(dx, y.shape, y.dtype, "dx (must have y's dtype)")
    _must(dr_out, y.shape, r_out.dtype, "dr_out (must have r_out's dtype)")
    if (dx is None) != (w_pre is None):
        raise ValueError("dx and w_pre go together")
    if dx is None and dr_out is None:
        raise ValueError("neither dx nor dr_out")
    a = _act(act, z)
    away = _elsewhere(y, stream)
    if away is not None:
        with away:
            return kda_block_norm_backward(
                y, r_out, dx=dx, dr_out=dr_out, w_post=w_post, z=z,
                w_pre=w_pre, act=act, res_scale=res_scale,
                branch_scale=branch_scale, eps=eps, workspace=workspace)
    dy, dr = torch.empty_like(y), torch.empty_like(r_out)
    dz, d1, d2 = (None if t is None else torch.empty_like(t)
                  for t in (z, w_post, w_pre))
    ws = _ws(workspace, kda_block_norm_backward_workspace_size(rows, C), y,
             "kda_block_norm_backward")
    dev = y.get_device()
    py, pr, pz, p1, p2, *rest, pk = _ptrs(
        dev, y, r_out, z, w_post, w_pre, dx, dr_out, dy, dr, dz, d1, d2, ws)
    _check(_block_bwd(py, io, pr, rt, pz, a, p1, p2, res_scale, branch_scale,
                      eps, *rest, rows, C, pk, ws.numel(), _raw_stream(dev)),
           "kda_block_norm_backward")
    return dy, dr, dz, d1, d2
