"""Binding of linear attention with one decay per head and of the norm and
rotation of queries and keys (``include/kda.h``).  Argument marshalling only;
devices, streams and what is allocated as in ``layer.py``.
"""
from __future__ import annotations

import functools

import torch

from . import _check, _f, _i, _io_dtype, _need, _sig, _sz, _vp
from .layer import (_CODE, _F32, _elsewhere, _int, _ll, _must, _ptrs,
                    _raw_stream, _size, _state, _ws)

KDA_GATE_FIXED = 32  # gate-dtype flag: g holds one log-decay per head, [H]

_lin = _sig("kda_linattn", _i,
            [_vp] * 3 + [_i, _vp, _i] + [_vp] * 4 + [_i] * 6 +
            [_f, _vp, _sz, _vp])
_lin_bwd = _sig("kda_linattn_backward", _i,
                [_vp] * 3 + [_i, _vp, _i] + [_vp] * 9 + [_i] * 6 +
                [_f, _vp, _sz, _vp])
_lin_step = _sig("kda_linattn_step", _i,
                 [_vp] * 3 + [_i, _vp, _i, _vp, _vp] + [_i] * 5 + [_f, _vp])
_lin_ws = _sig("kda_linattn_workspace_size", _sz, [_i] * 7)
_lin_bwd_ws = _sig("kda_linattn_backward_workspace_size", _sz, [_i] * 7)
_qk = _sig("kda_qk_norm_rope", _i,
           [_vp, _vp, _i, _ll, _ll] + [_vp] * 4 + [_i, _i, _f, _vp, _vp] +
           [_ll] * 3 + [_i] * 3 + [_vp])
_qk_bwd = _sig("kda_qk_norm_rope_backward", _i,
               [_vp, _vp, _i, _ll, _ll] + [_vp] * 4 + [_i, _i, _f, _vp, _vp,
                                                        _ll, _ll, _vp, _vp,
                                                        _ll, _ll, _vp, _vp,
                                                        _ll] +
               [_i] * 3 + [_vp, _sz, _vp])
_qk_bwd_ws = _sig("kda_qk_norm_rope_backward_workspace_size", _sz,
                  [_ll] + [_i] * 3)


def _lin_codes(q, k, v, g, nd):
    """Check q, k [*lead, Hk, Dk], v [*lead, H, Dv] and g [*lead, H] or [H]
    with nd leading dimensions; returns the dtype codes of q and of the gate
    and Hk, H, Dk, Dv."""
    qs, vs = q.shape, v.shape
    if len(qs) != nd + 2 or len(vs) != nd + 2:
        raise ValueError(f"q has {len(qs)} dimensions and v {len(vs)}, "
                         f"expected {nd + 2}")
    _int(max(max(qs), max(vs)), "size of q or v")
    io, gt = _CODE.get(q.dtype), _CODE.get(g.dtype)
    if io is None or gt is None:
        _io_dtype(q, "q")
        _io_dtype(g, "g")
    _must(k, qs, q.dtype, "k (must have q's shape and dtype)")
    if vs[:nd] != qs[:nd] or v.dtype is not q.dtype:
        _need(v, (*qs[:nd], *vs[nd:]), q.dtype, "v (must go with q)")
    if g.dim() == 1:
        _must(g, (vs[nd],), g.dtype, "g (one decay per head)")
        gt |= KDA_GATE_FIXED
    else:
        _must(g, vs[:-1], g.dtype, "g")
    return io, gt, qs[nd], vs[nd], qs[nd + 1], vs[nd + 1]


@functools.lru_cache(maxsize=256)
def kda_linattn_workspace_size(B, T, Hk, H, Dk, Dv, dtype) -> int:
    return _size(_lin_ws, B, T, Hk, H, Dk, Dv, _CODE.get(dtype, dtype))


@functools.lru_cache(maxsize=256)
def kda_linattn_backward_workspace_size(B, T, Hk, H, Dk, Dv, dtype) -> int:
    return _size(_lin_bwd_ws, B, T, Hk, H, Dk, Dv, _CODE.get(dtype, dtype))


def kda_linattn(q, k, v, g, *, s0=None, lengths=None, scale=1.0, o=None,
                s_out=None, want_state=True, workspace=None, stream=None):
    """S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over
    sequences.

    q, k [B,T,Hk,Dk]; v [B,T,H,Dv] with H a multiple of Hk (value head h has
    the queries and keys of head h // (H // Hk)); g [B,T,H], or [H] for a
    decay that every token of a head shares; s0 [B,H,Dk,Dv] fp32 or None
    (zeros); lengths [B] int32 on the GPU or None: tokens from lengths[b] on
    leave the state alone and give zeros.  s_out may be s0.  Returns
    (o [B,T,H,Dv], state after the last token [B,H,Dk,Dv] fp32 or None)."""
    io, gt, Hk, H, Dk, Dv = _lin_codes(q, k, v, g, 2)
    B, T = q.shape[:2]
    S = (B, H, Dk, Dv)
    _must(s0, S, _F32, "s0")
    _must(s_out, S, _F32, "s_out")
    _must(lengths, (B,), torch.int32, "lengths")
    _must(o, v.shape, v.dtype, "o")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return kda_linattn(q, k, v, g, s0=s0, lengths=lengths,
                               scale=scale, o=o, s_out=s_out,
                               want_state=want_state, workspace=workspace)
    ws = _ws(workspace,
             kda_linattn_workspace_size(B, T, Hk, H, Dk, Dv, io), q,
             "kda_linattn")
    if o is None:
        o = torch.empty_like(v)
    if s_out is None and want_state:
        s_out = _state(s0, S, q)
    dev = q.get_device()
    pq, pk, pv, pg, *rest, pw = _ptrs(dev, q, k, v, g, s0, lengths, o, s_out,
                                      ws)
    _check(_lin(pq, pk, pv, io, pg, gt, *rest, B, T, Hk, H, Dk, Dv, scale, pw,
                ws.numel(), _raw_stream(dev)), "kda_linattn")
    return o, s_out


def kda_linattn_backward(q, k, v, g, do, *, s0=None, dsT=None, lengths=None,
                         scale=1.0, want_dg=True, want_ds0=True,
                         workspace=None, stream=None):
    """Gradient of kda_linattn for the loss sum(o*do) + sum(s_out*dsT).
    Returns (dq, dk, dv, dg shaped like g or None, ds0 or None)."""
    io, gt, Hk, H, Dk, Dv = _lin_codes(q, k, v, g, 2)
    B, T = q.shape[:2]
    S = (B, H, Dk, Dv)
    _must(do, v.shape, v.dtype, "do (must have v's shape and dtype)")
    _must(s0, S, _F32, "s0")
    _must(dsT, S, _F32, "dsT")
    _must(lengths, (B,), torch.int32, "lengths")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return kda_linattn_backward(
                q, k, v, g, do, s0=s0, dsT=dsT, lengths=lengths, scale=scale,
                want_dg=want_dg, want_ds0=want_ds0, workspace=workspace)
    ws = _ws(workspace,
             kda_linattn_backward_workspace_size(B, T, Hk, H, Dk, Dv, io), q,
             "kda_linattn_backward")
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    dg = torch.empty_like(g) if want_dg else None
    ds0 = _state(s0, S, q) if want_ds0 else None
    dev = q.get_device()
    pq, pk, pv, pg, *rest, pw = _ptrs(dev, q, k, v, g, s0, lengths, do, dsT,
                                      dq, dk, dv, dg, ds0, ws)
    _check(_lin_bwd(pq, pk, pv, io, pg, gt, *rest, B, T, Hk, H, Dk, Dv, scale,
                    pw, ws.numel(), _raw_stream(dev)), "kda_linattn_backward")
    return dq, dk, dv, dg, ds0


def kda_linattn_step(q, k, v, g, state, *, scale=1.0, o=None, stream=None):
    """One token of kda_linattn per sequence: q, k [N,Hk,Dk], v [N,H,Dv],
    g [N,H] or [H]; `state` [N,H,Dk,Dv] fp32 is updated in place.  Returns
    o [N,H,Dv]."""
    io, gt, Hk, H, Dk, Dv = _lin_codes(q, k, v, g, 1)
    N = q.shape[0]
    _must(state, (N, H, Dk, Dv), _F32, "state")
    _must(o, v.shape, v.dtype, "o")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return kda_linattn_step(q, k, v, g, state, scale=scale, o=o)
    if o is None:
        o = torch.empty_like(v)
    dev = q.get_device()
    pq, pk, pv, pg, ps, po = _ptrs(dev, q, k, v, g, state, o)
    _check(_lin_step(pq, pk, pv, io, pg, gt, ps, po, N, Hk, H, Dk, Dv, scale,
                     _raw_stream(dev)), "kda_linattn_step")
    return o


def _token_stride(shape, st, name):
    """Values from token to token of a tensor [..., H, D] with these strides,
    whose last two dimensions are dense and whose others are one range of
    evenly spaced tokens."""
    if (st[-1] != 1 and shape[-1] != 1) or (st[-2] != shape[-1] and
                                            shape[-2] != 1):
        raise ValueError(f"{name}: the heads of a token must be dense")
    step = want = None
    for n, s in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != want:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        want = s * n
    return shape[-2] * shape[-1] if step is None else step


def _layout(t):
    """shape, strides and dtype of a tensor or None"""
    return None if t is None else (t.shape, t.stride(), t.dtype)


@functools.lru_cache(maxsize=1024)
def _qk_plan(q, k, positions, inv_freq, wq, wk, *more):
    """The sizes of a call from its tensors' layouts (kept for the layouts that
    came before: the checks take 6 us of a decode step's host time): dtype
    code, rows, Hq, Hk, D, rot, then the token strides of q, k and of `more`,
    (name, layout) of tensors shaped like q and k in turn."""
    def need(what, shape, dtype, name):
        if what is not None:
            if tuple(what[0]) != tuple(shape):
                raise ValueError(f"{name}: shape {tuple(what[0])}, expected "
                                 f"{tuple(shape)}")
            if what[2] != dtype:
                raise ValueError(f"{name}: dtype {what[2]}, expected {dtype}")

    qs, _, dtype = q
    if len(qs) < 3:
        raise ValueError(f"q has {len(qs)} dimensions, expected at least 3")
    lead, Hq, D = qs[:-2], qs[-2], qs[-1]
    io = _CODE.get(dtype)
    if io is None:
        raise ValueError(f"q: dtype {dtype}, expected float32 or bfloat16")
    Hk = 0
    if k is not None:
        Hk = k[0][-2] if len(k[0]) > 1 else 0
        need(k, (*lead, Hk, D), dtype, "k (must go with q)")
    elif wk is not None:
        raise ValueError("wk without k")
    need(wq, (D,), _F32, "wq")
    need(wk, (D,), _F32, "wk")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    rot = 0
    if inv_freq is not None:
        if len(inv_freq[0]) != 1:
            raise ValueError("inv_freq has one dimension")
        rot = 2 * inv_freq[0][0]
        if rot == 0:
            raise ValueError("inv_freq is empty")
        need(inv_freq, (rot // 2,), _F32, "inv_freq")
        need(positions, lead, torch.int32, "positions")
    rows = 1
    for n in lead:
        rows *= n
    _int(max(Hq, Hk, D, rot), "size of q or k")
    strides = [_token_stride(qs, q[1], "q"),
               0 if k is None else _token_stride(k[0], k[1], "k")]
    for i, (name, t) in enumerate(more):
        like = k if i % 2 else q
        if t is None:
            strides.append(like and like[0][-2] * D or 0)  # a new, dense one
        elif like is None:
            raise ValueError(f"{name} without k")
        else:
            need(t, like[0], dtype, name)
            strides.append(_token_stride(t[0], t[1], name))
    return (io, rows, Hq, Hk, D, rot), tuple(strides)


def _pointer(t, dev, name):
    """a strided tensor's data pointer (or None), on GPU number `dev`"""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} on {t.device}, expected cuda:{dev}")
    return t.data_ptr()


def _dense(like):
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def kda_qk_norm_rope(q, k, positions, inv_freq, *, wq=None, wk=None, eps=1e-6,
                     interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head (x / sqrt(mean(x^2) + eps) * w)
    and the rotation of the first 2 * len(inv_freq) channels by
    position * inv_freq, in one pass.

    q [..., Hq, D], k [..., Hk, D] or None; positions [...] int32 and
    inv_freq [rot / 2] fp32, or None for both (no rotation); wq, wk [D] fp32
    or None (that side is not normed).  Pairs are channels i and i + rot / 2,
    or with interleaved 2 i and 2 i + 1.  The heads of a token are dense;
    tokens may be apart, as parts of a fused projection are.  q_out, k_out may
    be q, k.  Returns (q_out, k_out or None)."""
    (io, rows, Hq, Hk, D, rot), (sq, sk, so, sko) = _qk_plan(
        _layout(q), _layout(k), _layout(positions), _layout(inv_freq),
        _layout(wq), _layout(wk), ("q_out", _layout(q_out)),
        ("k_out", _layout(k_out)))
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return kda_qk_norm_rope(q, k, positions, inv_freq, wq=wq, wk=wk,
                                    eps=eps, interleaved=interleaved,
                                    q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = _dense(q)
    if k_out is None and k is not None:
        k_out = _dense(k)
    dev = q.get_device()
    p1, p2, pp, pf = _ptrs(dev, wq, wk, positions, inv_freq)
    _check(_qk(q.data_ptr(), _pointer(k, dev, "k"), io, sq, sk, p1, p2, pp, pf,
               rot, 1 if interleaved else 0, eps,
               _pointer(q_out, dev, "q_out"), _pointer(k_out, dev, "k_out"),
               so, sko, rows, Hq, Hk, D, _raw_stream(dev)),
           "kda_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def kda_qk_norm_rope_backward_workspace_size(rows, Hq, Hk, D) -> int:
    return _size(_qk_bwd_ws, rows, Hq, Hk, D)


def kda_qk_norm_rope_backward(q, k, positions, inv_freq, dq_out, dk_out, *,
                              wq=None, wk=None, eps=1e-6, interleaved=False,
                              dq=None, dk=None, workspace=None, stream=None):
    """Gradient of kda_qk_norm_rope from the same inputs.  dq, dk: tensors to
    write the gradients into (as parts of a fused projection's, or dq_out and
    dk_out themselves), or None for new ones.  Returns (dq, dk or None,
    dwq [D] fp32 or None, dwk or None)."""
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    if dq_out is None:
        raise ValueError("dq_out is missing")
    (io, rows, Hq, Hk, D, rot), (sq, sk, so, sko, s1, s2) = _qk_plan(
        _layout(q), _layout(k), _layout(positions), _layout(inv_freq),
        _layout(wq), _layout(wk), ("dq_out", _layout(dq_out)),
        ("dk_out", _layout(dk_out)), ("dq", _layout(dq)),
        ("dk", _layout(dk)))
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return kda_qk_norm_rope_backward(
                q, k, positions, inv_freq, dq_out, dk_out, wq=wq, wk=wk,
                eps=eps, interleaved=interleaved, dq=dq, dk=dk,
                workspace=workspace)
    ws = _ws(workspace,
             kda_qk_norm_rope_backward_workspace_size(rows, Hq, Hk, D), q,
             "kda_qk_norm_rope_backward")
    if dq is None:
        dq = _dense(q)
    if dk is None and k is not None:
        dk = _dense(k)
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (wq, wk))
    dev = q.get_device()
    p1, p2, pp, pf, g1, g2, pw = _ptrs(dev, wq, wk, positions, inv_freq, dwq,
                                       dwk, ws)
    _check(_qk_bwd(q.data_ptr(), _pointer(k, dev, "k"), io, sq, sk, p1, p2, pp,
                   pf, rot, 1 if interleaved else 0, eps,
                   _pointer(dq_out, dev, "dq_out"),
                   _pointer(dk_out, dev, "dk_out"), so, sko,
                   _pointer(dq, dev, "dq"), _pointer(dk, dev, "dk"), s1, s2,
                   g1, g2, rows, Hq, Hk, D, pw, ws.numel(), _raw_stream(dev)),
           "kda_qk_norm_rope_backward")
    return dq, dk, dwq, dwk
