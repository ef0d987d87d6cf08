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


def _token_stride(t, name):
    """Values from token to token of t [..., H, D], whose last two dimensions
    are dense and whose others are one range of evenly spaced tokens."""
    if t.is_contiguous():
        return t.shape[-2] * t.shape[-1]
    shape, st = t.shape, t.stride()
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


def _qk_codes(q, k, positions, inv_freq, wq, wk):
    """Check the inputs; returns the dtype code, rows, Hq, Hk, D and rot."""
    if q.dim() < 3:
        raise ValueError(f"q has {q.dim()} dimensions, expected at least 3")
    lead, Hq, D = q.shape[:-2], q.shape[-2], q.shape[-1]
    io = _CODE.get(q.dtype)
    if io is None:
        _io_dtype(q, "q")
    Hk = 0
    if k is not None:
        if k.shape[:-2] != lead or k.shape[-1] != D or \
                k.dtype is not q.dtype or k.dim() != q.dim():
            _need(k, (*lead, k.shape[-2] if k.dim() > 1 else 0, D), q.dtype,
                  "k (must go with q)")
        Hk = k.shape[-2]
    elif wk is not None:
        raise ValueError("wk without k")
    _must(wq, (D,), _F32, "wq")
    _must(wk, (D,), _F32, "wk")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq has one dimension")
        rot = 2 * inv_freq.shape[0]
        if rot == 0:
            raise ValueError("inv_freq is empty")
        _must(inv_freq, (rot // 2,), _F32, "inv_freq")
        _must(positions, lead, torch.int32, "positions")
    rows = 1
    for n in lead:
        rows *= n
    _int(max(Hq, Hk, D, rot), "size of q or k")
    return io, rows, Hq, Hk, D, rot


def _strided(dev, *ts):
    """Data pointers and token strides of tensors (or None) on GPU `dev`."""
    ptrs, steps = [], []
    for t, name in ts:
        if t is None:
            ptrs.append(None)
            steps.append(0)
            continue
        if t.get_device() != dev:
            raise ValueError(f"{name} on {t.device}, expected cuda:{dev}")
        steps.append(_token_stride(t, name))
        ptrs.append(t.data_ptr())
    return ptrs, steps


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
    io, rows, Hq, Hk, D, rot = _qk_codes(q, k, positions, inv_freq, wq, wk)
    _must(q_out, q.shape, q.dtype, "q_out")
    if k is not None:
        _must(k_out, k.shape, k.dtype, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return kda_qk_norm_rope(q, k, positions, inv_freq, wq=wq, wk=wk,
                                    eps=eps, interleaved=interleaved,
                                    q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None and k is not None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    dev = q.get_device()
    (pq, pk, po, ko), (sq, sk, so, sko) = _strided(
        dev, (q, "q"), (k, "k"), (q_out, "q_out"), (k_out, "k_out"))
    p1, p2, pp, pf = _ptrs(dev, wq, wk, positions, inv_freq)
    _check(_qk(pq, pk, io, sq, sk, p1, p2, pp, pf, rot, int(bool(interleaved)),
               eps, po, ko, so, sko, rows, Hq, Hk, D, _raw_stream(dev)),
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
    io, rows, Hq, Hk, D, rot = _qk_codes(q, k, positions, inv_freq, wq, wk)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    if dk is not None and k is None:
        raise ValueError("dk without k")
    _need(dq_out, q.shape, q.dtype, "dq_out (must have q's shape and dtype)")
    _must(dq, q.shape, q.dtype, "dq")
    if k is not None:
        _must(dk_out, k.shape, k.dtype, "dk_out (must have k's shape and "
              "dtype)")
        _must(dk, k.shape, k.dtype, "dk")
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
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if dk is None and k is not None:
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (wq, wk))
    dev = q.get_device()
    (pq, pk, po, ko, d1, d2), (sq, sk, so, sko, s1, s2) = _strided(
        dev, (q, "q"), (k, "k"), (dq_out, "dq_out"), (dk_out, "dk_out"),
        (dq, "dq"), (dk, "dk"))
    p1, p2, pp, pf, g1, g2, pw = _ptrs(dev, wq, wk, positions, inv_freq, dwq,
                                       dwk, ws)
    _check(_qk_bwd(pq, pk, io, sq, sk, p1, p2, pp, pf, rot,
                   int(bool(interleaved)), eps, po, ko, so, sko, d1, d2, s1,
                   s2, g1, g2, rows, Hq, Hk, D, pw, ws.numel(),
                   _raw_stream(dev)), "kda_qk_norm_rope_backward")
    return dq, dk, dwq, dwk
