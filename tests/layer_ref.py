"""64-bit references of the layer operators (scan, gated head norm, norms
around a block), with the error that their fp32 evaluation may have.

Every reference returns (value, slack) pairs: `slack` bounds, element by
element, the distance of any fp32 evaluation in a sensible order from the
value, derived from magnitudes.  A result that is then rounded to a type t may
be off by a further half step, finfo(t).eps / 2 of its value (see `within`).

u = 2^-24 is the rounding of one fp32 operation.

Scan.  A token costs at most: the exp (1.5 ulp = 3u of a), the product into the
composed decay (u), the multiply-add (u), the product beta x (u), and below
one more for the composition of maps over groups of tokens: 8u of the
magnitudes covers it.  With |h|_t = a |h|_{t-1} + |u_t| (all terms positive),
the error obeys E_t <= a E_{t-1} + 8u |h|_t; the gradient's likewise, last to
first.
Sums of n terms in any order: n u of the sum of magnitudes.

Norms.  A sum of C squares is off by (C + 2)u of itself, its inverse root by
half of that and 4u; a gate by (|z| + 8) 2u (the hardware exponential's
argument is off by |z| u, and its result, the sum and the reciprocal by a few
u); every further product by u.  `_rel` collects them.
"""
import torch

U = 2.0 ** -24
F8 = torch.float64


def half(dtype):
    return torch.finfo(dtype).eps / 2


def within(name, got, ref, dtype=None):
    """got (of the kernel) against (value, slack), element by element."""
    want, slack = ref
    got = got.detach().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    r = half(dtype or got.dtype)
    tol = slack + r * (want.abs() + slack) + 1e-37
    err = (got.to(F8) - want).abs()
    bad = ~(err <= tol)  # NaN counts as bad
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err / tol, err * 0)
                             .nan_to_num(nan=1e30)))
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at flat "
            f"{i}: got {got.flatten()[i].item()}, want "
            f"{want.flatten()[i].item()}, tolerance {tol.flatten()[i].item()}")


def c8(t):
    return None if t is None else t.detach().cpu().to(F8)


def scan(x, g, beta=None, h0=None, lengths=None, dy=None, dhT=None):
    """dict of (value, slack): y, h, chunk (states before chunks of 128) and,
    with dy, dx, dg, dbeta, dh0.  x [B,T,H,D]."""
    x, g, beta, h0, dy, dhT = map(c8, (x, g, beta, h0, dy, dhT))
    B, T, H, D = x.shape
    head = g.dim() == 3
    a = torch.exp(g.unsqueeze(-1) if head else g).expand(B, T, H, D).clone()
    n = (torch.full((B,), T) if lengths is None
         else lengths.cpu().long().clamp(0, T))
    live = (torch.arange(T)[None] < n[:, None])[:, :, None, None]
    live = live.expand(B, T, H, D)
    b = torch.ones(B, T, H, 1, dtype=F8) if beta is None \
        else beta.unsqueeze(-1)
    zero = torch.zeros((), dtype=F8)
    a = torch.where(live, a, torch.ones((), dtype=F8))
    u = torch.where(live, b * x, zero)
    h = torch.zeros(B, H, D, dtype=F8) if h0 is None else h0
    m, e = h.abs(), torch.zeros_like(h)
    hs, ms, es, cs, ces = [], [], [], [], []
    for t in range(T):
        if t % 128 == 0:
            cs.append(h)
            ces.append(e)
        h = a[:, t] * h + u[:, t]
        m = a[:, t] * m + u[:, t].abs()
        e = a[:, t] * e + 8 * U * m
        hs.append(h)
        ms.append(m)
        es.append(e)
    hs, ms, es = (torch.stack(v, 1) for v in (hs, ms, es))
    out = dict(y=(torch.where(live, hs, zero), torch.where(live, es, zero)),
               h=(h, e), chunk=(torch.stack(cs, 1), torch.stack(ces, 1)))
    if dy is None:
        return out
    dy = torch.where(live, dy, zero)
    x = torch.where(live, x, zero)
    d = torch.zeros(B, H, D, dtype=F8) if dhT is None else dhT
    dm, de = d.abs(), torch.zeros_like(d)
    dh = torch.zeros_like(x)
    dhm, dhe = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T - 1, -1, -1):
        dh[:, t] = dy[:, t] + d
        dhm[:, t] = dy[:, t].abs() + dm
        dhe[:, t] = de + 8 * U * dhm[:, t]
        d = a[:, t] * dh[:, t]
        dm = a[:, t] * dhm[:, t]
        de = a[:, t] * dhe[:, t]
    out["dh0"] = (d, de + 8 * U * dm)
    s0 = torch.zeros(B, 1, H, D, dtype=F8) if h0 is None else h0[:, None]
    hp = torch.cat([s0, hs[:, :-1]], 1)
    mp = torch.cat([s0.abs(), ms[:, :-1]], 1)
    ep = torch.cat([torch.zeros_like(s0), es[:, :-1]], 1)
    dh, dhm, dhe = (torch.where(live, v, zero) for v in (dh, dhm, dhe))
    bb = torch.where(live[..., :1], b, zero)
    out["dx"] = (bb * dh, bb.abs() * dhe + 4 * U * bb.abs() * dhm)
    dg = dh * a * hp
    dge = a * (dhe * (mp + ep) + dhm * ep) + 8 * U * dhm * a * mp
    if head:
        dge = dge.sum(-1) + D * U * (dhm * a * mp).sum(-1)
        dg = dg.sum(-1)
    out["dg"] = (dg, dge)
    if beta is not None:
        out["dbeta"] = ((dh * x).sum(-1),
                        (dhe * x.abs() + (D + 4) * U * dhm * x.abs()).sum(-1))
    return out


def gate(z, act):
    """gate, derivative, magnitude of the derivative's terms, relative
    error"""
    if z is None:
        return None
    s = torch.sigmoid(z)
    m = torch.sigmoid(z) * torch.sigmoid(-z)
    rel = (z.abs() + 8) * 2 * U
    # 1 - s is off by u where s rounds to nearly one
    if act == "sigmoid":
        return s, m, m + s * U / rel, rel
    return z * s, s + z * m, s + z.abs() * (m + s * U / rel), rel


def _rms(v, eps):
    C = v.shape[-1]
    return 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps), \
        (C / 2 + 8) * U


def _norm_grad(v, r, rr, t, te):
    """gradient of v r for r = _rms(v) (relative error rr), and its slack;
    te: slack of t"""
    C = v.shape[-1]
    n = v * r
    m = (t * n).mean(-1, keepdim=True)
    am = (t * n).abs().mean(-1, keepdim=True)
    ame = (te * n.abs()).mean(-1, keepdim=True) + (2 * rr + (C + 4) * U) * am
    val = r * (t - n * m)
    slack = r * (te + n.abs() * ame) + \
        (2 * rr + 6 * U) * r * (t.abs() + n.abs() * am)
    return val, slack


def gated_norm(o, z, w, act, eps, dy=None):
    """y, or with dy (do, dz, dw), as (value, slack)."""
    o, z, w, dy = map(c8, (o, z, w, dy))
    r, rr = _rms(o, eps)
    g = gate(z, act)
    rel = rr + 6 * U
    if dy is None:
        y = o * r * w
        if g is not None:
            y, rel = y * g[0], rel + g[3]
        return y, rel * y.abs()
    n = o * r
    t, te = dy, torch.zeros_like(dy)
    dz = None
    if g is not None:
        t = dy * g[0]
        te = (g[3] + 2 * U) * t.abs()
        v = dy * n * w
        dz = (v * g[1], (rr + g[3] + 8 * U) * v.abs() * g[2])
    rows = o.numel() // o.shape[-1]
    lead = tuple(range(o.dim() - 1))
    dw = ((t * n).sum(lead),
          (te * n.abs() + (rr + 4 * U + rows * U) * (t * n).abs()).sum(lead))
    do = _norm_grad(o, r, rr, t * w, te * w.abs() + 2 * U * (t * w).abs())
    return do, dz, dw


def block_norm(y, r, w_post, z, w_pre, act, rs, bs, eps):
    """(r_out, x), each (value, slack) or None"""
    y, r, w_post, z, w_pre = map(c8, (y, r, w_post, z, w_pre))
    u, rel = y, 4 * U
    if w_post is not None:
        r1, rr = _rms(y, eps)
        u, rel = u * r1 * w_post, rel + rr + 2 * U
    g = gate(z, act)
    if g is not None:
        u, rel = u * g[0], rel + g[3]
    h = rs * r + bs * u
    he = abs(bs) * rel * u.abs() + 4 * U * ((rs * r).abs() + (bs * u).abs())
    if w_pre is None:
        return (h, he), None
    r2, rr = _rms(h, eps)
    # the root mean square moves by at most the root mean square of the error
    hr = he.square().mean(-1, keepdim=True).sqrt() * r2
    x = h * r2 * w_pre
    return (h, he), (x, r2 * w_pre.abs() * he + (rr + hr + 6 * U) * x.abs())


def block_norm_grad(y, r, dx, dr_out, w_post, z, w_pre, act, rs, bs, eps):
    """(dy, dr, dz, dw_post, dw_pre), each (value, slack) or None; r: the
    stream the forward left"""
    y, r, dx, dr_out, w_post, z, w_pre = map(
        c8, (y, r, dx, dr_out, w_post, z, w_pre))
    R = y.numel() // y.shape[-1]
    lead = tuple(range(y.dim() - 1))
    d = torch.zeros_like(r) if dr_out is None else dr_out
    de = torch.zeros_like(d)
    dz = dw_post = dw_pre = None
    if dx is not None:
        r2, rr = _rms(r, eps)
        t = dx * w_pre
        v, ve = _norm_grad(r, r2, rr, t, 2 * U * t.abs())
        dw = dx * r * r2
        dw_pre = (dw.sum(lead), (rr + 4 * U + R * U) * dw.abs().sum(lead))
        de = ve + 2 * U * (d.abs() + v.abs())
        d = d + v
    dr = (rs * d, abs(rs) * (de + 2 * U * d.abs()))
    du, due = bs * d, abs(bs) * (de + 2 * U * d.abs())
    n, nr = y, 0.0
    if w_post is not None:
        r1, rr = _rms(y, eps)
        n, nr = y * r1, rr + 2 * U
    w = 1.0 if w_post is None else w_post
    g = gate(z, act)
    if g is not None:
        v = du * n * w
        dz = (v * g[1], ((n * w).abs() * due + (nr + g[3] + 8 * U) * v.abs())
              * g[2])
        du, due = du * g[0], g[0].abs() * due + (g[3] + 2 * U) * \
            (du * g[0]).abs()
    if w_post is None:
        return (du, due), dr, dz, None, dw_pre
    dw_post = ((du * n).sum(lead),
               (due * n.abs() + (nr + 4 * U + R * U) * (du * n).abs())
               .sum(lead))
    dy = _norm_grad(y, r1, rr, du * w, due * w.abs() + 2 * U * (du * w).abs())
    return dy, dr, dz, dw_post, dw_pre
