"""64-bit references of linear attention with one decay per head and of the
norm and rotation of queries and keys, as (value, slack) pairs (see
``layer_ref``: `slack` bounds what an evaluation in the kernels' precision may
be off, element by element, before the result's own rounding).

Linear attention.  Every result is a sum of products that the recurrences over
magnitudes, M_t = a_t M_{t-1} + |k_t| |v_t|^T and N_t = |scale q_t| |do_t|^T +
a_{t+1} N_{t+1}, add up with their signs off.  A term's weight is a product of
decays over chunks of at least 32 tokens: one chunk's decay exp2(d) is off by
(0.7 |ln decay| + 3) u, the |ln|s add up to 88 before the weight is 0 in fp32,
and every chunk boundary costs at most 8 roundings; products over channels
and sums over a chunk's 64 tokens cost a rounding per term.  So `kappa` times
the magnitudes covers fp32 evaluation.  With bf16 data,
- the pair products and the state are rounded to bf16 where they enter o, dq,
  dk and dv: 2^-8 of the magnitudes;
- the state and the gate's gradient are made of two-part operands, whose rest
  is half a step of half a step: 2^-17 and (two states) 2^-16.
The gate's gradient takes the sum over the pairs across a chunk's end from that
across its start, so what those are off stays: 2 <N, M> at every boundary
behind the token is added to its magnitude.
"""
import torch

from layer_ref import F8, U, c8, _norm_grad, _rms


def _live(lengths, B, T):
    n = torch.full((B,), T) if lengths is None \
        else lengths.cpu().long().clamp(0, T)
    return torch.arange(T)[None] < n[:, None]


def linattn(q, k, v, g, s0=None, lengths=None, scale=1.0, do=None, dsT=None):
    """dict of (value, slack): o, s and, with do, dq, dk, dv, dg, ds0."""
    bf = q.dtype == torch.bfloat16
    q, k, v, g, s0, do, dsT = map(c8, (q, k, v, g, s0, do, dsT))
    B, T, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    G = H // Hk
    fixed = g.dim() == 1
    kappa = (256 + 8 * -(-T // 32) + 2 * (Dk + Dv)) * U
    r, s_r, g_r = (2.0 ** -8, 2.0 ** -17, 2.0 ** -16) if bf else (0, 0, 0)
    live = _live(lengths, B, T)
    zero = torch.zeros((), dtype=F8)
    a = torch.exp(g).expand(B, T, H)
    a = torch.where(live[..., None], a, torch.ones((), dtype=F8))
    dead = ~live[..., None, None]
    q, k = (torch.where(dead, zero, x.repeat_interleave(G, 2))
            for x in (q, k))
    v = torch.where(dead, zero, v)
    S = torch.zeros(B, H, Dk, Dv, dtype=F8) if s0 is None else s0
    M = S.abs()
    Ss, Ms, o, oe = [S], [M], [], []
    for t in range(T):
        A = a[:, t, :, None, None]
        S = A * S + k[:, t].unsqueeze(-1) * v[:, t].unsqueeze(-2)
        M = A * M + k[:, t].abs().unsqueeze(-1) * v[:, t].abs().unsqueeze(-2)
        Ss.append(S)
        Ms.append(M)
        o.append(scale * (q[:, t].unsqueeze(-1) * S).sum(-2))
        oe.append((r + kappa) * abs(scale) *
                  (q[:, t].abs().unsqueeze(-1) * M).sum(-2))
    out = dict(o=(torch.stack(o, 1), torch.stack(oe, 1)),
               s=(S, (kappa + s_r) * M))
    if do is None:
        return out
    do = scale * torch.where(dead, zero, do)
    dS = torch.zeros_like(S) if dsT is None else dsT
    N = dS.abs()
    res = {n: [None] * T for n in ("dq", "dk", "dv", "dg")}
    # what the sums across chunk boundaries behind a token may be off
    stay = torch.zeros(B, H, dtype=F8)
    for t in range(T - 1, -1, -1):
        if (t + 1) % 32 == 0 or t == T - 1:
            stay = stay + 2 * (N * Ms[t + 1]).sum((-1, -2))
        dS = dS + q[:, t].unsqueeze(-1) * do[:, t].unsqueeze(-2)
        N = N + q[:, t].abs().unsqueeze(-1) * do[:, t].abs().unsqueeze(-2)
        c = r + kappa

        def over(x, y, dim, w):
            return (x * w).sum(dim), c * (y * w.abs()).sum(dim)

        res["dq"][t] = over(Ss[t + 1], Ms[t + 1], -1, do[:, t].unsqueeze(-2))
        res["dk"][t] = over(dS, N, -1, v[:, t].unsqueeze(-2))
        res["dv"][t] = over(dS, N, -2, k[:, t].unsqueeze(-1))
        A = a[:, t, :, None, None]
        dS, N = A * dS, A * N
        on = live[:, t, None].expand(B, H)
        res["dg"][t] = (
            torch.where(on, (dS * Ss[t]).sum((-1, -2)), zero),
            torch.where(on, (kappa + g_r) * ((N * Ms[t]).sum((-1, -2)) + stay),
                        zero))
    out["ds0"] = (dS, (kappa + s_r) * N)
    for n, x in res.items():
        out[n] = tuple(torch.stack([y[i] for y in x], 1) for i in (0, 1))
    for n in ("dq", "dk"):
        out[n] = tuple(x.reshape(B, T, Hk, G, Dk).sum(3) for x in out[n])
    if fixed:
        out["dg"] = tuple(x.sum((0, 1)) for x in out["dg"])
    return out


def _turn(x, xe, cs, interleaved, back=False):
    """x (slack xe) rotated; a rotation in fp32 is off by 6 u of the pair's
    magnitudes (cosine and sine by 2 u each, products and sum)"""
    if cs is None:
        return x, xe
    c, s = cs
    s = -s if back else s
    n = c.shape[-1]

    def split(y):
        if interleaved:
            return y[..., 0:2 * n:2], y[..., 1:2 * n:2]
        return y[..., :n], y[..., n:2 * n]

    def join(a, b, y):
        z = torch.stack([a, b], -1).flatten(-2) if interleaved \
            else torch.cat([a, b], -1)
        return torch.cat([z, y[..., 2 * n:]], -1)

    a, b = split(x)
    ae, be = split(xe)
    e = 6 * U * (a.abs() + b.abs())
    return (join(a * c - b * s, b * c + a * s, x),
            join(ae * c.abs() + be * s.abs() + e,
                 be * c.abs() + ae * s.abs() + e, xe))


def _angles(positions, inv_freq):
    if inv_freq is None:
        return None
    a = positions.cpu().to(F8)[..., None, None] * inv_freq.cpu().to(F8)
    return a.cos(), a.sin()


def qk_norm(x, w, positions, inv_freq, interleaved, eps):
    """one side's output, (value, slack)"""
    x, w = c8(x), c8(w)
    y, e = x, torch.zeros_like(x)
    if w is not None:
        r, rr = _rms(x, eps)
        y = x * r * w
        e = (rr + 4 * U) * y.abs()
    return _turn(y, e, _angles(positions, inv_freq), interleaved)


def qk_norm_grad(x, w, positions, inv_freq, interleaved, eps, dy):
    """one side's (dx, dw), each (value, slack) or None"""
    x, w, dy = c8(x), c8(w), c8(dy)
    t, te = _turn(dy, torch.zeros_like(dy), _angles(positions, inv_freq),
                  interleaved, back=True)
    if w is None:
        return (t, te), None
    r, rr = _rms(x, eps)
    n = x * r
    lead = tuple(range(x.dim() - 1))
    rows = x.numel() // x.shape[-1]
    dw = ((t * n).sum(lead),
          (te * n.abs() + (rr + 4 * U + rows * U) * (t * n).abs()).sum(lead))
    return _norm_grad(x, r, rr, t * w,
                      te * w.abs() + 2 * U * (t * w).abs()), dw
