"""The gate's gradient of linear attention in 64 bits, with what an evaluation
from sums over chunks may be off.

dg_t is the sum of (q_i . k_j)(do_i . v_j) exp(G_i - G_j) over all pairs
i >= t > j: with dS the state's gradient as it leaves token t and S the state
before it, the product <dS, S>.  In chunks it is put together from sums over
parts of these pairs, whose fp32 roundings are independent of each other, so
that they add up by their squares: to K W, with

    W = |dS o S| + sqrt <N, M> + |<dS, S>|

(o element by element, N and M the recurrences of dS and S over squares: the
roots of the sums of squares of the elements' and of the pairs' products) and K
= 2^-18, 64 half steps: a state is rounded 4 times a chunk, over 64 chunks 16
half steps in the mean of squares; four times that.  (The sums begin anew every
8 chunks, which these bounds need not know.)

Z, the pairs around a whole chunk, is what is across its end less what reaches
into it, and the next chunk's E is what Z and the chunk's own make: each is off
by what the sums behind it were off in the same segment, and every boundary
adds its K W.  But Z is no more than exp(G) times the sum of the |S| and the
largest |dS|, and off by twice that at most.
"""
import torch

from layer_ref import F8, c8

K = 2.0 ** -18


class Parts:
    """Everything the gradient is put together from, of x (q, k, v, g, s0)
    and d (do, dsT), for chunks of C tokens in segments of `seg`."""

    def __init__(self, x, d, C, seg, lengths=None, scale=1.0):
        q, k, v, g, s0 = (c8(x.get(n)) for n in ("q", "k", "v", "g", "s0"))
        do, dsT = c8(d["do"]), c8(d.get("dsT"))
        B, T, Hk, Dk = q.shape
        H, Dv = v.shape[2:]
        self.fixed = g.dim() == 1
        self.C, self.seg, self.T = C, seg, T
        n = torch.full((B,), T) if lengths is None \
            else lengths.cpu().long().clamp(0, T)
        self.live = live = torch.arange(T)[None] < n[:, None]  # [B, T]
        dead = ~live[..., None, None]
        q, k = (x.repeat_interleave(H // Hk, 2) for x in (q, k))
        q, k, v, do = (x.masked_fill(dead, 0.0) for x in (q, k, v, do))
        do = scale * do
        g = g.expand(B, T, H).masked_fill(~live[..., None], 0.0)
        a = torch.exp(g)
        S = torch.zeros(B, H, Dk, Dv, dtype=F8) if s0 is None else s0
        M = S * S
        Ss, Ms = [S], [M]
        for t in range(T):
            A = a[:, t, :, None, None]
            k_, v_ = k[:, t].unsqueeze(-1), v[:, t].unsqueeze(-2)
            S = A * S + k_ * v_
            M = A * A * M + k_ ** 2 * v_ ** 2
            Ss.append(S)
            Ms.append(M)
        dS = torch.zeros_like(S) if dsT is None else dsT
        N = dS * dS

        def w(dS, N, t):
            e = (dS * Ss[t]).sum((-1, -2))
            return e, (dS * Ss[t]).norm(dim=(-1, -2)) + \
                (N * Ms[t]).sum((-1, -2)).sqrt() + e.abs()

        # at t: across the boundary before token t
        E, W = [None] * (T + 1), [None] * (T + 1)
        E[T], W[T] = w(dS, N, T)
        late, early, Z, cap = {}, {}, {}, {}
        for t in range(T - 1, -1, -1):
            c, t0 = t // C, t // C * C
            if t == T - 1 or (t + 1) % C == 0:
                G = g[:, t0:t + 1].sum(1)
                S0 = Ss[t0]
                Z[c] = torch.exp(G) * (dS * S0).sum((-1, -2))
                cap[c] = torch.exp(G) * dS.abs().amax((-1, -2)) * \
                    S0.abs().sum((-1, -2))
                end, reach = dS, torch.ones_like(G)
            # the token's query on the state before the chunk; its key on the
            # gradient behind it
            back = torch.exp(g[:, t0:t + 1].sum(1))
            late[t] = back * torch.einsum("bhd,bhde,bhe->bh", q[:, t], S0,
                                          do[:, t])
            early[t] = reach * torch.einsum("bhd,bhde,bhe->bh", k[:, t], end,
                                            v[:, t])
            reach = reach * a[:, t]
            A = a[:, t, :, None, None]
            q_, o_ = q[:, t].unsqueeze(-1), do[:, t].unsqueeze(-2)
            dS = A * (dS + q_ * o_)
            N = A * A * (N + q_ ** 2 * o_ ** 2)
            E[t], W[t] = w(dS, N, t)
        self.E, self.W, self.Z, self.cap = E, W, Z, cap
        self.late, self.early = late, early
        # what lies inside a chunk: the rest, of sums of a few in 64 bits
        self.pairs = {}
        for c in Z:
            t0, t1 = c * C, min(T, c * C + C)
            for t in range(t0, t1):
                x = sum(late[i] for i in range(t, t1))
                y = sum(early[j] for j in range(t0, t)) if t > t0 else 0.0
                self.pairs[t] = E[t] - x - y - Z[c]

    def gradient(self):
        """(value, slack), of the gate's shape"""
        on = self.live[..., None]
        T, C = self.T, self.C
        dg = torch.stack(self.E[:T], 1).masked_fill(~on, 0.0)
        slack = [None] * T
        for c in sorted(self.Z, reverse=True):
            t0, t1 = c * C, min(T, c * C + C)
            if t1 == T or t1 % self.seg == 0:
                off = (K * self.W[t1]) ** 2
            off = off + (K * self.W[t1]) ** 2
            off = torch.minimum(off, 4 * self.cap[c] ** 2)
            for t in range(t0, t1):
                slack[t] = off.sqrt() + K * self.W[t]
            off = off + (K * self.W[t0]) ** 2
        slack = torch.stack(slack, 1).masked_fill(~on, 0.0)
        return self.shape(dg), self.shape(slack)

    def shape(self, x):
        return x.sum((0, 1)) if self.fixed else x

    def chunked(self, dtype=F8, carry=None, Z=None):
        """The gradient from the sums over chunks, E from chunk to chunk in
        `dtype`.  carry: what becomes of E - early (of chunk c) instead of
        itself; Z: Z itself"""
        T, C = self.T, self.C
        out = [None] * T
        for c in sorted(self.Z, reverse=True):
            t0, t1 = c * C, min(T, c * C + C)
            if t1 == T or t1 % self.seg == 0:
                E = self.E[t1].to(dtype)
            y = sum(self.early[t] for t in range(t0, t1)).to(dtype)
            z = E - y
            if carry is not None:
                z = carry(c, z, E)
            if Z is not None:
                z = Z(c, z)
            x = torch.zeros_like(y)
            e = y
            for t in range(t1 - 1, t0 - 1, -1):
                x = x + self.late[t].to(dtype)
                e = e - self.early[t].to(dtype)
                out[t] = x + sum((self.early[j].to(dtype)
                                  for j in range(t0, t)),
                                 torch.zeros_like(e)) + z + \
                    self.pairs[t].to(dtype)
            E = z + x
        dg = torch.stack(out, 1).to(F8)
        return self.shape(dg.masked_fill(~self.live[..., None], 0.0))
