"""The 64-bit references of linear attention and of the norm and rotation of
queries and keys against autograd through the formulas, differences, and
planted mistakes that their slack must catch."""
import math

import pytest
import torch

import linattn_ref as ref
from layer_ref import F8, within


def _inputs(B=2, T=41, Hk=2, G=2, Dk=3, Dv=5, fixed=False, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=gen, dtype=F8)

    H = Hk * G
    x = dict(q=r(B, T, Hk, Dk), k=r(B, T, Hk, Dk), v=r(B, T, H, Dv),
             g=-torch.nn.functional.softplus(r(H) if fixed else r(B, T, H)),
             s0=r(B, H, Dk, Dv), scale=0.7)
    return x, dict(do=r(B, T, H, Dv), dsT=r(B, H, Dk, Dv))


def _plain(q, k, v, g, s0, scale, lengths):
    """the sum over all pairs of tokens, without a recurrence"""
    B, T, Hk, Dk = q.shape
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // Hk, 2) for x in (q, k))
    outs, states = [], []
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        gb = (g.expand(T, H) if g.dim() == 1 else g[b])[:n]
        G = torch.cat([torch.zeros(1, H, dtype=F8), gb.cumsum(0)])
        w = torch.exp(G[1:, None] - G[None, 1:])  # [i, j, H]
        w = w * torch.ones(n, n, dtype=F8).tril()[..., None]
        pairs = torch.einsum("ihd,jhd->ijh", q[b, :n], k[b, :n]) * w
        o = torch.einsum("ijh,jhe->ihe", pairs, v[b, :n]) + \
            torch.einsum("ih,ihd,hde->ihe", torch.exp(G[1:]), q[b, :n], s0[b])
        outs.append(torch.cat([scale * o,
                               torch.zeros(T - n, *o.shape[1:], dtype=F8)]))
        states.append(torch.exp(G[n])[:, None, None] * s0[b] +
                      torch.einsum("jh,jhd,jhe->hde",
                                   torch.exp(G[n] - G[1:]), k[b, :n],
                                   v[b, :n]))
    return torch.stack(outs), torch.stack(states)


@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("lengths", [None, [41, 7], [0, 1]])
def test_linattn_against_pairs_and_autograd(fixed, lengths):
    x, d = _inputs(fixed=fixed)
    if lengths is not None:
        lengths = torch.tensor(lengths, dtype=torch.int32)
    got = ref.linattn(**x, lengths=lengths, **d)
    leaves = {n: x[n].clone().requires_grad_() for n in "qkvg"}
    leaves["s0"] = x["s0"].clone().requires_grad_()
    o, s = _plain(**leaves, scale=x["scale"], lengths=lengths)
    torch.testing.assert_close(got["o"][0], o.detach(), rtol=1e-11, atol=1e-11)
    torch.testing.assert_close(got["s"][0], s.detach(), rtol=1e-11, atol=1e-11)
    loss = (o * d["do"]).sum() + (s * d["dsT"]).sum()
    grads = torch.autograd.grad(loss, list(leaves.values()))
    for n, w in zip(("dq", "dk", "dv", "dg", "ds0"), grads):
        torch.testing.assert_close(got[n][0], w, rtol=1e-10, atol=1e-10)


def test_linattn_gate_gradient_by_differences():
    x, d = _inputs(B=1, T=9, Hk=1, G=1)
    got = ref.linattn(**x, **d)["dg"][0]

    def loss(g):
        r = ref.linattn(**{**x, "g": g})
        return (r["o"][0] * d["do"]).sum() + (r["s"][0] * d["dsT"]).sum()

    for t in range(9):
        e = torch.zeros_like(x["g"])
        e[0, t, 0] = 1e-5
        num = (loss(x["g"] + e) - loss(x["g"] - e)) / 2e-5
        assert abs(num - got[0, t, 0]) < 1e-8 * (1 + abs(num))


def test_linattn_forgets_exactly():
    x, d = _inputs(T=12)
    x["g"][:, 5] = -math.inf
    r = ref.linattn(**x, **d)
    assert (r["dg"][0][:, 5] == 0).all() and torch.isfinite(r["dq"][0]).all()
    y = {n: (v[:, 5:] if n in ("q", "k", "v", "g") else v)
         for n, v in x.items()}
    assert torch.equal(r["o"][0][:, 5:], ref.linattn(**y)["o"][0])


@pytest.mark.parametrize("mistake", ["gate", "order", "head", "tail"])
def test_linattn_slack_catches(mistake):
    x, d = _inputs(T=40, Dk=16, Dv=16, seed=3)
    x = {n: (v.float() if torch.is_tensor(v) else v) for n, v in x.items()}
    n = torch.tensor([40, 23], dtype=torch.int32)
    right = ref.linattn(**x, lengths=n)
    y = dict(x)
    if mistake == "gate":      # the decay one token late
        y["g"] = x["g"].roll(1, 1)
    elif mistake == "order":   # the token itself left out
        y["v"] = x["v"].roll(1, 1)
    elif mistake == "head":    # heads shared the other way round
        y["k"] = x["k"].flip(2)
    wrong = ref.linattn(**y, lengths=n + (mistake == "tail"))
    with pytest.raises(AssertionError):
        within("o", wrong["o"][0].float(), right["o"])
    within("o", right["o"][0].float(), right["o"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
@pytest.mark.parametrize("norm", [False, True])
def test_qk_norm_against_autograd(interleaved, rot, norm):
    gen = torch.Generator().manual_seed(rot)
    x = torch.randn(3, 7, 2, 8, generator=gen, dtype=F8)
    dy = torch.randn(3, 7, 2, 8, generator=gen, dtype=F8)
    w = 1 + 0.1 * torch.randn(8, generator=gen, dtype=F8) if norm else None
    pos = inv = None
    if rot:
        pos = torch.randint(-5, 300000, (3, 7), generator=gen,
                            dtype=torch.int32)
        inv = torch.rand(rot // 2, generator=gen)
    leaves = [x.clone().requires_grad_()]
    y = leaves[0]
    if norm:
        leaves.append(w.clone().requires_grad_())
        y = y / (y.square().mean(-1, keepdim=True) + 1e-3).sqrt() * leaves[1]
    if rot:
        m = torch.eye(8, dtype=F8).expand(3, 7, 1, 8, 8).clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            t = (pos.to(F8) * inv[i].to(F8))[..., None]
            m[..., a, a], m[..., a, b] = t.cos(), -t.sin()
            m[..., b, b], m[..., b, a] = t.cos(), t.sin()
        y = (m @ y.unsqueeze(-1)).squeeze(-1)
    got = ref.qk_norm(x, w, pos, inv, interleaved, 1e-3)[0]
    torch.testing.assert_close(got, y.detach(), rtol=1e-12, atol=1e-12)
    grads = torch.autograd.grad(y, leaves, dy)
    dx, dw = ref.qk_norm_grad(x, w, pos, inv, interleaved, 1e-3, dy)
    torch.testing.assert_close(dx[0], grads[0], rtol=1e-10, atol=1e-10)
    assert (dw is None) == (not norm)
    if norm:
        torch.testing.assert_close(dw[0], grads[1], rtol=1e-10, atol=1e-10)


def test_qk_norm_slack_catches_fp32_angles():
    """angles made in fp32 are outside the slack at far positions"""
    x = torch.randn(50, 1, 16)
    pos = torch.arange(262144 - 50, 262144, dtype=torch.int32)
    inv = torch.pow(10000.0, -torch.arange(8) / 8.0)
    right = ref.qk_norm(x, None, pos, inv, False, 0.0)
    a = (pos.float()[:, None, None] * inv).double()
    c, s = a.cos(), a.sin()
    lo, hi = x[..., :8].double(), x[..., 8:].double()
    wrong = torch.cat([lo * c - hi * s, hi * c + lo * s], -1).float()
    with pytest.raises(AssertionError):
        within("y", wrong, right)
