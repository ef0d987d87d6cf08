"""The 64-bit references of the layer operators against central differences
of their own forward formulas, and the scan's against its closed form: what
the GPU tests compare with is checked here first (CPU)."""
import pytest
import torch

import layer_ref as ref

F8 = torch.float64


def rand(*shape, seed=0):
    gen = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=gen, dtype=F8)


def differences(loss, leaves, grads, eps=1e-5, tol=1e-7):
    """d loss along a random direction of each leaf = <grad, direction>"""
    for name, v in leaves.items():
        d = rand(*v.shape, seed=len(name))
        d = d / d.norm()
        up = loss(**dict(leaves, **{name: v + eps * d}))
        dn = loss(**dict(leaves, **{name: v - eps * d}))
        num = float(up - dn) / (2 * eps)
        got = float((grads[name] * d).sum())
        assert abs(num - got) <= tol * max(1.0, abs(num)), (name, num, got)


@pytest.mark.parametrize("head,lengths", [
    (False, None), (True, None), (False, [9, 0, 1]), (True, [3, 11, 0])])
def test_scan_gradient(head, lengths):
    B, T, H, D = 3, 11, 2, 4
    n = None if lengths is None else torch.tensor(lengths)
    leaves = dict(x=rand(B, T, H, D), beta=rand(B, T, H, seed=1),
                  g=-rand(*((B, T, H) if head else (B, T, H, D))).abs(),
                  h0=rand(B, H, D, seed=2))
    dy, dhT = rand(B, T, H, D, seed=3), rand(B, H, D, seed=4)

    def loss(x, g, beta, h0):
        o = ref.scan(x, g, beta, h0, n)
        return (o["y"][0] * dy).sum() + (o["h"][0] * dhT).sum()

    o = ref.scan(**leaves, lengths=n, dy=dy, dhT=dhT)
    differences(loss, leaves, {k: o["d" + k][0] for k in leaves})


def test_scan_closed_form():
    x, g = rand(2, 300, 1, 3), -rand(2, 300, 1, 3, seed=1).abs() / 50
    cum = g.cumsum(1)
    want = torch.stack([(torch.exp(cum[:, t:t + 1] - cum[:, :t + 1]) *
                         x[:, :t + 1]).sum(1) for t in range(300)], 1)
    got = ref.scan(x, g)
    torch.testing.assert_close(got["y"][0], want, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(got["chunk"][0][:, 2], want[:, 255])


@pytest.mark.parametrize("act", ["sigmoid", "silu", None])
def test_gated_norm_gradient(act):
    leaves = dict(o=rand(5, 2, 16), w=rand(16))
    if act:
        leaves["z"] = rand(5, 2, 16, seed=3)
    dy = rand(5, 2, 16, seed=1)

    def loss(o, w, z=None):
        return (ref.gated_norm(o, z, w, act, 1e-6)[0] * dy).sum()

    do, dz, dw = ref.gated_norm(leaves["o"], leaves.get("z"), leaves["w"],
                                act, 1e-6, dy)
    grads = dict(o=do[0], w=dw[0])
    if act:
        grads["z"] = dz[0]
    differences(loss, leaves, grads)


@pytest.mark.parametrize("act", ["sigmoid", "silu", None])
@pytest.mark.parametrize("post,pre", [(1, 1), (0, 1), (1, 0)])
def test_block_norm_gradient(act, post, pre):
    R, C, rs, bs = 4, 10, 0.7, 0.4
    leaves = dict(y=rand(R, C), r=rand(R, C, seed=1))
    if post:
        leaves["w_post"] = rand(C, seed=2)
    if pre:
        leaves["w_pre"] = rand(C, seed=3)
    if act:
        leaves["z"] = rand(R, C, seed=4)
    dx, dro = rand(R, C, seed=5), rand(R, C, seed=6)

    def fwd(y, r, w_post=None, w_pre=None, z=None):
        return ref.block_norm(y, r, w_post, z, w_pre, act, rs, bs, 1e-6)

    def loss(**kw):
        h, x = fwd(**kw)
        return (h[0] * dro).sum() + ((x[0] * dx).sum() if pre else 0)

    r_out = fwd(**leaves)[0][0]
    got = ref.block_norm_grad(
        leaves["y"], r_out, dx if pre else None, dro, leaves.get("w_post"),
        leaves.get("z"), leaves.get("w_pre"), act, rs, bs, 1e-6)
    names = ["y", "r", "z", "w_post", "w_pre"]
    differences(loss, leaves, {k: v[0] for k, v in zip(names, got)
                               if v is not None})
