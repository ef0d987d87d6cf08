"""The reference of linear attention's gate gradient against the recurrence's,
and the mistakes that its bounds have to catch."""
import pytest
import torch

import linattn_ref
from layer_ref import F8, within
from linattn_gate_ref import Parts

KINDS = ("slow", "weak", "fixed", "softplus")


def inputs(T, kind, Dk=16, Dv=16, Hk=1, H=2, B=1, seed=0):
    gen = torch.Generator().manual_seed(seed + T)

    def r(*s):
        return torch.randn(*s, generator=gen, dtype=F8)

    unit = torch.nn.functional.normalize
    x = dict(q=unit(r(B, T, Hk, Dk), dim=-1), k=unit(r(B, T, Hk, Dk), dim=-1),
             v=r(B, T, H, Dv), s0=r(B, H, Dk, Dv))
    x["g"] = {"slow": lambda: -0.002 * r(B, T, H).abs(),
              "weak": lambda: -0.3 * torch.rand(B, T, H, generator=gen,
                                                dtype=F8),
              "fixed": lambda: -torch.tensor([0.05, 0.002], dtype=F8)[:H],
              "softplus": lambda: -torch.nn.functional.softplus(r(B, T, H)),
              }[kind]()
    return x, dict(do=r(B, T, H, Dv), dsT=r(B, H, Dk, Dv))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths", [None, [90, 33]])
def test_is_the_recurrence(kind, lengths):
    x, d = inputs(90, kind, 3, 5, B=2)
    if lengths is not None:
        lengths = torch.tensor(lengths, dtype=torch.int32)
    p = Parts(x, d, 32, 64, lengths, scale=0.7)
    want = linattn_ref.linattn(**x, **d, lengths=lengths, scale=0.7)["dg"][0]
    torch.testing.assert_close(p.gradient()[0], want, rtol=1e-11, atol=1e-12)
    torch.testing.assert_close(p.chunked(), want, rtol=1e-9, atol=1e-11)


def bounded(p, c, z):
    """z, of chunk c, within the most that it can be"""
    cap = p.cap[c].to(z.dtype)
    return z.clamp(-cap, cap)


def weakly(kind):
    """whether chunks of 64 leave much of what is before them"""
    return kind in ("slow", "fixed")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [64, 577, 900])
def test_bounds_catch_mistakes(kind, T):
    x, d = inputs(T, kind)
    p = Parts(x, d, 64, 1 << 20)
    right = p.gradient()
    within("dg", right[0].float(), right)
    # fp32 sums, with a bound on Z or where chunks forget little without
    within("dg", p.chunked(torch.float32,
                           lambda c, z, E: bounded(p, c, z)), right,
           torch.float32)
    if weakly(kind):
        within("dg", p.chunked(torch.float32), right, torch.float32)
    wrong = {"nothing": torch.zeros_like(right[0]), "sign": -right[0],
             "late": right[0] * (1 + 2.0 ** -8)}
    if weakly(kind) and T > 64:
        wrong["no Z"] = p.chunked(Z=lambda c, z: 0 * z)
        wrong["no carry"] = p.chunked(
            carry=lambda c, z, E: p.E[T] - sum(
                p.early[t] for t in range(c * 64, min(T, c * 64 + 64))))
    for name, dg in wrong.items():
        with pytest.raises(AssertionError):
            within(name, dg.float(), right, torch.float32)


@pytest.mark.parametrize("g0", [-20.0, -27.0])
def test_bounds_catch_what_is_left_of_a_difference(g0):
    """one token that forgets nearly all among some that forget little: E less
    the chunk's own in fp32 is rounding alone"""
    x, d = inputs(512, "slow")
    x["g"][:, 300] = g0
    p = Parts(x, d, 64, 1 << 20)
    right = p.gradient()
    assert (right[0][0, 300].abs() < 1e-6).all()
    with pytest.raises(AssertionError):
        # 2^-22 of E: what fp32 sums leave
        within("dg", p.chunked(carry=lambda c, z, E: z + 2.0 ** -22 * E),
               right, torch.float32)
    within("dg", p.chunked(carry=lambda c, z, E: bounded(
        p, c, z + 2.0 ** -22 * E)), right, torch.float32)


def test_bounds_catch_what_a_later_loss_leaves():
    """a loss on the last tokens: what the sums across their chunk are off is
    not carried to the tokens before, whose gradients decay"""
    x, d = inputs(1500, "weak")
    x["g"] = torch.full_like(x["g"], -0.2)
    d["do"][:, :-8] = 0
    d["dsT"].zero_()
    p = Parts(x, d, 64, 1 << 20)
    right = p.gradient()
    assert (right[0][0, 100].abs() < 1e-80).all()
    noise = p.E[1500 - 1500 % 64].abs() * 2.0 ** -22
    with pytest.raises(AssertionError):
        within("dg", p.chunked(carry=lambda c, z, E: z + noise), right,
               torch.float32)
    within("dg", p.chunked(carry=lambda c, z, E: bounded(p, c, z + noise)),
           right, torch.float32)
