"""How many bits of a product linear attention keeps: results that consist of
one term each, so that every rounding on the way shows in full.

A result in bf16 may be off by its own rounding, 2^-8 of the value, and by what
an operand in two parts leaves, 2^-17 of the term; a factor exp(G) made of a
difference of 64-bit sums is off by 4 u (its argument's rounding, under one for
|G| <= 1, the hardware's exponential 2, a product 1) for each chunk that the
term passes through, u = 2^-24."""
import pytest
import torch

import linattn_ref as ref
from layer_ref import U, within

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_74_amd as m
    return m


def one_hot(gen, *shape):
    """exact in every type: a product with it picks one term"""
    i = torch.randint(0, shape[-1], shape[:-1], generator=gen)
    return torch.nn.functional.one_hot(i, shape[-1]).float()


def terms(name, got, want, T, r=2.0 ** -17):
    """got against values that are one term each"""
    within(name, got, (want, (r + (8 + 4 * -(-T // 32)) * U) * want.abs()))


def state_inputs(T, Dk, Dv, seed, H=3):
    gen = torch.Generator().manual_seed(seed + T + 3 * Dk + Dv)
    x = dict(q=one_hot(gen, 1, T, H, Dk), k=torch.zeros(1, T, H, Dk),
             v=one_hot(gen, 1, T, H, Dv))
    x = {n: t.to(BF) for n, t in x.items()}
    # all of them forget exp(-1) at most
    x["g"] = -torch.rand(1, T, H, generator=gen) / T
    x["s0"] = torch.randn(1, H, Dk, Dv, generator=gen)
    d = dict(do=one_hot(gen, 1, T, H, Dv).to(BF),
             dsT=torch.randn(1, H, Dk, Dv, generator=gen))
    return gen, x, d


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}


WIDTHS = [(16, 16), (32, 32), (64, 64), (128, 128), (128, 32), (16, 64)]


@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T", [1, 64, 130, 700])
def test_a_state_in_the_output(kda, Dk, Dv, T):
    """o = exp(G) s0^T q with nothing added: one element of s0 each"""
    _, x, _ = state_inputs(T, Dk, Dv, 1)
    want = ref.linattn(**x)["o"][0]
    y = cuda(x)
    o, _ = kda.kda_linattn(y["q"], y["k"], y["v"], y["g"], s0=y["s0"])
    terms("o", o, want, T)


@pytest.mark.parametrize("want_dg", [False, True])
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T", [1, 64, 130, 700])
def test_a_state_in_the_gradients(kda, Dk, Dv, T, want_dg):
    """dq of a state that nothing is added to, dk and dv of a state's gradient
    that nothing is added to"""
    gen, x, d = state_inputs(T, Dk, Dv, 2)
    want = ref.linattn(**x, **d)
    y, e = cuda(x), cuda(d)
    got = kda.kda_linattn_backward(y["q"], y["k"], y["v"], y["g"], e["do"],
                                   s0=y["s0"], want_dg=want_dg)
    terms("dq", got[0], want["dq"][0], T)
    x["k"] = one_hot(gen, *x["k"].shape).to(BF)
    d["do"].zero_()
    want = ref.linattn(**x, **d)
    y, e = cuda(x), cuda(d)
    got = kda.kda_linattn_backward(y["q"], y["k"], y["v"], y["g"], e["do"],
                                   dsT=e["dsT"], want_dg=want_dg)
    terms("dk", got[1], want["dk"][0], T)
    terms("dv", got[2], want["dv"][0], T)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("Hk", [1, 3])
@pytest.mark.parametrize("T", [70, 1100])
def test_gradients_do_not_depend_on_what_is_wanted(kda, io, Dk, Dv, Hk, T):
    """the same bits with and without the gate's gradient, and with and without
    the first state's"""
    gen = torch.Generator().manual_seed(T + Dk + Dv)

    def r(*s, dtype=io):
        return torch.randn(*s, generator=gen).to(dtype).cuda()

    four = (r(2, T, Hk, Dk), r(2, T, Hk, Dk), r(2, T, 3, Dv),
            -r(2, T, 3, dtype=F).abs())
    do, s0, dsT = r(2, T, 3, Dv), r(2, 3, Dk, Dv, dtype=F), r(2, 3, Dk, Dv,
                                                              dtype=F)
    full = kda.kda_linattn_backward(*four, do, s0=s0, dsT=dsT)
    for dg, ds0 in ((False, True), (True, False), (False, False)):
        part = kda.kda_linattn_backward(*four, do, s0=s0, dsT=dsT, want_dg=dg,
                                        want_ds0=ds0)
        for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), full, part):
            assert b is None or torch.equal(a, b), n


def pair_inputs(T, Dk, Dv, seed):
    """every tensor dense, log-decays that add up to -1 at most"""
    gen = torch.Generator().manual_seed(seed + T + 3 * Dk + Dv)
    H = 3

    def r(*s):
        return torch.randn(*s, generator=gen).to(BF)

    x = dict(q=r(1, T, H, Dk), k=r(1, T, H, Dk), v=r(1, T, H, Dv),
             g=-torch.rand(1, T, H, generator=gen) / T)
    return gen, x, dict(do=r(1, T, H, Dv))


def only(x, t):
    """x with zeros for all tokens but t"""
    y = torch.zeros_like(x)
    y[:, t] = x[:, t]
    return y


# the last chunk of 700 tokens begins at 640, for chunks of 32 and of 64
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T,t0", [(2, 0), (40, 0), (64, 0), (700, 640)])
def test_a_pair_product_in_the_output(kda, Dk, Dv, T, t0):
    """o_i = exp(G_i - G_0) (q_i . k_0) v_0 of a one-hot q"""
    gen, x, _ = pair_inputs(T, Dk, Dv, 3)
    x["q"] = one_hot(gen, *x["q"].shape).to(BF)
    x["v"] = only(x["v"], t0)
    want = ref.linattn(**x)["o"][0]
    y = cuda(x)
    o, _ = kda.kda_linattn(*y.values())
    terms("o", o, want, T)


@pytest.mark.parametrize("want_dg", [False, True])
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T,t0", [(2, 0), (40, 0), (64, 0), (700, 640)])
def test_a_pair_product_in_the_gradients(kda, Dk, Dv, T, t0, want_dg):
    """dq_i of one token's key; dk_j and dv_j of the last token's query and
    gradient, for the tokens of other chunks by way of the state"""
    gen, x, d = pair_inputs(T, Dk, Dv, 4)
    one = {n: one_hot(gen, *t.shape).to(BF) for n, t in {**x, **d}.items()
           if n != "g"}

    def grads(**over):
        y = {**x, **d, **over}
        want = ref.linattn(**y)
        y = cuda(y)
        return kda.kda_linattn_backward(y["q"], y["k"], y["v"], y["g"],
                                        y["do"], want_dg=want_dg), want

    got, want = grads(do=one["do"], k=only(x["k"], t0))
    terms("dq", got[0], want["dq"][0], T)
    got, want = grads(v=one["v"], q=only(x["q"], T - 1))
    terms("dk", got[1], want["dk"][0], T)
    got, want = grads(k=one["k"], do=only(d["do"], T - 1))
    terms("dv", got[2], want["dv"][0], T)


@pytest.mark.parametrize("kind", ["softplus", "slow"])
@pytest.mark.parametrize("Hk", [1, 2])
@pytest.mark.parametrize("T,Dk,Dv", [(512, 128, 128), (900, 32, 64)])
def test_errors_are_those_of_the_last_rounding(kda, kind, Hk, T, Dk, Dv):
    """Over a whole tensor: a rounded value's distance from the true one is at
    most its own rounding's (that of the true value, in the mean: to 1 % over
    60,000 of them) and what was off before, 2^-17 of its terms' magnitudes."""
    gen = torch.Generator().manual_seed(T + Hk)
    B, H = 1, 2

    def r(*s):
        return torch.randn(*s, generator=gen)

    x = dict(q=torch.nn.functional.normalize(r(B, T, Hk, Dk), dim=-1).to(BF),
             k=torch.nn.functional.normalize(r(B, T, Hk, Dk), dim=-1).to(BF),
             v=r(B, T, H, Dv).to(BF),
             g=-torch.nn.functional.softplus(r(B, T, H)) if kind == "softplus"
             else -0.002 * torch.rand(B, T, H, generator=gen),
             s0=r(B, H, Dk, Dv))
    d = dict(do=r(B, T, H, Dv).to(BF), dsT=r(B, H, Dk, Dv))
    want = ref.linattn(**x, **d)
    y, e = cuda(x), cuda(d)
    four = [y[n] for n in "qkvg"]
    got = [kda.kda_linattn(*four, s0=y["s0"])[0],
           *kda.kda_linattn_backward(*four, e["do"], s0=y["s0"],
                                     dsT=e["dsT"])[:3]]
    # ref's slack is (2^-8 + kappa) times the magnitudes
    kappa = (256 + 8 * -(-T // 32) + 2 * (Dk + Dv)) * U
    for n, t in zip(("o", "dq", "dk", "dv"), got):
        w, slack = want[n]
        own = (w.to(BF).double() - w).norm()
        before = slack.norm() / (2.0 ** -8 + kappa) * 2.0 ** -17
        assert (t.cpu().double() - w).norm() <= 1.01 * own + before, n


@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T", [1, 40, 130, 500])
def test_a_term_of_the_states_has_all_bits(kda, Dk, Dv, T):
    """the state of one token's key and value, the first state's gradient of
    one token's query and output: fp32 products of bf16 values"""
    gen, x, d = pair_inputs(T, Dk, Dv, 5)
    x["k"], x["v"] = only(x["k"], 0), only(x["v"], 0)
    x["q"], d["do"] = only(x["q"], T - 1), only(d["do"], T - 1)
    want = ref.linattn(**x, **d, dsT=torch.zeros(1, 3, Dk, Dv))
    y, e = cuda(x), cuda(d)
    _, s = kda.kda_linattn(*[y[n] for n in "qkvg"])
    terms("s", s, want["s"][0], T, 0)
    got = kda.kda_linattn_backward(*[y[n] for n in "qkvg"], e["do"])
    terms("ds0", got[4], want["ds0"][0], T, 0)


@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T", [1, 40, 130, 500])
def test_a_term_of_the_gate_gradient_has_all_bits(kda, Dk, Dv, T):
    """dg of the last token's query and the first state, which is one element
    of it for every token; of the first token's key and the last state's
    gradient, one element for every later one"""
    gen, x, d = state_inputs(T, Dk, Dv, 6)
    x["v"].zero_()
    x["q"], d["do"] = only(x["q"], T - 1), only(d["do"], T - 1)
    d["dsT"].zero_()
    want = ref.linattn(**x, **d)["dg"][0]
    y, e = cuda(x), cuda(d)
    got = kda.kda_linattn_backward(*[y[n] for n in "qkvg"], e["do"],
                                   s0=y["s0"])
    assert (want.abs().amax((0, 1)) > 0).all()
    terms("dg", got[3], want, T, 0)
    _, x, d = state_inputs(T, Dk, Dv, 7)
    x["k"] = only(one_hot(gen, *x["k"].shape).to(BF), 0)
    d["do"].zero_()
    x["s0"].zero_()
    want = ref.linattn(**x, **d)["dg"][0]
    y, e = cuda(x), cuda(d)
    got = kda.kda_linattn_backward(*[y[n] for n in "qkvg"], e["do"],
                                   dsT=e["dsT"])
    # the first token's is a difference of two of the others
    n = 8 + 4 * -(-T // 32)
    within("dg", got[3], (want, n * U * want.abs().amax(1, keepdim=True)
                          .expand_as(want)))


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("Dk,Dv", [(32, 32), (64, 128)])
def test_a_state_is_rounded_once_a_chunk(kda, io, Dk, Dv):
    """With decays of 0.001 a token in the mean a state remembers 1000 of them,
    31 chunks of 32.  Every chunk rounds it once (in the mean of squares u /
    sqrt 3 of its elements) and multiplies it by a rounded decay (within u,
    likewise), a token's own weight is within 3 u: sqrt(31 / 3 + 31 / 3 + 3) u,
    4.9 u of the state's norm."""
    gen = torch.Generator().manual_seed(Dk)
    T = 4096

    def r(*s):
        return torch.randn(*s, generator=gen).to(io)

    unit = torch.nn.functional.normalize
    x = dict(q=unit(r(1, T, 1, Dk), dim=-1), k=unit(r(1, T, 1, Dk), dim=-1),
             v=r(1, T, 1, Dv),
             g=-0.002 * torch.rand(1, T, 1, generator=gen))
    do = r(1, T, 1, Dv)
    # many of the same head: one segment a sequence; the sums of 64 chunks
    y = {n: t.repeat_interleave(600, 2).contiguous() for n, t in x.items()}
    y = cuda(y)
    want = ref.linattn(**x, do=do)
    _, s = kda.kda_linattn(*y.values())
    ds0 = kda.kda_linattn_backward(
        *y.values(), do.repeat_interleave(600, 2).contiguous().cuda())[4]
    for n, t in (("s", s), ("ds0", ds0)):
        w = want[n][0]
        assert (t[:, :1].cpu().double() - w).norm() <= 4.9 * U * w.norm(), n
