"""What include/kda.h says of linear attention at the ends of its range: where
an infinity or NaN goes, and from where on a decayed term may be nothing."""
import math

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


def inputs(io, B=2, T=200, Hk=2, H=4, D=32, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=gen).to(io).cuda()

    return dict(q=r(B, T, Hk, D), k=r(B, T, Hk, D), v=r(B, T, H, D),
                g=-0.01 * torch.rand(B, T, H, generator=gen).cuda()), \
        r(B, T, H, D)


def same(a, b):
    """element by element, as bits"""
    return (a == b) | (a.isnan() & b.isnan())


# token 100 lies in the chunk from 64 (fp32: 96) on
@pytest.mark.parametrize("io,first", [(BF, 64), (F, 96)])
@pytest.mark.parametrize("name,hurt", [("q", (2, 3)), ("k", (2, 3)),
                                       ("v", (3,)), ("s0", (3,))])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_where_a_bad_value_goes(kda, io, first, name, hurt, bad):
    x, _ = inputs(io)
    s0 = torch.randn(2, 4, 32, 32, device="cuda")
    four = list(x.values())
    o, s = kda.kda_linattn(*four, s0=s0)
    if name == "s0":
        s0[1, 3, 5, 6] = bad
        first = 0
    else:
        x[name][1, 100, 3 if name == "v" else 1, 7] = bad
    o2, s2 = kda.kda_linattn(*four, s0=s0)
    may = torch.zeros_like(o, dtype=torch.bool)
    may[1, first:, hurt] = True
    assert (same(o, o2) | may).all()
    may = torch.zeros_like(s, dtype=torch.bool)
    may[1, hurt] = True
    assert (same(s, s2) | may).all()
    # and does reach its own token, but for q every later one
    for h in hurt:
        assert not o2[1, 100:, h].isfinite().all(-1)[0]
        if name != "q":
            assert not o2[1, 100:, h].isfinite().all(-1).any()
            assert not s2[1, h].isfinite().all()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("T,reset", [(90, 80), (200, 150), (1500, 1400)])
def test_a_reset_does_not_clear_it(kda, io, T, reset):
    """as in the formula: 0 * inf; the step's too"""
    x, _ = inputs(io, 1, T, 1, 1)
    x["v"][0, 10, 0, 3] = math.inf
    x["g"][0, reset] = -math.inf
    o, s = kda.kda_linattn(*x.values())
    assert o[0, reset:, 0, 3].isnan().all() and s[0, 0, :, 3].isnan().all()
    s = torch.full((1, 1, 32, 32), math.inf, device="cuda")
    o = kda.kda_linattn_step(*[t[:, reset].clone() for t in x.values()],
                             s)
    assert o.isnan().all() and s.isnan().all()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("Hk", [2, 4])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "do", "dsT"])
def test_where_a_bad_value_goes_in_the_gradients(kda, io, Hk, name):
    x, do = inputs(io, Hk=Hk)
    dsT = torch.randn(2, 4, 32, 32, device="cuda")
    four = list(x.values())
    good = kda.kda_linattn_backward(*four, do, dsT=dsT)
    t = {**x, "do": do, "dsT": dsT}[name]
    shared = name in "qk" and Hk == 2
    if name == "dsT":
        t[1, 3, 5, 6] = math.nan
    elif name == "g":
        t[1, 100, 3] = math.nan
    else:
        t[1, 100, t.shape[2] - 1, 7] = math.nan
    bad = kda.kda_linattn_backward(*four, do, dsT=dsT)
    heads = (2, 3) if shared else (3,)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), good, bad):
        may = torch.zeros_like(a, dtype=torch.bool)
        if n == "ds0":
            may[1, heads] = True
        elif n in ("dq", "dk"):
            may[1, :, Hk - 1] = True
        else:
            may[1, :, heads] = True
        assert (same(a, b) | may).all(), n
    # what a gradient of the last state reaches is every token's
    if name == "dsT":
        assert bad[3][1, :, 3].isnan().all()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("T", [2, 40, 64, 130, 700])
@pytest.mark.parametrize("where", ["one", "all"])
def test_decayed_terms_stay_down_to_the_limit(kda, io, T, where):
    """a term of 2^100 decayed by 2^-125, by one gate or all of them, keeps its
    bits (4 u a chunk, and the argument of the exponential is rounded by 63 u
    of its 125 ln 2 once)"""
    x = {n: torch.zeros(1, T, 1, 16, dtype=io) for n in "qkv"}
    x["k"][0, 0, 0, 3], x["v"][0, 0, 0, 5] = 2.0 ** 50, 2.0 ** 50
    x["q"][0, T - 1, 0, 3] = 1.0
    x["g"] = torch.zeros(1, T, 1)
    ln = -125 * math.log(2.0)
    if where == "one":
        x["g"][0, T // 2] = ln
    else:
        x["g"][0, 1:] = ln / (T - 1)
    want = ref.linattn(**x)
    o, s = kda.kda_linattn(*[t.cuda() for t in x.values()])
    slack = (64 + 4 * -(-T // 32)) * U
    for n, t in (("o", o), ("s", s)):
        w = want[n][0]
        assert (w != 0).any()
        r = 2.0 ** -17 if n == "o" and io == BF else 0
        within(n, t, (w, (slack + r) * w.abs()))
