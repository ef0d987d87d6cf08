"""The gate's gradient of linear attention on the GPU where it is put together
over many chunks: against the 64-bit formula within the bounds of
linattn_gate_ref, which the mistakes that such sums can hold do not meet."""
import pytest
import torch

from layer_ref import U, within
from linattn_gate_ref import K, Parts

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
CHUNK = {BF: 64, F: 32}


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_74_amd as m
    return m


def inputs(B, T, Hk, H, Dk, Dv, io, kind, seed=0):
    gen = torch.Generator().manual_seed(seed + T + 31 * Dk + Dv)

    def r(*s):
        return torch.randn(*s, generator=gen)

    unit = torch.nn.functional.normalize
    x = dict(q=unit(r(B, T, Hk, Dk), dim=-1).to(io),
             k=unit(r(B, T, Hk, Dk), dim=-1).to(io), v=r(B, T, H, Dv).to(io),
             s0=r(B, H, Dk, Dv))
    x["g"] = {
        "slow": lambda: -0.002 * torch.rand(B, T, H, generator=gen),
        # chunks leave e^-5 to e^-10 of what is before them
        "weak": lambda: -0.3 * torch.rand(B, T, H, generator=gen),
        "fixed": lambda: -torch.exp2(-2.0 - 3 * torch.arange(H)),
        "softplus": lambda: -torch.nn.functional.softplus(r(B, T, H)),
    }[kind]()
    return x, dict(do=r(B, T, H, Dv).to(io), dsT=r(B, H, Dk, Dv))


def gradient(kda, x, d, times=1, lengths=None, scale=1.0):
    """dg of heads repeated `times` over, of the first of each; the others'
    must be the same"""
    def many(n, t):
        if t is None:
            return None
        dim = 0 if t.dim() == 1 else 1 if n in ("s0", "dsT") else 2
        return torch.cat([t.cuda()] * times, dim).contiguous()

    y = {n: many(n, t) for n, t in {**x, **d}.items()}
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32,
                                                  device="cuda")
    dg = kda.kda_linattn_backward(
        y["q"], y["k"], y["v"], y["g"], y["do"], s0=y.get("s0"),
        dsT=y.get("dsT"), lengths=n, scale=scale)[3]
    H = x["v"].shape[2]
    assert torch.equal(dg, torch.cat([dg[..., :H]] * times, -1))
    return dg[..., :H].cpu()


def check(kda, x, d, times=1, seg=1 << 20, lengths=None, scale=1.0,
          norm=False):
    """norm: also over the whole tensor, 16 half steps of the values.  A fixed
    decay's is the sum of its tokens' values, which cancel while their errors
    need not: a chunk's two sums are off by 2 half steps of W at its ends each,
    and those of 8 chunks stay until the product of the states is made anew,
    sqrt(16) * 2 = 8 half steps of the largest W that far for every token."""
    p = Parts(x, d, CHUNK[x["q"].dtype], seg,
              None if lengths is None else torch.tensor(lengths), scale)
    want = p.gradient()
    got = gradient(kda, x, d, times, lengths, scale)
    within("dg", got, want)
    if norm and p.fixed:
        ends = [*range(0, p.T, p.C), p.T]
        W = sum((b - a) * torch.stack([p.W[e] for e in ends[i:i + 9]]).amax(0)
                for i, (a, b) in enumerate(zip(ends, ends[1:])))
        assert ((got - want[0]).abs() <= 8 * U * W.sum(0)).all()
    elif norm:
        assert (got - want[0]).norm() <= 2.0 ** -20 * want[0].norm()
    return got, want


# 600 heads of 16 or 32 fill the GPU: a sequence is one segment, of 64 chunks at
# most
LENGTHS = [(1, 0), (2, -1), (16, 0), (17, 5), (64, -3), (65, 0)]


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind,chunks,over", [
    (kind, *n) for kind in ("slow", "fixed") for n in LENGTHS] + [
    (kind, *n) for kind in ("weak", "softplus") for n in LENGTHS[:4]])
def test_segments_of_chunks(kda, io, kind, chunks, over):
    C = CHUNK[io]
    T = chunks * C + over
    x, d = inputs(1, T, 2, 2, 16, 16 if chunks % 2 else 32, io, kind)
    check(kda, x, d, 300, 64 * C, norm=True)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind", ["slow", "fixed"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (32, 128)])
def test_segments_of_any_width(kda, io, kind, Dk, Dv):
    x, d = inputs(1, 9 * CHUNK[io] + 7, 1, 2, Dk, Dv, io, kind)
    check(kda, x, d, 300, norm=True)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind", ["slow", "fixed"])
@pytest.mark.parametrize("T", [577, 900, 1500])
def test_short_segments(kda, io, kind, T):
    """few heads: a segment is a chunk or two"""
    x, d = inputs(1, T, 1, 2, 32, 32, io, kind)
    check(kda, x, d, norm=True)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind", ["slow", "weak", "fixed"])
def test_ragged_segments(kda, io, kind):
    """lengths at and beside chunks' ends, of sequences of one segment each"""
    C = CHUNK[io]
    T = 20 * C
    n = [T, T - 1, 16 * C, 16 * C + 1, 5 * C - 1, 1, 0, T + 9]
    x, d = inputs(len(n), T, 1, 1, 16, 16, io, kind)
    got, _ = check(kda, x, d, 80, lengths=n)
    if kind != "fixed":
        for b, m in enumerate(n):
            assert (got[b, m:] == 0).all()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("g0", [-5.0, -10.0, -16.0, -20.0, -27.0, -60.0])
@pytest.mark.parametrize("later", [1.0, 1000.0])
def test_one_token_that_forgets(kda, io, times, g0, later):
    """a token that forgets nearly all among some that forget little, as a new
    document in a packed row; with gradients that are larger behind it"""
    x, d = inputs(1, 512, 1, 2, 16, 16, io, "slow", seed=1)
    x["g"][:, 300] = g0
    d["do"][:, 300:] = (later * d["do"][:, 300:].float()).to(io)
    d["dsT"] *= later
    check(kda, x, d, times)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("g", [-0.2, -0.02])
def test_a_loss_on_the_last_tokens(kda, io, times, g):
    """a prompt without a loss: gradients decay from its end on, in long
    segments far below what they begin with; the sum over all tokens, of a
    fixed decay, has no more of them than there is"""
    C = CHUNK[io]
    T = 40 * C + 3
    x, d = inputs(1, T, 1, 2, 16, 16, io, "slow", seed=2)
    x["g"] = torch.full_like(x["g"], g)
    d["do"][:, :-8] = 0
    d["dsT"] = None
    got, (want, _) = check(kda, x, d, times)
    if g == -0.2:
        assert (got[0, :20 * C].abs() < 1e-30).all()
    total = want.sum((0, 1))
    x["g"] = torch.full((2,), g)
    _, (want, _) = check(kda, x, d, times, norm=True)
    torch.testing.assert_close(want, total, rtol=1e-9, atol=0)


@pytest.mark.parametrize("io", [BF, F])
def test_a_state_that_is_nothing(kda, io):
    """no first state and a first token that forgets: nothing crosses it"""
    x, d = inputs(1, 200, 1, 2, 32, 32, io, "slow", seed=3)
    x["s0"] = None
    x["g"][:, 0] = -float("inf")
    got, _ = check(kda, x, d)
    assert (got[:, 0] == 0).all()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("big", [1e-12, 1e12])
def test_states_of_any_size(kda, io, big):
    """squares of states far from 1, and of gradients as far the other way"""
    x, d = inputs(1, 700, 1, 2, 32, 32, io, "slow", seed=4)
    x["v"], x["s0"] = (x["v"].float() * big).to(io), x["s0"] * big
    d["do"] = (d["do"].float() / big).to(io)
    d["dsT"] = d["dsT"] / big
    check(kda, x, d, 300)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind", ["slow", "softplus", "fixed"])
def test_what_a_workspace_holds_does_not_matter(kda, io, kind):
    """sequences of several marks, of lengths before, at and behind them; the
    marks that nothing is asked of are not read; captured and replayed too"""
    C = CHUNK[io]
    T = 27 * C
    n = torch.tensor([T, 8 * C, 8 * C + 1, 16 * C - 1, 3, 0, 24 * C, 25 * C],
                     dtype=torch.int32, device="cuda")
    x, d = inputs(8, T, 1, 1, 32, 64, io, kind, seed=6)
    y = {k: t.cuda().repeat_interleave(70, 0 if t.dim() == 1 else 1 if k in
                                       ("s0", "dsT") else 2).contiguous()
         for k, t in {**x, **d}.items()}
    size = kda.kda_linattn_backward_workspace_size(8, T, 70, 70, 32, 64, io)

    def run(ws):
        return kda.kda_linattn_backward(
            *[y[k] for k in "qkvg"], y["do"], s0=y["s0"], dsT=y["dsT"],
            lengths=n, workspace=ws)

    base = run(torch.zeros(size, dtype=torch.uint8, device="cuda"))
    # NaNs, and values like any
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(base, run(ws)))
    ws.fill_(63)
    assert all(torch.equal(a, b) for a, b in zip(base, run(ws)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(ws)
    for fill in (255, 63, 0):
        ws.fill_(fill)
        for t in got:
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(base, got))
        run(None)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("g0", [-18.0, -20.0, -24.0])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_no_gradient_is_rounding_alone(kda, io, D, g0, seed):
    """A token that forgets so much that what crosses its chunk, exp(g0) of what
    is across its end (2^-26 at most, 8 half steps of fp32 are 2^-21), cannot be
    told from rounding: it counts as nothing, and the rest is the token's own to
    its accuracy."""
    C = CHUNK[io]
    x, d = inputs(1, 512, 1, 2, D, D, io, "slow", seed=seed)
    x["g"][:, 300] = g0
    p = Parts(x, d, C, 1 << 20)
    want = p.gradient()[0][0, 300]
    got = gradient(kda, x, d, 1 if D == 128 else 300)[0, 300]
    off = p.Z[300 // C][0].abs() + K * p.W[300][0]
    assert ((got - want).abs() <= off).all()
