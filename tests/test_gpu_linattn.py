"""kda_linattn, its gradient and its single-token step on the GPU against the
64-bit recurrence, element by element within derived bounds (linattn_ref)."""
import math

import pytest
import torch

import layer_ref
import linattn_ref as ref
from layer_ref import within

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
GRADS = ("dq", "dk", "dv", "dg", "ds0")


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_74_amd as m
    return m


def inputs(B, T, Hk, H, Dk, Dv, io=BF, gate=F, kind="softplus", s0=True,
           seed=0):
    gen = torch.Generator().manual_seed(seed * 7919 + T + 31 * Dk + Dv)

    def r(*s):
        return torch.randn(*s, generator=gen)

    q, k = (torch.nn.functional.normalize(r(B, T, Hk, Dk), dim=-1)
            for _ in range(2))
    if kind == "fixed":
        g = -torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    elif kind == "slow":
        g = -0.002 * torch.rand(B, T, H, generator=gen)
    else:
        g = -torch.nn.functional.softplus(r(B, T, H))
        g[torch.rand(g.shape, generator=gen) < 0.02] = -math.inf
    x = dict(q=q.to(io), k=k.to(io), v=r(B, T, H, Dv).to(io), g=g.to(gate))
    x = {n: t.cuda() for n, t in x.items()}
    x["s0"] = r(B, H, Dk, Dv).cuda() if s0 else None
    d = dict(do=r(B, T, H, Dv).to(io).cuda(),
             dsT=r(B, H, Dk, Dv).cuda() if s0 else None)
    return x, d


def check(kda, x, d, scale=1.0, lengths=None, want=None):
    """forward and gradient against the reference; returns the results"""
    kw = dict(s0=x["s0"], scale=scale, lengths=lengths)
    four = [x[n] for n in "qkvg"]
    o, s = kda.kda_linattn(*four, **kw)
    if want is None:
        want = ref.linattn(**x, scale=scale, lengths=lengths, **d)
    within("o", o, want["o"])
    within("s", s, want["s"])
    got = kda.kda_linattn_backward(*four, d["do"], dsT=d["dsT"], **kw)
    for n, t in zip(GRADS, got):
        within(n, t, want[n])
    return (o, s, *got)


@pytest.mark.parametrize("io,gate", [(BF, F), (BF, BF), (F, F)])
@pytest.mark.parametrize("Dk", [16, 32, 64, 128])
@pytest.mark.parametrize("Dv", [16, 32, 64, 128])
def test_widths_and_types(kda, io, gate, Dk, Dv):
    x, d = inputs(2, 71, 1, 2, Dk, Dv, io, gate)
    check(kda, x, d, scale=0.5)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 128,
                               129])
def test_lengths_of_a_chunk(kda, io, T):
    x, d = inputs(1, T, 2, 2, 32, 64, io, seed=1)
    check(kda, x, d)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind", ["softplus", "slow", "fixed"])
@pytest.mark.parametrize("T,Dk,Dv", [(577, 32, 16), (1500, 16, 32),
                                     (900, 128, 128)])
def test_segments(kda, io, kind, T, Dk, Dv):
    """sequences cut into several segments, with and without a first state"""
    x, d = inputs(1, T, 1, 1, Dk, Dv, io, kind=kind, s0=T != 1500, seed=2)
    check(kda, x, d, scale=Dk ** -0.5)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("Hk,H", [(1, 4), (3, 6), (2, 2)])
@pytest.mark.parametrize("kind", ["softplus", "fixed"])
def test_shared_heads(kda, io, Hk, H, kind):
    x, d = inputs(2, 200, Hk, H, 32, 32, io, kind=kind, seed=3)
    check(kda, x, d)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("kind", ["softplus", "fixed"])
def test_ragged(kda, io, kind):
    """lengths of 0, 1, inside and at the end of chunks and segments, past T
    and negative; what lies behind a sequence's end is not read"""
    T = 700
    n = torch.tensor([0, 1, 64, 65, 333, 700, 701, -3], dtype=torch.int32,
                     device="cuda")
    x, d = inputs(8, T, 1, 1, 16, 32, io, kind=kind, seed=4)
    dead = torch.arange(T, device="cuda")[None] >= n[:, None]
    for t in (x["q"], x["k"], x["v"], d["do"], x["g"]):
        if t.dim() > 1:
            t[dead] = math.nan
    y = {m: (t.nan_to_num(0.0, neginf=-math.inf) if t is not None else None)
         for m, t in x.items()}
    want = ref.linattn(**y, lengths=n, do=d["do"].nan_to_num(0.0),
                       dsT=d["dsT"])
    res = check(kda, x, d, lengths=n, want=want)
    for t in (res[0], res[2], res[3], res[4]):
        assert (t[dead] == 0).all()
    if kind == "softplus":
        assert (res[5][dead] == 0).all()
    assert torch.equal(res[6][0], d["dsT"][0])
    assert torch.equal(res[1][0], x["s0"][0])


@pytest.mark.parametrize("io", [BF, F])
def test_everything_forgotten(kda, io):
    """each token forgets all; then a whole chunk of -inf and lowest values"""
    x, d = inputs(1, 130, 1, 2, 32, 32, io, seed=5)
    x["g"][:] = -math.inf
    res = check(kda, x, d)
    assert (res[5] == 0).all() and (res[6] == 0).all()
    x, d = inputs(1, 300, 1, 2, 32, 32, io, seed=6)
    x["g"][:, 64:128] = torch.finfo(F).min
    x["g"][:, 200] = -math.inf
    x["g"][:, 250:] = 0.0
    x["g"][:, 20:40] = -30.0
    check(kda, x, d)


def test_growing_gates(kda):
    """g > 0 is the caller's business, but counts as what it is"""
    x, d = inputs(1, 100, 1, 1, 16, 16, F, seed=7)
    x["g"] = 0.02 * torch.rand_like(x["g"])
    check(kda, x, d)


@pytest.mark.parametrize("io", [BF, F])
def test_gate_gradient_across_weak_chunks(kda, io):
    """chunks that forget most, but not all, of what is before them: the sums
    across their ends stay accurate"""
    x, d = inputs(1, 1024, 1, 1, 32, 32, io, seed=8)
    x["g"] = -0.3 * torch.rand_like(x["g"])
    check(kda, x, d)


def test_rms_error_of_bf16(kda):
    """Over a whole tensor errors are random: the output's own rounding, the
    pair products' and the state's are three of at most 2^-8 each, so their
    root mean square is under 2^-8 of the values' (uniform in a step: 2^-8 /
    sqrt 3 each at most, and only two of them meet in one term)."""
    x, d = inputs(1, 512, 2, 2, 128, 128, kind="slow", seed=9)
    four = [x[n] for n in "qkvg"]
    want = ref.linattn(**x, **d)
    o, _ = kda.kda_linattn(*four, s0=x["s0"])
    got = kda.kda_linattn_backward(*four, d["do"], s0=x["s0"], dsT=d["dsT"])
    for n, t in zip(("o", *GRADS[:3]), (o, *got[:3])):
        w = want[n][0]
        assert (t.cpu().double() - w).norm() < 2.0 ** -8 * w.norm(), n


def test_state_in_place_and_wants(kda):
    for T in (40, 1500):
        x, d = inputs(1, T, 1, 2, 64, 64, seed=10)
        four = [x[n] for n in "qkvg"]
        o, s = kda.kda_linattn(*four, s0=x["s0"])
        again = x["s0"].clone()
        o2, s2 = kda.kda_linattn(*four, s0=again, s_out=again)
        assert s2 is again and torch.equal(o, o2) and torch.equal(s, again)
        o3, s3 = kda.kda_linattn(*four, s0=x["s0"], want_state=False,
                                 o=torch.empty_like(o))
        assert s3 is None and torch.equal(o, o3)
        full = kda.kda_linattn_backward(*four, d["do"], s0=x["s0"],
                                        dsT=d["dsT"])
        part = kda.kda_linattn_backward(*four, d["do"], s0=x["s0"],
                                        dsT=d["dsT"], want_dg=False,
                                        want_ds0=False)
        assert part[3] is None and part[4] is None
        # without the gate's gradient the state takes part rounded alone
        r = 2.0 ** -8
        for n, a, b in zip(GRADS, full[:3], part[:3]):
            a, b = a.double(), b.double()
            assert (a - b).norm() <= 2 * r * a.norm(), n


@pytest.mark.parametrize("io,gate", [(BF, F), (BF, BF), (F, F)])
def test_same_from_call_to_call(kda, io, gate):
    x, d = inputs(2, 1100, 1, 2, 64, 32, io, gate, seed=11)
    four = [x[n] for n in "qkvg"]

    def run():
        return (*kda.kda_linattn(*four, s0=x["s0"]),
                *kda.kda_linattn_backward(*four, d["do"], s0=x["s0"],
                                          dsT=d["dsT"]))

    first = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_prompt_in_parts(kda):
    """a prompt in two calls, the state handed on, is the prompt in one"""
    x, d = inputs(2, 500, 2, 4, 32, 64, F, seed=12)
    four = [x[n] for n in "qkvg"]
    want = ref.linattn(**x)
    a, s = kda.kda_linattn(*[t[:, :213].contiguous() for t in four],
                           s0=x["s0"])
    b, s = kda.kda_linattn(*[t[:, 213:].contiguous() for t in four], s0=s)
    within("o", torch.cat([a, b], 1), want["o"])
    within("s", s, want["s"])


@pytest.mark.parametrize("io,gate", [(BF, F), (BF, BF), (F, F)])
@pytest.mark.parametrize("Dk", [16, 32, 64, 128])
@pytest.mark.parametrize("Dv", [16, 32, 64, 128])
def test_step(kda, io, gate, Dk, Dv):
    """one token: an odd count of heads, shared in threes, one that forgets.
    fp32: the state costs an exponential (2 u) and a multiply-add, the output a
    sum of Dk products."""
    N, Hk, H = 5, 1, 3
    x, _ = inputs(N, 1, Hk, H, Dk, Dv, io, gate, seed=13)
    x["g"][1] = -math.inf
    q, k, v, g = (x[n][:, 0].contiguous() for n in "qkvg")
    st = x["s0"].clone()
    o = kda.kda_linattn_step(q, k, v, g, st, scale=0.3)
    u = layer_ref.U
    Q, K = (t.cpu().double().repeat_interleave(3, 1) for t in (q, k))
    a = torch.exp(g.cpu().double())[..., None, None]
    S0, kv = x["s0"].cpu().double(), K.unsqueeze(-1) * \
        v.cpu().double().unsqueeze(-2)
    S, M = a * S0 + kv, a * S0.abs() + kv.abs()
    within("state", st, (S, 4 * u * M))
    within("o", o, (0.3 * (Q.unsqueeze(-1) * S).sum(-2),
                    0.3 * (Dk + 8) * u * (Q.abs().unsqueeze(-1) * M).sum(-2)))


def test_step_follows_the_prompt(kda):
    """a prompt, then token by token, with a decay per head that stays"""
    x, _ = inputs(3, 90, 2, 4, 64, 128, F, kind="fixed", seed=14)
    want = ref.linattn(**x)
    four = [x[n] for n in "qkv"]
    o, st = kda.kda_linattn(*[t[:, :70].contiguous() for t in four], x["g"],
                            s0=x["s0"])
    outs = [o]
    for t in range(70, 90):
        outs.append(kda.kda_linattn_step(
            *[y[:, t].contiguous() for y in four], x["g"], st).unsqueeze(1))
    within("o", torch.cat(outs, 1), want["o"])
    within("s", st, want["s"])


def test_many_heads_without_segments(kda):
    """more heads than workgroups are wanted; few are checked"""
    B, T, H = 3, 130, 200
    x, d = inputs(B, T, H, H, 16, 16, seed=15)
    o, s = kda.kda_linattn(*[x[n] for n in "qkvg"], s0=x["s0"])
    got = kda.kda_linattn_backward(*[x[n] for n in "qkvg"], d["do"],
                                   s0=x["s0"], dsT=d["dsT"])
    pick = [0, 77, 199]
    y = {n: (t[:, :, pick] if n != "s0" else t[:, pick])
         for n, t in x.items()}
    want = ref.linattn(**y, do=d["do"][:, :, pick], dsT=d["dsT"][:, pick])
    within("o", o[:, :, pick], want["o"])
    within("s", s[:, pick], want["s"])
    for n, t in zip(GRADS, got):
        within(n, t[:, pick] if n == "ds0" else t[:, :, pick], want[n])


def test_long_segments_of_the_gradient(kda):
    """enough heads that a sequence would be one segment, but long enough that
    the gradient cuts it: chunks of 32 and 64 tokens, 64 of them at most"""
    x, d = inputs(1, 4500, 1, 1, 16, 16, F, kind="slow", seed=16)
    # the same head many times over fills the GPU; one of them is checked
    H = 600
    y = {n: t.repeat_interleave(H, 1 if n == "s0" else 2).contiguous()
         for n, t in x.items()}
    do = d["do"].repeat_interleave(H, 2).contiguous()
    dsT = d["dsT"].repeat_interleave(H, 1).contiguous()
    want = ref.linattn(**x, **d)
    got = kda.kda_linattn_backward(*[y[n] for n in "qkvg"], do, s0=y["s0"],
                                   dsT=dsT)
    for n, t in zip(GRADS, got):
        t = t if n != "ds0" else t.transpose(0, 1)
        a = t[:, :, 5:6] if n != "ds0" else t[5:6].transpose(0, 1)
        within(n, a, want[n])


def test_segments_that_forget(kda):
    """enough heads that segments are several chunks long, and gates that
    forget their first ones by their end"""
    x, d = inputs(1, 1500, 1, 1, 128, 128, seed=23)
    H = 64
    y = {n: t.repeat_interleave(H, 1 if n == "s0" else 2).contiguous()
         for n, t in x.items()}
    do = d["do"].repeat_interleave(H, 2).contiguous()
    dsT = d["dsT"].repeat_interleave(H, 1).contiguous()
    want = ref.linattn(**x, **d)
    four = [y[n] for n in "qkvg"]
    o, s = kda.kda_linattn(*four, s0=y["s0"])
    within("o", o[:, :, 5:6], want["o"])
    within("s", s[:, 5:6], want["s"])
    got = kda.kda_linattn_backward(*four, do, s0=y["s0"], dsT=dsT)
    for n, t in zip(GRADS, got):
        within(n, t[:, 5:6] if n == "ds0" else t[:, :, 5:6], want[n])


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("Dk,Dv", [(64, 32), (16, 128), (128, 16), (32, 32)])
@pytest.mark.parametrize("want_dg", [False, True])
def test_shared_heads_of_any_width(kda, io, Dk, Dv, want_dg):
    """with and without the gate's gradient, whose sums other kernels make"""
    x, d = inputs(1, 330, 2, 6, Dk, Dv, io, seed=24)
    want = ref.linattn(**x, **d)
    got = kda.kda_linattn_backward(*[x[n] for n in "qkvg"], d["do"],
                                   s0=x["s0"], dsT=d["dsT"], want_dg=want_dg)
    for n, t in zip(GRADS, got):
        if n != "dg" or want_dg:
            within(n, t, want[n])


@pytest.mark.parametrize("io,gate", [(BF, F), (BF, BF), (F, F)])
def test_fixed_decays_of_many_sequences(kda, io, gate):
    x, d = inputs(130, 40, 1, 2, 16, 16, io, gate, kind="fixed", seed=25)
    check(kda, x, d)


@pytest.mark.parametrize("io", [BF, F])
def test_one_token_of_many_sequences(kda, io):
    x, d = inputs(300, 1, 2, 4, 32, 16, io, seed=26)
    check(kda, x, d)


def test_offsets_past_32_bits(kda):
    """More than 2^31 values in each tensor.  With exp(-1) a token, what is 150
    tokens away is 1e-65 of itself: both ends are those of a short sequence."""
    T, H, D, n, keep = (1 << 19) + 77, 32, 128, 300, 150
    gen = torch.Generator(device="cuda").manual_seed(27)

    def r():
        return torch.randn(1, T, H, D, generator=gen, device="cuda", dtype=BF)

    q, k, v, do = r() * 0.125, r() * 0.125, r(), r()
    g = torch.full((1, T, H), -1.0, device="cuda")
    o, s = kda.kda_linattn(q, k, v, g)
    got = kda.kda_linattn_backward(q, k, v, g, do)
    last = slice(T - n, T)
    pick = [0, 31]
    for part, inner in ((slice(0, n), slice(0, keep)),
                        (last, slice(n - keep, n))):
        def cut(t):
            return t[:, part][:, :, pick].contiguous()
        want = ref.linattn(cut(q), cut(k), cut(v), cut(g), do=cut(do))
        for m, t in zip(("o", *GRADS), (o, *got[:4])):
            within(m, cut(t)[:, inner],
                   tuple(w[:, inner] for w in want[m]))
        if part is last:
            within("s", s[:, pick], want["s"])


def test_own_stream_and_workspaces(kda):
    """two calls at once on two streams, each with its workspace"""
    x, d = inputs(1, 1500, 1, 2, 64, 64, seed=17)
    four = [x[n] for n in "qkvg"]
    base = kda.kda_linattn(*four, s0=x["s0"])
    grads = kda.kda_linattn_backward(*four, d["do"], s0=x["s0"],
                                     dsT=d["dsT"])
    n1 = kda.kda_linattn_workspace_size(1, 1500, 1, 2, 64, 64, BF)
    n2 = kda.kda_linattn_backward_workspace_size(1, 1500, 1, 2, 64, 64, BF)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for s in streams:
        for _ in range(3):
            # the workspace's contents do not matter
            w = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                 for n in (n1, n2)]
            s.wait_stream(torch.cuda.current_stream())
            res.append((kda.kda_linattn(*four, s0=x["s0"], workspace=w[0],
                                        stream=s),
                        kda.kda_linattn_backward(
                            *four, d["do"], s0=x["s0"], dsT=d["dsT"],
                            workspace=w[1], stream=s), w))
    torch.cuda.synchronize()
    for a, b, _ in res:
        assert all(torch.equal(p, q) for p, q in zip(a, base))
        assert all(torch.equal(p, q) for p, q in zip(b, grads))
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_linattn(*four, workspace=torch.empty(16, dtype=torch.uint8,
                                                     device="cuda"))


def test_captured_and_replayed(kda):
    """two graphs side by side, replayed with eager work in between"""
    x, d = inputs(1, 1100, 1, 2, 32, 32, seed=18)
    y, e = inputs(1, 1100, 1, 2, 32, 32, kind="fixed", seed=19)

    def run(x, d):
        four = [x[n] for n in "qkvg"]
        o, s = kda.kda_linattn(*four, s0=x["s0"])
        step = kda.kda_linattn_step(
            *[t[:, 0].contiguous() for t in four[:3]],
            four[3] if four[3].dim() == 1 else four[3][:, 0].contiguous(), s)
        return (o, s, step, *kda.kda_linattn_backward(
            *four, d["do"], s0=x["s0"], dsT=d["dsT"]))

    want = [run(x, d), run(y, e)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in ((x, d), (y, e)):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(*a)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*a))
        graphs.append(g)
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            for t in o:
                t.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, w))
        run(x, d)
    x["v"].copy_(x["v"].roll(1, 1))
    graphs[0].replay()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], run(x, d)))


def test_outputs_lie_within_their_tensors(kda):
    """what lies before and behind an output stays as it was"""
    x, d = inputs(1, 130, 1, 2, 16, 32, seed=20)
    four = [x[n] for n in "qkvg"]
    n, m = x["v"].numel(), x["s0"].numel()
    ob = torch.full((n + 128,), 3.0, dtype=BF, device="cuda")
    sb = torch.full((m + 128,), 3.0, device="cuda")
    o, s = kda.kda_linattn(*four, s0=x["s0"], o=ob[64:-64].view_as(x["v"]),
                           s_out=sb[64:-64].view_as(x["s0"]))
    want = kda.kda_linattn(*four, s0=x["s0"])
    assert torch.equal(o, want[0]) and torch.equal(s, want[1])
    for b in (ob, sb):
        assert (b[:64] == 3).all() and (b[-64:] == 3).all()


def test_a_nan_stays_in_its_chunk_and_head(kda):
    """a NaN in v reaches its own and later tokens, and at most the 63 before
    it, of its own head"""
    x, _ = inputs(1, 320, 2, 2, 16, 16, seed=21)
    x["g"].clamp_(min=-1.0)
    four = [x[n] for n in "qkvg"]
    good, _ = kda.kda_linattn(*four)
    x["v"][0, 200, 0, 3] = math.nan
    o, _ = kda.kda_linattn(*four)
    assert torch.equal(o[:, :, 1], good[:, :, 1])
    assert torch.equal(o[:, :137], good[:, :137])
    assert torch.isnan(o[0, 200:, 0, 3]).all()


def test_refusals(kda):
    x, d = inputs(1, 8, 1, 1, 16, 16, seed=22)
    four = [x[n] for n in "qkvg"]
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_linattn(*four, o=four[2])
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_linattn(*four, scale=math.inf)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_linattn(four[0].transpose(1, 2).expand(1, 1, 8, 16)
                        .transpose(1, 2), four[1], four[2],
                        torch.zeros(1, 16, 1, device="cuda")[:, ::2])
    q = torch.randn(1, 8, 1, 48, device="cuda")
    with pytest.raises(kda.KdaError, match="unsupported"):
        kda.kda_linattn(q, q, q, torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_linattn(*four, s0=torch.zeros(1, 1, 16, 16))
