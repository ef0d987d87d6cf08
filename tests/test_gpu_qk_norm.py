"""kda_qk_norm_rope and its gradient on the GPU against the 64-bit formulas,
element by element within derived bounds (linattn_ref), and a block with
linear attention run through the operators it is made of."""
import math

import pytest
import torch

import layer_ref
import linattn_ref as ref
from layer_ref import within

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_74_amd as m
    return m


def rn(*shape, seed=0, dtype=F, scale=1.0):
    gen = torch.Generator().manual_seed(seed * 7919 + sum(shape))
    return (scale * torch.randn(*shape, generator=gen)).to(dtype).cuda()


def turns(lead, rot, far=False, seed=0):
    if not rot:
        return None, None
    gen = torch.Generator().manual_seed(seed)
    pos = torch.randint(-7, 262144 if far else 500, lead, generator=gen,
                        dtype=torch.int32)
    inv = torch.pow(10000.0, -torch.arange(0, rot, 2) / rot)
    return pos.cuda(), inv.float().cuda()


def check(kda, q, k, pos, inv, wq, wk, interleaved=False, eps=EPS, dq=None,
          dk=None):
    """forward, and with dq the gradient"""
    kw = dict(wq=wq, wk=wk, interleaved=interleaved, eps=eps)
    sides = [("q", q, wq, dq)] + ([("k", k, wk, dk)] if k is not None else [])
    out = kda.kda_qk_norm_rope(q, k, pos, inv, **kw)
    for (n, x, w, _), y in zip(sides, out):
        within(n, y, ref.qk_norm(x, w, pos, inv, interleaved, eps))
    if dq is None:
        return out
    got = kda.kda_qk_norm_rope_backward(q, k, pos, inv, dq, dk, **kw)
    for i, (n, x, w, dy) in enumerate(sides):
        dx, dw = ref.qk_norm_grad(x, w, pos, inv, interleaved, eps, dy)
        within("d" + n, got[i], dx)
        if w is None:
            assert got[2 + i] is None
        else:
            within("dw" + n, got[2 + i], dw)
    return out, got


@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("part", [0, 1, 2])
def test_widths(kda, D, dtype, interleaved, part):
    """no rotation, a part of the channels, all"""
    rot = [0, max(16, D // 4), D][part]
    lead = (3, 5)
    pos, inv = turns(lead, rot, far=True)
    q, k = rn(*lead, 6, D, seed=1, dtype=dtype), rn(*lead, 2, D, seed=2,
                                                    dtype=dtype)
    check(kda, q, k, pos, inv, 1 + 0.1 * rn(D, seed=3), 1 + 0.1 * rn(D, seed=4),
          interleaved, dq=rn(*lead, 6, D, seed=5, dtype=dtype),
          dk=rn(*lead, 2, D, seed=6, dtype=dtype))


@pytest.mark.parametrize("rot,interleaved", [(48, False), (80, False),
                                             (112, False), (8, True),
                                             (24, True), (104, True)])
def test_odd_rotations(kda, rot, interleaved):
    """rotated parts that are no power of two"""
    pos, inv = turns((9,), rot)
    q, k = rn(9, 3, 128, seed=7), rn(9, 1, 128, seed=8)
    check(kda, q, k, pos, inv, rn(128, seed=9), None, interleaved,
          dq=rn(9, 3, 128, seed=10), dk=rn(9, 1, 128, seed=11))


@pytest.mark.parametrize("Hq,Hk", [(1, 0), (1, 1), (7, 3), (32, 32), (33, 2)])
@pytest.mark.parametrize("rows", [1, 2, 63, 300])
@pytest.mark.parametrize("D", [16, 128])
def test_heads_and_rows(kda, Hq, Hk, rows, D):
    pos, inv = turns((rows,), 16)
    q = rn(rows, Hq, D, seed=12, dtype=BF)
    k = rn(rows, Hk, D, seed=13, dtype=BF) if Hk else None
    w = 1 + 0.1 * rn(D, seed=14)
    check(kda, q, k, pos, inv, w, w if Hk else None,
          dq=rn(rows, Hq, D, seed=15, dtype=BF),
          dk=rn(rows, Hk, D, seed=16, dtype=BF) if Hk else None)


def test_more_tokens_than_a_pass(kda):
    """the gradient's workgroups take several tokens each"""
    pos, inv = turns((9001,), 32)
    q, k = rn(9001, 2, 64, seed=17, dtype=BF), rn(9001, 1, 64, seed=18,
                                                  dtype=BF)
    w = rn(64, seed=19)
    check(kda, q, k, pos, inv, w, w, dq=rn(9001, 2, 64, seed=20, dtype=BF),
          dk=rn(9001, 1, 64, seed=21, dtype=BF))


@pytest.mark.parametrize("sides", ["q", "k", ""])
def test_one_side_normed(kda, sides):
    pos, inv = turns((21,), 32)
    q, k = rn(21, 4, 64, seed=22), rn(21, 4, 64, seed=23)
    w = rn(64, seed=24)
    check(kda, q, k, pos, inv, w if "q" in sides else None,
          w if "k" in sides else None, dq=rn(21, 4, 64, seed=25),
          dk=rn(21, 4, 64, seed=26))


@pytest.mark.parametrize("dtype", [BF, F])
def test_fused_projection_and_in_place(kda, dtype):
    """q and k as parts of one projection: read there, written elsewhere or
    there; what lies between stays as it was"""
    B, T, Hq, Hk, D = 2, 17, 4, 2, 32
    fused = rn(B, T, (Hq + 2 * Hk) * D, seed=27, dtype=dtype)

    def parts(x):
        return (x[..., :Hq * D].unflatten(-1, (Hq, D)),
                x[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)))

    q, k = parts(fused)
    pos, inv = turns((B, T), 32, far=True)
    w = 1 + 0.1 * rn(D, seed=28)
    kw = dict(wq=w, wk=w, eps=EPS)
    keep = fused.clone()
    a, b = check(kda, q, k, pos, inv, w, w)
    dense = kda.kda_qk_norm_rope(q.contiguous(), k.contiguous(), pos, inv,
                                 **kw)
    assert torch.equal(a, dense[0]) and torch.equal(b, dense[1])
    assert torch.equal(fused, keep)
    grad = rn(B, T, (Hq + 2 * Hk) * D, seed=29, dtype=dtype)
    dqo, dko = parts(grad)
    want = kda.kda_qk_norm_rope_backward(q, k, pos, inv, dqo.contiguous(),
                                         dko.contiguous(), **kw)
    into = torch.full_like(grad, 5.0)
    dq, dk = parts(into)
    got = kda.kda_qk_norm_rope_backward(q, k, pos, inv, dqo, dko, dq=dq,
                                        dk=dk, **kw)
    assert got[0] is dq and got[1] is dk
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert (into[..., (Hq + Hk) * D:] == 5).all()
    kept = grad.clone()
    got = kda.kda_qk_norm_rope_backward(q, k, pos, inv, dqo, dko, dq=dqo,
                                        dk=dko, **kw)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(grad[..., (Hq + Hk) * D:], kept[..., (Hq + Hk) * D:])
    kda.kda_qk_norm_rope(q, k, pos, inv, q_out=q, k_out=k, **kw)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(fused[..., (Hq + Hk) * D:], keep[..., (Hq + Hk) * D:])
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_qk_norm_rope(q, k, pos, inv, q_out=k.expand(B, T, Hk, D)
                             if Hq == Hk else q.as_strided(
                                 q.shape, (T * Hq * D, Hq * D, D, 1)), **kw)


def test_offsets_past_32_bits(kda):
    """tokens 65536 values apart: more than 2^31 values from first to last"""
    rows, D = 40001, 64
    x = torch.empty(rows, 65536, dtype=BF, device="cuda")
    x[:, :6 * D] = rn(rows, 6 * D, seed=40, dtype=BF)
    q, k = (t.unflatten(-1, (2, D)) for t in (x[:, :2 * D], x[:, 2 * D:4 * D]))
    dq = x[:, 4 * D:6 * D].unflatten(-1, (2, D))
    w = rn(D, seed=41)
    pos, inv = turns((rows,), 32)
    kw = dict(wq=w, wk=w, eps=EPS)
    dense = [t.contiguous() for t in (q, k, dq)]
    want = kda.kda_qk_norm_rope_backward(dense[0], dense[1], pos, inv,
                                         dense[2], dense[2], **kw)
    got = kda.kda_qk_norm_rope_backward(q, k, pos, inv, dq, dq, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = kda.kda_qk_norm_rope(dense[0], dense[1], pos, inv, **kw)
    got = kda.kda_qk_norm_rope(q, k, pos, inv, q_out=q, k_out=k, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_far_positions(kda):
    """up to the largest int: the angles are exact in 64 bits.  At 2^31 the
    reference's own product is off by 2^-22, so there the bound is wider by
    2^-21 of the pair."""
    x = rn(6, 1, 16, seed=30)
    inv = torch.pow(10000.0, -torch.arange(0, 16, 2) / 16).float().cuda()
    pos = torch.tensor([0, 1, 262143, 10 ** 6, -10 ** 6, 2 ** 24 + 1],
                       dtype=torch.int32, device="cuda")
    check(kda, x, None, pos, inv, None, None)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 2 ** 30,
                        2 ** 30 + 1, -2 ** 30], dtype=torch.int32,
                       device="cuda")
    y, _ = kda.kda_qk_norm_rope(x, None, pos, inv)
    want, slack = ref.qk_norm(x, None, pos, inv, False, EPS)
    m = x.cpu().double().abs()
    within("y", y, (want, slack + 2.0 ** -21 * (m + m.roll(8, -1))))


def test_exact_quarters(kda):
    """positions that are whole quarter turns"""
    x = rn(9, 1, 16, seed=31)
    inv = torch.full((8,), math.pi / 2, device="cuda")
    pos = torch.arange(-4, 5, dtype=torch.int32, device="cuda")
    check(kda, x, None, pos, inv, None, None)
    check(kda, x, None, pos, inv, None, None, interleaved=True)


@pytest.mark.parametrize("dtype", [BF, F])
def test_special_rows(kda, dtype):
    """rows of zeros, tiny and huge values; an infinity or NaN stays in its
    head, and in channels that pass by where there is no norm"""
    q = rn(8, 2, 64, seed=32, dtype=dtype)
    q[0] = 0
    q[1] *= 1e-4
    q[2] *= 1e12
    pos, inv = turns((8,), 32)
    w = rn(64, seed=33)
    check(kda, q, None, pos, inv, w, None, dq=rn(8, 2, 64, seed=34,
                                                 dtype=dtype))
    good, _ = kda.kda_qk_norm_rope(q, None, pos, inv)
    q[3, 0, 40] = math.inf
    q[4, 1, 50] = math.nan
    q[5, 0, 3] = math.inf   # turned with channel 19
    y, _ = kda.kda_qk_norm_rope(q, None, pos, inv)
    same = torch.ones_like(y, dtype=torch.bool)
    for i, h, c in ((3, 0, [40]), (4, 1, [50]), (5, 0, [3, 19])):
        same[i, h, c] = False
    assert torch.equal(y[same], good[same])
    assert torch.isinf(y[3, 0, 40]) and torch.isnan(y[4, 1, 50])
    assert not torch.isfinite(y[5, 0, 3])


def test_squares_below_the_normal_range(kda):
    """eps = 0 and squares of about 2^-130, multiples of 2^-149: the mean is off
    by two half steps, 2^-149, of at least 2^-132, its root by 2^-18"""
    q = torch.where(rn(5, 3, 64, seed=35) < 0, -2.0 ** -65, 2.0 ** -65.5)
    w = rn(64, seed=36)
    y, _ = kda.kda_qk_norm_rope(q, None, None, None, wq=w, eps=0.0)
    x = q.double()
    want = x / (x * x).mean(-1, keepdim=True).sqrt() * w.double()
    assert ((y.double() - want).abs() <= 2.0 ** -17 * want.abs()).all()
    z, _ = kda.kda_qk_norm_rope(torch.zeros_like(q), None, None, None, wq=w,
                                eps=0.0)
    assert torch.isnan(z).all()


def test_streams_and_graphs(kda):
    q, k = rn(130, 4, 128, seed=35, dtype=BF), rn(130, 2, 128, seed=36,
                                                  dtype=BF)
    dq, dk = rn(130, 4, 128, seed=37, dtype=BF), rn(130, 2, 128, seed=38,
                                                    dtype=BF)
    pos, inv = turns((130,), 128)
    kw = dict(wq=rn(128, seed=39), wk=rn(128, seed=40))

    def run(**more):
        return (*kda.kda_qk_norm_rope(q, k, pos, inv, **kw, **more),
                *kda.kda_qk_norm_rope_backward(q, k, pos, inv, dq, dk, **kw,
                                               **more))

    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for _ in range(3):
        for t in got:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        run()
    q.neg_()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_refusals(kda):
    q, k = rn(5, 2, 32, seed=41, dtype=BF), rn(5, 2, 32, seed=42, dtype=BF)
    pos, inv = turns((5,), 32)
    with pytest.raises(kda.KdaError, match="unsupported"):
        kda.kda_qk_norm_rope(q, k, pos, inv[:12])
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_qk_norm_rope(q, k, pos, inv, q_out=k)
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_qk_norm_rope(q, k, None, None)
    with pytest.raises(ValueError, match="evenly"):
        kda.kda_qk_norm_rope(q.expand(3, 5, 2, 32), None,
                             pos.expand(3, 5).contiguous(), inv)
    with pytest.raises(kda.KdaError, match="invalid"):
        kda.kda_qk_norm_rope(q[:1].expand(5, 2, 32), None, pos, inv)
    with pytest.raises(ValueError, match="cpu|GPU"):
        kda.kda_qk_norm_rope(q, k.cpu(), pos, inv)


def test_a_block_of_the_operators(kda):
    """Projections read as parts of one buffer, normed and rotated, linear
    attention over a prompt and then token by token, its output normed and
    gated, the norms around the block: each step against its reference on what
    it was given, and the prompt's last token against the same token as a
    step."""
    B, T, Hk, H, D, C = 2, 100, 2, 4, 32, 128
    fused = rn(B, T, (2 * Hk + H) * D, seed=43, dtype=BF)
    q, k = (fused[..., i * Hk * D:(i + 1) * Hk * D].unflatten(-1, (Hk, D))
            for i in range(2))
    v = fused[..., 2 * Hk * D:].unflatten(-1, (H, D)).contiguous()
    pos = torch.arange(1000, 1000 + T, dtype=torch.int32,
                       device="cuda").expand(B, T).contiguous()
    inv = turns((1,), D)[1]
    # an L2 norm: w = 1 / sqrt(D), eps = e / D
    w = torch.full((D,), D ** -0.5, device="cuda")
    kw = dict(wq=w, wk=w, eps=EPS / D)
    qn, kn = check(kda, q, k, pos, inv, w, w, eps=EPS / D)
    assert ((qn.float().norm(dim=-1) - 1).abs() < 2 ** -7).all()
    g = -torch.exp2(-torch.arange(1.0, H + 1, device="cuda"))
    want = ref.linattn(qn, kn, v, g)
    o, s = kda.kda_linattn(qn, kn, v, g)
    within("o", o, want["o"])
    z, wo = rn(B, T, H, D, seed=44, dtype=BF), 1 + 0.1 * rn(D, seed=45)
    y = kda.kda_gated_norm(o, z, wo, act="silu")
    within("y", y, layer_ref.gated_norm(o, z, wo, "silu", EPS))
    r, wr = rn(B, T, C, seed=46), rn(C, seed=47)
    r2, x = kda.kda_block_norm(y.view(B, T, C), r, w_pre=wr)
    w1, w2 = layer_ref.block_norm(y.view(B, T, C), r, None, None, wr, None,
                                  1.0, 1.0, EPS)
    within("r", r2, w1)
    within("x", x, w2)
    # back through the block: the gradient of each step is the next one's
    dy, dr, _, _, _ = kda.kda_block_norm_backward(
        y.view(B, T, C), r2, dx=torch.ones_like(x), w_pre=wr)
    do, dz, dw = kda.kda_gated_norm_backward(o, z, wo, dy.view_as(o),
                                             act="silu")
    grads = kda.kda_linattn_backward(qn, kn, v, g, do)
    want = ref.linattn(qn, kn, v, g, do=do)
    for n, a in zip(("dq", "dk", "dv", "dg"), grads):
        within(n, a, want[n])
    into = torch.empty_like(fused)
    dq, dk = (into[..., i * Hk * D:(i + 1) * Hk * D].unflatten(-1, (Hk, D))
              for i in range(2))
    kda.kda_qk_norm_rope_backward(q, k, pos, inv, grads[0], grads[1], dq=dq,
                                  dk=dk, **kw)
    for n, a, b, c in (("dq", dq, q, grads[0]), ("dk", dk, k, grads[1])):
        within(n, a, ref.qk_norm_grad(b, w, pos, inv, False, EPS / D, c)[0])
    # the last tokens one by one, behind the others' state
    m = 90
    _, st = kda.kda_linattn(*[t[:, :m].contiguous() for t in (qn, kn, v)], g)
    want = ref.linattn(qn, kn, v, g)
    outs = []
    for t in range(m, T):
        a, b = kda.kda_qk_norm_rope(q[:, t:t + 1], k[:, t:t + 1],
                                    pos[:, t:t + 1].contiguous(), inv, **kw)
        assert torch.equal(a[:, 0], qn[:, t]) and torch.equal(b[:, 0],
                                                             kn[:, t])
        outs.append(kda.kda_linattn_step(a[:, 0], b[:, 0],
                                         v[:, t].contiguous(), g, st))
    within("steps", torch.stack(outs, 1),
           tuple(t[:, m:] for t in want["o"]))
    within("state", st, want["s"])
