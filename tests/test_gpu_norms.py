"""kda_gated_norm, kda_block_norm and their gradients on the GPU against the
64-bit references, element by element within derived bounds (layer_ref), and
a block of such a model run through them and the mixers."""
import math

import pytest
import torch

import layer_ref as ref
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


def gated(kda, o, z, w, act, dy):
    y = kda.kda_gated_norm(o, z, w, act=act, eps=EPS)
    within("y", y, ref.gated_norm(o, z, w, act, EPS))
    got = kda.kda_gated_norm_backward(o, z, w, dy, act=act, eps=EPS)
    want = ref.gated_norm(o, z, w, act, EPS, dy)
    for n, a, b in zip(("do", "dz", "dw"), got, want):
        if b is None:
            assert a is None
        else:
            within(n, a, b)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("act", ["sigmoid", "silu", None])
@pytest.mark.parametrize("lead", [(1, 1), (3, 5), (129, 7)])
def test_gated_norm(kda, D, dtype, act, lead):
    o = rn(*lead, D, seed=1, dtype=dtype, scale=3.0)
    z = rn(*lead, D, seed=2, dtype=dtype) if act else None
    gated(kda, o, z, 1 + 0.1 * rn(D, seed=3), act or "sigmoid",
          rn(*lead, D, seed=4, dtype=dtype))


def test_gated_norm_more_rows_than_a_pass(kda):
    """the gradient's workgroups take several rows each"""
    o = rn(40001, 1, 128, seed=5, dtype=BF)
    z = rn(40001, 1, 128, seed=6, dtype=BF)
    gated(kda, o, z, rn(128, seed=7), "silu", rn(40001, 1, 128, seed=8,
                                                 dtype=BF))


@pytest.mark.parametrize("dtype", [BF, F])
def test_gated_norm_far_values(kda, dtype):
    """rows of zeros, of tiny and of huge values, gates far out"""
    o = rn(8, 1, 64, seed=9, dtype=dtype)
    o[0] = 0
    o[1] *= 1e-4
    o[2] *= 1e12
    o[3, 0, 1:] = 0
    z = rn(8, 1, 64, seed=10, dtype=dtype)
    z[4], z[5], z[6] = 60.0, -60.0, -10.0
    gated(kda, o, z, rn(64, seed=11), "silu", rn(8, 1, 64, seed=12,
                                                 dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, F])
def test_gate_gradient_far_out(kda, dtype):
    """dz of the sigmoid gate keeps its relative accuracy where the gate is
    nearly 1 or 0: with a row norm off by rr, the derivative's exponential by
    (|z| + 8) 2u (its argument |z| u, a few u for the rest) and the products,
    the value is off by that share of itself and its own rounding."""
    o = rn(24, 1, 32, seed=60, dtype=dtype)
    z = rn(24, 1, 32, seed=61, dtype=dtype)
    z += (torch.arange(24, device="cuda") * 6.0 - 69.0).view(24, 1, 1).to(dtype)
    w, dy = rn(32, seed=62), rn(24, 1, 32, seed=63, dtype=dtype)
    _, dz, _ = kda.kda_gated_norm_backward(o, z, w, dy, eps=EPS)
    o8, z8, w8, dy8 = map(ref.c8, (o, z, w, dy))
    r, rr = ref._rms(o8, EPS)
    want = dy8 * o8 * r * w8 * torch.sigmoid(z8) * torch.sigmoid(-z8)
    rel = rr + (z8.abs() + 8) * 2 * ref.U + 8 * ref.U
    within("dz", dz, (want, rel * want.abs()))


def test_gated_norm_nan_stays_in_its_row(kda):
    o, z = rn(50, 3, 32, seed=13, dtype=BF), rn(50, 3, 32, seed=14, dtype=BF)
    w, dy = rn(32, seed=15), rn(50, 3, 32, seed=16, dtype=BF)
    y = kda.kda_gated_norm(o, z, w)
    do, dz, _ = kda.kda_gated_norm_backward(o, z, w, dy)
    o[7, 1, 3] = math.nan
    y2 = kda.kda_gated_norm(o, z, w)
    do2, dz2, _ = kda.kda_gated_norm_backward(o, z, w, dy)
    for a, b in ((y, y2), (do, do2), (dz, dz2)):
        assert bool(torch.isnan(b[7, 1]).all())
        b[7, 1] = a[7, 1]
        assert torch.equal(a, b)


def block(kda, R, C, io=BF, res=F, post=True, pre=True, act="sigmoid",
          dr=True, rs=1.0, bs=0.5, seed=20):
    y, r = rn(R, C, seed=seed, dtype=io), rn(R, C, seed=seed + 1, dtype=res,
                                             scale=4.0)
    z = rn(R, C, seed=seed + 2, dtype=io) if act else None
    wp = 1 + 0.1 * rn(C, seed=seed + 3) if post else None
    wq = 1 + 0.1 * rn(C, seed=seed + 4) if pre else None
    kw = dict(z=z, w_post=wp, w_pre=wq, act=act or "sigmoid", res_scale=rs,
              branch_scale=bs, eps=EPS)
    h, x = kda.kda_block_norm(y, r, **kw)
    wh, wx = ref.block_norm(y, r, wp, z, wq, act, rs, bs, EPS)
    within("r_out", h, wh)
    if pre:
        within("x", x, wx)
    else:
        assert x is None
    r2 = r.clone()
    h2, x2 = kda.kda_block_norm(y, r2, r_out=r2, **kw)
    assert h2 is r2 and torch.equal(h, r2)
    assert x is None or torch.equal(x, x2)
    dx = rn(R, C, seed=seed + 5, dtype=io) if pre else None
    dro = rn(R, C, seed=seed + 6, dtype=res) if dr else None
    got = kda.kda_block_norm_backward(y, h, dx=dx, dr_out=dro, **kw)
    want = ref.block_norm_grad(y, h, dx, dro, wp, z, wq, act, rs, bs, EPS)
    for n, a, b in zip(("dy", "dr", "dz", "dw_post", "dw_pre"), got, want):
        if b is None:
            assert a is None, n
        else:
            within(n, a, b)


@pytest.mark.parametrize("C", [1, 7, 8, 63, 64, 100, 512, 520, 1001, 2048,
                               4096, 4097, 5000, 8192, 8200, 10001, 16384])
def test_block_norm_widths(kda, C):
    block(kda, 5, C)


@pytest.mark.parametrize("io,res", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("act", ["sigmoid", "silu", None])
@pytest.mark.parametrize("C", [96, 333])
def test_block_norm_types(kda, io, res, act, C):
    block(kda, 17, C, io, res, act=act, rs=0.75, seed=30)


@pytest.mark.parametrize("post,pre,dr", [(1, 1, 0), (0, 1, 1), (0, 1, 0),
                                         (1, 0, 1), (0, 0, 1)])
@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("C", [256, 77])
def test_block_norm_parts(kda, post, pre, dr, act, C):
    block(kda, 9, C, post=bool(post), pre=bool(pre), dr=bool(dr), act=act,
          seed=40)


@pytest.mark.parametrize("R", [1, 2, 511, 512, 513, 3001])
def test_block_norm_rows(kda, R):
    """fewer and more rows than the gradient's workgroups"""
    block(kda, R, 136, BF, BF, seed=50)


def test_block_norm_largest_rows(kda):
    for io, res, C in ((F, F, 16384), (BF, F, 16383), (F, F, 16383)):
        block(kda, 3, C, io, res, act="silu", seed=60)


@pytest.mark.parametrize("C", [2, 4, 6, 9, 15, 71, 72, 135, 136, 137, 263,
                               264, 519, 527, 4095, 4104, 4107, 8191, 8199,
                               8200, 8201, 12296])
@pytest.mark.parametrize("io,res", [(F, F), (BF, F), (BF, BF)])
def test_block_norm_layout_borders(kda, C, io, res):
    """widths where the lanes of a row, the pieces of a thread or the tail
    change, with rows that do not fill the last workgroup's lanes"""
    block(kda, 37 if C < 4000 else 5, C, io, res, act="silu", seed=130)


@pytest.mark.parametrize("C", [1, 3, 65, 129, 777, 8197])
@pytest.mark.parametrize("dtype", [BF, F])
def test_block_norm_writes_rows_only(kda, C, dtype):
    """what lies behind the last row stays as it was, the tail's stores and
    the vectors at odd addresses included"""
    R, n = 13, 13 * C
    y, r = rn(R, C, seed=140, dtype=dtype), rn(R, C, seed=141, dtype=dtype)
    w = rn(C, seed=142)
    h, x = kda.kda_block_norm(y, r, w_post=w, w_pre=w)
    bufs = [torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
            for _ in range(2)]
    ho, xo = (b[:n].view(R, C) for b in bufs)
    kda.kda_block_norm(y, r, w_post=w, w_pre=w, r_out=ho, x=xo)
    assert torch.equal(h, ho) and torch.equal(x, xo)
    for b in bufs:
        assert bool((b[n:] == 7).all())


def test_norms_repeatable_and_captured(kda):
    o, z, dy = (rn(700, 4, 64, seed=70 + i, dtype=BF) for i in range(3))
    w = rn(64, seed=74)
    y, r, g, dx = (rn(600, 256, seed=75 + i, dtype=BF) for i in range(4))
    wp, wq = rn(256, seed=79), rn(256, seed=80)
    kw = dict(z=g, w_post=wp, w_pre=wq)

    def work():
        h, x = kda.kda_block_norm(y, r, **kw)
        return (h, x, *kda.kda_block_norm_backward(y, h, dx=dx, dr_out=r,
                                                   **kw),
                kda.kda_gated_norm(o, z, w),
                *kda.kda_gated_norm_backward(o, z, w, dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = work()
    for i in range(5):
        y.copy_(rn(600, 256, seed=90 + i, dtype=BF))
        o.copy_(rn(700, 4, 64, seed=95 + i, dtype=BF))
        gr.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        for _ in range(2):
            for a, b in zip(got, work()):
                assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_norms_on_another_stream(kda):
    y, r = rn(2000, 512, seed=100, dtype=BF), rn(2000, 512, seed=101)
    w = rn(512, seed=102)
    want = kda.kda_block_norm(y, r, w_pre=w)
    grads = kda.kda_block_norm_backward(y, want[0], dx=y, w_pre=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_block_norm(y, r, w_pre=w, stream=s)
    g2 = kda.kda_block_norm_backward(y, got[0], dx=y, w_pre=w, stream=s)
    torch.cuda.synchronize()
    for a, b in zip((*want, *grads), (*got, *g2)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_rows_past_32_bits(kda):
    """more than 2^31 elements: the last rows as on their own"""
    R, C = 140000, 16384
    assert R * C > 2 ** 31
    y = torch.zeros(R, C, dtype=BF, device="cuda")
    tail = rn(5, C, seed=110, dtype=BF)
    y[-5:] = tail
    w = 1 + 0.1 * rn(C, seed=111)
    h, x = kda.kda_block_norm(y, y, w_pre=w)
    h2, x2 = kda.kda_block_norm(tail, tail, w_pre=w)
    assert torch.equal(h[-5:], h2) and torch.equal(x[-5:], x2)
    o = y.view(-1, 128)
    z = h.view(-1, 128)
    n = kda.kda_gated_norm(o, z, w[:128].contiguous())
    n2 = kda.kda_gated_norm(tail.view(-1, 128), h2.view(-1, 128),
                            w[:128].contiguous())
    assert torch.equal(n[-n2.shape[0]:], n2)


def test_block_of_a_model(kda):
    """prefill of one block on two mixers (the KDA layer, then the scan) with
    the norms between, then decode steps of the same block continuing it: the
    steps equal the prefill of the longer sequence.

    fp32 throughout; KDA's own fp32 bar is 1e-4 of the largest value, and the
    norms keep relative errors (their rows' roots are near 1 here), so the
    chain is held to that bar for each of its two mixers."""
    B, T, H, D, L = 2, 150, 2, 64, 6
    C, N = H * D, 150 + 6
    a = dict(h=rn(B, N, C, seed=120), gate=rn(B, N, H, D, seed=121),
             g=-rn(B, N, H, D, seed=122).abs(),
             beta=torch.sigmoid(rn(B, N, H, seed=123)))
    w, wp, wq = (1 + 0.1 * rn(n, seed=124 + i)
                 for i, n in enumerate((D, C, C)))

    def unit(v):
        return torch.nn.functional.normalize(v, dim=-1).contiguous()

    def pieces(lo, hi):
        return {k: v[:, lo:hi].contiguous() for k, v in a.items()}

    def run(p, s, hs, step):
        """one block; s, hs: the two mixers' states"""
        q = unit(p["h"].view(B, -1, H, D))
        k = unit(p["gate"])
        v = p["h"].view(B, -1, H, D)
        if step:
            o = kda.kda_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(),
                                    v[:, 0].contiguous(),
                                    p["g"][:, 0].contiguous(),
                                    p["beta"][:, 0].contiguous(), s)[:, None]
        else:
            o, s = kda.kda_prefill(q, k, v, p["g"], p["beta"], s0=s)
        o = kda.kda_gated_norm(o.contiguous(), p["gate"], w)
        r, x = kda.kda_block_norm(o.view(B, -1, C), p["h"], w_post=wp,
                                  w_pre=wq, branch_scale=0.5)
        x = x.view(B, -1, H, D)
        if step:
            y = kda.kda_scan_step(x[:, 0].contiguous(),
                                  p["g"][:, 0].contiguous(),
                                  p["beta"][:, 0].contiguous(), hs)[:, None]
        else:
            y, hs, _ = kda.kda_scan(x, p["g"], p["beta"], h0=hs)
        y = kda.kda_gated_norm(y.contiguous(), p["gate"], w, act="silu")
        r, x = kda.kda_block_norm(y.view(B, -1, C), r, w_pre=wq)
        return r, x, s, hs

    s0 = torch.zeros(B, H, D, D, device="cuda")
    h0 = torch.zeros(B, H, D, device="cuda")
    want = run(a, s0, h0, False)
    r, x, s, hs = run(pieces(0, T), s0, h0, False)
    rs, xs = [r], [x]
    for t in range(T, T + L):
        r, x, s, hs = run(pieces(t, t + 1), s, hs, True)
        rs.append(r)
        xs.append(x)
    for name, got, ref_ in (("r", torch.cat(rs, 1), want[0]),
                            ("x", torch.cat(xs, 1), want[1]),
                            ("S", s, want[2]), ("h", hs, want[3])):
        err = float((got - ref_).abs().max() / ref_.abs().max())
        assert err <= 2e-4, (name, err)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gate_of_an_fp32_stream(kda, act):
    """bf16 gates that reach fp32 results are good to fp32: with y = 1, r = 0
    and no norms r_out is the gate itself, and dw of a head of equal values the
    gate times its norm.

    u = 2^-24.  exp(-|z|) is within 1.5 ulp = 3u, 1 + e then within 1.5u + u,
    its reciprocal 2u more, the product with e (z < 0) 4u more; silu's product
    u: 10u.  dw: the norm of 16 values (16 / 2 + 8) u, products 2u."""
    z = torch.arange(-80, 80, 1 / 16).to(BF)
    z = z[:len(z) // 16 * 16].view(-1, 16)
    z8 = z.double()
    want = torch.sigmoid(z8) * (z8 if act == "silu" else 1.0)
    one = torch.ones(z.shape, dtype=BF, device="cuda")
    r, _ = kda.kda_block_norm(one, torch.zeros(z.shape, device="cuda"),
                              z=z.cuda(), act=act)
    within("r_out", r, (want, 10 * ref.U * want.abs()))
    # one row a call: dw is then the row's own term
    w = torch.ones(16, device="cuda")
    for i in range(0, z.shape[0], 8):
        _, _, dw = kda.kda_gated_norm_backward(one[i:i + 1], z[i:i + 1].cuda(),
                                               w, one[i:i + 1], act=act,
                                               eps=EPS)
        n = want[i] / math.sqrt(1 + EPS)
        within("dw", dw, (n, 28 * ref.U * n.abs()))


@pytest.mark.parametrize("dtype", [BF, F])
def test_gates_at_the_ends_of_the_range(kda, dtype):
    """gates that are infinite, huge or NaN: the formula's limits"""
    z = torch.tensor([math.inf, 3e38, 100.0, 0.0, -100.0, -3e38, -math.inf,
                      math.nan], device="cuda").to(dtype).view(1, -1)
    one = torch.ones(1, 8, dtype=dtype, device="cuda")
    r = torch.zeros(1, 8, device="cuda")
    s = torch.tensor([1, 1, 1, 0.5, 0, 0, 0, math.nan])
    got = kda.kda_block_norm(one, r, z=z)[0].cpu()[0]
    assert torch.allclose(got, s, rtol=0, atol=1e-37, equal_nan=True)
    silu = kda.kda_block_norm(one, r, z=z, act="silu")[0].cpu()[0]
    want = s * z.cpu().float()[0]  # -inf * 0 is NaN
    assert torch.allclose(silu, want, rtol=0, atol=1e-37, equal_nan=True)
    dz = kda.kda_block_norm_backward(one, r, dr_out=r + 1, z=z)[2].cpu()[0]
    want = torch.tensor([0, 0, 0, 0.25, 0, 0, 0, math.nan])
    assert torch.allclose(dz.float(), want, rtol=0, atol=1e-37, equal_nan=True)
