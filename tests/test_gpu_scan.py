"""kda_scan, kda_scan_backward and kda_scan_step on the GPU against the
64-bit reference, element by element within derived bounds (layer_ref)."""
import math

import pytest
import torch

import layer_ref as ref
from gpu_common import say
from layer_ref import within

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_74_amd as m
    return m


def inputs(B, T, H, D, io=BF, gt=F, head=False, beta=True, h0=True,
           lengths=None, kind="softplus", seed=0, reset=1 / 64):
    gen = torch.Generator().manual_seed(seed + 13 * T + D)

    def rn(*s):
        return torch.randn(*s, generator=gen)
    z = rn(B, T, H) if head else rn(B, T, H, D)
    g = torch.log1p(-0.002 * torch.sigmoid(z)) if kind == "slow" else \
        -torch.nn.functional.softplus(z)
    g[torch.rand(B, T, H, generator=gen) < reset] = -math.inf
    return dict(
        x=rn(B, T, H, D).to(io).cuda(), g=g.to(gt).cuda(),
        beta=torch.sigmoid(rn(B, T, H)).to(gt).cuda() if beta else None,
        h0=rn(B, H, D).cuda() if h0 else None,
        lengths=None if lengths is None else
        torch.tensor(lengths, dtype=torch.int32, device="cuda"),
        dy=rn(B, T, H, D).to(io).cuda(), dhT=rn(B, H, D).cuda())


def forward(kda, q, **kw):
    return kda.kda_scan(q["x"], q["g"], q["beta"], h0=q["h0"],
                        lengths=q["lengths"], **kw)


def backward(kda, q, **kw):
    return kda.kda_scan_backward(q["x"], q["g"], q["beta"], q["dy"],
                                 h0=q["h0"], dhT=q["dhT"],
                                 lengths=q["lengths"], **kw)


def check(kda, q):
    want = ref.scan(**q)
    y, h, cs = forward(kda, q, chunk_states=True)
    within("y", y, want["y"])
    within("h_out", h, want["h"])
    within("chunk_states", cs, want["chunk"])
    for states in (None, cs):
        dx, dg, db, d0 = backward(kda, q, chunk_states=states)
        within("dx", dx, want["dx"])
        within("dg", dg, want["dg"])
        within("dh0", d0, want["dh0"])
        if db is not None:
            within("dbeta", db, want["dbeta"])


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 127, 128, 129, 257, 640])
def test_lengths_from_one(kda, T):
    check(kda, inputs(2, T, 3, 32))


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("io,gt", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("head", [False, True])
def test_types_and_heads(kda, D, io, gt, head):
    # 5 heads: channel blocks that end inside a workgroup's 128 channels
    check(kda, inputs(2, 133, 5, D, io, gt, head, seed=1))


@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("head", [False, True])
def test_optional_inputs(kda, beta, h0, head):
    q = inputs(1, 200, 2, 64, head=head, beta=beta, h0=h0, seed=2)
    check(kda, q)
    q["dhT"] = None
    check(kda, q)


def test_one_head_of_16(kda):
    check(kda, inputs(3, 70, 1, 16, F, F, seed=3))


@pytest.mark.parametrize("head", [False, True])
def test_ragged(kda, head):
    """empty sequences, lengths on and beside chunk ends, out-of-range ones
    (clamped); what lies behind a sequence's end is never used"""
    n = [0, 1, 127, 128, 129, 300, -5, 900]
    q = inputs(8, 300, 3, 32, head=head, lengths=n, seed=4)
    for b, m in enumerate(n):
        m = min(max(m, 0), 300)
        for k in ("x", "g", "beta", "dy"):
            q[k][b, m:] = math.nan
        q["x"][b, m + 1:] = math.inf
    check(kda, q)
    y = forward(kda, q)[0]
    dx, dg, db, _ = backward(kda, q)
    for b, m in enumerate(n):
        m = min(max(m, 0), 300)
        for v in (y, dx, dg, db):
            assert bool((v[b, m:] == 0).all()), b


def test_slow_forgetting(kda):
    check(kda, inputs(1, 2000, 1, 32, F, F, kind="slow", reset=0, seed=5))


def test_long_and_few_channels(kda):
    """many chunks in one column: the states' hand-over from chunk to
    chunk"""
    q = inputs(1, 40000, 1, 16, kind="slow", reset=1 / 20000, seed=6)
    check(kda, q)


def test_forgetting_is_exact(kda):
    """g = -inf cuts the sequence: what comes after equals a fresh start, bit
    for bit where the chunks line up"""
    q = inputs(1, 512, 2, 64, seed=7, reset=0)
    q["g"][:, 256] = -math.inf
    y, _, _ = forward(kda, q)
    r = {k: (v[:, 256:].contiguous() if v is not None and v.dim() > 2 and
             k not in ("h0", "dhT") else v) for k, v in q.items()}
    r["h0"] = torch.full_like(q["h0"], 7.0)
    y2, _, _ = forward(kda, r)
    assert torch.equal(y[:, 256:], y2)


def test_infinite_state_forgotten_is_nan(kda):
    """0 * inf: as the formula has it"""
    q = inputs(1, 6, 1, 16, F, F, seed=8, reset=0)
    q["h0"][:] = math.inf
    q["g"][:, 3] = -math.inf
    y, h, _ = forward(kda, q)
    assert bool(torch.isinf(y[:, :3]).all()) and bool(torch.isnan(h).all())


def test_nan_stays_in_its_channel(kda):
    q = inputs(1, 400, 2, 64, seed=9, reset=0)
    want = forward(kda, q)[0]
    q["x"][0, 150, 1, 5] = math.nan
    y, h, _ = forward(kda, q)
    assert bool(torch.isnan(y[0, 150:, 1, 5]).all())
    assert bool(torch.isnan(h[0, 1, 5]))
    y[0, 150:, 1, 5] = want[0, 150:, 1, 5]
    assert torch.equal(y, want)


def test_repeatable(kda):
    q = inputs(2, 3000, 3, 128, kind="slow", seed=10)
    a = (*forward(kda, q, chunk_states=True), *backward(kda, q))
    for _ in range(5):
        b = (*forward(kda, q, chunk_states=True), *backward(kda, q))
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_states_given_or_recomputed_agree(kda):
    q = inputs(2, 1000, 3, 64, seed=11)
    cs = forward(kda, q, chunk_states=True)[2]
    for u, v in zip(backward(kda, q), backward(kda, q, chunk_states=cs)):
        assert torch.equal(u, v)


def test_state_in_place_and_pieces(kda):
    """h_out may be h0; a sequence run in pieces, its end token by token, is
    the sequence"""
    q = inputs(2, 300, 3, 64, F, F, seed=12)
    want = ref.scan(q["x"], q["g"], q["beta"], q["h0"])
    h = q["h0"].clone()
    ys = []
    for lo, hi in [(0, 130), (130, 131), (131, 290)]:
        s = slice(lo, hi)
        y, h2, _ = kda.kda_scan(
            q["x"][:, s].contiguous(), q["g"][:, s].contiguous(),
            q["beta"][:, s].contiguous(), h0=h, h_out=h)
        assert h2 is h
        ys.append(y)
    for t in range(290, 300):
        ys.append(kda.kda_scan_step(
            q["x"][:, t].contiguous(), q["g"][:, t].contiguous(),
            q["beta"][:, t].contiguous(), h)[:, None])
    within("y", torch.cat(ys, 1), want["y"])
    within("h", h, want["h"])


@pytest.mark.parametrize("N,H,D", [(1, 1, 16), (3, 5, 32), (7, 3, 128),
                                   (256, 32, 128)])
@pytest.mark.parametrize("io,gt", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("head,beta", [(False, True), (True, False)])
def test_step(kda, N, H, D, io, gt, head, beta):
    q = inputs(N, 1, H, D, io, gt, head, beta, seed=13)
    want = ref.scan(q["x"], q["g"], q["beta"], q["h0"])
    h = q["h0"].clone()
    y = kda.kda_scan_step(q["x"][:, 0].contiguous(), q["g"][:, 0].contiguous(),
                          None if not beta else
                          q["beta"][:, 0].contiguous(), h)
    within("y", y, (want["y"][0][:, 0], want["y"][1][:, 0]))
    within("h", h, want["h"])


def guarded(shape, dtype, fill=-77.0, pad=64):
    n = math.prod(shape)
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape)


def test_writes_only_its_outputs(kda):
    """the elements around y, h_out, the chunk states and the workspace stay
    as they were; every element of the outputs is written"""
    B, T, H, D = 2, 261, 5, 16
    q = inputs(B, T, H, D, lengths=[261, 100], seed=14)
    want = forward(kda, q, chunk_states=True)
    bufs = [guarded(s, d) for s, d in [
        ((B, T, H, D), BF), ((B, H, D), F), ((B, 3, H, D), F)]]
    need = kda.kda_scan_workspace_size(B, T, H, D)
    wb = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    forward(kda, q, y=bufs[0][1], h_out=bufs[1][1], chunk_states=bufs[2][1],
            workspace=wb[256:256 + need])
    for (buf, view), w in zip(bufs, want):
        assert torch.equal(view, w)
        assert bool((buf[:64] == -77).all()) and bool((buf[-64:] == -77).all())
    assert bool((wb[:256] == 0x5a).all()) and bool((wb[-256:] == 0x5a).all())
    need = kda.kda_scan_backward_workspace_size(B, T, H, D)
    wb = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    backward(kda, q, workspace=wb[256:256 + need])
    assert bool((wb[:256] == 0x5a).all()) and bool((wb[-256:] == 0x5a).all())


def test_dirty_workspace(kda):
    q = inputs(1, 1500, 2, 64, seed=15)
    a, d = forward(kda, q), backward(kda, q)
    n = kda.kda_scan_backward_workspace_size(1, 1500, 2, 64)
    for v in (0, 0xff, 0x7f):
        ws = torch.full((n,), v, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            b = forward(kda, q, workspace=ws)
            e = backward(kda, q, workspace=ws)
            assert all(torch.equal(u, w) for u, w in zip(a[:2], b[:2]))
            assert all(torch.equal(u, w) for u, w in zip(d, e))


def test_streams_side_by_side(kda):
    """two sequences' scans on two streams at once, each with its own
    workspace"""
    qs = [inputs(1, 6000, 4, 128, seed=16 + i) for i in range(2)]
    want = [(forward(kda, q), backward(kda, q)) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append((forward(kda, qs[i], stream=s),
                           backward(kda, qs[i], stream=s)))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for f, b in runs:
            assert all(torch.equal(u, v) for u, v in zip(w[0][:2], f[:2]))
            assert all(torch.equal(u, v) for u, v in zip(w[1], b))


def test_captured_and_replayed(kda):
    """forward, backward and steps in one graph, two graphs over one
    workspace, new inputs between replays, eager calls in between"""
    q = inputs(2, 700, 3, 64, seed=20)
    n = kda.kda_scan_backward_workspace_size(2, 700, 3, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    h = q["h0"].clone()

    def work():
        y, ho, cs = forward(kda, q, chunk_states=True, workspace=ws)
        h.copy_(ho)
        s = kda.kda_scan_step(q["x"][:, 0].contiguous(),
                              q["g"][:, 0].contiguous(),
                              q["beta"][:, 0].contiguous(), h)
        return (y, ho, cs, s, h,
                *backward(kda, q, chunk_states=cs, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = work()
        graphs.append((gr, out))
    for r in range(6):
        new = inputs(2, 700, 3, 64, seed=30 + r)
        for k in q:
            if q[k] is not None:
                q[k].copy_(new[k])
        gr, out = graphs[r % 2]
        gr.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        want = work()
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v), r


def test_offsets_past_32_bits(kda):
    """more than 2^31 elements: the last tokens, behind a cut, against the
    reference; and their gradients"""
    T, H, D = 540000, 32, 128
    assert T * H * D > 2 ** 31
    x = torch.zeros(1, T, H, D, dtype=BF, device="cuda")
    g = torch.full((1, T, H), -0.5, dtype=BF, device="cuda")
    q = inputs(1, 200, H, D, BF, BF, head=True, seed=40)
    q["g"][:, 0] = -math.inf
    for name, dst in (("x", x), ("g", g)):
        dst[:, T - 200:] = q[name]
    beta = torch.ones(1, T, H, dtype=BF, device="cuda")
    beta[:, T - 200:] = q["beta"]
    say("offsets: forward")
    y, h, _ = kda.kda_scan(x, g, beta)
    q["h0"] = None
    q["dhT"] = None
    want = ref.scan(**q)
    within("y", y[:, T - 200:], want["y"])
    within("h", h, want["h"])
    assert bool((y[:, T - 400:T - 200] == 0).all())
    dy = y.zero_()
    dy[:, T - 200:] = q["dy"]
    say("offsets: backward")
    dx, dg, db, _ = kda.kda_scan_backward(x, g, beta, dy)
    within("dx", dx[:, T - 200:], want["dx"])
    within("dg", dg[:, T - 200:], want["dg"])
    within("dbeta", db[:, T - 200:], want["dbeta"])


@pytest.mark.parametrize("T", [896, 1024, 1025, 1152, 4096, 4097, 4224, 8193])
def test_chunk_groups(kda, T):
    """chunk counts on and beside the hand-over's groups (8 chunks) and
    supergroups (4 groups), forward and from the other end"""
    check(kda, inputs(1, T, 2, 16, kind="slow", reset=0, seed=50))


@pytest.mark.parametrize("B,T,H,D", [(300, 3, 1, 16), (3, 1100, 5, 128),
                                     (65, 130, 3, 32), (1, 129, 40, 64)])
def test_many_columns(kda, B, T, H, D):
    check(kda, inputs(B, T, H, D, seed=51))


def test_small_call_after_a_large_one(kda):
    """a workspace that held a longer call's words serves a shorter one"""
    big, small = inputs(2, 5000, 2, 64, seed=52), inputs(2, 200, 2, 64, seed=53)
    want = (forward(kda, small), backward(kda, small))
    n = kda.kda_scan_backward_workspace_size(2, 5000, 2, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        forward(kda, big, workspace=ws)
        backward(kda, big, workspace=ws)
        f, b = (forward(kda, small, workspace=ws),
                backward(kda, small, workspace=ws))
        assert all(torch.equal(u, v) for u, v in zip(want[0][:2], f[:2]))
        assert all(torch.equal(u, v) for u, v in zip(want[1], b))


def test_graphs_side_by_side(kda):
    """two captured scans with workspaces of their own, replayed on two
    streams at once"""
    qs = [inputs(1, 5000, 4, 128, seed=60 + i) for i in range(2)]
    want = [forward(kda, q) for q in qs]
    n = kda.kda_scan_workspace_size(1, 5000, 4, 128)
    work = []
    for q in qs:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = forward(kda, q, workspace=ws)
        work.append((gr, out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for gr, _, _, s in work:
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for w, (_, out, _, _) in zip(want, work):
            assert all(torch.equal(u, v) for u, v in zip(w[:2], out[:2]))


def test_refuses_strided_tensors(kda):
    q = inputs(2, 10, 2, 32, seed=70)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_scan(q["x"].transpose(0, 1).contiguous().transpose(0, 1),
                     q["g"])
    h = torch.zeros(2, 2, 64, device="cuda")[..., ::2]
    x, g = q["x"][:, 0].contiguous(), q["g"][:, 0].contiguous()
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_scan_step(x, g, None, h)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_scan_step(x, g.cpu(), None, q["h0"])
    with pytest.raises(kda.KdaError):  # a workspace that is too small
        kda.kda_scan(q["x"], q["g"], workspace=torch.empty(
            16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kda.KdaError):  # y is x
        kda.kda_scan(q["x"], q["g"], y=q["x"])


@pytest.mark.parametrize("T", [129, 300, 1500, 5000])
def test_state_in_place_over_many_chunks(kda, T):
    """the final state written over the initial one while other chunks of the
    sequence are still to read it: every chunk starts from the initial one"""
    q = inputs(3, T, 3, 128, kind="slow", reset=0, seed=80)
    q["h0"] *= 100  # a chunk that started elsewhere would show
    y, h, _ = forward(kda, q)
    for _ in range(20):
        st = q["h0"].clone()
        y2, h2, _ = kda.kda_scan(q["x"], q["g"], q["beta"], h0=st, h_out=st)
        assert h2 is st and torch.equal(h, st) and torch.equal(y, y2)


@pytest.mark.parametrize("T", [1, 100, 128, 129, 700])
def test_gradient_from_chunk_states_alone(kda, T):
    """the chunk states take the place of h0, which the forward call may have
    overwritten (h_out = h0)"""
    q = inputs(2, T, 3, 64, seed=92, reset=0)
    want = backward(kda, q)
    h = q["h0"].clone()
    _, _, cs = kda.kda_scan(q["x"], q["g"], q["beta"], h0=h, h_out=h,
                            chunk_states=True)
    for h0 in (h, None):
        got = backward(kda, dict(q, h0=h0), chunk_states=cs)
        for u, v in zip(want, got):
            assert torch.equal(u, v)


def test_decay_within_one_and_a_half_ulp(kda):
    """exp(g) as a step makes it from a state of ones and no input: the
    hardware's 2^t is off by at most an ulp, the last multiply-add by half of
    one, and what the correction of t leaves out is under 2^-10 of one"""
    gen = torch.Generator().manual_seed(93)
    N = 1 << 16
    g = -87.3 * torch.rand(N, 1, 16, generator=gen) ** 3
    g[0], g[1], g[2] = 0.0, -math.inf, -1e-8
    state = torch.ones(N, 1, 16, device="cuda")
    kda.kda_scan_step(torch.zeros(N, 1, 16, device="cuda"), g.cuda(), None,
                      state)
    want = torch.exp(g.double())
    ulp = torch.exp2(torch.floor(torch.log2(want.clamp_min(2.0 ** -126))) - 23)
    err = (state.cpu().double() - want).abs() / ulp
    assert bool((state[0] == 1).all()) and bool((state[1] == 0).all())
    assert float(err.max()) <= 1.5 + 2.0 ** -10, float(err.max())
