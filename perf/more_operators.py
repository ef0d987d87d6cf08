"""The operators of a block whose mixer is linear attention with one decay per
head, as a user calls them:

- linattn: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over
  sequences, backwards, and for one new token per sequence;
- qk_norm_rope: RMS norm of every query and key head and the rotation by
  position in one pass, and its gradient.

``run`` takes the plain form in torch operations, or with ``own`` the calls of
this repository's package.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token for a handful of sequences: interactive serving
        dict(name="linattn_step_n8_h32_d128", op="linattn", way="step", B=8,
             T=1, H=32, Hk=32, Dk=128, Dv=128, io="bf16", gate="f32",
             kind="softplus", s0=True, ragged=False),
        # one new token for a full decode batch
        dict(name="linattn_step_n256_h32_d128", op="linattn", way="step",
             B=256, T=1, H=32, Hk=32, Dk=128, Dv=128, io="bf16", gate="bf16",
             kind="softplus", s0=True, ragged=False),
        # a short prompt behind a cached state
        dict(name="linattn_b1_t200_h32_d128", op="linattn", way="fwd", B=1,
             T=200, H=32, Hk=32, Dk=128, Dv=128, io="bf16", gate="f32",
             kind="softplus", s0=True, ragged=False),
        # the prompt of one 8K context
        dict(name="linattn_b1_t8192_h32_d128", op="linattn", way="fwd", B=1,
             T=8192, H=32, Hk=32, Dk=128, Dv=128, io="bf16", gate="f32",
             kind="slow", s0=True, ragged=False),
        # the served context length on the heads of one of eight ranks, a
        # fixed decay for each head
        dict(name="linattn_b1_t262144_h4_d128", op="linattn", way="fwd", B=1,
             T=262144, H=4, Hk=4, Dk=128, Dv=128, io="bf16", gate="f32",
             kind="fixed", s0=False, ragged=False),
        # gradient of one 8K context
        dict(name="linattn_bwd_b1_t8192_h32_d128", op="linattn", way="bwd",
             B=1, T=8192, H=32, Hk=32, Dk=128, Dv=128, io="bf16", gate="f32",
             kind="softplus", s0=True, ragged=False),
        # a padded fp32 training batch of odd lengths whose value heads share
        # queries and keys in pairs, forward and backward
        dict(name="linattn_train_b6_t1531_h6_hk3_d64", op="linattn",
             way="train", B=6, T=1531, H=6, Hk=3, Dk=64, Dv=64, io="f32",
             gate="f32", kind="softplus", s0=True, ragged=True),
        # the queries and keys of a decode batch, rotary fraction 0.25
        dict(name="qk_norm_rope_n64_h16_2_d128", op="qk", way="fwd", rows=64,
             Hq=16, Hk=2, D=128, rot=32, io="bf16", pair="half",
             far=True, fused=True),
        # of one 8K context, as many keys as queries, every channel rotated
        dict(name="qk_norm_rope_n8192_h32_32_d128", op="qk", way="fwd",
             rows=8192, Hq=32, Hk=32, D=128, rot=128, io="bf16", pair="half",
             far=False, fused=False),
        # of a training batch, B8 T4096, read out of the fused projection
        dict(name="qk_norm_rope_n32768_h16_2_d128", op="qk", way="fwd",
             rows=32768, Hq=16, Hk=2, D=128, rot=32, io="bf16", pair="half",
             far=False, fused=True),
        # its gradient over an odd count of tokens at far positions, the
        # other layout of pairs
        dict(name="qk_norm_rope_bwd_n8191_h32_8_d128", op="qk", way="bwd",
             rows=8191, Hq=32, Hk=8, D=128, rot=128, io="bf16",
             pair="interleaved", far=True, fused=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(
        rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linattn", "linattn", "linattn", "qk", "qk"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "linattn":
        way = rng.choice(["step", "fwd", "fwd", "bwd", "train"])
        Dk, Dv = (rng.choice([16, 32, 64, 128, 128]) for _ in range(2))
        share = rng.choice([1, 1, 2, 4])
        Hk = rng.randint(1, 32 // share)
        H = Hk * share
        if way == "step":
            B, T = _log(rng, 1, 256), 1
        else:
            B = rng.randint(1, 8)
            T = _log(rng, 1, min(65536, (1 << 25) // (B * H * max(Dk, Dv))))
        return dict(op=op, way=way, B=B, T=T, H=H, Hk=Hk, Dk=Dk, Dv=Dv, io=io,
                    gate="f32" if io == "f32" else rng.choice(["bf16", "f32"]),
                    kind=rng.choice(["softplus", "slow", "fixed"]),
                    s0=way == "step" or rng.random() < 0.6,
                    ragged=way != "step" and rng.random() < 0.4)
    D = rng.choice([16, 32, 64, 128, 128, 256])
    Hk = rng.randint(1, 16)
    Hq = Hk * rng.choice([1, 2, 4, 8]) if Hk <= 4 else Hk
    return dict(op=op, way=rng.choice(["fwd", "bwd"]),
                rows=_log(rng, 1, min(65536, (1 << 25) // ((Hq + Hk) * D))),
                Hq=Hq, Hk=Hk, D=D,
                rot=rng.choice([r for r in (0, 16, D // 4, D // 2, D)
                                if r % 16 == 0]),
                io=io, pair=rng.choice(["half", "interleaved"]),
                far=rng.random() < 0.5, fused=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * seed + 29)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda",
                           dtype=torch.float32).to(dtype)

    def unit(*shape, dtype):
        x = randn(*shape)
        return x.div_(x.norm(dim=-1, keepdim=True)).to(dtype)

    io = _DT[case["io"]]
    st = {"case": case}
    if case["op"] == "linattn":
        B, T, H, Hk, Dk, Dv = (case[n] for n in ("B", "T", "H", "Hk", "Dk",
                                                 "Dv"))
        gt = _DT[case["gate"]]
        lead = (B,) if case["way"] == "step" else (B, T)
        st["q"] = unit(*lead, Hk, Dk, dtype=io)
        st["k"] = unit(*lead, Hk, Dk, dtype=io)
        st["v"] = randn(*lead, H, Dv, dtype=io)
        if case["kind"] == "fixed":
            # from about 1/2 a token to 1/256, a little off for each seed
            h = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
            g = -torch.exp2(-8.0 * h / H) * (1 + 0.1 * torch.rand(
                H, generator=gen, device="cuda"))
        else:
            z = randn(*lead, H)
            g = torch.log1p(-0.002 * torch.sigmoid(z)) \
                if case["kind"] == "slow" else \
                -torch.nn.functional.softplus(z)
            # the first token of a new document in a packed row forgets all
            reset = torch.rand(g.shape, generator=gen, device="cuda") < 1 / 512
            g[reset] = -math.inf
        st["g"] = g.to(gt)
        st["s0"] = 0.1 * randn(B, H, Dk, Dv) if case["s0"] else None
        st["lengths"] = None
        if case["ragged"]:
            n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda",
                              dtype=torch.int32)
            n[seed % B] = T
            st["lengths"] = n
        if case["way"] in ("bwd", "train"):
            st["do"] = randn(B, T, H, Dv, dtype=io)
            st["dsT"] = 0.1 * randn(B, H, Dk, Dv)
        st["scale"] = Dk ** -0.5 if case["kind"] == "fixed" else 1.0
        return st
    R, Hq, Hk, D = case["rows"], case["Hq"], case["Hk"], case["D"]
    if case["fused"]:
        # the projection of queries, keys and values as one matrix product
        # leaves it
        x = randn(R, (Hq + 2 * Hk) * D, dtype=io)
        st["q"] = x[:, :Hq * D].view(R, Hq, D)
        st["k"] = x[:, Hq * D:(Hq + Hk) * D].view(R, Hk, D)
    else:
        st["q"] = randn(R, Hq, D, dtype=io)
        st["k"] = randn(R, Hk, D, dtype=io)
    st["wq"] = 1.0 + 0.1 * randn(D)
    st["wk"] = 1.0 + 0.1 * randn(D)
    st["inv_freq"] = st["positions"] = None
    if case["rot"]:
        i = torch.arange(0, case["rot"], 2, device="cuda",
                         dtype=torch.float64)
        st["inv_freq"] = torch.pow(10000.0, -i / case["rot"]).float()
        st["positions"] = torch.randint(
            0, 262144 if case["far"] else 8192, (R,), generator=gen,
            device="cuda", dtype=torch.int32)
    if case["way"] == "bwd":
        st["dq"] = randn(R, Hq, D, dtype=io)
        st["dk"] = randn(R, Hk, D, dtype=io)
    return st


# ---------------------------------------------------------------------------
# the plain forms

def _pairs(G):
    """exp(G_i - G_j) for i >= j, else 0, of the last dimension (64 bits),
    in 32 bits"""
    d = G.unsqueeze(-1) - G.unsqueeze(-2)
    n = G.shape[-1]
    keep = torch.ones(n, n, dtype=torch.bool, device=G.device).tril()
    return torch.where(keep, d, -math.inf).exp().float()


def _chunks(st):
    """q, k, v (and do) as [B, H, n, C, D] in 32 bits with zeros behind each
    sequence, and the log-decays summed inside the chunks in 64 bits: 32 lose
    them where a chunk forgets and where the axis is long"""
    case = st["case"]
    B, T, H, Hk = case["B"], case["T"], case["H"], case["Hk"]
    C = 128 if T > 16384 else 64
    n = -(-T // C)
    live = None
    if st["lengths"] is not None:
        t = torch.arange(T, device="cuda")
        live = t[None, :] < st["lengths"][:, None]

    def cut(x):
        x = x.float()
        if live is not None:
            x = torch.where(live[:, :, None, None], x, 0.0)
        if x.shape[2] != H:
            x = x.repeat_interleave(H // Hk, 2)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - T))
        return x.reshape(B, n, C, H, -1).permute(0, 3, 1, 2, 4).contiguous()

    # exp(-1e4) is 0, and differences of finite sums are never NaN
    g = st["g"].double().clamp(min=-1e4).expand(B, T, H)
    if live is not None:
        g = torch.where(live[:, :, None], g, 0.0)
    g = torch.nn.functional.pad(g, (0, 0, 0, n * C - T))
    G = g.reshape(B, n, C, H).permute(0, 3, 1, 2).cumsum(-1)
    return {"C": C, "live": live, "G": G, "cut": cut, "q": cut(st["q"]),
            "k": cut(st["k"]), "v": cut(st["v"])}


def _back(x, case):
    """[B, H, n, C, D] as [B, T, H, D]"""
    B, H, D = x.shape[0], x.shape[1], x.shape[-1]
    return x.permute(0, 2, 3, 1, 4).reshape(B, -1, H, D)[:, :case["T"]]


def _tr(x):
    return x.transpose(-1, -2).contiguous()


def _states(c, kv, first):
    """the states before every chunk and behind the last one, from what each
    chunk adds (kv) and the state before the first"""
    B, H, n = kv.shape[:3]
    total = c["G"][..., -1].cumsum(-1)              # behind chunk i
    A = _pairs(total)                               # [B, H, n, n]
    flat = kv.reshape(B, H, n, -1)
    ends = A @ flat
    if first is not None:
        ends += total.exp().float()[..., None] * \
            first.reshape(B, H, 1, -1)
    ends = ends.reshape(kv.shape)
    head = torch.zeros_like(kv[:, :, :1]) if first is None \
        else first.unsqueeze(2)
    return torch.cat([head, ends[:, :, :-1]], 2), ends[:, :, -1]


def _states_back(c, kv, last):
    """the same for gradients, which come from behind: those that reach the
    end of every chunk, and the one that leaves the first"""
    r = {"G": c["G"].flip(2)}
    ends, out = _states(r, kv.flip(2), last)
    return ends.flip(2), out


def _linattn_fwd(st, c):
    G, last = c["G"], c["G"][..., -1:]
    inside = _pairs(G)
    kv = _tr(c["k"] * (last - G).exp().float()[..., None]) @ c["v"]
    starts, end = _states(c, kv, st["s0"])
    qk = c["q"] @ _tr(c["k"])
    o = (qk * inside) @ c["v"] + G.exp().float()[..., None] * \
        (c["q"] @ starts)
    return o * st["scale"], end, starts, qk, inside


def _linattn_bwd(st, c, starts, end, qk, inside):
    case, G, last = st["case"], c["G"], c["G"][..., -1:]
    do = c["cut"](st["do"]) * st["scale"]
    eG, wC = G.exp().float()[..., None], (last - G).exp().float()[..., None]
    dkv = _tr(c["q"] * eG) @ do
    dends, ds0 = _states_back(c, dkv, st["dsT"])
    dA = (do @ _tr(c["v"])) * inside
    A = qk * inside
    dq_far = eG * (do @ _tr(starts))
    dk_far = wC * (c["v"] @ _tr(dends))
    dq = dA @ c["k"] + dq_far
    dk = _tr(dA) @ c["q"] + dk_far
    dv = _tr(A) @ do + wC * (c["k"] @ dends)
    # the pairs of tokens that lie on both sides of the gate
    M = dA * qk
    M = M.flip(-2).cumsum(-2).flip(-2).tril(-1).sum(-1)
    late = (c["q"] * dq_far).sum(-1)
    early = (c["k"] * dk_far).sum(-1)
    both = last.exp().float()[..., 0] * (starts * dends).sum((-1, -2))
    dg = M + late.flip(-1).cumsum(-1).flip(-1) + \
        early.cumsum(-1) - early + both.unsqueeze(-1)
    return dq, dk, dv, _back(dg.unsqueeze(-1), case)[..., 0], ds0


def _linattn_grads(st, c, fwd):
    case = st["case"]
    io, gt = _DT[case["io"]], _DT[case["gate"]]
    dq, dk, dv, dg, ds0 = _linattn_bwd(st, c, *fwd)
    B, T, H, Hk = case["B"], case["T"], case["H"], case["Hk"]

    def heads(x):
        x = _back(x, case)
        if Hk != H:
            x = x.reshape(B, T, Hk, H // Hk, -1).sum(3)
        return x.to(io)

    if c["live"] is not None:
        dg = torch.where(c["live"][:, :, None], dg, 0.0)
    if case["kind"] == "fixed":
        dg = dg.double().sum((0, 1))
    return heads(dq), heads(dk), _back(dv, case).to(io), dg.to(gt), ds0


def _linattn(st):
    case = st["case"]
    io = _DT[case["io"]]
    if case["way"] == "step":
        many = case["H"] // case["Hk"]
        q, k = (st[n].float().repeat_interleave(many, 1) for n in "qk")
        a = torch.exp(st["g"].float()).expand(case["B"], case["H"])
        s = st["s0"]
        s.mul_(a[..., None, None])
        s += k.unsqueeze(-1) * st["v"].float().unsqueeze(-2)
        o = st["scale"] * (q.unsqueeze(-1) * s).sum(-2)
        return o.to(io), s
    c = _chunks(st)
    o, end, starts, qk, inside = _linattn_fwd(st, c)
    out = (_back(o, case).to(io), end)
    if case["way"] == "fwd":
        return out
    grads = _linattn_grads(st, c, (starts, end, qk, inside))
    return grads if case["way"] == "bwd" else (*out, *grads)


def _turns(st):
    """cosine and sine [rows, 1, rot / 2]; the angles of far positions need
    64 bits"""
    a = st["positions"].double()[:, None] * st["inv_freq"].double()
    return a.cos().float().unsqueeze(1), a.sin().float().unsqueeze(1)


def _rotate(x, turns, pair, back=False):
    if turns is None:
        return x
    c, s = turns
    s = -s if back else s
    n = c.shape[-1]
    if pair == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _rms(x):
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _qk(st):
    case = st["case"]
    io = _DT[case["io"]]
    turns = _turns(st) if case["rot"] else None
    q, k = st["q"].float(), st["k"].float()
    if case["way"] == "fwd":
        return tuple(_rotate(x * _rms(x) * w, turns, case["pair"]).to(io)
                     for x, w in ((q, st["wq"]), (k, st["wk"])))

    def grad(x, w, dy):
        t = _rotate(dy.float(), turns, case["pair"], back=True)
        r = _rms(x)
        n = x * r
        dw = (t * n).sum((0, 1))
        t = t * w
        return (r * (t - n * (t * n).mean(-1, keepdim=True))).to(io), dw

    dq, dwq = grad(q, st["wq"], st["dq"])
    dk, dwk = grad(k, st["wk"], st["dk"])
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------
# the framework's operators

def _own(st):
    import gated_delta_rule_74_amd as kda

    case = st["case"]
    if case["op"] == "linattn":
        q, k, v, g, scale = (st[n] for n in ("q", "k", "v", "g", "scale"))
        if case["way"] == "step":
            return kda.kda_linattn_step(q, k, v, g, st["s0"],
                                        scale=scale), st["s0"]
        kw = dict(s0=st["s0"], lengths=st["lengths"], scale=scale)
        out = ()
        if case["way"] != "bwd":
            out = kda.kda_linattn(q, k, v, g, **kw)
        if case["way"] == "fwd":
            return out
        return (*out, *kda.kda_linattn_backward(q, k, v, g, st["do"],
                                                dsT=st["dsT"], **kw))
    kw = dict(wq=st["wq"], wk=st["wk"], eps=EPS,
              interleaved=case["pair"] == "interleaved")
    if case["way"] == "fwd":
        return kda.kda_qk_norm_rope(st["q"], st["k"], st["positions"],
                                    st["inv_freq"], **kw)
    return kda.kda_qk_norm_rope_backward(
        st["q"], st["k"], st["positions"], st["inv_freq"], st["dq"],
        st["dk"], **kw)


def run(state):
    if own:
        return _own(state)
    return _linattn(state) if state["case"]["op"] == "linattn" \
        else _qk(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    s = _BYTES[case["io"]]
    if case["op"] == "linattn":
        B, T, H, Hk, Dk, Dv = (case[n] for n in ("B", "T", "H", "Hk", "Dk",
                                                 "Dv"))
        qk, v = 2 * B * T * Hk * Dk * s, B * T * H * Dv * s
        g = _BYTES[case["gate"]] * (H if case["kind"] == "fixed"
                                    else B * T * H)
        S = 4 * B * H * Dk * Dv
        n = B * T * H
        if case["way"] == "step":
            return {"bytes": qk + 2 * v + g + 2 * S, "flops": 5 * n * Dk * Dv}
        # the recurrence's products, or those of chunks of 64 where less
        fwd = {"bytes": qk + 2 * v + g + S * (2 if case["s0"] else 1),
               "flops": n * min(5 * Dk * Dv,
                                4 * Dk * Dv + 64 * (Dk + Dv))}
        bwd = {"bytes": 2 * qk + 3 * v + 2 * g + S * (3 if case["s0"] else 2),
               "flops": n * (10 * Dk * Dv + 64 * (3 * Dk + 2 * Dv))}
        if case["way"] == "fwd":
            return fwd
        if case["way"] == "bwd":
            return bwd
        return {"bytes": bwd["bytes"] + v + S,
                "flops": bwd["flops"] + fwd["flops"]}
    n = case["rows"] * (case["Hq"] + case["Hk"]) * case["D"]
    small = 4 * case["rows"] + 8 * case["D"] + 2 * case["rot"]
    if case["way"] == "fwd":
        return {"bytes": 2 * s * n + small, "flops": 8 * n}
    return {"bytes": 3 * s * n + small + 8 * case["D"], "flops": 16 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_linattn(case, st):
    """token by token; the states of 128 tokens at a time are kept for the
    gradients"""
    f8 = torch.float64
    B, T, H = case["B"], case["T"], case["H"]
    many = H // case["Hk"]
    step = case["way"] == "step"

    def first(x):
        x = x.to(f8)
        x = x.unsqueeze(1) if step else x
        x = x.transpose(0, 1)
        if x.shape[2] != H:
            x = x.repeat_interleave(many, 2)
        return x.contiguous()

    q, k, v = (first(st[n]) for n in "qkv")
    g = st["g"].to(f8)
    g = g.expand(T, B, H) if g.dim() == 1 else first(st["g"])
    a = g.exp()
    ends = None
    if st["lengths"] is not None:
        n = st["lengths"].long()
        ends = torch.arange(T, device="cuda")[:, None] >= n[None]
        a = torch.where(ends[..., None], 1.0, a)
        dead = ends[..., None, None]
        q, k, v = (torch.where(dead, 0.0, x) for x in (q, k, v))
    a = a[..., None, None]
    S = q.new_zeros(B, H, case["Dk"], case["Dv"]) if st["s0"] is None \
        else st["s0"].to(f8)
    scale = st["scale"]
    k = k.unsqueeze(-1)
    v = v.unsqueeze(-2)
    kept = []
    o = torch.empty_like(v)
    for t in range(T):
        if t % 128 == 0:
            kept.append(S)
        S = torch.addcmul(a[t] * S, k[t], v[t])
        if case["way"] != "bwd":
            o[t] = q[t].unsqueeze(-2) @ S
    o = (scale * o.squeeze(-2)).transpose(0, 1)
    if step:
        return o[:, 0].contiguous(), S
    out = (o.contiguous(), S)
    if case["way"] == "fwd":
        return out
    do = scale * first(st["do"])
    if ends is not None:
        do = torch.where(dead, 0.0, do)
    do = do.unsqueeze(-2)
    q = q.unsqueeze(-1)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dv = torch.empty_like(v)
    dg = torch.empty_like(a)
    dS = st["dsT"].to(f8)
    for t0 in range((T - 1) // 128 * 128, -1, -128):
        t1 = min(T, t0 + 128)
        Ss = [kept[t0 // 128]]
        for t in range(t0, t1):
            Ss.append(torch.addcmul(a[t] * Ss[-1], k[t], v[t]))
        for t in range(t1 - 1, t0 - 1, -1):
            dS = torch.addcmul(dS, q[t], do[t])
            dq[t] = (Ss[t - t0 + 1] * do[t]).sum(-1, keepdim=True)
            dk[t] = (dS * v[t]).sum(-1, keepdim=True)
            dv[t] = k[t].transpose(-1, -2) @ dS
            dS = a[t] * dS
            dg[t] = (dS * Ss[t - t0]).sum((-1, -2), keepdim=True)

    def last(x, many=1):
        x = x.transpose(0, 1)
        return x.unflatten(2, (-1, many)).sum(3) if many > 1 \
            else x.contiguous()

    dg = dg[..., 0, 0]
    if ends is not None:
        dg = torch.where(ends[..., None], 0.0, dg)
    dg = dg.sum((0, 1)) if case["kind"] == "fixed" else last(dg)
    grads = (last(dq.squeeze(-1), many), last(dk.squeeze(-1), many),
             last(dv.squeeze(-2)), dg, dS)
    return grads if case["way"] == "bwd" else (*out, *grads)


def _exact_rotate(x, st, pair):
    """complex multiplication"""
    if st["inv_freq"] is None:
        return x
    rot = 2 * st["inv_freq"].numel()
    angle = st["positions"].double()[:, None, None] * \
        st["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)
    z, rest = x[..., :rot], x[..., rot:]
    if pair == "half":
        z = torch.complex(*z.chunk(2, -1)) * turn
        z = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(z.unflatten(-1, (-1, 2)).contiguous())
        z = torch.view_as_real(z * turn).flatten(-2)
    return torch.cat([z, rest], -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linattn":
        return _exact_linattn(case, st)
    back = case["way"] == "bwd"
    leaf = {n: st[n].double().requires_grad_(back)
            for n in ("q", "k", "wq", "wk")}
    outs = [_exact_rotate(
        leaf[n] / (leaf[n].square().mean(-1, keepdim=True) + EPS).sqrt() *
        leaf["w" + n], st, case["pair"]) for n in "qk"]
    if not back:
        return tuple(outs)
    return torch.autograd.grad(outs, [leaf[n] for n in ("q", "k", "wq", "wk")],
                               [st["dq"].double(), st["dk"].double()])
