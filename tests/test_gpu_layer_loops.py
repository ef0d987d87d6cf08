"""The layer operators where a workgroup goes through its loop several times:
several tiles of the scan, several turns of rows of the block norm's gradient,
the last one partial.  Against the 64-bit references, element by element."""
import pytest
import torch

import layer_ref as ref
from gpu_common import say
from layer_ref import within
from test_gpu_norms import EPS, rn
from test_gpu_scan import backward, forward, inputs

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_74_amd as m
    return m


# ---------------------------------------------------------------------------
# block norm

def turn(kda, C):
    """(rows that a workgroup of the gradient takes at once, the most
    workgroups there are): from the workspace, 2 partial rows per workgroup"""
    def groups(rows):
        return kda.kda_block_norm_backward_workspace_size(rows, C) // (8 * C)
    per = 1
    while groups(2 * per) == 1:
        per *= 2
    return per, groups((1 << 22) - 1)


# The weights' gradients are sums over all rows.  Here a thread adds at most 4
# rows, a workgroup at most 32 threads' sums, and the sum over at most 1024
# workgroups takes 16 + 16 + 2 additions: 70 in a chain, whatever the rows.
# The reference's bound counts one rounding per row, so it is taken over pieces
# of 80 rows, values and bounds added in 64 bits.  A row left out or counted
# twice then shows.
PIECE = 80


def pieces(R, tensors):
    tensors = list(tensors)
    for lo in range(0, R, PIECE):
        yield [None if t is None else t[lo:lo + PIECE] for t in tensors]


def joined(parts, sums):
    """the pieces' (value, slack) pairs, one behind the other or added up"""
    out = []
    for i, p in enumerate(zip(*parts)):
        if p[0] is None:
            out.append(None)
        else:
            f = (lambda v: torch.stack(v).sum(0)) if i in sums else torch.cat
            out.append(tuple(f([q[j] for q in p]) for j in (0, 1)))
    return out


@pytest.mark.parametrize("C", [65, 136, 520, 777, 4096, 4097, 8192, 8200,
                               8201])
@pytest.mark.parametrize("io,res", [(F, F), (BF, F), (BF, BF)])
def test_block_norm_turns(kda, C, io, res):
    per, most = turn(kda, C)
    R = 3 * most * per + per // 2 + 1  # three whole turns and a partial one
    say(f"C {C}: {R} rows, {per} a workgroup, {most} workgroups")
    y, z, dx = (rn(R, C, seed=150 + i, dtype=io) for i in range(3))
    r, dro = (rn(R, C, seed=160 + i, dtype=res) for i in range(2))
    wp, wq = (1 + 0.1 * rn(C, seed=170 + i) for i in range(2))
    kw = dict(z=z, w_post=wp, w_pre=wq, act="silu", res_scale=0.75,
              branch_scale=0.5, eps=EPS)
    h, x = kda.kda_block_norm(y, r, **kw)
    wh, wx = joined([ref.block_norm(a, b, wp, c, wq, "silu", 0.75, 0.5, EPS)
                     for a, b, c in pieces(R, map(ref.c8, (y, r, z)))], ())
    within("r_out", h, wh)
    within("x", x, wx)
    got = kda.kda_block_norm_backward(y, h, dx=dx, dr_out=dro, **kw)
    want = joined([ref.block_norm_grad(a, b, c, d, wp, e, wq, "silu", 0.75,
                                       0.5, EPS)
                   for a, b, c, d, e in pieces(
                       R, map(ref.c8, (y, h, dx, dro, z)))], (3, 4))
    for n, a, b in zip(("dy", "dr", "dz", "dw_post", "dw_pre"), got, want):
        within(n, a, b)


# ---------------------------------------------------------------------------
# scan

def heads(q, hs):
    """the inputs of some heads"""
    out = dict(q)
    for k, v in q.items():
        if v is None or k == "lengths":
            continue
        out[k] = (v[:, hs] if k in ("h0", "dhT") else v[:, :, hs]).contiguous()
    return out


def check_heads(kda, q, hs):
    """all outputs of heads hs, of a call on all heads"""
    want = ref.scan(**heads(q, hs))
    y, h, cs = forward(kda, q, chunk_states=True)
    within("y", y[:, :, hs], want["y"])
    within("h_out", h[:, hs], want["h"])
    within("chunk_states", cs[:, :, hs], want["chunk"])
    for states in (None, cs):
        dx, dg, db, d0 = backward(kda, q, chunk_states=states)
        within("dx", dx[:, :, hs], want["dx"])
        within("dg", dg[:, :, hs], want["dg"])
        within("dh0", d0[:, hs], want["dh0"])
        within("dbeta", db[:, :, hs], want["dbeta"])


@pytest.mark.parametrize("io,gt", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("lengths", [None, [1337, 2100]])
def test_scan_tiles_in_many_chunks(kda, io, gt, head, lengths):
    """1088 tiles: 17 chunks of 64 columns, carried values far from zero"""
    q = inputs(2, 2100, 32, 128, io, gt, head, kind="slow", reset=0,
               lengths=lengths, seed=90)
    q["h0"] *= 10
    check_heads(kda, q, [0, 7, 18, 31])


@pytest.mark.parametrize("io,gt", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("T", [5, 128])
def test_scan_tiles_of_one_chunk(kda, io, gt, head, T):
    """1300 sequences of at most one chunk, some of them empty or short"""
    n = [(7 * b) % (T + 1) for b in range(1300)]
    q = inputs(1300, T, 1, 16, io, gt, head, kind="slow", lengths=n, seed=91)
    check_heads(kda, q, [0])
