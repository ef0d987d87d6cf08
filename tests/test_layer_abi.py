"""CPU checks of the layer operators' boundary: workspace sizes, the C
functions' refusals (nothing is launched, so no GPU is needed), and the
binding's checks of shapes, dtypes and combinations."""
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

import gated_delta_rule_74_amd as kda
from gated_delta_rule_74_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # a 16-byte aligned fake device address (never dereferenced)
BF, F, HEAD = kda.KDA_BF16, kda.KDA_F32, kda.KDA_GATE_HEAD
INV, UNS = kda.KDA_EINVAL, kda.KDA_EUNSUPPORTED


def adr(i):
    return A + 0x10000 * i


def test_workspace_sizes():
    for f in (kda.kda_scan_workspace_size,
              kda.kda_scan_backward_workspace_size):
        assert f(1, 8192, 32, 128) > 0
        assert f(2, 1, 1, 16) > 0
        for bad in [(0, 8, 1, 16), (1, 0, 1, 16), (1, 8, 1, 48),
                    (1, 8, 1, 256), (1, (1 << 30) + 1, 1, 16),
                    (1 << 20, 1 << 20, 1, 16), (1, 8, 1 << 28, 16)]:
            assert f(*bad) == 0, bad
    assert kda.kda_gated_norm_backward_workspace_size(1, 16) > 0
    assert kda.kda_gated_norm_backward_workspace_size(0, 16) == 0
    assert kda.kda_gated_norm_backward_workspace_size(5, 24) == 0
    assert kda.kda_gated_norm_backward_workspace_size(1 << 40, 16) == 0
    assert kda.kda_block_norm_backward_workspace_size(3, 5) > 0
    for bad in [(0, 5), (3, 0), (3, 16385), (1 << 22, 8)]:
        assert kda.kda_block_norm_backward_workspace_size(*bad) == 0


def _scan(**kw):
    a = dict(x=adr(0), io=BF, g=adr(1), beta=adr(2), gt=F, h0=None,
             lengths=None, y=adr(3), h_out=None, cs=None, B=2, T=300, H=3,
             D=64, ws=adr(9), wsb=1 << 40, stream=None)
    a.update(kw)
    return layer._scan(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INV), (dict(T=0), INV), (dict(H=-1), INV), (dict(D=0), INV),
    (dict(x=None), INV), (dict(g=None), INV), (dict(y=None), INV),
    (dict(ws=None), INV), (dict(wsb=16), INV), (dict(x=A + 8), INV),
    (dict(h0=A + 4), INV), (dict(cs=A + 4), INV), (dict(lengths=A + 2), INV),
    (dict(io=5), INV), (dict(gt=2), INV), (dict(io=BF | HEAD), INV),
    (dict(y=adr(0)), INV), (dict(y=adr(1)), INV), (dict(h_out=adr(2)), INV),
    (dict(h_out=adr(3)), INV), (dict(cs=adr(3)), INV),
    (dict(h_out=adr(5), cs=adr(5)), INV),
    (dict(D=48), UNS), (dict(D=256), UNS), (dict(io=F, gt=BF), UNS),
    (dict(io=F, gt=BF | HEAD), UNS), (dict(T=(1 << 30) + 1), UNS),
    (dict(B=1 << 20, T=1 << 20), UNS), (dict(H=1 << 25), UNS),
])
def test_scan_rejects(kw, want):
    assert _scan(**kw) == want


def _scan_bwd(**kw):
    a = dict(x=adr(0), io=BF, g=adr(1), beta=adr(2), gt=F, h0=None,
             lengths=None, dy=adr(3), dhT=None, cs=None, dx=adr(4),
             dg=adr(5), dbeta=adr(6), dh0=None, B=2, T=300, H=3, D=64,
             ws=adr(9), wsb=1 << 40, stream=None)
    a.update(kw)
    return layer._scan_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), INV), (dict(dy=None), INV), (dict(dx=None), INV),
    (dict(dg=None), INV), (dict(dbeta=None), INV), (dict(beta=None), INV),
    (dict(dx=adr(0)), INV), (dict(dg=adr(3)), INV), (dict(dg=adr(4)), INV),
    (dict(dh0=adr(7), dhT=adr(7)), INV), (dict(dh0=adr(7), cs=adr(7)), INV),
    (dict(dhT=A + 4), INV), (dict(wsb=0), INV), (dict(D=8), UNS),
    (dict(io=F, gt=BF), UNS),
])
def test_scan_backward_rejects(kw, want):
    assert _scan_bwd(**kw) == want


def _step(**kw):
    a = dict(x=adr(0), io=BF, g=adr(1), beta=adr(2), gt=BF, state=adr(3),
             y=adr(4), N=4, H=2, D=16, stream=None)
    a.update(kw)
    return layer._scan_step(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), INV), (dict(state=None), INV), (dict(y=None), INV),
    (dict(y=adr(3)), INV), (dict(state=adr(0)), INV), (dict(g=A + 2), INV),
    (dict(gt=7), INV), (dict(D=24), UNS), (dict(io=F), UNS),
    (dict(N=1 << 30, H=1 << 10), UNS),
])
def test_scan_step_rejects(kw, want):
    assert _step(**kw) == want


def _gated(**kw):
    a = dict(o=adr(0), z=adr(1), io=BF, w=adr(2), act=1, eps=1e-6, y=adr(3),
             rows=10, D=128, stream=None)
    a.update(kw)
    return layer._gated(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), INV), (dict(o=None), INV), (dict(w=None), INV),
    (dict(y=None), INV), (dict(z=None), INV), (dict(act=0), INV),
    (dict(act=3), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(y=adr(0)), INV), (dict(y=adr(1)), INV), (dict(z=A + 8), INV),
    (dict(io=2), INV), (dict(D=96), UNS), (dict(rows=1 << 40), UNS),
])
def test_gated_norm_rejects(kw, want):
    assert _gated(**kw) == want


def _gated_bwd(**kw):
    a = dict(o=adr(0), z=adr(1), io=BF, w=adr(2), act=2, eps=1e-6, dy=adr(3),
             do=adr(4), dz=adr(5), dw=adr(6), rows=10, D=128, ws=adr(9),
             wsb=1 << 30, stream=None)
    a.update(kw)
    return layer._gated_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INV), (dict(dz=None), INV), (dict(z=None, act=0), INV),
    (dict(dw=None), INV), (dict(do=adr(3)), INV), (dict(do=adr(5)), INV),
    (dict(wsb=100), INV), (dict(ws=None), INV), (dict(D=100), UNS),
])
def test_gated_norm_backward_rejects(kw, want):
    assert _gated_bwd(**kw) == want


def _block(**kw):
    a = dict(y=adr(0), io=BF, r=adr(1), rt=F, z=adr(2), act=1, wp=adr(3),
             wq=adr(4), rs=1.0, bs=1.0, eps=1e-6, ro=adr(5), x=adr(6),
             rows=10, C=100, stream=None)
    a.update(kw)
    return layer._block(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), INV), (dict(C=0), INV), (dict(y=None), INV),
    (dict(r=None), INV), (dict(ro=None), INV), (dict(x=None), INV),
    (dict(wq=None), INV), (dict(z=None), INV), (dict(act=0), INV),
    (dict(rs=float("inf")), INV), (dict(bs=float("nan")), INV),
    (dict(eps=-1.0), INV), (dict(x=adr(1)), INV), (dict(x=adr(0)), INV),
    (dict(ro=adr(0)), INV), (dict(x=adr(5)), INV), (dict(rt=9), INV),
    (dict(r=A + 4), INV), (dict(io=F, rt=BF), UNS), (dict(C=16385), UNS),
    (dict(rows=1 << 22), UNS),
])
def test_block_norm_rejects(kw, want):
    assert _block(**kw) == want


def _block_bwd(**kw):
    a = dict(y=adr(0), io=BF, r=adr(1), rt=F, z=adr(2), act=1, wp=adr(3),
             wq=adr(4), rs=1.0, bs=1.0, eps=1e-6, dx=adr(5), dro=adr(6),
             dy=adr(7), dr=adr(8), dz=adr(10), dwp=adr(11), dwq=adr(12),
             rows=10, C=100, ws=adr(9), wsb=1 << 30, stream=None)
    a.update(kw)
    return layer._block_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(dx=None), INV), (dict(wq=None), INV), (dict(dwq=None), INV),
    (dict(dwp=None), INV), (dict(dz=None), INV), (dict(dy=None), INV),
    (dict(dr=None), INV), (dict(ws=None), INV), (dict(wsb=64), INV),
    (dict(dx=None, wq=None, dwq=None, dro=None), INV),
    (dict(dr=adr(6)), INV), (dict(dy=adr(8)), INV), (dict(dr=adr(1)), INV),
    (dict(C=16385), UNS),
])
def test_block_norm_backward_rejects(kw, want):
    assert _block_bwd(**kw) == want


# ---------------------------------------------------------------------------
# the binding, with CPU tensors: the mismatch is named before the device

def t(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


F32 = torch.float32


def test_binding_rejects_scan():
    B, T, H, D = 2, 130, 3, 16
    x, g, b = t(B, T, H, D), t(B, T, H, D, dt=F32), t(B, T, H, dt=F32)
    bad = [
        (dict(x=t(B, T, D)), "x has"), (dict(g=t(B, T, H, 8, dt=F32)), "g"),
        (dict(g=t(B, T, dt=F32)), "per-head"), (dict(beta=t(B, T, H)), "beta"),
        (dict(h0=t(B, H, D)), "h0"), (dict(h_out=t(B, H, 8, dt=F32)), "h_out"),
        (dict(lengths=torch.zeros(B, dtype=torch.int64)), "lengths"),
        (dict(lengths=torch.zeros(3, dtype=torch.int32)), "lengths"),
        (dict(y=t(B, T, H, D, dt=F32)), "y"),
        (dict(chunk_states=t(B, 1, H, D, dt=F32)), "chunk_states"),
        (dict(x=x.half()), "x"), ({}, "GPU"),
    ]
    for over, what in bad:
        a = dict(x=x, g=g, beta=b)
        a.update(over)
        with pytest.raises(ValueError, match=what):
            kda.kda_scan(a.pop("x"), a.pop("g"), a.pop("beta"), **a)
    dy = t(B, T, H, D)
    for over, what in [(dict(dy=t(B, T, H, D, dt=F32)), "dy"),
                       (dict(dhT=t(B, H, D)), "dhT"),
                       (dict(chunk_states=t(B, 3, H, D, dt=F32)),
                        "chunk_states"), ({}, "GPU")]:
        a = dict(dy=dy)
        a.update(over)
        with pytest.raises(ValueError, match=what):
            kda.kda_scan_backward(x, g, b, a.pop("dy"), **a)
    st = t(B, H, D, dt=F32)
    with pytest.raises(ValueError, match="state"):
        kda.kda_scan_step(x[:, 0], g[:, 0], b[:, 0], st[:1])
    with pytest.raises(ValueError, match="beta"):
        kda.kda_scan_step(x[:, 0], g[:, 0], b, st)


def test_binding_rejects_norms():
    o, w = t(4, 3, 32), t(32, dt=F32)
    for a, kw, what in [
            ((o, t(4, 3, 16), w), {}, "z"), ((o, o.float(), w), {}, "z"),
            ((o, o, t(32)), {}, "w"), ((o, o, w), dict(act="gelu"), "act"),
            ((o, o, w), dict(y=t(4, 3, 32, dt=F32)), "y"),
            ((o, o, w), {}, "GPU")]:
        with pytest.raises(ValueError, match=what):
            kda.kda_gated_norm(*a, **kw)
    with pytest.raises(ValueError, match="dy"):
        kda.kda_gated_norm_backward(o, o, w, o[:1])
    y, r, c = t(5, 40), t(5, 40, dt=F32), t(40, dt=F32)
    for kw, what in [(dict(z=t(5, 39)), "z"), (dict(w_post=t(40)), "w_post"),
                     (dict(w_pre=t(39, dt=F32)), "w_pre"),
                     (dict(r_out=t(5, 40)), "r_out"), (dict(x=y), "x"),
                     (dict(w_pre=c, x=r), "x"), ({}, "GPU")]:
        with pytest.raises(ValueError, match=what):
            kda.kda_block_norm(y, r, **kw)
    with pytest.raises(ValueError, match="r"):
        kda.kda_block_norm(y, r[:4])
    for kw, what in [(dict(dx=y), "dx and w_pre"), ({}, "neither"),
                     (dict(w_pre=c), "dx and w_pre"),
                     (dict(dr_out=y), "dr_out"),
                     (dict(dx=r, w_pre=c), "dx")]:
        with pytest.raises(ValueError, match=what):
            kda.kda_block_norm_backward(y, r, **kw)


def test_binding_refuses_sizes_past_an_int():
    """A size above 2^31 - 1 is refused, not cut to its lower 32 bits (these
    would be calls of 5 rows, 3 tokens, one sequence, 16 values)."""
    def m(*s, dt=torch.bfloat16):
        return torch.empty(*s, dtype=dt, device="meta")

    P = 1 << 32
    y = m(P + 5, 1)
    calls = [
        lambda: kda.kda_block_norm(y, y),
        lambda: kda.kda_block_norm_backward(y, y, dr_out=y),
        lambda: kda.kda_scan(m(1, P + 3, 1, 16), m(1, P + 3, 1)),
        lambda: kda.kda_scan_backward(m(1, P + 3, 1, 16), m(1, P + 3, 1), None,
                                      m(1, P + 3, 1, 16)),
        lambda: kda.kda_scan_step(m(P + 1, 1, 16), m(P + 1, 1), None,
                                  m(P + 1, 1, 16, dt=F32)),
        lambda: kda.kda_gated_norm(m(2, P + 16), None, m(P + 16, dt=F32)),
    ]
    for call in calls:
        with pytest.raises(kda.KdaError, match="unsupported"):
            call()


def test_workspace_sizes_past_an_int():
    """no workspace, rather than that of the sizes' lower 32 bits"""
    P = 1 << 32
    for f in (kda.kda_scan_workspace_size,
              kda.kda_scan_backward_workspace_size):
        for n in ((P + 1, 8, 1, 16), (1, P + 8, 1, 16), (1, 8, P + 1, 16),
                  (1, 8, 1, P + 16), (1 - P, 8, 1, 16)):
            assert f(*n) == 0, n
    f = kda.kda_gated_norm_backward_workspace_size
    assert f(5, P + 16) == 0 and f((1 << 64) + 5, 16) == 0
    f = kda.kda_block_norm_backward_workspace_size
    assert f(P + 3, 8) == 0 and f(3, P + 8) == 0


@pytest.mark.parametrize("nc", [2, 7, 8, 9, 10, 16, 17, 32, 33, 34, 65, 1000])
def test_most_tiles_can_be_cleared(nc):
    """the two passes' words of the most tiles there may be: 16 bytes a thread,
    and a launch of at most 2^32 - 1 threads"""
    B = ((1 << 23) - 1) // nc
    size = kda.kda_scan_backward_workspace_size(B, nc * 128, 1, 16)
    words = size - B * 16 * nc * 4
    assert size > 0 and 0 < words // 16 < 2 ** 32 - 256
    assert kda.kda_scan_backward_workspace_size(B + nc, nc * 128, 1, 16) == 0


@pytest.mark.skipif(shutil.which("hipcc") is None and
                    not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc not available")
def test_layer_abi_clean_under_asan_ubsan():
    """The boundary's host code under AddressSanitizer and
    UndefinedBehaviorSanitizer, its launchers replaced by stubs."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    csrc = os.path.join(ROOT, "gated_delta_rule_74_amd", "csrc")
    with tempfile.TemporaryDirectory(prefix="kda_san_") as tmp:
        exe = os.path.join(tmp, "layer_abi_san")
        r = subprocess.run(
            [hipcc, "-O1", "-g", "-std=c++17", "--offload-arch=gfx950",
             "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xclang",
             "-target-feature", "-Xclang", "-packed-fp32-ops", "-I",
             os.path.join(ROOT, "include"), "-I", csrc,
             os.path.join(csrc, "kda_layer_api.hip"),
             os.path.join(ROOT, "tests", "sanitize", "layer_abi_driver.cpp"),
             "-o", exe], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                   UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
        r = subprocess.run([exe], capture_output=True, text=True, env=env,
                           timeout=300)
        assert r.returncode == 0 and "0 mismatches" in r.stdout, \
            r.stdout + r.stderr
