"""CPU checks of the boundary of linear attention and of the norm and rotation
of queries and keys: workspace sizes, the C functions' refusals (nothing is
launched, so no GPU is needed), the binding's checks."""
import ctypes
import os
import re
import shutil
import subprocess
import tempfile

import pytest
import torch

import gated_delta_rule_74_amd as kda
from gated_delta_rule_74_amd import linattn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # a 16-byte aligned fake device address (never dereferenced)
BF, F = kda.KDA_BF16, kda.KDA_F32
HEAD, FIXED = kda.KDA_GATE_HEAD, kda.KDA_GATE_FIXED
INV, UNS = kda.KDA_EINVAL, kda.KDA_EUNSUPPORTED
P = 1 << 32


def adr(i):
    return A + 0x10000 * i


def test_signatures_match_the_header():
    """every argument's type, as the header declares it"""
    with open(os.path.join(ROOT, "include", "kda.h")) as f:
        h = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for f in (linattn._lin, linattn._lin_bwd, linattn._lin_step,
              linattn._lin_ws, linattn._lin_bwd_ws, linattn._qk,
              linattn._qk_bwd, linattn._qk_bwd_ws):
        args = re.search(r"\b" + f.__name__ + r"\(([^)]*)\)", h).group(1)
        want = [ctypes.c_void_p if "*" in a else
                ctypes.c_longlong if "long long" in a else
                ctypes.c_size_t if "size_t" in a else
                ctypes.c_float if "float" in a else ctypes.c_int
                for a in args.split(",")]
        assert list(f.argtypes) == want, f.__name__


def test_workspace_sizes():
    for f in (kda.kda_linattn_workspace_size,
              kda.kda_linattn_backward_workspace_size):
        for dt in (torch.bfloat16, torch.float32):
            assert f(1, 8192, 32, 32, 128, 128, dt) > 0
            assert f(1, 1, 1, 1, 16, 128, dt) >= 256
            assert f((1 << 20) - 1, 4, 1, 4, 16, 16, dt) > 0
        for bad in [(0, 8, 1, 1, 16, 16), (1, 0, 1, 1, 16, 16),
                    (1, 8, 0, 1, 16, 16), (1, 8, 2, 3, 16, 16),
                    (1, 8, 2, 1, 16, 16), (1, 8, 1, 1, 48, 16),
                    (1, 8, 1, 1, 16, 256), (1, (1 << 30) + 1, 1, 1, 16, 16),
                    (1, 8, 1 << 20, 1 << 20, 16, 16),
                    (1 << 12, 1 << 20, 4, 4, 16, 16), (P + 1, 8, 1, 1, 16, 16),
                    (1 << 20, 4, 4, 4, 16, 16), (1, 8, 1, 1, P + 16, 16),
                    (1, P + 8, 1, 1, 16, 16)]:
            assert f(*bad, torch.bfloat16) == 0, bad
    f = kda.kda_qk_norm_rope_backward_workspace_size
    assert f(1, 1, 0, 16) > 0 and f(100000, 32, 8, 256) > 0
    for bad in [(0, 1, 1, 16), (1, 0, 1, 16), (1, 1, -1, 16), (1, 1, 1, 48),
                (1 << 26, 1, 1, 16), (1 << 25, 64, 64, 128),
                (1, 1 << 20, 1, 16), (P + 1, 1 << 31, 1, 16)]:
        assert f(*bad) == 0, bad


def _lin(**kw):
    a = dict(q=adr(0), k=adr(1), v=adr(2), io=BF, g=adr(3), gt=F, s0=None,
             lengths=None, o=adr(4), s_out=None, B=2, T=300, Hk=2, H=4, Dk=64,
             Dv=128, scale=1.0, ws=adr(9), wsb=1 << 40, stream=None)
    a.update(kw)
    return linattn._lin(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INV), (dict(T=0), INV), (dict(Hk=0), INV), (dict(H=-1), INV),
    (dict(Dk=0), INV), (dict(Dv=0), INV), (dict(Hk=3), INV),
    (dict(Hk=8), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(g=None), INV), (dict(o=None), INV),
    (dict(ws=None), INV), (dict(wsb=16), INV), (dict(q=A + 8), INV),
    (dict(s0=A + 4), INV), (dict(s_out=A + 4), INV),
    (dict(lengths=A + 2), INV), (dict(io=5), INV), (dict(gt=2), INV),
    (dict(gt=4 | FIXED), INV), (dict(io=BF | FIXED), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(o=adr(0)), INV), (dict(o=adr(3)), INV), (dict(s_out=adr(2)), INV),
    (dict(s_out=adr(4)), INV), (dict(s0=adr(4)), INV), (dict(o=adr(9)), INV),
    (dict(s_out=adr(9)), INV),
    (dict(Dk=48), UNS), (dict(Dv=256), UNS), (dict(io=F, gt=BF), UNS),
    (dict(io=F, gt=BF | FIXED), UNS), (dict(T=(1 << 30) + 1), UNS),
    (dict(B=1 << 20, T=1 << 20), UNS), (dict(H=1 << 20), UNS),
    (dict(B=1 << 21), UNS), (dict(B=1 << 20, T=4, Dv=64), UNS),
])
def test_linattn_rejects(kw, want):
    assert _lin(**kw) == want


def _lin_bwd(**kw):
    a = dict(q=adr(0), k=adr(1), v=adr(2), io=BF, g=adr(3), gt=F, s0=None,
             lengths=None, do=adr(4), dsT=None, dq=adr(5), dk=adr(6),
             dv=adr(7), dg=adr(8), ds0=None, B=2, T=300, Hk=2, H=4, Dk=64,
             Dv=128, scale=1.0, ws=adr(9), wsb=1 << 40, stream=None)
    a.update(kw)
    return linattn._lin_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), INV), (dict(do=None), INV), (dict(dq=None), INV),
    (dict(dk=None), INV), (dict(dv=None), INV), (dict(dq=adr(6)), INV),
    (dict(dq=adr(0)), INV), (dict(dg=adr(3)), INV), (dict(dv=adr(4)), INV),
    (dict(dsT=adr(10), ds0=adr(10)), INV), (dict(dsT=A + 4), INV),
    (dict(ds0=A + 4), INV), (dict(wsb=0), INV), (dict(Hk=3), INV),
    (dict(Dk=8), UNS), (dict(io=F, gt=BF), UNS),
])
def test_linattn_backward_rejects(kw, want):
    assert _lin_bwd(**kw) == want


def _step(**kw):
    a = dict(q=adr(0), k=adr(1), v=adr(2), io=BF, g=adr(3), gt=BF,
             state=adr(4), o=adr(5), N=4, Hk=1, H=2, Dk=16, Dv=32, scale=1.0,
             stream=None)
    a.update(kw)
    return linattn._lin_step(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), INV), (dict(Hk=0), INV), (dict(H=3, Hk=2), INV),
    (dict(state=None), INV), (dict(o=None), INV), (dict(o=adr(4)), INV),
    (dict(state=adr(2)), INV), (dict(g=A + 2), INV), (dict(gt=7), INV),
    (dict(scale=float("nan")), INV), (dict(Dk=24), UNS), (dict(Dv=256), UNS),
    (dict(io=F), UNS), (dict(N=1 << 21), UNS),
])
def test_linattn_step_rejects(kw, want):
    assert _step(**kw) == want


def _qk(**kw):
    a = dict(q=adr(0), k=adr(1), io=BF, sq=512, sk=256, wq=adr(2), wk=adr(3),
             pos=adr(4), inv=adr(5), rot=32, il=0, eps=1e-6, qo=adr(6),
             ko=adr(7), so=512, sko=256, rows=10, Hq=4, Hk=2, D=128,
             stream=None)
    a.update(kw)
    return linattn._qk(*a.values())


NO_K = dict(k=None, wk=None, ko=None, Hk=0)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV),
    (dict(D=0), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(Hk=0), INV), (dict(qo=None), INV), (dict(ko=None), INV),
    (dict(NO_K, wk=adr(3)), INV), (dict(NO_K, ko=adr(7)), INV),
    (dict(pos=None), INV), (dict(inv=None), INV), (dict(rot=0), INV),
    (dict(rot=-16), INV), (dict(rot=144), INV), (dict(il=2), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(wq=None, wk=None, pos=None, inv=None, rot=0), INV),
    (dict(sq=504), INV), (dict(sq=516), INV), (dict(sk=128), INV),
    (dict(so=-512), INV), (dict(sko=0), INV), (dict(q=A + 8), INV),
    (dict(pos=A + 2), INV), (dict(io=9), INV), (dict(qo=adr(1)), INV),
    (dict(ko=adr(0)), INV), (dict(qo=adr(7)), INV), (dict(qo=adr(2)), INV),
    (dict(qo=adr(0), so=1024), INV), (dict(ko=adr(4)), INV),
    (dict(D=96, sq=1024, so=1024, sk=512, sko=512), UNS),
    (dict(rot=24), UNS), (dict(rot=20, il=1), UNS), (dict(rows=1 << 26), UNS),
    (dict(Hq=1 << 16, sq=1 << 23, so=1 << 23), UNS),
])
def test_qk_norm_rope_rejects(kw, want):
    assert _qk(**kw) == want


def _qk_bwd(**kw):
    a = dict(q=adr(0), k=adr(1), io=BF, sq=512, sk=256, wq=adr(2), wk=adr(3),
             pos=adr(4), inv=adr(5), rot=32, il=0, eps=1e-6, dqo=adr(6),
             dko=adr(7), s1=512, s2=256, dq=adr(8), dk=adr(10), s3=512, s4=256,
             dwq=adr(11), dwk=adr(12), rows=10, Hq=4, Hk=2, D=128, ws=adr(9),
             wsb=1 << 30, stream=None)
    a.update(kw)
    return linattn._qk_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(dqo=None), INV), (dict(dko=None), INV), (dict(dq=None), INV),
    (dict(dk=None), INV), (dict(dwq=None), INV), (dict(dwk=None), INV),
    (dict(wk=None), INV), (dict(ws=None), INV), (dict(wsb=64), INV),
    (dict(dq=adr(10)), INV), (dict(dq=adr(0)), INV), (dict(dq=adr(7)), INV),
    (dict(dwq=adr(6)), INV), (dict(dk=adr(7), s4=512), INV),
    (dict(s1=500), INV), (dict(s4=128), INV), (dict(rot=8), UNS),
    (dict(D=48), UNS),
])
def test_qk_norm_rope_backward_rejects(kw, want):
    assert _qk_bwd(**kw) == want


# ---------------------------------------------------------------------------
# the binding, with CPU tensors: the mismatch is named before the device

F32, I32 = torch.float32, torch.int32


def t(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def test_binding_rejects_linattn():
    B, T, Hk, H, D, E = 2, 70, 2, 4, 16, 32
    x = dict(q=t(B, T, Hk, D), k=t(B, T, Hk, D), v=t(B, T, H, E),
             g=t(B, T, H, dt=F32))
    s = t(B, H, D, E, dt=F32)
    for over, what in [
            (dict(q=t(B, T, D)), "q has"), (dict(k=t(B, T, H, D)), "k"),
            (dict(k=x["k"].float()), "k"), (dict(v=t(B, T + 1, H, E)), "v"),
            (dict(v=x["v"].float()), "v"), (dict(g=t(B, T, Hk, dt=F32)), "g"),
            (dict(g=t(Hk, dt=F32)), "one decay"),
            (dict(g=t(B, T, H, E, dt=F32)), "g"), (dict(q=x["q"].half()), "q"),
            (dict(g=x["g"].double()), "g"), (dict(s0=s[:1]), "s0"),
            (dict(s_out=s.bfloat16()), "s_out"),
            (dict(o=t(B, T, H, D)), "o"),
            (dict(lengths=torch.zeros(B, dtype=torch.int64)), "lengths"),
            (dict(lengths=torch.zeros(3, dtype=I32)), "lengths"),
            ({}, "GPU")]:
        a = {**x, **over}
        four = [a.pop(n) for n in "qkvg"]
        with pytest.raises(ValueError, match=what):
            kda.kda_linattn(*four, **a)
    for over, what in [(dict(do=t(B, T, H, D)), "do"),
                       (dict(dsT=s[0]), "dsT"), ({}, "GPU")]:
        a = {"do": t(B, T, H, E), **over}
        with pytest.raises(ValueError, match=what):
            kda.kda_linattn_backward(*x.values(), **a)
    one = [v[:, 0].contiguous() for v in x.values()]
    with pytest.raises(ValueError, match="state"):
        kda.kda_linattn_step(*one, s[:1])
    with pytest.raises(ValueError, match="o"):
        kda.kda_linattn_step(*one, s, o=t(B, H, D))
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_linattn_step(*one, s)


def test_binding_rejects_qk_norm_rope():
    q, k, w = t(5, 4, 32), t(5, 2, 32), t(32, dt=F32)
    pos, inv = t(5, dt=I32), t(16, dt=F32)
    for a, kw, what in [
            ((q[0], k, pos, inv), {}, "q has"),
            ((q, k[:4], pos, inv), {}, "k"),
            ((q, t(5, 2, 16), pos, inv), {}, "k"),
            ((q, k.float(), pos, inv), {}, "k"),
            ((q.half(), None, pos, inv), {}, "q"),
            ((q, k, pos, None), {}, "go together"),
            ((q, k, None, inv), {}, "go together"),
            ((q, k, pos.long(), inv), {}, "positions"),
            ((q, k, pos[:3], inv), {}, "positions"),
            ((q, k, pos, inv.double()), {}, "inv_freq"),
            ((q, k, pos, inv[:0]), {}, "empty"),
            ((q, k, pos, inv), dict(wq=w[:16]), "wq"),
            ((q, k, pos, inv), dict(wk=w.bfloat16()), "wk"),
            ((q, None, pos, inv), dict(wk=w), "wk without k"),
            ((q, None, pos, inv), dict(k_out=k), "k_out"),
            ((q, k, pos, inv), dict(q_out=k), "q_out"),
            ((q, k, pos, inv), {}, "GPU")]:
        with pytest.raises(ValueError, match=what):
            kda.kda_qk_norm_rope(*a, **kw)
    for over, what in [(dict(dq_out=q[:4]), "dq_out"),
                       (dict(dk_out=None), "go together"),
                       (dict(dk_out=q), "dk_out"), (dict(dq=k), "dq"),
                       (dict(dk=q), "dk"), ({}, "GPU")]:
        a = dict(dq_out=q, dk_out=k)
        a.update(over)
        with pytest.raises(ValueError, match=what):
            kda.kda_qk_norm_rope_backward(q, k, pos, inv, a.pop("dq_out"),
                                          a.pop("dk_out"), wq=w, wk=w, **a)


def test_token_strides():
    x = t(3, 5, 96)  # [B, T, fused]

    def f(t, name):
        return linattn._token_stride(t.shape, t.stride(), name)

    q = x[..., :64].unflatten(-1, (4, 16))
    assert f(q, "q") == 96
    assert f(q.contiguous(), "q") == 64
    assert f(q[:1], "q") == 96 and f(q[:, :1], "q") == 480
    assert f(q[1, 2][None], "q") == 64  # one token
    for bad, what in [(q.transpose(0, 1), "evenly"),
                      (q[:, ::2].unflatten(1, (3, 1)).transpose(0, 1),
                       "evenly"),
                      (q.transpose(-1, -2), "dense"),
                      (x[..., :64].unflatten(-1, (16, 4)).transpose(-1, -2),
                       "dense"), (q[..., ::2], "dense"), (q[:, :, ::2],
                                                          "dense")]:
        with pytest.raises(ValueError, match=what):
            f(bad, "q")


def test_binding_refuses_sizes_past_an_int():
    def m(*s, dt=torch.bfloat16):
        return torch.empty(*s, dtype=dt, device="meta")

    q = m(1, P + 3, 1, 16)
    calls = [
        lambda: kda.kda_linattn(q, q, q, m(1, dt=F32)),
        lambda: kda.kda_linattn_backward(q, q, q, m(1, dt=F32), q),
        lambda: kda.kda_linattn_step(q[0], q[0], q[0], m(1, dt=F32), q),
        lambda: kda.kda_qk_norm_rope(m(1, P + 1, 16), None, None, None),
    ]
    for call in calls:
        with pytest.raises(kda.KdaError, match="unsupported"):
            call()


@pytest.mark.skipif(shutil.which("hipcc") is None and
                    not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc not available")
def test_linattn_abi_clean_under_asan_ubsan():
    """The boundary's host code under AddressSanitizer and
    UndefinedBehaviorSanitizer, its launchers replaced by stubs."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    csrc = os.path.join(ROOT, "gated_delta_rule_74_amd", "csrc")
    with tempfile.TemporaryDirectory(prefix="kda_san_") as tmp:
        exe = os.path.join(tmp, "linattn_abi_san")
        r = subprocess.run(
            [hipcc, "-O1", "-g", "-std=c++17", "--offload-arch=gfx950",
             "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xclang",
             "-target-feature", "-Xclang", "-packed-fp32-ops", "-I",
             os.path.join(ROOT, "include"), "-I", csrc,
             os.path.join(csrc, "kda_linattn_api.hip"),
             os.path.join(ROOT, "tests", "sanitize",
                          "linattn_abi_driver.cpp"),
             "-o", exe], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                   UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
        r = subprocess.run([exe], capture_output=True, text=True, env=env,
                           timeout=300)
        assert r.returncode == 0 and "0 mismatches" in r.stdout, \
            r.stdout + r.stderr
