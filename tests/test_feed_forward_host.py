"""Refusals of the feed-forward operators' C entry points, on the host: every invalid argument is
answered with its documented status before any HIP call."""
import ctypes as C
import math

import pytest

FAKE = 0x10000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import os

    import block_scaled_precision_nvfp4_amd as bsq
    if not os.path.exists(bsq.LIB_PATH):
        from block_scaled_precision_nvfp4_amd import build
        build.build()
    return bsq.lib()


def mv(L, gated=False, **kw):
    a = dict(flags=0, act=0, M=2, N=64, K=64, x=FAKE, ldx=64, c=FAKE, s=FAKE, e=FAKE, uc=FAKE, us=FAKE, ue=FAKE, y=FAKE,
             dt=0)
    a.update(kw)
    if gated:
        return L.nvfp4_gated_matvec(a["flags"], a["act"], a["M"], a["N"], a["K"], a["x"], a["ldx"], a["c"], a["s"],
                                    a["e"], a["uc"], a["us"], a["ue"], a["y"], None)
    return L.nvfp4_matvec(a["flags"], a["M"], a["N"], a["K"], a["x"], a["ldx"], a["c"], a["s"], a["e"], a["y"], a["dt"],
                          None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(flags=0x10), 3, "flags"), (dict(M=-1), 2, "negative"), (dict(N=-1), 2, "negative"),
    (dict(K=-16), 2, "negative"), (dict(K=24), 2, "multiple of 16"), (dict(K=1 << 24, ldx=1 << 24), 2, "exceeds"),
    (dict(M=(1 << 20) + 1), 2, "tokens"), (dict(N=(1 << 31) + 1), 2, "rows"), (dict(y=None), 1, "output"),
    (dict(e=None), 1, "tensor scale"), (dict(x=None), 1, "NULL"), (dict(c=None), 1, "NULL"), (dict(s=None), 1, "NULL"),
    (dict(ldx=56), 2, "ldx"), (dict(ldx=68), 2, "ldx"), (dict(x=FAKE + 2), 6, "aligned"), (dict(c=FAKE + 8), 6, "aligned"),
    (dict(s=FAKE + 4), 6, "aligned"), (dict(y=FAKE + 2), 6, "aligned"),
])
def test_matvec_refusals(L, gated, kw, status, needle):
    assert mv(L, gated, **kw) == status
    assert needle in L.bsq_last_error().decode()


def test_matvec_types_and_activations(L):
    assert mv(L, dt=2) == 3
    assert mv(L, True, act=3) == 3 and mv(L, True, act=-1) == 3
    for k in ("uc", "us", "ue"):
        assert mv(L, True, **{k: None}) == 1
    assert mv(L, True, uc=FAKE + 4) == 6


def test_grad_workspace(L):
    assert L.grad_workspace_bytes(-1) == -1
    assert L.grad_workspace_bytes((1 << 24) + 1) == -1
    assert L.grad_workspace_bytes(0) > 0
    assert L.grad_workspace_bytes(1000) >= L.grad_workspace_bytes(1)


def clip(L, sumsq_only=False, **kw):
    a = dict(p=[FAKE, FAKE], o=None, n=[8, 8], d=[1, 0], count=None, s=FAKE, max_norm=1.0, norm=FAKE, ws=FAKE)
    a.update(kw)
    arr = lambda t, v: None if v is None else (t * len(v))(*v)   # noqa: E731
    count = len(a["p"]) if a["count"] is None else a["count"]
    P, O, N, D = arr(C.c_void_p, a["p"]), arr(C.c_void_p, a["o"]), arr(C.c_int64, a["n"]), arr(C.c_int, a["d"])
    if sumsq_only:
        return L.grad_sumsq(P, N, D, count, a["s"], a["ws"], None)
    return L.grad_clip(P, O, N, D, count, a["s"], a["max_norm"], a["norm"], None)


@pytest.mark.parametrize("sumsq_only", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), 2), (dict(count=(1 << 24) + 1), 2), (dict(n=None), 1), (dict(d=None), 1),
    (dict(n=[8, -1]), 2), (dict(n=[1 << 40, 1]), 2), (dict(d=[1, 2]), 3), (dict(p=[FAKE, None]), 1),
    (dict(p=[FAKE + 2, FAKE]), 6), (dict(p=[FAKE, FAKE + 1]), 6), (dict(s=None), 1), (dict(s=FAKE + 4), 6),
])
def test_grad_refusals(L, sumsq_only, kw, status):
    assert clip(L, sumsq_only, **kw) == status


def test_grad_only_refusals(L):
    assert clip(L, True, ws=None) == 1 and clip(L, True, ws=FAKE + 8) == 6
    assert clip(L, max_norm=-0.5) == 3 and clip(L, max_norm=math.nan) == 3
    assert clip(L, norm=None) == 1 and clip(L, norm=FAKE + 2) == 6
    assert clip(L, o=[FAKE, None]) == 1 and clip(L, o=[FAKE, FAKE + 1]) == 6


def gated(L, backward=False, **kw):
    a = dict(fmt=0, act=0, M=4, F=64, K=512, a=FAKE, as_=FAKE, ae=FAKE, g=FAKE, gs=FAKE, ge=FAKE, u=FAKE, us=FAKE,
             ue=FAKE, h=FAKE, gu=FAKE)
    a.update(kw)
    if backward:
        return L.blockscaled_gated_gemm_backward(a["fmt"], a["act"], a["M"], a["F"], a["K"], a["a"], a["as_"], a["ae"],
                                                 a["g"], a["gs"], a["ge"], a["gu"], a["h"], None)
    return L.blockscaled_gated_gemm(a["fmt"], a["act"], a["M"], a["F"], a["K"], a["a"], a["as_"], a["ae"], a["g"],
                                    a["gs"], a["ge"], a["u"], a["us"], a["ue"], a["h"], a["gu"], None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(fmt=2), 3, "fmt"), (dict(fmt=0x11), 3, "row-scaled"), (dict(fmt=0x40), 3, "slab"),
    (dict(fmt=0xC1, K=544), 2, "512"), (dict(act=3), 3, "act"), (dict(act=-1), 3, "act"), (dict(M=-1), 2, "negative"),
    (dict(F=-1), 2, "negative"), (dict(K=-32), 2, "negative"), (dict(K=48), 2, "multiple of 32"),
    (dict(K=1 << 24), 2, "exceeds"), (dict(fmt=1, K=1 << 23), 2, "exceeds"), (dict(M=1 << 30, F=1 << 30), 2, "large"),
    (dict(M=1 << 62, F=8), 2, "large"), (dict(h=None), 1, "NULL"), (dict(h=FAKE + 8), 6, "aligned"),
    (dict(gu=FAKE + 2), 6, "aligned"), (dict(a=None), 1, "NULL"), (dict(as_=None), 1, "NULL"), (dict(ae=None), 1, "scale"),
    (dict(g=None), 1, "NULL"), (dict(ge=None), 1, "scale"), (dict(g=FAKE + 4), 6, "aligned"), (dict(gs=FAKE + 8), 6, "aligned"),
])
def test_gated_refusals(L, backward, kw, status, needle):
    assert gated(L, backward, **kw) == status
    assert needle in L.bsq_last_error().decode()


def test_gated_only_refusals(L):
    assert gated(L, u=None) == 1 and gated(L, ue=None) == 1 and gated(L, us=FAKE + 1) == 6
    assert gated(L, True, gu=None) == 1
    assert gated(L, M=0, h=None) == 0 and gated(L, True, F=0, gu=None) == 0   # nothing to do


@pytest.mark.parametrize("act", [0, 1, 2])
def test_plain_derivatives_against_differences(act):
    import torch

    from tests.plain64 import act64
    g = torch.linspace(-12, 12, 2001, dtype=torch.float64)
    e = 1e-5
    d = (act64(g + e, act)[0] - act64(g - e, act)[0]) / (2 * e)
    assert float((d - act64(g, act)[1]).abs().max()) < 1e-8


def test_clip_in_one_call_refusals(L):
    def call(**kw):
        a = dict(p=[FAKE], n=[8], d=[1], m=1.0, norm=FAKE, ws=FAKE)
        a.update(kw)
        P, N, D = (C.c_void_p * 1)(*a["p"]), (C.c_int64 * 1)(*a["n"]), (C.c_int * 1)(*a["d"])
        return L.clip_grad_norm(P, None, N, D, 1, a["m"], a["norm"], a["ws"], None)
    assert call(m=-1.0) == 3 and call(m=math.nan) == 3 and call(d=[2]) == 3
    assert call(norm=None) == 1 and call(ws=None) == 1 and call(p=[None]) == 1
    assert call(norm=FAKE + 1) == 6 and call(ws=FAKE + 8) == 6 and call(p=[FAKE + 2]) == 6
