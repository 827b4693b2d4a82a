"""blockscaled_gated_gemm and blockscaled_gated_gemm_backward against a plain binary64 form.

Tolerance: the fp32 accumulation of a product is off by at most twice (K + 4) 2^-24 S, S = sum |a b| (any
order, the output factors' roundings among it); MXFP8 products are compared with the model of the
scaled MFMA's own truncation (gpu_common.mxfp8_mfma_model).  The activation's bound is act_rel, and each
output is off by half a bf16 step more."""
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import mxfp8_mfma_model, note
from tests.plain64 import (BF16, F32, act64, act_grad_terms, act_rel, assert_within, mxfp8_values, nvfp4_values,
                           product)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NV, MX, SLAB = bsq.FMT_NVFP4, bsq.FMT_MXFP8, bsq.FMT_MX_SLAB
AR, BR = bsq.FMT_A_ROWSCALED, bsq.FMT_B_ROWSCALED


def gauss(R, K, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((R, K), generator=g) * std).to(torch.bfloat16).to(DEV)


def operand(fmt, rowscaled, slab, R, K, std, seed):
    """(codes, scales, s_enc) as the library's own casts make them."""
    x = gauss(R, K, std, seed)
    if fmt & 0xF == MX:
        q = bsq.mxfp8_quantize(x, bsq.ROW | (bsq.MX_SLAB if fmt & slab else 0))
        return q["row_codes"], q["row_scales"], None
    if fmt & rowscaled:
        q = bsq.nvfp4_quantize_rowscaled(x)
        return q["codes"], q["scales"], q["s_enc"]
    q = bsq.nvfp4_quantize(x)
    return q["row_codes"], q["row_scales"], q["s_enc"][:1].clone()


def product64(fmt, a, b, slab_a, slab_b, rows, cols):
    """(product of the rows and columns asked for, its error bound)."""
    K = a[0].shape[1] * (2 if fmt & 0xF == NV else 1)
    if fmt & 0xF == NV:
        va, vb = nvfp4_values(*a), nvfp4_values(*b)
        p, S = product(va[rows], vb[cols])
        return p, 2 * (K + 4) * F32 * S
    va, vb = mxfp8_values(a[0], a[1], slab_a), mxfp8_values(b[0], b[1], slab_b)
    _, S = product(va[rows], vb[cols])

    def row_major(q, slab):
        c = q[0].cpu()
        if slab:
            R, k = c.shape
            f = c.reshape(-1)
            c = torch.cat([f[i * k:min(R, i + 256) * k].reshape(k // 64, -1, 64).transpose(0, 1).reshape(-1, k)
                           for i in range(0, R, 256)])
        return c.numpy()
    m = mxfp8_mfma_model(row_major(a, slab_a), a[1].cpu().numpy(), row_major(b, slab_b), b[1].cpu().numpy(),
                         rows.numpy(), cols.numpy())
    return torch.from_numpy(m), 2 * (K + 4) * F32 * S


def sample(n, most, seed):
    """All indices, or `most` of them with the ends of every 64 rows preferred."""
    if n <= most:
        return torch.arange(n)
    r = np.random.default_rng(seed)
    edges = [i for i in range(n) if i % 64 in (0, 63) or i == n - 1]
    pick = r.choice(edges, min(len(edges), most // 2), replace=False).tolist() + r.choice(n, most // 2, replace=False).tolist()
    return torch.from_numpy(np.unique(np.asarray(pick + [0, n - 1], np.int64)))


def rounded(v, e):
    """Bound of a bf16 output whose fp32 value is within e of v."""
    return e + (v.abs() + e) * BF16 + 2.0 ** -133


def forward(fmt, act, M, F, K, save, seed=1, most=192):
    note("gated fmt=%#x act=%d %d %d %d save=%s" % (fmt, act, M, F, K, save))
    a = operand(fmt, AR, bsq.FMT_MX_SLAB_A, M, K, 1.0, seed)
    wg = operand(fmt, BR, bsq.FMT_MX_SLAB_B, F, K, 2.0 / K ** 0.5, seed + 1)
    wu = operand(fmt, BR, bsq.FMT_MX_SLAB_B, F, K, 1.0 / K ** 0.5, seed + 2)
    r = bsq.blockscaled_gated_gemm(fmt, act, *a, *wg, *wu, save_gate_up=save)
    torch.cuda.synchronize()
    h, gu = r if save else (r, None)
    rows, cols = sample(M, most, seed), sample(F, most, seed + 1)
    sa, sb = bool(fmt & bsq.FMT_MX_SLAB_A), bool(fmt & bsq.FMT_MX_SLAB_B)
    g, eg = product64(fmt, a, wg, sa, sb, rows, cols)
    u, eu = product64(fmt, a, wu, sa, sb, rows, cols)
    at = lambda t: t.cpu()[rows][:, cols]   # noqa: E731
    f, _ = act64(g, act)
    want = f * u
    e = 1.13 * eg * (u.abs() + eu) + f.abs() * eu + want.abs() * (act_rel(g.abs() + eg, act) + 2 * F32)
    assert_within(at(h), want, rounded(want, e), "h")
    if save:
        assert_within(at(gu[:, :F]), g, rounded(g, eg), "gate")
        assert_within(at(gu[:, F:]), u, rounded(u, eu), "up")
    return h


SIZES = [(1, 1, 32), (3, 7, 64), (64, 128, 256), (255, 129, 288), (257, 200, 512), (130, 264, 1056), (300, 384, 768)]


@pytest.mark.parametrize("fmt", [NV, NV | AR, NV | BR, NV | AR | BR, MX])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_forward(fmt, M, F, K):
    forward(fmt, M % 3, M, F, K, True)


@pytest.mark.parametrize("fmt", [MX | SLAB, MX | bsq.FMT_MX_SLAB_A, MX | bsq.FMT_MX_SLAB_B])
@pytest.mark.parametrize("M,F,K", [(1, 1, 512), (129, 130, 512), (257, 513, 1024), (300, 392, 1536)])
def test_forward_slab(fmt, M, F, K):
    forward(fmt, F % 3, M, F, K, F % 2 == 0)


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("fmt", [NV, MX])
def test_forward_not_saved_has_the_same_h(fmt, act):
    h0 = forward(fmt, act, 200, 136, 512, True)
    h1 = forward(fmt, act, 200, 136, 512, False)
    assert torch.equal(h0, h1)


@pytest.mark.parametrize("fmt,M,F,K", [(NV, 2500, 4104, 512), (NV | AR, 1030, 2056, 768), (MX | SLAB, 1500, 4104, 512),
                                       (NV, 4200, 2048, 1280)])
def test_forward_many_tiles(fmt, M, F, K):
    forward(fmt, 0, M, F, K, True, most=96)
    forward(fmt, 2, M, F, K, False, most=96)


# just below and above the sizes where the kernels change over from 64 x 64 to 256 x 256 tiles
@pytest.mark.parametrize("fmt,M,F,K", [(NV, 2048, 1024, 256), (NV, 2049, 1032, 256), (NV, 2049, 1033, 288), (MX, 1536, 512, 512),
                                       (MX, 1537, 520, 512), (MX, 1537, 517, 512), (MX, 2049, 1033, 544),
                                       (MX | SLAB, 1537, 520, 512), (MX | bsq.FMT_MX_SLAB_A, 1537, 517, 1024),
                                       (MX | bsq.FMT_MX_SLAB_B, 1800, 700, 512), (NV | AR | BR, 2049, 1033, 256),
                                       (NV | BR, 2100, 1041, 96)])
def test_forward_large_and_small_tiles(fmt, M, F, K):
    forward(fmt, K % 3, M, F, K, True, most=96)


@pytest.mark.parametrize("fmt,M,F,K", [(NV, 2048, 2048, 256), (NV, 2049, 2056, 256), (NV, 2049, 2057, 288), (MX, 2048, 1024, 512),
                                       (MX, 2049, 1032, 512), (MX, 2049, 1033, 512), (MX, 2049, 2059, 544),
                                       (MX | SLAB, 2049, 1037, 512), (MX | bsq.FMT_MX_SLAB_A, 2100, 1032, 1024),
                                       (MX | bsq.FMT_MX_SLAB_B, 2049, 1036, 512), (NV | AR | BR, 2049, 2051, 256),
                                       (NV | AR, 2100, 2064, 96)])
def test_backward_large_and_small_tiles(fmt, M, F, K):
    backward(fmt, F % 3, M, F, K, most=96)


def backward(fmt, act, M, F, K, seed=5, most=192, in_place=False, gate_std=1.5):
    note("gated backward fmt=%#x act=%d %d %d %d" % (fmt, act, M, F, K))
    dy = operand(fmt, AR, bsq.FMT_MX_SLAB_A, M, K, 0.01, seed)
    w = operand(fmt, BR, bsq.FMT_MX_SLAB_B, F, K, 0.02, seed + 1)
    gu = gauss(M, 2 * F, gate_std, seed + 2)
    keep = gu.clone()
    d = bsq.blockscaled_gated_gemm_backward(fmt, act, *dy, *w, gu, out=gu if in_place else None)
    torch.cuda.synchronize()
    assert in_place or torch.equal(gu, keep)
    rows, cols = sample(M, most, seed), sample(F, most, seed + 1)
    dh, e = product64(fmt, dy, w, bool(fmt & bsq.FMT_MX_SLAB_A), bool(fmt & bsq.FMT_MX_SLAB_B), rows, cols)
    at = lambda t: t.cpu()[rows][:, cols]   # noqa: E731
    g, u = at(keep[:, :F]).double(), at(keep[:, F:]).double()
    f, df = act64(g, act)
    rel = act_rel(g, act) + 4 * F32
    want_g, want_u = dh * u * df, dh * f
    eg = e * (u * df).abs() + (dh.abs() + e) * u.abs() * act_grad_terms(g, act) * rel
    eu = e * f.abs() + (dh.abs() + e) * f.abs() * rel
    assert_within(at(d[:, :F]), want_g, rounded(want_g, eg), "d_gate")
    assert_within(at(d[:, F:]), want_u, rounded(want_u, eu), "d_up")
    # the same against differences of sum(dh act(g) u)
    step = 1e-5
    diff = dh * u * (act64(g + step, act)[0] - act64(g - step, act)[0]) / (2 * step)
    slack = 1e-8 * (1 + (dh * u).abs())
    assert_within(at(d[:, :F]), diff, rounded(diff, eg + slack), "d_gate against differences")
    return d


@pytest.mark.parametrize("fmt", [NV, NV | AR, NV | BR, NV | AR | BR, MX])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_backward(fmt, M, F, K):
    backward(fmt, F % 3, M, F, K)


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("fmt", [NV, MX | SLAB])
def test_backward_activations(fmt, act):
    backward(fmt, act, 200, 264, 512)
    backward(fmt, act, 100, 72, 512, gate_std=20.0)   # gates far out on both sides


@pytest.mark.parametrize("fmt", [MX | SLAB, MX | bsq.FMT_MX_SLAB_A, MX | bsq.FMT_MX_SLAB_B])
@pytest.mark.parametrize("M,F,K", [(1, 1, 512), (257, 513, 1024), (300, 392, 1536)])
def test_backward_slab(fmt, M, F, K):
    backward(fmt, M % 3, M, F, K)


def test_backward_many_tiles_and_in_place():
    backward(MX | SLAB, 0, 1500, 4104, 512, most=96)
    a = backward(NV, 1, 2500, 2056, 768, most=96)
    assert torch.equal(a, backward(NV, 1, 2500, 2056, 768, most=96, in_place=True))


def test_empty_and_k0():
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)   # noqa: E731
    one = torch.ones(1, device=DEV)
    h, gu = bsq.blockscaled_gated_gemm(NV, 0, e8(0, 16), e8(0, 2), one, e8(8, 16), e8(8, 2), one, e8(8, 16), e8(8, 2),
                                       one, save_gate_up=True)
    assert tuple(h.shape) == (0, 8) and tuple(gu.shape) == (0, 16)
    for fmt, s in ((NV, one), (MX, None)):
        h, gu = bsq.blockscaled_gated_gemm(fmt, 1, e8(5, 0), e8(5, 0), s, e8(9, 0), e8(9, 0), s, e8(9, 0), e8(9, 0), s,
                                           save_gate_up=True)
        assert not h.any() and not gu.any()
        d = bsq.blockscaled_gated_gemm_backward(fmt, 0, e8(5, 0), e8(5, 0), s, e8(9, 0), e8(9, 0), s,
                                                torch.ones((5, 18), dtype=torch.bfloat16, device=DEV))
        assert not d.any()


@pytest.mark.parametrize("fmt", [NV, MX])
def test_nothing_outside_the_outputs_is_written(fmt):
    M, F, K = 70, 75, 288
    a, wg, wu = (operand(fmt, 0, 0, r, K, 0.5, s) for r, s in ((M, 1), (F, 2), (F, 3)))
    pad = 4096
    buf = torch.full((M * 3 * F + 3 * pad,), 9.0, dtype=torch.bfloat16, device=DEV)
    h0, g0 = pad, 2 * pad + M * F + (-(M * F)) % 8
    h = buf[h0:h0 + M * F].view(M, F)
    gu = buf[g0:g0 + 2 * M * F].view(M, 2 * F)
    bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu, save_gate_up=True, out=h, gate_up=gu)
    dy, w = operand(fmt, 0, 0, M, K, 0.5, 4), operand(fmt, 0, 0, F, K, 0.5, 5)
    bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, gu, out=gu)
    rest = torch.cat([buf[:h0], buf[h0 + M * F:g0], buf[g0 + 2 * M * F:]])
    assert (rest == 9.0).all()


def test_non_finite_values_stay_in_their_row_and_column():
    M, F, K = 40, 48, 512
    for fmt in (NV, MX):
        a, wg, wu = (operand(fmt, 0, 0, r, K, 0.5, s) for r, s in ((M, 1), (F, 2), (F, 3)))
        clean = bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu).cpu()
        a[1][3, 1] = 0x7F if fmt == NV else 0xFF    # NaN scales: a token, a gate row, an up row
        wg[1][5, 0] = 0x7F if fmt == NV else 0xFF
        wu[1][7, 2] = 0x7F if fmt == NV else 0xFF
        h = bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu).cpu()
        bad = torch.zeros((M, F), dtype=torch.bool)
        bad[3], bad[:, 5], bad[:, 7] = True, True, True
        assert torch.equal(h[~bad], clean[~bad])
        if fmt == MX:   # the NVFP4 products take the scale code without a value, which no cast writes, as 480
            assert torch.isnan(h[bad]).all()
    g = torch.tensor([[math.inf, -math.inf, math.nan, 0.0] + [1.0] * 4], dtype=torch.bfloat16, device=DEV)
    u = torch.ones((1, 8), dtype=torch.bfloat16, device=DEV)
    dy, w = operand(MX, 0, 0, 1, 64, 0.5, 6), operand(MX, 0, 0, 8, 64, 0.5, 7)
    for act in (0, 1, 2):
        d = bsq.blockscaled_gated_gemm_backward(MX, act, *dy, *w, torch.cat([g, u], 1)).cpu()
        assert torch.isfinite(d[0, 3:8]).all() and torch.isfinite(d[0, 11:]).all()
        assert torch.isnan(d[0, 2]) and torch.isnan(d[0, 10])


def test_other_stream_and_graph_replays():
    M, F, K = 300, 264, 512
    wg, wu = operand(NV, 0, 0, F, K, 0.05, 2), operand(NV, 0, 0, F, K, 0.05, 3)
    wd = operand(MX, 0, 0, F, K, 0.05, 4)
    a, dy = operand(NV, 0, 0, M, K, 1.0, 1), operand(MX, 0, 0, M, K, 1.0, 5)

    def step(h=None, gu=None, d=None):
        h, gu = bsq.blockscaled_gated_gemm(NV, 0, *a, *wg, *wu, save_gate_up=True, out=h, gate_up=gu)
        return h, gu, bsq.blockscaled_gated_gemm_backward(MX, 0, *dy, *wd, gu, out=d)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*got)
    for seed in (11, 12, 13):
        for t, n in zip(a + dy, operand(NV, 0, 0, M, K, 1.0, seed) + operand(MX, 0, 0, M, K, 1.0, seed + 50)):
            if t is not None:
                t.copy_(n)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_python_refusals():
    M, F, K = 16, 24, 64
    a, wg, wu = (operand(NV, 0, 0, r, K, 0.5, s) for r, s in ((M, 1), (F, 2), (F, 3)))
    small = operand(NV, 0, 0, F - 8, K, 0.5, 3)
    other_k = operand(NV, 0, 0, F, 2 * K, 0.5, 3)
    for bad in (small, other_k, (wu[0], wu[1][:, :2].contiguous(), wu[2]), (wu[0], wu[1], torch.ones(2, device=DEV))):
        with pytest.raises(ValueError):
            bsq.blockscaled_gated_gemm(NV, 0, *a, *wg, *bad)
    with pytest.raises(TypeError):
        bsq.blockscaled_gated_gemm(NV, 0, a[0].cpu(), a[1], a[2], *wg, *wu)
    with pytest.raises(TypeError):
        bsq.blockscaled_gated_gemm(NV, 0, *a, *wg, wu[0], wu[1], None)
    with pytest.raises(bsq.BsqError):
        bsq.blockscaled_gated_gemm(NV, 3, *a, *wg, *wu)
    with pytest.raises(ValueError):
        bsq.blockscaled_gated_gemm(NV, 0, *a, *wg, *wu, gate_up=torch.empty((M, 2 * F), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        bsq.blockscaled_gated_gemm_backward(NV, 0, *a, *wg, torch.empty((M, F), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        bsq.blockscaled_gated_gemm_backward(NV, 0, *a, *wg, torch.empty((M, 2 * F), device=DEV))
    with pytest.raises(ValueError):
        bsq.blockscaled_gated_gemm_backward(NV, 0, *a, *other_k, torch.empty((M, 2 * F), dtype=torch.bfloat16, device=DEV))


# outputs past 2^31 elements: 76800 x 2 * 14336
@pytest.mark.parametrize("fmt,K", [(NV, 512), (NV, 96), (MX, 96)])
def test_outputs_past_2_to_the_31_elements(fmt, K):
    M, F = 76800, 14336
    a, wg, wu = (operand(fmt, 0, 0, r, K, std, s) for r, std, s in ((M, 1.0, 1), (F, 2.0 / K ** 0.5, 2), (F, 1.0 / K ** 0.5, 3)))
    h, gu = bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu, save_gate_up=True)
    rows = torch.tensor([0, 255, 256, 37449, 37450, 74898, 74899, M - 257, M - 2, M - 1])   # 37449 * 2F < 2^30 < 37450 * 2F
    cols = torch.tensor([0, 127, 128, F - 129, F - 1])
    part = tuple(t[rows.to(DEV)] if t is not None and t.dim() == 2 else t for t in a)
    every = torch.arange(len(rows))
    g, eg = product64(fmt, part, wg, False, False, every, cols)
    u, eu = product64(fmt, part, wu, False, False, every, cols)
    f, _ = act64(g, 0)
    want = f * u
    e = 1.13 * eg * (u.abs() + eu) + f.abs() * eu + want.abs() * (act_rel(g.abs() + eg, 0) + 2 * F32)
    at = lambda t: t[rows.to(DEV)][:, cols.to(DEV)].cpu()   # noqa: E731
    assert_within(at(h), want, rounded(want, e), "h")
    assert_within(at(gu[:, :F]), g, rounded(g, eg), "gate")
    assert_within(at(gu[:, F:]), u, rounded(u, eu), "up")
    keep = gu[rows.to(DEV)].cpu()
    dy, w = operand(fmt, 0, 0, M, K, 0.01, 4), operand(fmt, 0, 0, F, K, 0.02, 5)
    d = bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, gu, out=gu)
    part = tuple(t[rows.to(DEV)] if t is not None and t.dim() == 2 else t for t in dy)
    dh, e = product64(fmt, part, w, False, False, every, cols)
    g, u = keep[:, :F][:, cols].double(), keep[:, F:][:, cols].double()
    f, df = act64(g, 0)
    rel = act_rel(g, 0) + 4 * F32
    eg = e * (u * df).abs() + (dh.abs() + e) * u.abs() * act_grad_terms(g, 0) * rel
    eu = e * f.abs() + (dh.abs() + e) * f.abs() * rel
    assert_within(at(d[:, :F]), dh * u * df, rounded(dh * u * df, eg), "d_gate")
    assert_within(at(d[:, F:]), dh * f, rounded(dh * f, eu), "d_up")


# K-blocks even and odd, slices even and odd, K ending inside a slice; the sizes take the large tiles
@pytest.mark.parametrize("fmt,K", [(NV, 512), (NV, 544), (NV, 96), (MX, 512), (MX, 544), (MX, 576), (MX, 608), (MX, 160)])
def test_non_finite_scales_stay_in_their_row_and_column_of_large_tiles(fmt, K):
    M, F = 2310, 2057
    a, wg, wu = (operand(fmt, 0, 0, r, K, 0.5, s) for r, s in ((M, 1), (F, 2), (F, 3)))
    dy, w, gu = operand(fmt, 0, 0, M, K, 0.5, 4), operand(fmt, 0, 0, F, K, 0.5, 5), gauss(M, 2 * F, 1.0, 6)
    run = lambda: (bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu).cpu(),   # noqa: E731
                   bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, gu).cpu())
    h0, d0 = run()
    nan = 0x7F if fmt == NV else 0xFF
    last = a[1].shape[1] - 1
    for t in (a, dy):
        t[1][3, 0] = t[1][259, 1] = t[1][2305, last] = nan
    wg[1][5, 0] = wg[1][200, last] = wu[1][7, 1] = wu[1][1030, 0] = nan
    w[1][5, 0] = w[1][200, last] = w[1][1030, 1] = nan
    h, d = run()
    rows, cols, wcols = [3, 259, 2305], [5, 200, 7, 1030], [5, 200, 1030]
    keep = torch.ones((M, F), dtype=torch.bool)
    keep[rows] = False
    back = keep.clone()
    keep[:, cols] = False
    back[:, wcols] = False
    assert torch.equal(h[keep], h0[keep])
    for half in (slice(0, F), slice(F, 2 * F)):
        assert torch.equal(d[:, half][back], d0[:, half][back])
    if fmt == MX:   # the NVFP4 products take the scale code without a value, which no cast writes, as 480
        assert torch.isnan(h[rows]).all() and torch.isnan(d[rows]).all()
