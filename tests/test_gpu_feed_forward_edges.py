"""Edges of the feed-forward operators: stores of the large tiles and of the token kernels stay inside their
outputs, values that are not finite go where the binary64 form has them, and the gated products around the sizes
where one tile hands over to the other.

The guarded outputs lie in a buffer with at least a tile's rows before and after them, filled with a value
that no output takes; the results are those of the same call on buffers of its own, bit for bit."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.plain64 import assert_within, nvfp4_values, product, store_error, sum_error
from tests.test_gpu_gated import AR, BR, DEV, MX, NV, SLAB, backward, forward, gauss, operand
from tests.test_gpu_matvec import tokens, weights

pytestmark = pytest.mark.gpu
MARK = 12345.0   # 12352 in bf16


def guarded(shapes, dtype):
    """Views of one marked buffer, 16-byte aligned, and a check that nothing around them changed."""
    pads = [max(4096, 264 * s[1]) // 8 * 8 for s in shapes]
    at, spans = 0, []
    for s, p in zip(shapes, pads):
        at += p
        spans.append((at, s))
        at += -(-s[0] * s[1] // 8) * 8
    buf = torch.full((at + pads[-1],), MARK, dtype=dtype, device=DEV)
    views = [buf[a:a + s[0] * s[1]].view(s) for a, s in spans]

    def intact():
        end = 0
        for a, s in spans:
            assert (buf[end:a] == buf[0]).all(), "written before an output"
            end = a + s[0] * s[1]
        assert (buf[end:] == buf[0]).all(), "written after an output"
        assert buf[0] == torch.tensor(MARK, dtype=dtype)
    return views, intact


# rows of the last tile: 1 .. 128 (half of its waves have none) and 129 .. 255; widths of whole 16-byte chunks and
# others; every loop.  All sizes take the 256 x 256 tiles.
GUARDED = [(NV, 2100, 2568, 512), (NV, 2239, 2568, 768), (NV, 2100, 2571, 512), (NV | AR | BR, 2239, 2568, 256),
           (NV, 2177, 2563, 288), (NV, 2100, 2564, 96), (MX, 2100, 2568, 512), (MX, 2239, 2563, 512),
           (MX, 2177, 2568, 544), (MX, 2050, 2561, 160), (MX | SLAB, 2100, 2568, 512), (MX | SLAB, 2239, 2565, 1024)]


@pytest.mark.parametrize("fmt,M,F,K", GUARDED)
def test_large_tiles_write_nothing_outside_their_outputs(fmt, M, F, K):
    note("guarded gated %#x %d %d %d" % (fmt, M, F, K))
    a = operand(fmt, AR, bsq.FMT_MX_SLAB_A, M, K, 1.0, 1)
    wg, wu = (operand(fmt, BR, bsq.FMT_MX_SLAB_B, F, K, 1.0 / K ** 0.5, s) for s in (2, 3))
    h, gu = bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu, save_gate_up=True)
    (vh, vgu), intact = guarded([(M, F), (M, 2 * F)], torch.bfloat16)
    bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu, save_gate_up=True, out=vh, gate_up=vgu)
    intact()
    assert torch.equal(vh, h) and torch.equal(vgu, gu)
    (vh,), intact = guarded([(M, F)], torch.bfloat16)
    bsq.blockscaled_gated_gemm(fmt, 0, *a, *wg, *wu, out=vh)
    intact()
    assert torch.equal(vh, h)
    dy, w = operand(fmt, AR, bsq.FMT_MX_SLAB_A, M, K, 0.01, 4), operand(fmt, BR, bsq.FMT_MX_SLAB_B, F, K, 0.02, 5)
    d = bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, gu)
    (vd, vgu), intact = guarded([(M, 2 * F), (M, 2 * F)], torch.bfloat16)
    vgu.copy_(gu)
    bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, vgu, out=vd)
    intact()
    assert torch.equal(vd, d) and torch.equal(vgu, gu)
    bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, vgu, out=vgu)
    intact()
    assert torch.equal(vgu, d)


@pytest.mark.parametrize("M", [1, 3, 20, 67])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens_write_nothing_outside_their_outputs(M, dtype):
    N, K = 1033, 528
    x, w, wu = tokens(M, K, 1), weights(N, K, 2), weights(N, K, 3)
    (y,), intact = guarded([(M, N)], dtype)
    bsq.nvfp4_matvec(x, *w, out_dtype=dtype, out=y)
    intact()
    assert torch.equal(y, bsq.nvfp4_matvec(x, *w, out_dtype=dtype))
    if dtype == torch.bfloat16:
        (h,), intact = guarded([(M, N)], dtype)
        bsq.nvfp4_gated_matvec(bsq.ACT_GELU, x, *w, *wu, out=h)
        intact()
        assert torch.equal(h, bsq.nvfp4_gated_matvec(bsq.ACT_GELU, x, *w, *wu))


# K below 64, of whole pieces of 64, and ending inside one
@pytest.mark.parametrize("M", [1, 6])
@pytest.mark.parametrize("K", [48, 512, 272])
def test_tokens_that_are_not_finite(M, K):
    N = 40
    clean, (c, s, se) = tokens(M, K, 9), weights(N, K, 10)
    s[7, K // 16 - 1] = 0x7F
    for value in (float("nan"), float("inf"), -float("inf")):
        for k in (0, K // 2 + 3, K - 1):
            x = clean.clone()
            x[M - 1, k] = value
            want, S = product(x.cpu().double(), nvfp4_values(c, s, se))
            y = bsq.nvfp4_matvec(x, c, s, se, out_dtype=torch.float32)
            assert_within(y, want, sum_error(K, S) + store_error(want, torch.float32), "y")


@pytest.mark.parametrize("M", [1, 6])
@pytest.mark.parametrize("K", [48, 512, 272])
def test_gated_tokens_that_are_not_finite(M, K):
    F = 40
    x, wg, wu = tokens(M, K, 9), weights(F, K, 10), weights(F, K, 11)
    clean = bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, *wg, *wu).cpu()
    assert torch.isfinite(clean).all()
    wg[1][5, 0] = wu[1][7, K // 16 - 1] = 0x7F
    bad = torch.zeros((M, F), dtype=torch.bool)
    bad[:, 5] = bad[:, 7] = True
    h = bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, *wg, *wu).cpu()
    assert torch.equal(torch.isnan(h), bad) and torch.equal(h[~bad], clean[~bad])
    if M > 1:
        x[2, K - 1] = float("nan")
        bad[2] = True
        h = bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, *wg, *wu).cpu()
        assert torch.equal(torch.isnan(h), bad) and torch.equal(h[~bad], clean[~bad])


# the last size that the 64 x 64 tiles take and the next one, of each loop, and large ones of the loops whose
# change-over lies highest
@pytest.mark.parametrize("fmt,M,F,K", [(NV, 1024, 2048, 256), (NV, 1024, 2049, 256), (NV, 2048, 1536, 288), (NV, 2049, 1536, 288),
                                       (MX, 2048, 1024, 512), (MX, 2049, 1024, 512), (MX, 1024, 512, 4096), (MX, 1024, 513, 4096),
                                       (MX, 2048, 1280, 1056), (MX, 2049, 1280, 1056), (MX, 2048, 1536, 544), (MX, 2049, 1536, 544),
                                       (MX | SLAB, 1536, 1024, 1024), (MX | SLAB, 1537, 1024, 1024),
                                       (MX | bsq.FMT_MX_SLAB_B, 1024, 1024, 4096), (MX | bsq.FMT_MX_SLAB_B, 1025, 1024, 4096)])
def test_forward_around_the_change_of_tiles(fmt, M, F, K):
    forward(fmt, K % 3, M, F, K, True, most=96)


@pytest.mark.parametrize("fmt,M,F,K", [(NV, 2048, 2560, 256), (NV, 2049, 2560, 256), (NV, 1536, 4096, 288), (NV, 1537, 4096, 288),
                                       (MX, 2048, 2048, 512), (MX, 2049, 2048, 512), (MX, 1024, 1024, 4096), (MX, 1025, 1024, 4096),
                                       (MX, 2048, 2560, 1056), (MX, 2049, 2560, 1056), (MX, 1536, 4096, 544), (MX, 1537, 4096, 544),
                                       (MX | SLAB, 1536, 2048, 1024), (MX | SLAB, 1537, 2048, 1024),
                                       (MX | bsq.FMT_MX_SLAB_A, 1024, 2048, 4096), (MX | bsq.FMT_MX_SLAB_A, 1025, 2048, 4096),
                                       (NV, 2305, 2571, 288), (NV | AR, 2305, 2568, 96), (MX, 2305, 2563, 544),
                                       (MX, 2305, 2568, 160)])
def test_backward_around_the_change_of_tiles(fmt, M, F, K):
    backward(fmt, K % 3, M, F, K, most=96)


# K-blocks even and odd, slices even and odd, K ending inside a slice; the size takes the large tiles
@pytest.mark.parametrize("fmt,K", [(NV, 512), (NV, 544), (NV, 96), (MX, 512), (MX, 544), (MX, 576), (MX, 608), (MX, 160)])
def test_scales_that_are_not_finite_in_the_backward_of_large_tiles(fmt, K):
    M, F = 2566, 2057
    dy, w, gu = operand(fmt, 0, 0, M, K, 0.5, 4), operand(fmt, 0, 0, F, K, 0.5, 5), gauss(M, 2 * F, 1.0, 6)
    d0 = bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, gu).cpu()
    nan, last = 0x7F if fmt == NV else 0xFF, dy[1].shape[1] - 1
    dy[1][3, 0] = dy[1][259, 1] = dy[1][2561, last] = nan
    w[1][5, 0] = w[1][200, last] = w[1][1030, 1] = nan
    d = bsq.blockscaled_gated_gemm_backward(fmt, 0, *dy, *w, gu).cpu()
    rows, cols = [3, 259, 2561], [5, 200, 1030]
    keep = torch.ones((M, F), dtype=torch.bool)
    keep[rows] = False
    keep[:, cols] = False
    for half in (slice(0, F), slice(F, 2 * F)):
        assert torch.equal(d[:, half][keep], d0[:, half][keep])
    if fmt == MX:   # the NVFP4 products take the scale code without a value as 480
        assert torch.isnan(d[rows]).all() and torch.isnan(d[:, cols]).all()
