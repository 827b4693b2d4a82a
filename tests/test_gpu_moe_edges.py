"""Experts' operators where they can go wrong: row-scaled NVFP4 gathers at the widths of every kernel, MXFP8 blocks at the bottom
of the scales' range and of negative zeros, and outputs of all operators in guarded buffers through the C entry points."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.test_gpu_moe import DEV, gauss, ids, order_of, rows_of

pytestmark = pytest.mark.gpu


# a wave a token up to 2048 and up to 4096 wide, a workgroup a token above; tokens that end inside a workgroup
@pytest.mark.parametrize("T", [2051, 2048, 2047])
@pytest.mark.parametrize("H", [1040, 2048, 2064, 4096, 4112])
def test_nvfp4_gathers_of_many_wide_tokens(T, H):
    note("gather nvfp4 %d %d" % (T, H))
    p, s = order_of(T, 3, 7, 32, T + H)
    x = gauss(T, H, seed=H)
    x[3] = 0
    x[5, H // 2:] = 0
    x[7] *= 2.0 ** -100
    x[9, -16:] *= 2.0 ** 30   # the largest magnitude in the last block
    x[T - 1, :16] = -3.0e38
    xd = x.to(DEV)
    got = bsq.moe_gather(xd, p, s)
    assert torch.equal(got.cpu(), rows_of(x, s, 3))
    q, ref = bsq.moe_gather_nvfp4_rowscaled(xd, p, s), bsq.nvfp4_quantize_rowscaled(got)
    for n in ("codes", "scales", "s_enc"):
        assert torch.equal(q[n], ref[n]), n


@pytest.mark.parametrize("T", [0, 3, 3000])
def test_nvfp4_gathers_of_width_zero(T):
    """Rows without elements have a scale all the same, the cast's, by which a product along them divides."""
    note("gather nvfp4 width 0, %d tokens" % T)
    p, s = order_of(T, 2, 4, 32, 5) if T else order_of(0, 2, 4, 1, 5)
    if T == 0:
        s = torch.full((5,), -1, dtype=torch.int32, device=DEV)   # rows of padding only
    x, R = torch.zeros((T, 0), dtype=torch.bfloat16, device=DEV), s.numel()
    ref = bsq.nvfp4_quantize_rowscaled(bsq.moe_gather(x, p, s))
    assert (ref["s_enc"] == 1).all()
    s_enc, intact = guard((R,), torch.float32)
    s_enc.fill_(float("nan"))
    call("moe_gather_nvfp4_rowscaled", T, 2, 0, None, 0, p, s, R, None, None, s_enc)
    intact()
    assert torch.equal(s_enc, ref["s_enc"])
    q = bsq.moe_gather_nvfp4_rowscaled(x, p, s)
    assert all(torch.equal(q[n], ref[n]) for n in ("codes", "scales", "s_enc"))
    b = bsq.nvfp4_quantize(torch.zeros((16, 0), dtype=torch.bfloat16, device=DEV))
    y = bsq.blockscaled_gemm(bsq.FMT_NVFP4 | bsq.FMT_A_ROWSCALED, q["codes"], q["scales"], q["s_enc"], b["row_codes"],
                             b["row_scales"], b["s_enc"][:1])
    assert y.shape == (R, 16) and not y.any()


def tiny_blocks(T, H, seed):
    """Ordinary blocks of 32, and among them blocks of 2^-112 (the least scale byte above 0 is that of 2^-118) down to bf16's
    smallest subnormals, blocks of negative zeros, of zeros of both signs, and of one value among negative zeros."""
    g = torch.Generator().manual_seed(seed)
    x = gauss(T, H, seed=seed).double().reshape(T, H // 32, 32)
    kind = torch.randint(0, 8, (T, H // 32), generator=g)
    kind[0], kind[1] = 0, 1   # a token of ordinary blocks only, one of tiny ones only
    scale = torch.pow(2.0, -torch.randint(112, 134, (T, H // 32), generator=g).double())
    scale[1] = 2.0 ** -125
    x = torch.where((kind == 1).unsqueeze(2), x * scale.unsqueeze(2), x)
    lone = torch.full_like(x, -0.0)
    lone[..., 13] = scale * 1.5
    signs = torch.where(torch.rand(x.shape, generator=g) < 0.5, 0.0, -0.0).double()
    for k, v in ((2, torch.full_like(x, -0.0)), (3, lone), (4, signs), (5, torch.where(signs == 0, x, signs))):
        x = torch.where((kind == k).unsqueeze(2), v, x)
    x[kind == 6, ::3] = -0.0   # negative zeros in ordinary blocks
    return x.reshape(T, H).float().to(torch.bfloat16)


@pytest.mark.parametrize("T,k,E,H", [(6, 2, 4, 32), (40, 2, 8, 288), (65, 3, 5, 4128), (3000, 2, 8, 512)])
def test_mxfp8_gathers_of_tiny_blocks(T, k, E, H):
    note("gather mxfp8 tiny %d %d %d %d" % (T, k, E, H))
    import oracle
    p, s = order_of(T, k, E, 32, T, drop=0.0)
    x = tiny_blocks(T, H, T)
    got = bsq.moe_gather(x.to(DEV), p, s)
    assert torch.equal(got.cpu().view(torch.int16), rows_of(x.view(torch.int16), s, k))
    q, ref = bsq.moe_gather_mxfp8(x.to(DEV), p, s), bsq.mxfp8_quantize(got)
    assert (q["row_scales"] == 0).any() and (q["row_codes"][(q["row_scales"] == 0).repeat_interleave(32, 1)] & 127).any()
    for n in ("row_codes", "row_scales"):
        assert torch.equal(q[n], ref[n]), n
    want = oracle.mxfp8_quantize(got.cpu()[:400], direction=oracle.ROW)
    for n in ("row_codes", "row_scales"):
        assert np.array_equal(q[n].cpu().numpy()[:400], want[n]), n


def guard(shape, dtype):
    """A 16-byte aligned tensor inside a marked buffer, and a check that nothing around it changed."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    pad = max(4096, 272 * int(shape[-1]) * 4) // 16 * 16
    buf = torch.full((pad + n + pad,), 0xA5, dtype=torch.uint8, device=DEV)

    def intact():
        assert (buf[:pad] == 0xA5).all(), "written before an output"
        assert (buf[pad + n:] == 0xA5).all(), "written after an output"
    return buf[pad:pad + n].view(dtype).view(shape), intact


def call(fn, *args):
    at = [t.data_ptr() if isinstance(t, torch.Tensor) else t for t in args]
    assert getattr(bsq.lib(), fn)(*at, torch.cuda.current_stream().cuda_stream) == 0, bsq.lib().bsq_last_error()


# rows that end inside a wave's or a lane's part, few and many tokens, each kernel of the gathers, rows without a slot at the end
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 32), (3, 2, 4, 96), (37, 3, 8, 1056), (100, 2, 5, 4128), (2050, 2, 6, 608), (2050, 2, 6, 2080),
                                     (9, 4, 8, 8224)])
def test_nothing_is_written_outside_the_outputs(T, k, E, H):
    note("guarded routed outputs %d %d %d %d" % (T, k, E, H))
    e = ids(T, k, E, T, drop=0.1).to(DEV)
    n, L = T * k, bsq.lib()
    R = L.moe_sort_rows(n, E, 16)
    ws = torch.empty(max(L.moe_sort_workspace_bytes(n, E), 16), dtype=torch.uint8, device=DEV)
    (offs, a), (p, b), (s, c) = guard((E + 1,), torch.int64), guard((T, k), torch.int32), guard((R,), torch.int32)
    call("moe_sort", e, 8, n, E, 16, R, offs, p, s, ws)
    checks, want = [a, b, c], bsq.moe_sort(e, E, 16)
    assert torch.equal(offs, want["offsets"]) and torch.equal(p, want["positions"]) and torch.equal(s, want["source"])
    x, w = gauss(T, H, seed=1).to(DEV), gauss(T, k, seed=2, dtype=torch.float32).to(DEV)
    (codes, a), (scales, b), (s_enc, c) = guard((R, H // 2), torch.uint8), guard((R, H // 16), torch.uint8), guard((R,), torch.float32)
    call("moe_gather_nvfp4_rowscaled", T, k, H, x, H, p, s, R, codes, scales, s_enc)
    checks += [a, b, c]
    q = bsq.moe_gather_nvfp4_rowscaled(x, p, s)
    assert torch.equal(codes, q["codes"]) and torch.equal(scales, q["scales"]) and torch.equal(s_enc, q["s_enc"])
    (codes, a), (scales, b) = guard((R, H), torch.uint8), guard((R, H // 32), torch.uint8)
    call("moe_gather_mxfp8", T, k, H, x, H, p, s, R, codes, scales)
    checks += [a, b]
    q = bsq.moe_gather_mxfp8(x, p, s)
    assert torch.equal(codes, q["row_codes"]) and torch.equal(scales, q["row_scales"])
    for code, dtype in ((bsq.OUT_BF16, torch.bfloat16), (bsq.OUT_F32, torch.float32)):
        y = gauss(R, H, seed=3, dtype=dtype).to(DEV)
        (dy, a), (dw, b) = guard((R, H), dtype), guard((T, k), torch.float32)
        call("moe_combine_backward", T, k, H, x, y, code, R, p, s, w, dy, dw)
        checks += [a, b]
        want_dy, want_dw = bsq.moe_combine_backward(x, y, p, s, w)
        assert torch.equal(dy, want_dy) and torch.equal(dw, want_dw)
    for intact in checks:
        intact()


def test_large_outputs_stay_inside_their_buffers():
    """Outputs that are stored past the caches."""
    T, k, E, H = 33003, 2, 5, 2048
    p, s = order_of(T, k, E, 32, 1)
    x, w = gauss(T, H, seed=1).to(DEV), gauss(T, k, seed=2, dtype=torch.float32).to(DEV)
    R = s.numel()
    for code, dtype in ((bsq.OUT_BF16, torch.bfloat16), (bsq.OUT_F32, torch.float32)):
        y = bsq.moe_gather(x, p, s).to(dtype)
        (dy, a), (dw, b) = guard((R, H), dtype), guard((T, k), torch.float32)
        call("moe_combine_backward", T, k, H, x, y, code, R, p, s, w, dy, dw)
        a()
        b()
        want_dy, want_dw = bsq.moe_combine_backward(x, y, p, s, w)
        assert torch.equal(dy, want_dy) and torch.equal(dw, want_dw)
