"""Experts' operators where they can go wrong: row-scaled NVFP4 gathers at the widths of every kernel, and MXFP8 blocks at the
bottom of the scales' range and of negative zeros."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.test_gpu_moe import DEV, gauss, order_of, rows_of

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
