"""Experts' operators where they can go wrong: row-scaled NVFP4 gathers at the widths of every kernel."""
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
