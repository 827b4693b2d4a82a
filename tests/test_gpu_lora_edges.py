"""Adapters where the kernels of many tokens can go wrong: every shape of their launches with K of several pieces.

Tolerances as in test_gpu_lora."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.plain64 import F32, assert_within, nvfp4_values, product, store_error, sum_error
from tests.test_gpu_feed_forward_edges import guarded
from tests.test_gpu_lora import DEV, case, gauss, lora64
from tests.test_gpu_matvec import weights

pytestmark = pytest.mark.gpu

# 64, 32 and 16 ranks a workgroup, alone with their tokens (which then pass the caches by) and one of several; whole blocks of 64
# columns for each number of 32-rank steps, one and two of them a workgroup; K that ends inside a piece, and enough
# pieces that every wave has more of them than it holds at once
SHAPES = [(4100, 704, 1544, 64, 9, True), (4100, 64, 520, 64, 3, False), (4100, 704, 4168, 32, 4, False),
          (4100, 192, 2120, 16, 8, True), (600, 320, 712, 256, 5, True), (150, 128, 712, 128, 4, False),
          (2100, 576, 456, 256, 3, False), (1000, 640, 840, 64, 7, True), (70, 64, 8264, 16, 70, False)]


@pytest.mark.parametrize("M,N,K,r,L,runs", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_add_in_every_shape_of_the_launch(M, N, K, r, L, runs, dtype):
    note("lora add %d %d %d %d %d runs=%s %s" % (M, N, K, r, L, runs, dtype))
    x, ad, a, b, s = case(M, N, K, r, L, seed=M + K, runs=runs)
    y = gauss(M, N, seed=9, dtype=dtype)
    v, e = lora64(x, ad, a, b, s)
    want = y.cpu().double() + v
    (o,), intact = guarded([(M, N)], dtype)
    got = bsq.lora_add(y, x, ad, a, b, s, out=o)
    intact()
    assert_within(got, want, e + want.abs() * F32 + store_error(want, dtype), "out")
    none = ((ad < 0) | (ad >= L)).cpu()
    assert none.any() and torch.equal(got.cpu()[none], y.cpu()[none])
    o.copy_(y)
    bsq.lora_add(o, x, ad, a, b, s)
    intact()
    assert torch.equal(o, got)


@pytest.mark.parametrize("M,N,K,r,L", [(100, 128, 272, 24, 3), (100, 192, 1040, 64, 5), (90, 128, 272, 128, 4), (130, 64, 528, 256, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matvec_in_whole_blocks_of_columns(M, N, K, r, L, dtype):
    note("nvfp4 lora matvec %d %d %d %d %d %s" % (M, N, K, r, L, dtype))
    x, ad, a, b, s = case(M, N, K, r, L, seed=M)
    w = weights(N, K, 4)
    base, S = product(x.cpu().double(), nvfp4_values(*w))
    v, e = lora64(x, ad, a, b, s)
    (o,), intact = guarded([(M, N)], dtype)
    got = bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s, out_dtype=dtype, out=o)
    intact()
    want = base + v
    assert_within(got, want, sum_error(K, S) + e + want.abs() * F32 + store_error(want, dtype), "y")
