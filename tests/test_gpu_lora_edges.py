"""Adapters where the kernels of many tokens can go wrong: every shape of their launches with K of several pieces, values
that are not finite and values at the ends of fp32's range among mixed adapters, and the gradient towards the tokens.

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


@pytest.mark.parametrize("M,r", [(100, 24), (300, 64), (4100, 64)])
def test_values_that_are_not_finite_among_many_tokens(M, r):
    """Tiles of 16 tokens with four adapters each: a value spoils its token, or its adapter's tokens, and no bit of another."""
    N, K, L = 72, 272, 4
    x, ad, a, b, s = case(M, N, K, r, L, none=0.1)
    ad[:5] = torch.tensor([0, 1, 2, 3, 1], dtype=torch.int32)
    y, w = gauss(M, N, seed=8), weights(N, K, 4)
    f = lambda: (bsq.lora_add(y, x, ad, a, b, s, out=torch.empty_like(y)).cpu(),   # noqa: E731
                 bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s).cpu())
    clean = f()
    assert all(torch.isfinite(t).all() for t in clean)
    for value in (float("nan"), float("inf"), -float("inf")):
        for m in (2, 31, M - 1):
            ad_m = int(ad[m])
            ad[m] = 2
            want = f()
            keep = x[m, 7].clone()
            x[m, 7] = value   # a token
            for got, ref in zip(f(), want):
                assert not torch.isfinite(got[m]).any()
                got[m] = ref[m]
                assert torch.equal(got, ref)
            x[m, 7] = keep
            ad[m] = ad_m
        mine = (ad == 1).cpu().nonzero().reshape(-1)
        for t, at, cols in ((a, (1, 5, K - 1), slice(None)), (b, (1, 11, r - 1), 11)):   # a value of adapter 1
            keep = t[at].clone()
            t[at] = value
            for got, want in zip(f(), clean):
                assert not torch.isfinite(got[mine][:, cols]).any()
                got[mine, cols] = want[mine, cols]
                assert torch.equal(got, want)
            t[at] = keep
    s[3] = float("nan")
    for got, want in zip(f(), clean):
        mine = (ad == 3).cpu()
        assert torch.isnan(got[mine]).all() and torch.equal(got[~mine], want[~mine])


@pytest.mark.parametrize("M", [40, 100, 300])
def test_large_and_small_down_products_side_by_side(M):
    """Down products of up to 2^127, whose bf16 rounding would be infinite, beside some of 2^-97 and of 2^-115 in the same tiles.
    Parts of a down product below 2^-133, bf16's smallest value, are cut off: r 2^-133 |b| a column more."""
    N, K, r, L = 64, 64, 8, 3
    x, a, b = gauss(M, K, seed=1), gauss(L, r, K, seed=2), gauss(L, N, r, seed=3)
    ad = (torch.arange(M) * 7 % 5 % 4).to(torch.int32).to(DEV)   # 3: none
    for i, (ex, ea, eb) in enumerate(((2.0 ** 60, 2.0 ** 62, 2.0 ** -100), (2.0 ** -50, 2.0 ** -50, 2.0 ** 90),
                                      (2.0 ** -59, 2.0 ** -59, 2.0 ** 100))):
        x[ad == i] *= ex
        a[i] *= ea
        b[i] *= eb
    v, e = lora64(x, ad, a, b, None)
    id_, on = ad.cpu().long(), (ad < 3).cpu()
    cut = torch.zeros(M, N, dtype=torch.float64)
    cut[on] = 2.0 ** -133 * b.cpu().double().abs().sum(2)[id_[on]]
    y = torch.zeros((M, N), device=DEV)
    got = bsq.lora_add(y, x, ad, a, b, out=torch.empty_like(y))
    assert_within(got, v, e + cut + v.abs() * 2 * F32, "out")
    assert (v[on].abs().amax(1) > 0).all() and float((x[ad == 0].cpu().double() @ a[0].cpu().double().t()).abs().max()) > 2.0 ** 126


def towards_tokens(dy, ad, a, b, s):
    """The gradient of lora_add with respect to x, fp32: lora_add with A^T and B^T in each other's place, K and N as well; N is
    then along the products, so dy and B get columns of zeros up to a multiple of 8."""
    N = dy.shape[1]
    pad = -N % 8
    dy = torch.nn.functional.pad(dy, (0, pad))
    bt = torch.nn.functional.pad(b.transpose(1, 2), (0, pad)).contiguous()
    dx = torch.zeros((dy.shape[0], a.shape[2]), device=DEV)
    return bsq.lora_add(dx, dy, ad, bt, a.transpose(1, 2).contiguous(), s)


@pytest.mark.parametrize("M,N,K,r,L", [(1, 64, 64, 8, 2), (5, 100, 136, 16, 3), (40, 257, 72, 24, 4), (100, 130, 520, 64, 5),
                                       (300, 64, 200, 40, 3)])
def test_gradient_towards_the_tokens(M, N, K, r, L):
    note("lora gradient %d %d %d %d %d" % (M, N, K, r, L))
    x, ad, a, b, s = case(M, N, K, r, L, seed=M + N)
    dy = gauss(M, N, seed=5)
    dx = towards_tokens(dy, ad, a, b, s).cpu().double()
    want, e = lora64(dy, ad, b.transpose(1, 2), a.transpose(1, 2), s)   # (dy B) A
    assert_within(dx, want, e + want.abs() * F32, "dx")
    # <f(x1) - f(x2), dy> = <x1 - x2, dx>, f being linear in x: exact but for f's errors on either side, each weighted
    # by |dy|, and dx's, weighted by |x1 - x2|.  f starts from zeros, in fp32: one rounding more of the output.
    x1, x2 = (x + gauss(M, K, seed=6)), (x - gauss(M, K, seed=7))
    zeros = torch.zeros((M, N), device=DEV)
    f = lambda t: bsq.lora_add(zeros, t, ad, a, b, s, out=torch.empty_like(zeros)).cpu().double()   # noqa: E731
    (v1, e1), (v2, e2) = (lora64(t, ad, a, b, s) for t in (x1, x2))
    step, d = x1.cpu().double() - x2.cpu().double(), dy.cpu().double()
    tol = ((e1 + e2 + (v1.abs() + v2.abs()) * F32) * d.abs()).sum() + (step.abs() * (e + want.abs() * F32)).sum()
    assert abs(float(((f(x1) - f(x2)) * d).sum() - (step * dx).sum())) <= float(tol) * (1 + 2.0 ** -20)


def test_the_gradient_needs_whole_pieces_of_the_columns():
    x, ad, a, b, s = case(4, 100, 64, 16, 2)
    dx, dy = torch.zeros((4, 64), device=DEV), gauss(4, 100, seed=1)
    with pytest.raises(bsq.BsqError):   # 100 columns are not a multiple of 8
        bsq.lora_add(dx, dy, ad, b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous(), s)
    assert not dx.any()
