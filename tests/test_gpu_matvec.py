"""nvfp4_matvec and nvfp4_gated_matvec against a plain binary64 form of the decoded weights.

Tolerance: every product of a bf16 token and an exactly decoded weight is exact in fp32, so the sum is
off by at most (K + 2) 2^-24 S with S = sum |x w| (any order; two more roundings for the division), and
the output by half a step of its type."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.plain64 import (act64, assert_within, gated_error, nvfp4_values, product, store_error, sum_error)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def tokens(M, K, seed, ld=None, std=1.0):
    g = torch.Generator().manual_seed(seed)
    buf = torch.zeros((M, ld or K), dtype=torch.bfloat16)
    buf[:, :K] = (torch.randn((M, K), generator=g) * std).to(torch.bfloat16)
    if ld:
        buf[:, K:] = float("nan")   # what lies between tokens is not read into any sum
    return buf.to(DEV)[:, :K]


def weights(N, K, seed, rows=False):
    """Any code and any finite scale byte (subnormal and negative ones among them)."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0, 255, (N, K // 16), generator=g, dtype=torch.uint8)
    scales[scales == 127] = 126
    s = torch.rand(N if rows else 1, generator=g) * 900 + 100
    return codes.to(DEV), scales.to(DEV), s.to(DEV)


def check(M, N, K, rows=False, out_dtype=torch.bfloat16, ld=None, seed=1):
    note("matvec %d %d %d rows=%s %s ld=%s" % (M, N, K, rows, out_dtype, ld))
    x, w = tokens(M, K, seed, ld), weights(N, K, seed + 1, rows)
    y = bsq.nvfp4_matvec(x, *w, out_dtype=out_dtype)
    torch.cuda.synchronize()
    want, S = product(x.cpu().double(), nvfp4_values(*w))
    assert_within(y, want, sum_error(K, S) + store_error(want, out_dtype), "y")


SIZES = [(1, 1, 16), (1, 16, 128), (1, 17, 48), (2, 33, 144), (3, 256, 256), (1, 300, 4112), (15, 31, 1040),
         (16, 64, 2048), (17, 64, 528), (33, 47, 2064), (64, 128, 1024), (65, 20, 272), (100, 1030, 640),
         (1, 2048, 14336)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("rows", [False, True])
def test_sizes(M, N, K, rows):
    check(M, N, K, rows)
    check(M, N, K, rows, torch.float32)


def test_strided_tokens():
    check(5, 100, 272, ld=280)
    check(40, 64, 1024, ld=2048, out_dtype=torch.float32)


def check_gated(act, M, F, K, rows=False, ld=None, seed=3):
    note("gated matvec act=%d %d %d %d rows=%s" % (act, M, F, K, rows))
    x, wg, wu = tokens(M, K, seed, ld), weights(F, K, seed + 1, rows), weights(F, K, seed + 2, rows)
    # bring gate values to the curved part of the activation
    sg = wg[2] * float((x.float().norm() / M ** 0.5).item()) * 150 / 900
    h = bsq.nvfp4_gated_matvec(act, x, wg[0], wg[1], sg, *wu)
    torch.cuda.synchronize()
    g, Sg = product(x.cpu().double(), nvfp4_values(wg[0], wg[1], sg))
    u, Su = product(x.cpu().double(), nvfp4_values(*wu))
    want = act64(g, act)[0] * u
    e = gated_error(g, u, sum_error(K, Sg), sum_error(K, Su), act)
    assert_within(h, want, e * (1 + 2.0 ** -8) + store_error(want, torch.bfloat16), "h")


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("M,F,K", [(1, 16, 64), (1, 1033, 2064), (5, 40, 4096), (16, 129, 272), (48, 70, 1040)])
def test_gated(act, M, F, K):
    check_gated(act, M, F, K)


def test_gated_rows_and_strides():
    check_gated(0, 3, 65, 528, rows=True)
    check_gated(2, 20, 33, 160, rows=True, ld=176)


def test_empty_and_k0():
    w = weights(32, 64, 5)
    y = bsq.nvfp4_matvec(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), *w)
    assert tuple(y.shape) == (0, 32)
    e = [t.to(DEV) for t in (torch.empty((8, 0), dtype=torch.uint8), torch.empty((8, 0), dtype=torch.uint8),
                             torch.ones(1))]
    out = torch.full((3, 8), 7.0, dtype=torch.bfloat16, device=DEV)
    x0 = torch.empty((3, 0), dtype=torch.bfloat16, device=DEV)
    assert not bsq.nvfp4_matvec(x0, *e, out=out).any()
    out.fill_(7.0)
    assert not bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x0, *e, *e, out=out).any()


def test_nan_and_infinity_stay_in_their_token_and_row():
    M, N, K = 6, 40, 272
    x, (c, s, se) = tokens(M, K, 9).clone(), weights(N, K, 10)
    x[2, K - 1] = float("nan")
    x[4, 0] = float("inf")
    s[7, K // 16 - 1] = 0x7F   # NaN scale in one row, in the block that ends K
    y = bsq.nvfp4_matvec(x, c, s, se).cpu()
    bad = torch.isnan(y) | torch.isinf(y)
    want = torch.zeros_like(bad)
    want[2, :] = want[4, :] = True
    want[:, 7] = True
    assert torch.equal(bad | want, want), "a value outside the NaN's token and row is not finite"
    assert torch.isnan(y[2]).all() and torch.isnan(y[:, 7]).all() and not torch.isfinite(y[4]).any()
    clean = bsq.nvfp4_matvec(tokens(M, K, 9), *weights(N, K, 10)).cpu()
    keep = ~want
    assert torch.equal(y[keep], clean[keep]), "the other outputs changed"


def test_same_bits_out_buffer_and_stream():
    x, w = tokens(4, 4096, 20), weights(512, 4096, 21)
    y = bsq.nvfp4_matvec(x, *w)
    out = torch.empty_like(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert bsq.nvfp4_matvec(x, *w, out=out) is out
    side.synchronize()
    assert torch.equal(out, y)


def test_graph_replays():
    x, w, wu = tokens(1, 1024, 30), weights(256, 1024, 31), weights(256, 1024, 32)
    y = torch.empty((1, 256), dtype=torch.bfloat16, device=DEV)
    h = torch.empty_like(y)
    bsq.nvfp4_matvec(x, *w, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsq.nvfp4_matvec(x, *w, out=y)
        bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, *w, *wu, out=h)
    for seed in (41, 42, 43):
        x.copy_(tokens(1, 1024, seed))
        want = (bsq.nvfp4_matvec(x, *w), bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, *w, *wu))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


def test_python_refusals():
    x, (c, s, se) = tokens(2, 64, 50), weights(8, 64, 51)
    for bad, exc in [((x.float(), c, s, se), TypeError), ((x[:, :32], c, s, se), ValueError),
                     ((x, c, s[:, :2].contiguous(), se), ValueError), ((x, c, s, torch.ones(3, device=DEV)), ValueError),
                     ((x, c.int(), s, se), TypeError), ((x.cpu(), c, s, se), TypeError),
                     ((torch.empty((64, 2), dtype=torch.bfloat16, device=DEV).t(), c, s, se), ValueError),
                     ((x.flatten(), c, s, se), ValueError)]:
        with pytest.raises(exc):
            bsq.nvfp4_matvec(*bad)
    with pytest.raises(bsq.BsqError):
        bsq.nvfp4_gated_matvec(3, x, c, s, se, c, s, se)
    with pytest.raises(bsq.BsqError):   # a token pitch that is no multiple of 8
        bsq.nvfp4_matvec(torch.empty((2, 67), dtype=torch.bfloat16, device=DEV)[:, :64], c, s, se)
    with pytest.raises(ValueError):
        bsq.nvfp4_matvec(x, c, s, se, out=torch.empty((2, 9), dtype=torch.bfloat16, device=DEV))


# the tile of tokens changes with their number and with the rows; K of one block, of a part of a chunk, of many
# chunks; every way that a row's last 64 elements lie
@pytest.mark.parametrize("M,N,K", [(1, 40, 32), (70, 33, 48), (2, 40, 80), (4, 100, 8208), (1, 33, 16400), (1, 4099, 1136),
                                   (5, 2000, 4128), (16, 70, 8272), (20, 7000, 336), (33, 3100, 1104), (64, 3300, 2128),
                                   (64, 500, 4096), (130, 3100, 528), (3, 9000, 512)])
def test_every_shape_of_a_launch(M, N, K):
    check(M, N, K, True, torch.float32, seed=60)
    check_gated(1, M, (N + 1) // 2, K, seed=61)


def test_tokens_far_apart():
    big = torch.zeros((3, 70, 272), dtype=torch.bfloat16, device=DEV)
    big[:, -1] = torch.randn((3, 272), generator=torch.Generator().manual_seed(71)).to(torch.bfloat16).to(DEV)
    w = weights(48, 272, 72)
    assert torch.equal(bsq.nvfp4_matvec(big[:, -1], *w), bsq.nvfp4_matvec(big[:, -1].contiguous(), *w))


def test_one_token_gives_what_a_token_of_several_gives_within_rounding():
    x, w = tokens(8, 1024, 73), weights(300, 1024, 74)
    many = bsq.nvfp4_matvec(x, *w, out_dtype=torch.float32).cpu().double()
    want, S = product(x.cpu().double(), nvfp4_values(*w))
    for m in range(8):
        one = bsq.nvfp4_matvec(x[m:m + 1], *w, out_dtype=torch.float32).cpu().double()
        assert_within(one, want[m:m + 1], sum_error(1024, S[m:m + 1]) + store_error(want[m:m + 1], torch.float32), "one")
        assert float((one - many[m:m + 1]).abs().max() / S[m].max()) < 2 * (1024 + 3) * 2.0 ** -24


@pytest.mark.parametrize("M", [1, 3])
def test_weights_past_2_to_the_32_bytes(M):
    N, K = 530000, 16400   # 4.3 GB of codes, rows of neither 16 nor 64 bytes
    g = torch.Generator(device=DEV).manual_seed(80)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    scales = torch.randint(0, 127, (N, K // 16), generator=g, dtype=torch.uint8, device=DEV)
    s = torch.rand(N, generator=g, device=DEV) * 900 + 100
    x = tokens(M, K, 81)
    y = bsq.nvfp4_matvec(x, codes, scales, s, out_dtype=torch.float32)
    rows = torch.tensor([0, 15, 16, 261870, 261888, 523760, 523776, N - 17, N - 1], device=DEV)
    want, S = product(x.cpu().double(), nvfp4_values(codes[rows], scales[rows], s[rows]))
    assert_within(y[:, rows], want, sum_error(K, S) + store_error(want, torch.float32), "y")


# values whose products with the codes alone leave fp32's range, while the weights (codes times scales) keep them in it
@pytest.mark.parametrize("M", [1, 3])
@pytest.mark.parametrize("N,K", [(40, 48), (33, 256), (70, 528)])
def test_largest_tokens_times_small_scales(M, N, K):
    g = torch.Generator().manual_seed(90)
    x = (torch.randn((M, K), generator=g).clamp(-3, 3) * 2.0 ** 126).to(torch.bfloat16).to(DEV)   # |x| < 2^128
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).to(DEV)
    scales = torch.randint(1, 3, (N, K // 16), generator=g, dtype=torch.uint8).to(DEV)   # 2^-9 and 2^-8
    w = (codes, scales, torch.full((1,), 2.0 ** 10, device=DEV))
    want, S = product(x.cpu().double(), nvfp4_values(*w))
    assert float(S.max()) * 2.0 ** 10 < 2.0 ** 128   # no partial sum of the products leaves the range
    for dt in (torch.float32, torch.bfloat16):
        y = bsq.nvfp4_matvec(x, *w, out_dtype=dt)
        assert_within(y, want, sum_error(K, S) + store_error(want, dt), "y")
    s = torch.full((1,), 2.0 ** 115, device=DEV)
    gate, up = product(x.cpu().double(), nvfp4_values(codes, scales, s)), product(x.cpu().double(), nvfp4_values(codes, scales, s))
    h = bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, codes, scales, s, codes, scales, s)
    want = act64(gate[0], 0)[0] * up[0]
    e = gated_error(gate[0], up[0], sum_error(K, gate[1]), sum_error(K, up[1]), 0)
    assert_within(h, want, e * (1 + 2.0 ** -8) + store_error(want, torch.bfloat16), "h")
