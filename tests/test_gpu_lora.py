"""Low-rank adapters of many requests, beside a given output and beside NVFP4 weights, against a binary64 form.

Tolerance: products of bf16 values are exact, so a down product is off by (K + 2) 2^-24 sum |x a|; it enters the up
product exactly (three bf16 parts, or fp32), whose 3 rank terms add up with (3 rank + 2) 2^-24 sum |t b|, besides the down
products' own errors times |b|; one rounding of the sum with y, and half a step of the output's type."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.plain64 import F32, assert_within, nvfp4_values, product, store_error, sum_error
from tests.test_gpu_feed_forward_edges import guarded
from tests.test_gpu_matvec import weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gauss(*shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def adapters(M, L, seed, none=0.2, runs=False):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(0, max(L, 1), (M,), generator=g)
    if runs:
        a = a.sort().values
    out = torch.rand(M, generator=g) < none
    wrong = torch.tensor([-1, L, -(1 << 31), (1 << 31) - 1])[torch.randint(0, 4, (M,), generator=g)]
    return torch.where(out, wrong, a).to(torch.int32).to(DEV)


def lora64(x, ad, a, b, s):
    """(sum, its error before y is added) of the adapters' part, in binary64."""
    M, K = x.shape
    L, r, N = a.shape[0], a.shape[1], b.shape[1]
    x, ad = x.cpu().double(), ad.cpu().long()
    v, e = torch.zeros((M, N), dtype=torch.float64), torch.zeros((M, N), dtype=torch.float64)
    for i in range(L):
        at = (ad == i).nonzero().reshape(-1)
        if at.numel():
            A, B = a[i].cpu().double(), b[i].cpu().double()
            sc = 1.0 if s is None else float(s[i])
            t, S = product(x[at], A)
            v[at] = t @ B.t() * sc
            e[at] = ((K + 2) * F32 * S @ B.abs().t() + (3 * r + 2) * F32 * (t.abs() @ B.abs().t())) * abs(sc)
    return v, e


def case(M, N, K, r, L, seed=1, runs=False, none=0.2):
    return (gauss(M, K, seed=seed), adapters(M, L, seed + 1, none, runs), gauss(L, r, K, seed=seed + 2, std=max(K, 1) ** -0.5),
            gauss(L, N, r, seed=seed + 3, std=r ** -0.5), torch.rand(L, generator=torch.Generator().manual_seed(seed)).to(DEV) + 0.5)


SIZES = [(1, 1, 8, 8, 1), (1, 17, 64, 8, 2), (3, 33, 72, 24, 4), (16, 64, 512, 16, 16), (17, 100, 1040, 16, 3), (40, 257, 136, 64, 5),
         (100, 300, 264, 128, 7), (5, 64, 16, 256, 2), (64, 1000, 2064, 40, 40), (300, 130, 520, 64, 8), (33, 72, 4096, 72, 2),
         (2, 16, 0, 8, 1), (4, 24, 64, 16, 0), (1, 4100, 4104, 16, 3), (520, 24, 64, 8, 600)]


@pytest.mark.parametrize("M,N,K,r,L", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_add(M, N, K, r, L, dtype):
    note("lora add %d %d %d %d %d %s" % (M, N, K, r, L, dtype))
    for runs in (False, True):
        x, ad, a, b, s = case(M, N, K, r, L, seed=M + N, runs=runs)
        y = gauss(M, N, seed=9, dtype=dtype)
        for scales in (s, None):
            v, e = lora64(x, ad, a, b, scales)
            want = y.cpu().double() + v
            tol = e + want.abs() * F32 + store_error(want, dtype)
            (o,), intact = guarded([(M, N)], dtype)
            before = y.clone()
            got = bsq.lora_add(y, x, ad, a, b, scales, out=o)
            intact()
            assert torch.equal(y, before)
            assert_within(got, want, tol, "out")
            none = ((ad < 0) | (ad >= L)).cpu()
            assert torch.equal(got.cpu()[none], y.cpu()[none])
            o.copy_(y)
            assert bsq.lora_add(o, x, ad, a, b, scales) is o   # in place
            intact()
            assert torch.equal(o, got)


def test_add_to_slices_of_a_wider_output():
    M, K, r, L = 21, 264, 16, 3
    wide = gauss(M, 400, seed=1)
    x = gauss(M, 2 * K, seed=2)[:, K:]
    for n0, N in ((0, 128), (128, 64), (192, 201), (393, 7), (3, 50)):
        _, ad, a, b, s = case(M, N, K, r, L, seed=n0 + 3)
        y = wide.clone()
        bsq.lora_add(y[:, n0:n0 + N], x, ad, a, b, s)
        v, e = lora64(x, ad, a, b, s)
        want = wide.cpu().double()
        want[:, n0:n0 + N] += v
        tol = torch.zeros_like(want)
        tol[:, n0:n0 + N] = e + want[:, n0:n0 + N].abs() * F32 + store_error(want[:, n0:n0 + N], torch.bfloat16)
        assert_within(y, want, tol, "slice")
        other = torch.zeros((M, 512), dtype=torch.bfloat16, device=DEV)
        bsq.lora_add(wide[:, n0:n0 + N], x, ad, a, b, s, out=other[:, 5:5 + N])
        assert torch.equal(other[:, 5:5 + N], y[:, n0:n0 + N]) and (other[:, 5 + N:] == 0).all() and (other[:, :5] == 0).all()


MATVECS = [(1, 1, 16, 8, 1), (1, 64, 256, 16, 1), (1, 1000, 4096, 64, 4), (2, 33, 48, 8, 3), (4, 100, 272, 24, 2), (5, 1033, 2064, 8, 4),
           (16, 256, 512, 16, 16), (17, 300, 1040, 32, 5), (33, 47, 4096, 128, 3), (64, 2048, 256, 16, 64), (70, 100, 528, 256, 2),
           (3, 16, 0, 8, 2), (130, 64, 64, 8, 7), (4, 40, 64, 8, 0)]


@pytest.mark.parametrize("M,N,K,r,L", MATVECS)
@pytest.mark.parametrize("rows", [False, True])
def test_matvec(M, N, K, r, L, rows):
    note("nvfp4 lora matvec %d %d %d %d %d rows=%s" % (M, N, K, r, L, rows))
    x, ad, a, b, s = case(M, N, K, r, L, seed=M + N)
    w = weights(N, K, 4, rows)
    base, S = product(x.cpu().double(), nvfp4_values(*w))
    for scales in (s, None):
        v, e = lora64(x, ad, a, b, scales)
        want = base + v
        for dtype in (torch.bfloat16, torch.float32):
            (o,), intact = guarded([(M, N)], dtype)
            got = bsq.nvfp4_lora_matvec(x, *w, ad, a, b, scales, out_dtype=dtype, out=o)
            intact()
            assert_within(got, want, sum_error(K, S) + e + want.abs() * F32 + store_error(want, dtype), "y")


@pytest.mark.parametrize("M", [1, 3, 16, 40, 100])
def test_without_adapters_it_is_the_matvec(M):
    N, K, r, L = 300, 1040, 16, 4
    x, _, a, b, s = case(M, N, K, r, L)
    ad, w = adapters(M, L, 3, none=1.0), weights(N, K, 4)
    a[:] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        assert torch.equal(bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s, out_dtype=dtype), bsq.nvfp4_matvec(x, *w, out_dtype=dtype))


@pytest.mark.parametrize("M", [5, 40])
def test_values_that_are_not_finite_stay_where_they_belong(M):
    N, K, r, L = 72, 272, 24, 4
    x, ad, a, b, s = case(M, N, K, r, L, none=0.0)
    ad[:4] = torch.arange(4, dtype=torch.int32)
    ad[4] = 1
    w, y = weights(N, K, 4), gauss(M, N, seed=8)
    f = lambda: (bsq.lora_add(y, x, ad, a, b, s, out=torch.empty_like(y)).cpu(),   # noqa: E731
                 bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s).cpu())
    clean = f()
    for value in (float("nan"), float("inf"), -float("inf")):
        keep = x[2, 7].clone()
        x[2, 7] = value   # a token
        for got, want in zip(f(), clean):
            assert not torch.isfinite(got[2]).any()
            got[2] = want[2]
            assert torch.equal(got, want)
        x[2, 7] = keep
        mine = (ad == 1).cpu()
        for t, at, cols in ((a, (1, 5, K - 1), slice(None)), (b, (1, 11, r - 1), 11)):   # a value of adapter 1
            keep = t[at].clone()
            t[at] = value
            for got, want in zip(f(), clean):
                assert not torch.isfinite(got[mine][:, cols]).any()
                got[mine.nonzero().reshape(-1), cols] = want[mine.nonzero().reshape(-1), cols]
                assert torch.equal(got, want)
            t[at] = keep
    s[3] = float("nan")
    for got, want in zip(f(), clean):
        mine = (ad == 3).cpu()
        assert torch.isnan(got[mine]).all() and torch.equal(got[~mine], want[~mine])


def test_large_and_small_down_products():
    """t of up to 2^126, whose bf16 rounding would be infinite, and of down to 2^-100."""
    M, N, K, r = 4, 32, 64, 8
    x, a, b = gauss(M, K, seed=1), gauss(1, r, K, seed=2), gauss(1, N, r, seed=3)
    ad = torch.zeros(M, dtype=torch.int32, device=DEV)
    y = torch.zeros((M, N), device=DEV)
    for ex, ea, eb in ((2.0 ** 60, 2.0 ** 62, 2.0 ** -100), (2.0 ** -50, 2.0 ** -50, 2.0 ** 90)):
        xs, as_, bs = x * ex, a * ea, b * eb
        v, e = lora64(xs, ad, as_, bs, None)
        got = bsq.lora_add(y, xs, ad, as_, bs, out=torch.empty_like(y))
        assert_within(got, v, e + v.abs() * 2 * F32, "out")


def test_refusals_of_the_binding():
    x, ad, a, b, s = case(4, 32, 64, 16, 2)
    y, w = gauss(4, 32, seed=3), weights(32, 64, 4)
    for bad in (lambda: bsq.lora_add(y[:3], x, ad, a, b), lambda: bsq.lora_add(y, x, ad[:3], a, b),
                lambda: bsq.lora_add(y, x, ad, a[:, :, :32], b), lambda: bsq.lora_add(y, x, ad, a, b[:1]),
                lambda: bsq.lora_add(y, x, ad, a, b, s[:1]), lambda: bsq.lora_add(y.t(), x, ad, a, b),
                lambda: bsq.lora_add(y, x, ad, a, b, out=y[:, :16]), lambda: bsq.nvfp4_lora_matvec(x, *w, ad, a, b[:, :16]),
                lambda: bsq.lora_add(y, x, ad, a, b, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bsq.lora_add(y.half(), x, ad, a, b), lambda: bsq.lora_add(y, x.float(), ad, a, b),
                lambda: bsq.lora_add(y, x, ad.long(), a, b), lambda: bsq.lora_add(y, x, ad, a.float(), b),
                lambda: bsq.lora_add(y, x, ad, a, b, out=y.float()), lambda: bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s.double())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(bsq.BsqError):   # rank 12
        bsq.lora_add(y, x, ad, gauss(2, 12, 64, seed=1), gauss(2, 32, 12, seed=1))


def test_captured_and_replayed():
    M, N, K, r, L = 24, 200, 272, 16, 5
    x, ad, a, b, s = case(M, N, K, r, L)
    y, w = gauss(M, N, seed=8), weights(N, K, 4)
    f = lambda: (bsq.lora_add(y, x, ad, a, b, s, out=torch.empty_like(y)), bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s))   # noqa: E731
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = f()
    for seed in (3, 4, 5):
        x.copy_(gauss(M, K, seed=seed))
        ad.copy_(adapters(M, L, seed))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, f()):
            assert torch.equal(got, want)


def test_two_streams_at_once():
    M, N, K, r, L = 600, 1024, 1024, 16, 4
    cases = [case(M, N, K, r, L, seed=s) for s in (1, 2)]
    y = gauss(M, N, seed=8)
    f = lambda c: bsq.lora_add(y, *c, out=torch.empty_like(y))   # noqa: E731
    want = [f(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(f(c))
        torch.cuda.synchronize()
        assert all(torch.equal(g, t) for g, t in zip(got, want))


def test_adapters_past_two_to_the_31_elements():
    M, N, K, r, L = 3, 4096, 4096, 256, 2200   # 2.3 G elements in each of a and b
    a = torch.zeros((L, r, K), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros((L, N, r), dtype=torch.bfloat16, device=DEV)
    x, y = gauss(M, K, seed=1), gauss(M, N, seed=2)
    a[L - 1], b[L - 1], a[0], b[0] = (gauss(*sh, seed=s, std=0.05) for s, sh in ((3, (r, K)), (4, (N, r)), (5, (r, K)), (6, (N, r))))
    ad = torch.tensor([L - 1, 0, L - 2], dtype=torch.int32, device=DEV)
    few = torch.tensor([1, 0, -1], dtype=torch.int32, device=DEV)
    small_a, small_b = torch.stack([a[0], a[L - 1]]), torch.stack([b[0], b[L - 1]])
    got = bsq.lora_add(y, x, ad, a, b, out=torch.empty_like(y))
    assert torch.equal(got, bsq.lora_add(y, x, few, small_a, small_b, out=torch.empty_like(y)))
    w = weights(N, K, 4)
    got = bsq.nvfp4_lora_matvec(x, *w, ad, a, b)
    assert torch.equal(got, bsq.nvfp4_lora_matvec(x, *w, few, small_a, small_b))


def test_tokens_are_used_once_each_in_matching_ways():
    """A token's result does not depend on its neighbours: any order of tokens gives each the same bits."""
    M, N, K, r, L = 50, 130, 264, 16, 6
    x, ad, a, b, s = case(M, N, K, r, L)
    y = gauss(M, N, seed=8)
    got = bsq.lora_add(y, x, ad, a, b, s, out=torch.empty_like(y))
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(DEV)
    assert torch.equal(bsq.lora_add(y[perm].contiguous(), x[perm].contiguous(), ad[perm].contiguous(), a, b, s), got[perm])


# above 64 tokens: every number of 32-rank steps, ranks that end inside one, columns that end inside 64 and inside 4, tiles
# of tokens that end inside one, and enough of them that a workgroup takes several columns and its adapters in turn
MANY = [(65, 70, 72, 8, 2, True), (66, 64, 64, 24, 66, False), (80, 200, 136, 32, 3, False), (129, 131, 200, 40, 5, True),
        (200, 68, 264, 72, 4, False), (100, 256, 128, 200, 3, False), (257, 320, 512, 256, 9, True), (1100, 72, 4104, 16, 3, True),
        (4200, 1000, 72, 16, 9, True), (4200, 260, 64, 128, 3, False), (2100, 2052, 64, 256, 4, True)]


@pytest.mark.parametrize("M,N,K,r,L,runs", MANY)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_add_to_many_tokens(M, N, K, r, L, runs, dtype):
    note("lora add %d %d %d %d %d runs=%s %s" % (M, N, K, r, L, runs, dtype))
    x, ad, a, b, s = case(M, N, K, r, L, seed=M + r, runs=runs)
    y = gauss(M, N, seed=9, dtype=dtype)
    v, e = lora64(x, ad, a, b, s)
    want = y.cpu().double() + v
    (o,), intact = guarded([(M, N)], dtype)
    got = bsq.lora_add(y, x, ad, a, b, s, out=o)
    intact()
    assert_within(got, want, e + want.abs() * F32 + store_error(want, dtype), "out")
    none = ((ad < 0) | (ad >= L)).cpu()
    assert torch.equal(got.cpu()[none], y.cpu()[none])
    o.copy_(y)
    bsq.lora_add(o, x, ad, a, b, s)
    intact()
    assert torch.equal(o, got)


@pytest.mark.parametrize("M,N,K,r,L", [(65, 130, 80, 24, 3), (300, 1033, 272, 64, 5), (1500, 96, 4112, 136, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matvec_of_many_tokens(M, N, K, r, L, dtype):
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


@pytest.mark.parametrize("M", [20, 300])
def test_what_lies_in_the_workspace_does_not_matter(M):
    N, K, r, L = 100, 200, 24, 5
    x, ad, a, b, s = case(M, N, K - K % 16, r, L)
    y, w = gauss(M, N, seed=8), weights(N, K - K % 16, 4)
    n = max(bsq.lib().nvfp4_lora_workspace_bytes(M, N, r, bsq.OUT_BF16), bsq.lib().lora_workspace_bytes(M, r))
    outs = []
    for fill in (0, 255, 127):   # zeros, NaN, large values
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        outs.append((bsq.lora_add(y, x, ad, a, b, s, out=torch.empty_like(y), workspace=ws),
                     bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s, workspace=ws)))
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])


@pytest.mark.parametrize("M", [3, 100])
def test_no_token_with_an_adapter(M):
    N, K, r = 132, 64, 16
    x, _, a, b, s = case(M, N, K, r, 2)
    ad = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    for dtype in (torch.bfloat16, torch.float32):
        y = gauss(M, N, seed=8, dtype=dtype)
        y[0, 0], y[1, 1] = float("nan"), float("inf")
        before = y.clone()
        got = bsq.lora_add(y, x, ad, a, b, s, out=torch.zeros_like(y))
        assert torch.equal(got.view(torch.uint8), before.view(torch.uint8))
        bsq.lora_add(y, x, ad, a, b, s)
        assert torch.equal(y.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 2, 3, 61, 62, 63, 64, 65, 66, 67, 190])
def test_ends_of_rows_at_any_alignment(N, dtype):
    """Every number of columns past a piece, in a slice of a wider y that starts and continues at odd elements: the bits of
    the same columns of a wide call, and nothing beside the slice."""
    M, K, r, L, W = 83, 96, 24, 3, 192
    x, ad, a, b, s = case(M, W, K, r, L, seed=4)
    y = gauss(M, W, seed=9, dtype=dtype)
    want = bsq.lora_add(y, x, ad, a, b, s, out=torch.empty_like(y))[:, :N]
    for left in (0, 1, 3):
        wide = gauss(M, left + N + 2 - (left + N) % 2 + 1, seed=2, dtype=dtype)   # an odd number of elements between rows
        wide[:, left:left + N] = y[:, :N]
        before, out = wide.clone(), wide.clone()
        bsq.lora_add(wide[:, left:left + N], x, ad, a, b[:, :N].contiguous(), s, out=out[:, left:left + N])
        bsq.lora_add(wide[:, left:left + N], x, ad, a, b[:, :N].contiguous(), s)
        for t in (out, wide):
            assert torch.equal(t[:, left:left + N], want)
            assert torch.equal(t[:, :left], before[:, :left]) and torch.equal(t[:, left + N:], before[:, left + N:])


@pytest.mark.parametrize("M,N,K,r,L", [(16, 4096, 272, 16, 5), (5, 4090, 528, 128, 3), (20, 4111, 96, 8, 2), (33, 8192, 80, 64, 40)])
def test_matvec_that_fills_the_chip(M, N, K, r, L):
    """Weights that leave no compute unit idle: the down products go first."""
    test_matvec(M, N, K, r, L, False)


def test_replays_of_a_matvec_that_fills_the_chip():
    M, N, K, r, L = 16, 4096, 512, 16, 5
    x, ad, a, b, s = case(M, N, K, r, L, seed=3)
    w = weights(N, K, 4)
    bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s)
    for seed in range(4):
        x.copy_(gauss(M, K, seed=50 + seed))
        ad.copy_(adapters(M, L, 60 + seed, 0.2))
        want = bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
