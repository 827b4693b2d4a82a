"""grad_sumsq, grad_clip and clip_grad_norm against a plain binary64 form.

Tolerance: squares are summed in binary64 (relative error below n 2^-53), so the norm is off by its
rounding to fp32, 2^-24, and that sum's half; a clipped gradient is g times c, c rounded to fp32 and the
product rounded once (fp32) or twice (fp32, then bf16): 2 2^-24, or 2^-8 (1 + 2^-14) for bf16."""
import math

import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.plain64 import assert_within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(sizes, kinds, seed, std=0.02, offset=0):
    """Gradients as views of flat buckets, tensor i of kind kinds[i % len], starting `offset` elements in."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = {"f": torch.float32, "b": torch.bfloat16}[kinds[i % len(kinds)]]
        out.append(((torch.randn(n + offset, generator=g) * std).to(dt).to(DEV))[offset:])
    return out


def norm64(grads):
    return math.sqrt(math.fsum(float(t.cpu().double().square().sum()) for t in grads))


def check(grads, max_norm, in_place=False):
    before = [t.clone() for t in grads]
    n = norm64(grads)
    c = min(1.0, max_norm / (n + 1e-6))
    out = None if in_place else [torch.empty_like(t) for t in grads]
    norm = bsq.clip_grad_norm(grads, max_norm, out=out)
    torch.cuda.synchronize()
    assert abs(float(norm) - n) <= n * (2.0 ** -24 + sum(t.numel() for t in grads) * 2.0 ** -53)
    for i, (b, o) in enumerate(zip(before, grads if in_place else out)):
        want = b.cpu().double() * c
        if c == 1.0:
            assert torch.equal(o, b), "gradient %d changed" % i
            continue
        rel = 2.0 ** -8 * (1 + 2.0 ** -14) if b.dtype == torch.bfloat16 else 2 * 2.0 ** -24
        tiny = 2.0 ** -134 if b.dtype == torch.bfloat16 else 2.0 ** -149
        assert_within(o, want, want.abs() * rel + tiny, "gradient %d" % i)
        if not in_place:
            assert torch.equal(grads[i], b), "the input changed"


CASES = [([1], "f"), ([1], "b"), ([7, 0, 1, 13], "fb"), ([8192], "f"), ([8193, 8191, 16384, 5], "bf"),
         ([0, 0, 3], "f"), (list(range(1, 131)), "fbb"), ([100003], "b"), ([3_000_001, 17, 40960], "fb")]


@pytest.mark.parametrize("sizes,kinds", CASES)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_sizes(sizes, kinds, offset):
    note("clip %s %s offset %d" % (sizes[:5], kinds, offset))
    g = make(sizes, kinds, 11, offset=offset)
    n = norm64(g)
    check(g, 0.3 * n)
    check(g, 2 * n)
    check(g, 2 * n, in_place=True)
    check(g, 0.3 * n, in_place=True)


def test_many_tensors_and_same_bits():
    g = make([37 + 11 * (i % 97) for i in range(500)], "fb", 12)
    check(g, 0.01)
    a, b = bsq.grad_sumsq(g), bsq.grad_sumsq(g)
    assert torch.equal(a, b)


def test_neither_overflow_nor_underflow():
    big = [torch.full((1000,), 3e38, device=DEV), torch.full((50,), 1e30, dtype=torch.bfloat16, device=DEV)]
    s = bsq.grad_sumsq(big)
    assert abs(float(s) / (sum(float(t.double().square().sum()) for t in big)) - 1) < 1e-12
    out = [torch.empty_like(t) for t in big]
    norm = bsq.clip_grad_norm(big, 1.0, out=out)   # the norm itself is beyond fp32
    assert math.isinf(float(norm))
    assert abs(float(out[0][0]) * math.sqrt(1000) - 1) < 1e-5
    small = [torch.full((1000,), 1e-30, device=DEV)]
    assert abs(float(bsq.grad_sumsq(small)) / float(small[0].double().square().sum()) - 1) < 1e-12
    tiny = [torch.full((4,), 2.0 ** -149, device=DEV)]
    assert float(bsq.grad_sumsq(tiny)) == 4 * 2.0 ** -298


def test_zero_bounds_nan_and_infinity():
    g = make([100, 2000], "fb", 13)
    out = [torch.empty_like(t) for t in g]
    bsq.clip_grad_norm(g, 0.0, out=out)
    assert not any(t.any() for t in out)
    z = [torch.zeros(100, device=DEV)]
    assert float(bsq.clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    check(g, math.inf, in_place=True)
    g[0][5] = math.inf
    norm = bsq.clip_grad_norm(g, 1.0, out=out)
    assert math.isinf(float(norm)) and math.isnan(float(out[0][5]))
    assert not out[0][:5].any() and not out[1].any()
    g[1][7] = math.nan
    norm = bsq.clip_grad_norm(g, 1.0)
    assert math.isnan(float(norm)) and all(torch.isnan(t).all() for t in g)


def test_two_ranks_add_their_sums():
    a, b = make([1000, 50], "fb", 14), make([3000], "f", 15)
    total = bsq.grad_sumsq(a) + bsq.grad_sumsq(b)
    n = norm64(a + b)
    out = [torch.empty_like(t) for t in a]
    norm = bsq.grad_clip(a, total, 0.5 * n, out=out)
    assert abs(float(norm) - n) <= n * 2.0 ** -23
    assert_within(out[0], a[0].cpu().double() * (0.5 * n / (n + 1e-6)), a[0].cpu().double().abs() * 2.0 ** -22, "out")


def test_other_stream_workspace_and_graph():
    g = make([5000, 333], "fb", 16)
    ws = torch.empty(bsq.lib().grad_workspace_bytes(2), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in g]
    want = [torch.empty_like(t) for t in g]
    n0 = bsq.clip_grad_norm(g, 0.1, out=want)
    with torch.cuda.stream(side):
        n1 = bsq.clip_grad_norm(g, 0.1, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = bsq.clip_grad_norm(g, 0.1, out=out, workspace=ws)
    for seed in (17, 18, 19):
        for t, s in zip(g, make([5000, 333], "fb", seed)):
            t.copy_(s)
        n = bsq.clip_grad_norm(g, 0.1, out=want)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, n) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_python_refusals():
    g = make([10, 20], "fb", 20)
    with pytest.raises(ValueError):
        bsq.clip_grad_norm([], 1.0)
    with pytest.raises(TypeError):
        bsq.clip_grad_norm([g[0].double()], 1.0)
    with pytest.raises(ValueError):
        bsq.clip_grad_norm([g[0].cpu()], 1.0)
    with pytest.raises(ValueError):
        bsq.clip_grad_norm([torch.zeros((4, 6), device=DEV).t()], 1.0)
    with pytest.raises(ValueError):
        bsq.clip_grad_norm(g, 1.0, out=[g[0]])
    with pytest.raises(ValueError):
        bsq.clip_grad_norm(g, 1.0, out=[g[0], g[1].float()])
    with pytest.raises(bsq.BsqError):
        bsq.clip_grad_norm(g, -1.0)
    with pytest.raises(bsq.BsqError):
        bsq.clip_grad_norm(g, math.nan)
    with pytest.raises(ValueError):
        bsq.clip_grad_norm(g, 1.0, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_tables_that_spill_into_more_launches():
    # 280 tensors to a launch, 176 with outputs; chunks of 8192; every start in a flat bucket
    sizes = [1 + (i * 7919) % 20000 for i in range(561)]
    g = make(sizes, "fbf", 21, offset=1)
    n = norm64(g)
    check(g, 0.5 * n)
    check(g, 0.5 * n, in_place=True)


def test_clip_in_one_call_and_in_two_agree():
    g = make([70001, 5, 8192, 333], "fb", 22)
    a, b = [torch.empty_like(t) for t in g], [torch.empty_like(t) for t in g]
    na = bsq.clip_grad_norm(g, 0.01, out=a)
    nb = bsq.grad_clip(g, bsq.grad_sumsq(g), 0.01, out=b)
    assert torch.equal(na, nb) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_outputs_at_another_offset_than_their_gradients():
    g = make([20011, 9000], "fb", 23)
    buf = {t.dtype: torch.full((40000,), 5.0, dtype=t.dtype, device=DEV) for t in g}
    out = [buf[t.dtype][3:3 + t.numel()] for t in g]
    want = [torch.empty_like(t) for t in g]
    bsq.clip_grad_norm(g, 0.01, out=out)
    bsq.clip_grad_norm(g, 0.01, out=want)
    for t, o, w in zip(g, out, want):
        assert torch.equal(o, w)
        assert (buf[t.dtype][:3] == 5.0).all() and (buf[t.dtype][3 + t.numel():] == 5.0).all()


def test_a_tensor_past_2_to_the_31_elements():
    n = (1 << 31) + 4099
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    g[-1] = 2.0
    norm = bsq.clip_grad_norm([g], 1.0)
    want = math.sqrt(0.25 * (n - 1) + 4.0)
    assert abs(float(norm) - want) <= want * 2.0 ** -23
    c = 1.0 / (want + 1e-6)
    for i, v in ((0, 0.5), (1 << 30, 0.5), ((1 << 31) - 1, 0.5), (1 << 31, 0.5), (n - 2, 0.5), (n - 1, 2.0)):
        assert abs(float(g[i]) - v * c) <= v * c * (2.0 ** -8 + 2.0 ** -20), i


# a factor below fp32's normal range: the gradients it scales are large enough for their products to matter
@pytest.mark.parametrize("max_norm", [1e-3, 1e-6, 1e-9])
@pytest.mark.parametrize("in_place", [False, True])
def test_factor_below_the_normal_range(max_norm, in_place):
    g = torch.Generator().manual_seed(24)
    v = torch.randn(9001, generator=g).clamp(-3, 3)
    grads = [(v * 1e38).to(DEV), (v[:777] * 9e37).to(torch.bfloat16).to(DEV), torch.ones(5, device=DEV)]
    before = [t.cpu().double() for t in grads]
    n = math.sqrt(math.fsum(float(t.square().sum()) for t in before))
    out = grads if in_place else [torch.empty_like(t) for t in grads]
    bsq.clip_grad_norm(grads, max_norm, out=None if in_place else out)
    for i, (b, o) in enumerate(zip(before, out)):
        want = b * (max_norm / (n + 1e-6))
        rel = 2.0 ** -8 * (1 + 2.0 ** -14) if o.dtype == torch.bfloat16 else 2 * 2.0 ** -24
        tiny = 2.0 ** -134 if o.dtype == torch.bfloat16 else 2.0 ** -149
        assert_within(o, want, want.abs() * rel + tiny, "gradient %d" % i)
