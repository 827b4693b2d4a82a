"""The order of token slots by expert, the gathers and the weighted combination with its gradients, against plain forms
on the CPU (whole numbers and copies equal, quantized rows bit for bit those of the casts, sums against binary64).

Tolerances: the combination adds k products by fused multiply-adds in fp32, each off by half a step of a partial sum, so
by k 2^-24 S with S = sum |w y|; a weight's gradient adds `width` exact products in some order, width 2^-24 S; a row's
gradient is one product rounded to fp32, 2^-24 of itself; then half a step of the output's type."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq
from tests.gpu_common import note
from tests.plain64 import F32, assert_within, store_error
from tests.test_gpu_feed_forward_edges import guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ids(T, k, E, seed, drop=0.0, one=None, dtype=torch.int64):
    """k different experts of each token where there are as many, some favoured; some dropped by ids out of range."""
    g = torch.Generator().manual_seed(seed)
    if one is not None:
        e = torch.full((T, k), one)
    elif k <= E and T * E <= 1 << 24:
        e = (torch.rand((T, E), generator=g) + torch.rand(E, generator=g)).topk(k, 1).indices
    else:
        e = torch.randint(0, E, (T, k), generator=g)
    if drop:
        out = torch.rand((T, k), generator=g) < drop
        far = (1 << 40) if dtype == torch.int64 else (1 << 30)
        wrong = torch.tensor([-1, E, -far, far + 1])[torch.randint(0, 4, (T, k), generator=g)]
        e = torch.where(out, wrong, e)
    return e.to(dtype)


def sorted_plain(e, E, align):
    """offsets, positions, source by numpy's stable sort."""
    flat = e.reshape(-1).numpy().astype(np.int64)
    n = flat.size
    rows = (n + min(n, E) * (align - 1)) // align * align
    kept = (flat >= 0) & (flat < E)
    counts = np.bincount(flat[kept], minlength=E)
    offsets = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)])
    order = np.nonzero(kept)[0]
    order = order[np.argsort(flat[order], kind="stable")]
    first = np.concatenate([[0], np.cumsum(counts)])[:-1]
    at = offsets[flat[order]] + np.arange(order.size) - first[flat[order]]
    positions, source = np.full(n, -1, np.int64), np.full(rows, -1, np.int64)
    positions[order] = at
    source[at] = order
    return offsets, positions.reshape(e.shape), source


def check_sort(e, E, align, ws=None):
    note("sort %s of %d align %d %s" % (tuple(e.shape), E, align, e.dtype))
    o = bsq.moe_sort(e.to(DEV), E, align, workspace=ws)
    torch.cuda.synchronize()
    for got, want in zip((o["offsets"], o["positions"], o["source"]), sorted_plain(e, E, align)):
        assert np.array_equal(got.cpu().numpy(), want)
    return o


# one workgroup and several; a lone slot, no slot, more experts than slots, every number of experts' bits
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (0, 2, 4), (5, 0, 4), (1, 8, 8), (37, 2, 8), (63, 1, 3), (65, 3, 1024), (1000, 4, 513),
                                   (16384, 1, 64), (16385, 1, 64), (8193, 2, 7), (4099, 8, 128), (3001, 6, 1000), (100003, 2, 1),
                                   (50021, 6, 60), (300007, 4, 256)])
@pytest.mark.parametrize("align", [1, 32, 256])
def test_sort(T, k, E, align):
    check_sort(ids(T, k, E, T + k), E, align)
    check_sort(ids(T, k, E, T + k, drop=0.2, dtype=torch.int32), E, align)


@pytest.mark.parametrize("T", [100, 40000])
def test_sort_of_one_expert_and_of_none(T):
    for E in (1, 8, 1024):
        check_sort(ids(T, 2, E, 1, one=E - 1), E, 64)
        check_sort(ids(T, 2, E, 1, one=-1), E, 64)
        check_sort(ids(T, 2, E, 1, one=E), E, 1)


def test_sort_with_a_workspace_of_the_caller():
    n = bsq.lib().moe_sort_workspace_bytes(80000, 64)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    for seed in (1, 2):   # what an earlier call left there does not matter
        check_sort(ids(40000, 2, 64, seed), 64, 32, ws)
    with pytest.raises(ValueError):
        bsq.moe_sort(ids(40000, 2, 64, 1).to(DEV), 64, workspace=ws[:-16])


def order_of(T, k, E, align, seed, drop=0.1):
    o = bsq.moe_sort(ids(T, k, E, seed, drop).to(DEV), E, align)
    return o["positions"], o["source"]


def rows_of(x, source, k):
    """x[source // k] with zero rows, on the CPU."""
    s = source.cpu().long()
    out = x.cpu()[s.clamp(min=0) // max(k, 1)]
    out[s < 0] = 0
    return out


def gauss(*shape, seed=0, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


GATHERS = [(1, 1, 1, 32, 1), (3, 2, 4, 64, 32), (37, 2, 8, 96, 1), (100, 8, 128, 288, 32), (65, 3, 5, 4096, 16), (7, 6, 9, 4128, 1),
           (20, 2, 3, 8192, 32), (9, 4, 8, 8224, 1), (5, 3, 2, 20000, 256), (2000, 4, 64, 512, 128)]


@pytest.mark.parametrize("T,k,E,H,align", GATHERS)
def test_gathers(T, k, E, H, align):
    note("gather %d %d %d %d %d" % (T, k, E, H, align))
    p, s = order_of(T, k, E, align, T)
    x = gauss(T, H, seed=T + H)
    x[0, :64] = 0            # blocks of zeros
    x[T // 2] *= 2.0 ** -60  # a tiny row
    want = rows_of(x, s, k)
    xd, R = x.to(DEV), s.numel()
    got = bsq.moe_gather(xd, p, s)
    assert torch.equal(got.cpu(), want)
    (v,), intact = guarded([(R, H)], torch.bfloat16)
    assert bsq.moe_gather(xd, p, s, out=v) is v
    intact()
    assert torch.equal(v.cpu(), want)
    if H % 16 == 0:
        q, ref = bsq.moe_gather_nvfp4_rowscaled(xd, p, s), bsq.nvfp4_quantize_rowscaled(got)
        for n in ("codes", "scales", "s_enc"):
            assert torch.equal(q[n], ref[n]), n
    if H % 32 == 0:
        q, ref = bsq.moe_gather_mxfp8(xd, p, s), bsq.mxfp8_quantize(got)
        for n in ("row_codes", "row_scales"):
            assert torch.equal(q[n], ref[n]), n


def test_quantized_gathers_against_the_oracle():
    import oracle
    p, s = order_of(50, 3, 6, 32, 3)
    x = gauss(50, 416, seed=4)
    want = rows_of(x, s, 3)
    q, ref = bsq.moe_gather_nvfp4_rowscaled(x.to(DEV), p, s), oracle.nvfp4_quantize_rowscaled(want)
    for n in ("codes", "scales", "s_enc"):
        assert np.array_equal(q[n].cpu().numpy(), ref[n]), n
    q, ref = bsq.moe_gather_mxfp8(x.to(DEV), p, s), oracle.mxfp8_quantize(want, direction=oracle.ROW)
    for n in ("row_codes", "row_scales"):
        assert np.array_equal(q[n].cpu().numpy(), ref[n]), n


def test_gathers_of_values_that_are_not_finite():
    p, s = order_of(40, 2, 4, 32, 5)
    x = gauss(40, 128, seed=6)
    x[3, 5], x[7, 100], x[9, 0], x[11] = float("nan"), float("inf"), -float("inf"), float("nan")
    got = bsq.moe_gather(x.to(DEV), p, s)
    assert torch.equal(got.cpu().view(torch.int16), rows_of(x.view(torch.int16), s, 2))
    q, ref = bsq.moe_gather_nvfp4_rowscaled(x.to(DEV), p, s), bsq.nvfp4_quantize_rowscaled(got)
    assert all(torch.equal(q[n].view(torch.uint8), ref[n].view(torch.uint8)) for n in ("codes", "scales", "s_enc"))
    # The MXFP8 cast encodes 512 adjacent elements together, in one of two ways that differ in what becomes of values
    # that are not finite, by whether all of the blocks among them have a scale byte above 0: its codes of such a
    # block depend on its neighbours, so there is no equality to ask for.  The gather makes such a value the NaN code
    # under the scale byte of 2^120, and every other block is the cast's.
    q, ref = bsq.moe_gather_mxfp8(x.to(DEV), p, s), bsq.mxfp8_quantize(got)
    bad = ~torch.isfinite(got)
    block = bad.reshape(-1, 4, 32).any(2)
    assert (q["row_codes"][bad] & 127 == 127).all() and (q["row_scales"][block] == 247).all()
    assert torch.equal(q["row_scales"][~block], ref["row_scales"][~block])
    fine = ~block.repeat_interleave(32, 1)
    assert torch.equal(q["row_codes"][fine], ref["row_codes"][fine])


def test_strided_tokens():
    p, s = order_of(30, 2, 4, 32, 8)
    buf = gauss(30, 200, seed=9)
    x = buf[:, 8:168]
    d = buf.to(DEV)[:, 8:168]
    want = rows_of(x, s, 2)
    got = bsq.moe_gather(d, p, s)
    assert torch.equal(got.cpu(), want)
    assert torch.equal(bsq.moe_gather_mxfp8(d, p, s)["row_codes"], bsq.mxfp8_quantize(got)["row_codes"])
    assert torch.equal(bsq.moe_gather_nvfp4_rowscaled(d, p, s)["codes"], bsq.nvfp4_quantize_rowscaled(got)["codes"])
    with pytest.raises(bsq.BsqError):
        bsq.moe_gather(buf.to(DEV)[:, 4:164], p, s)   # not 16-byte aligned
    with pytest.raises(ValueError):
        bsq.moe_gather(d.t(), p, s)


def combined64(y, p, w):
    """(sum w y, sum |w y|) over a token's slots, in binary64."""
    p = p.cpu().long()
    live = (p >= 0).unsqueeze(2)
    rows = y.cpu().double()[p.clamp(min=0).reshape(-1)].reshape(*p.shape, -1) if y.shape[0] else torch.zeros(*p.shape, y.shape[1]).double()
    v = rows * (1.0 if w is None else w.cpu().double().unsqueeze(2))
    v = torch.where(live, v, torch.zeros((), dtype=torch.float64))
    return v.sum(1), v.abs().sum(1)


COMBINES = [(1, 1, 1, 8), (1, 2, 8, 4096), (37, 2, 8, 64), (3, 64, 70, 136), (100, 8, 16, 520), (333, 6, 60, 1032), (5, 0, 4, 64),
            (9, 3, 4, 8200), (2000, 4, 64, 512)]


@pytest.mark.parametrize("T,k,E,H", COMBINES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine(T, k, E, H, dtype):
    note("combine %d %d %d %d %s" % (T, k, E, H, dtype))
    p, s = order_of(T, k, E, 16, T)
    y = gauss(s.numel(), H, seed=H, dtype=dtype)
    y[s.cpu() < 0] = float("nan")   # rows without a token belong to no sum
    w = gauss(T, k, seed=3, dtype=torch.float32)
    for weights in (w, None):
        want, S = combined64(y, p, weights)
        for od in (torch.bfloat16, torch.float32):
            (v,), intact = guarded([(T, H)], od)
            got = bsq.moe_combine(y.to(DEV), p, None if weights is None else weights.to(DEV), out_dtype=od, out=v)
            intact()
            assert_within(got, want, k * F32 * S + store_error(want, od), "out")


@pytest.mark.parametrize("T,k,E,H", COMBINES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine_backward(T, k, E, H, dtype):
    note("combine backward %d %d %d %d %s" % (T, k, E, H, dtype))
    p, s = order_of(T, k, E, 16, T)
    y, d, w = gauss(s.numel(), H, seed=H, dtype=dtype), gauss(T, H, seed=4), gauss(T, k, seed=5, dtype=torch.float32)
    dy, dw = bsq.moe_combine_backward(d.to(DEV), y.to(DEV), p, s, w.to(DEV))
    src = s.cpu().long()
    want = d.double()[src.clamp(min=0) // max(k, 1)] * (w.reshape(-1).double()[src.clamp(min=0)] if k else torch.zeros(0)).unsqueeze(1)
    want[src < 0] = 0
    assert dy.dtype == dtype
    assert_within(dy, want, want.abs() * F32 + store_error(want, dtype), "dy")
    pl = p.cpu().long()
    rows = y.double()[pl.clamp(min=0).reshape(-1)].reshape(T, k, H) if k else torch.zeros(T, 0, H).double()
    prod = torch.where((pl >= 0).unsqueeze(2), rows * d.double().unsqueeze(1), torch.zeros((), dtype=torch.float64))
    assert_within(dw, prod.sum(2), H * F32 * prod.abs().sum(2) + store_error(prod.sum(2), torch.float32), "dweights")


def test_gradients_against_differences():
    """The combination is linear in y and in the weights, so a central difference of any step is exact but for roundings:
    of the fp32 outputs, 2^-24 S each and k 2^-24 S of the sums, added up over the difference's two sides and divided
    by its step; the gradients' own as above."""
    T, k, E, H = 23, 3, 5, 72
    p, s = order_of(T, k, E, 16, 11)
    y, d, w = gauss(s.numel(), H, seed=1, dtype=torch.float32), gauss(T, H, seed=2), gauss(T, k, seed=3, dtype=torch.float32)
    dy, dw = bsq.moe_combine_backward(d.to(DEV), y.to(DEV), p, s, w.to(DEV))
    vy, vw = gauss(s.numel(), H, seed=4, dtype=torch.float32), gauss(T, k, seed=5, dtype=torch.float32)
    h = 0.5

    def loss(y_, w_):
        out = bsq.moe_combine(y_.to(DEV), p, w_.to(DEV), out_dtype=torch.float32).cpu().double()
        return float((out * d.double()).sum()), float((combined64(y_, p, w_)[1] * d.double().abs()).sum())
    for got, v, step in ((dy, vy, lambda t: (y + t * vy, w)), (dw, vw, lambda t: (y, w + t * vw))):
        (up, su), (down, sd) = loss(*step(h)), loss(*step(-h))
        # y + t v and w + t v are themselves rounded: 2^-24 of the sum's terms once more
        tol = (k + 2) * F32 * (su + sd) / (2 * h) + H * F32 * float((got.cpu().double() * v.double()).abs().sum() + su + sd)
        assert abs((up - down) / (2 * h) - float((got.cpu().double() * v.double()).sum())) <= tol


def test_gathers_gradient_is_the_combination():
    """<moe_gather(x), d> = <x, moe_combine(d)> for any x and d, in the copies' exact values and fp32 sums."""
    T, k, E, H = 50, 4, 8, 64
    p, s = order_of(T, k, E, 32, 12)
    x, d = gauss(T, H, seed=1), gauss(s.numel(), H, seed=2)
    a = (bsq.moe_gather(x.to(DEV), p, s).cpu().double() * d.double()).sum()
    dx = bsq.moe_combine(d.to(DEV), p, out_dtype=torch.float32).cpu().double()
    S = (combined64(d, p, None)[1] * x.double().abs()).sum()
    assert abs(float(a - (dx * x.double()).sum())) <= k * F32 * float(S)


def test_values_that_are_not_finite_stay_with_their_token():
    T, k, E, H = 30, 3, 6, 64
    e = ids(T, k, E, 13)
    e[4, 1] = -1
    o = bsq.moe_sort(e.to(DEV), E)
    p, s = o["positions"], o["source"]
    y, w, d = gauss(s.numel(), H, seed=1), gauss(T, k, seed=2, dtype=torch.float32), gauss(T, H, seed=3)
    clean = bsq.moe_combine(y.to(DEV), p, w.to(DEV)).cpu()
    dyc, dwc = (t.cpu() for t in bsq.moe_combine_backward(d.to(DEV), y.to(DEV), p, s, w.to(DEV)))
    w[4, 1] = float("nan")                          # of a dropped slot: adds nothing
    assert torch.equal(bsq.moe_combine(y.to(DEV), p, w.to(DEV)).cpu(), clean)
    dy, dw = (t.cpu() for t in bsq.moe_combine_backward(d.to(DEV), y.to(DEV), p, s, w.to(DEV)))
    assert torch.equal(dy, dyc) and torch.equal(dw, dwc) and dw[4, 1] == 0
    y[int(p[7, 2]), 5] = float("nan")
    w[9, 0] = float("inf")
    got, want = bsq.moe_combine(y.to(DEV), p, w.to(DEV)).cpu(), clean.clone()
    assert torch.isnan(got[7, 5]) and not torch.isfinite(got[9]).any()
    got[7, 5], got[9], want[7, 5], want[9] = 0, 0, 0, 0
    assert torch.equal(got, want)
    dy, dw = (t.cpu() for t in bsq.moe_combine_backward(d.to(DEV), y.to(DEV), p, s, w.to(DEV)))
    assert torch.isnan(dw[7, 2]) and not torch.isfinite(dy[int(p[9, 0])]).any()
    dw[7, 2], dwc[7, 2] = 0, 0
    dy[int(p[9, 0])], dyc[int(p[9, 0])] = 0, 0
    assert torch.equal(dw, dwc) and torch.equal(dy, dyc)


def test_positions_out_of_range_count_as_none():
    """Entries that no sort writes: nothing outside the tensors is read or written."""
    T, H, R = 6, 64, 10
    p = torch.tensor([[0, 1], [2, 10], [3, 1 << 30], [-7, 4], [5, 6], [7, 8]], dtype=torch.int32, device=DEV)
    s = torch.tensor([0, 1, 2, 4, 7, 8, 9, 10, 11, 12], dtype=torch.int32, device=DEV)   # 12: behind the last slot
    x, w = gauss(T, H, seed=1), gauss(T, 2, seed=2, dtype=torch.float32)
    (v,), intact = guarded([(R, H)], torch.bfloat16)
    bsq.moe_gather(x.to(DEV), p, s, out=v)
    intact()
    want = x[s.cpu().long().clamp(max=11) // 2].clone()
    want[9] = 0
    assert torch.equal(v.cpu(), want)
    y = gauss(R, H, seed=3)
    got = bsq.moe_combine(y.to(DEV), p, w.to(DEV), out_dtype=torch.float32)
    live = torch.where((p >= 0) & (p < R), p, -1)
    want, S = combined64(y, live, w)
    assert_within(got, want, 2 * F32 * S + store_error(want, torch.float32), "out")
    _, dw = bsq.moe_combine_backward(x.to(DEV), y.to(DEV), p, s, w.to(DEV))
    assert (dw.cpu()[live.cpu() < 0] == 0).all()


def test_refusals_of_the_binding():
    p, s = order_of(8, 2, 4, 1, 1, drop=0)
    x, y, w = gauss(8, 64).to(DEV), gauss(16, 64).to(DEV), torch.ones((8, 2), device=DEV)
    for bad in (lambda: bsq.moe_gather(x[:7], p, s), lambda: bsq.moe_gather(x, p.reshape(-1), s),
                lambda: bsq.moe_gather(x, p, s.reshape(4, 4)), lambda: bsq.moe_combine(y, p, w[:, :1]),
                lambda: bsq.moe_combine_backward(x, y[:15], p, s, w), lambda: bsq.moe_combine_backward(x[:, :32], y, p, s, w),
                lambda: bsq.moe_sort(p.reshape(-1), 4), lambda: bsq.moe_combine(y, p, out=x[:7]),
                lambda: bsq.moe_sort(p.t(), 4)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bsq.moe_gather(x.float(), p, s), lambda: bsq.moe_gather(x, p.long(), s),
                lambda: bsq.moe_combine(y, p, w.double()), lambda: bsq.moe_combine(y.half(), p, w),
                lambda: bsq.moe_combine(y, p, w, out_dtype=torch.float16), lambda: bsq.moe_combine_backward(x, y, p, s, None)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bsq.moe_sort(p, 0), lambda: bsq.moe_sort(p, 2000), lambda: bsq.moe_sort(p, 4, align=3),
                lambda: bsq.moe_gather(gauss(8, 60).to(DEV), p, s), lambda: bsq.moe_gather_mxfp8(gauss(8, 48).to(DEV), p, s)):
        with pytest.raises(bsq.BsqError):
            bad()


def test_captured_and_replayed():
    """A graph of the whole way, replayed on new inputs with eager calls in between."""
    T, k, E, H = 5000, 4, 16, 96   # several workgroups of the sort
    e = ids(T, k, E, 1).to(DEV)
    x, w = gauss(T, H, seed=1).to(DEV), gauss(T, k, seed=2, dtype=torch.float32).to(DEV)

    def way():
        o = bsq.moe_sort(e, E, 32)
        p, s = o["positions"], o["source"]
        xs = bsq.moe_gather(x, p, s)
        return (*o.values(), xs, *bsq.moe_gather_mxfp8(x, p, s).values(), *bsq.moe_gather_nvfp4_rowscaled(x, p, s).values(),
                bsq.moe_combine(xs, p, w), *bsq.moe_combine_backward(x, xs, p, s, w))
    way()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = way()
    for seed in (3, 4, 5, 6):
        e.copy_(ids(T, k, E, seed, drop=0.1))
        x.copy_(gauss(T, H, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, way()):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_two_streams_at_once():
    T, k, E, H = 20000, 2, 8, 512
    cases = [(ids(T, k, E, s).to(DEV), gauss(T, H, seed=s).to(DEV)) for s in (1, 2)]
    w = torch.rand((T, k), device=DEV)

    def way(e, x):
        o = bsq.moe_sort(e, E, 32)
        xs = bsq.moe_gather(x, o["positions"], o["source"])
        return o["source"], bsq.moe_combine(xs, o["positions"], w)
    want = [way(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(way(*c))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_past_two_to_the_31_elements():
    T, k, E, H = 270000, 2, 4, 4096   # 2.2 G elements in rows
    g = torch.Generator(device=DEV).manual_seed(1)
    e = torch.rand((T, E), device=DEV, generator=g).topk(k, 1).indices
    x = torch.randn((T, H), device=DEV, generator=g, dtype=torch.bfloat16)
    o = bsq.moe_sort(e, E, 32)
    p, s = o["positions"], o["source"]
    xs = bsq.moe_gather(x, p, s)
    assert xs.numel() > 1 << 31
    pick = torch.cat([torch.arange(s.numel() - 4000, s.numel(), device=DEV), torch.arange(0, s.numel(), 997, device=DEV)])
    src = s[pick].long()
    assert torch.equal(xs[pick], torch.where((src < 0).unsqueeze(1), 0, x[src.clamp(min=0) // k]))
    q = bsq.moe_gather_mxfp8(x, p, s)
    ref = bsq.mxfp8_quantize(xs[pick])
    assert torch.equal(q["row_codes"][pick], ref["row_codes"]) and torch.equal(q["row_scales"][pick], ref["row_scales"])
    del q
    w = torch.rand((T, k), device=DEV, generator=g)
    out = bsq.moe_combine(xs, p, w)
    some = torch.arange(0, T, 499, device=DEV)
    want = (xs[p[some].long().reshape(-1)].reshape(-1, k, H).double() * w[some].double().unsqueeze(2)).sum(1)
    assert ((out[some].double() - want).abs() <= want.abs() * (2.0 ** -8 + 4 * F32)).all()
    dy, dw = bsq.moe_combine_backward(x, xs, p, s, w)
    live = pick[src >= 0]
    sl = s[live].long()
    want = (x[sl // k].float() * w.reshape(-1)[sl].unsqueeze(1)).to(torch.bfloat16)
    assert torch.equal(dy[live], want) and (dy[pick[src < 0]] == 0).all()


# over 1024 slots a wave: counted twice instead of kept; with 16 waves a workgroup and with 8
@pytest.mark.parametrize("T,k,E", [(1200007, 2, 8), (400003, 3, 700)])
def test_sort_of_many_slots(T, k, E):
    check_sort(ids(T, k, E, 3, drop=0.05), E, 64)


# outputs of 128 MiB and more, in rows of whole lines and of others, go past the caches
@pytest.mark.parametrize("H", [2048, 2056])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_outputs(H, dtype):
    T, k, E = 33000, 2, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    e = torch.rand((T, E), device=DEV, generator=g).topk(k, 1).indices
    e[torch.rand((T, k), device=DEV, generator=g) < 0.02] = -1
    o = bsq.moe_sort(e, E, 32)
    p, s = o["positions"], o["source"]
    x = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    w = torch.rand((T, k), device=DEV, generator=g)
    src = s.long()
    none = (src < 0).unsqueeze(1)
    xs = bsq.moe_gather(x, p, s)
    assert torch.equal(xs, torch.where(none, 0, x[src.clamp(min=0) // k]))
    y = xs.to(dtype)
    live = (p >= 0).unsqueeze(2)
    rows = torch.where(live, y[p.clamp(min=0).reshape(-1).long()].reshape(T, k, H).double(), 0)
    want, S = (rows * w.unsqueeze(2)).sum(1), (rows.abs() * w.unsqueeze(2)).sum(1)
    for od in (torch.bfloat16, torch.float32):
        got = bsq.moe_combine(y, p, w, out_dtype=od).double()
        step = 2.0 ** -8 if od == torch.bfloat16 else F32
        assert ((got - want).abs() <= k * F32 * S + want.abs() * step + 2.0 ** -134).all()
    dy, dw = bsq.moe_combine_backward(x, y, p, s, w)
    prod = x.float()[src.clamp(min=0) // k] * w.reshape(-1)[src.clamp(min=0)].unsqueeze(1)   # one rounding to fp32
    assert torch.equal(dy, torch.where(none, 0, prod).to(dtype))
    dots = rows * x.double().unsqueeze(1)
    assert ((dw.double() - dots.sum(2)).abs() <= (H + 1) * F32 * dots.abs().sum(2)).all()


def test_few_and_many_tokens_agree():
    """The kernels fetch a token's slots in another way where tokens are few: the same bits either way."""
    T, k, E, H = 3000, 5, 12, 512
    p, s = order_of(T, k, E, 32, 21)
    y, w = gauss(s.numel(), H, seed=1).to(DEV), torch.rand((T, k), device=DEV)
    many = bsq.moe_combine(y, p, w)
    for a in range(0, T, 700):
        assert torch.equal(bsq.moe_combine(y, p[a:a + 700].contiguous(), w[a:a + 700].contiguous()), many[a:a + 700])
    # 2900 of the tokens dropped: the same rows of the first 100 from both gathers
    x = gauss(T, H, seed=2).to(DEV)
    e = ids(T, k, E, 22).to(DEV)
    e[100:] = -1
    few, all_ = bsq.moe_sort(e[:100].contiguous(), E, 32), bsq.moe_sort(e, E, 32)
    for f in (bsq.moe_gather_mxfp8, bsq.moe_gather_nvfp4_rowscaled):
        a = f(x[:100], few["positions"], few["source"])
        b = f(x, all_["positions"], all_["source"])
        n = min(few["source"].numel(), all_["source"].numel())
        assert all(torch.equal(a[key][:n], b[key][:n]) for key in a)


def test_on_another_stream():
    T, k, E, H = 200, 2, 8, 256
    e, x, w = ids(T, k, E, 1).to(DEV), gauss(T, H, seed=1).to(DEV), torch.rand((T, k), device=DEV)
    o = bsq.moe_sort(e, E)
    want = bsq.moe_combine(bsq.moe_gather(x, o["positions"], o["source"]), o["positions"], w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2 = x * 2   # only the side stream's order makes it ready
        o = bsq.moe_sort(e, E)
        got = bsq.moe_combine(bsq.moe_gather(x2, o["positions"], o["source"]), o["positions"], w)
    side.synchronize()
    assert torch.equal(got, want * 2)


def test_combination_of_the_most_tokens():
    """The largest call: 2^23 tokens of 2048, fp32 rows, one slot each."""
    T, H, rows = 1 << 23, 2048, 64
    y = gauss(rows, H, seed=3, dtype=torch.float32).to(DEV)
    p = (torch.arange(T, dtype=torch.int32, device=DEV) * 7 % (rows + 1)).reshape(T, 1)   # row 64 is out of range
    note("combine %d x %d" % (T, H))
    out = bsq.moe_combine(y, p)
    want = torch.cat([y, torch.zeros(1, H, device=DEV)]).to(torch.bfloat16)
    for t0 in range(0, T, 1 << 20):
        assert torch.equal(out[t0:t0 + (1 << 20)], want[p[t0:t0 + (1 << 20), 0].long()])


@pytest.mark.parametrize("T,k,E", [(6, 4, 126), (4, 5, 63), (1, 8, 1024), (2, 1, 17), (64, 8, 128), (65, 3, 33)])
@pytest.mark.parametrize("align", [1, 16, 256])
def test_sort_of_few_slots_for_many_experts(T, k, E, align):
    check_sort(ids(T, k, E, T + E), E, align)
    check_sort(ids(T, k, E, T + E, drop=0.3, dtype=torch.int32), E, align)
