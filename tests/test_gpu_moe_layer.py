"""A layer of experts on quantized operands, forward and backward, from its parts as a user joins them: the order by
expert, tokens gathered into the products' operands, the grouped products, the weighted way back, and the gradients.

The fused gathers are compared bit for bit with the same layer built from indexing by torch and the casts; the whole
with a layer in fp32.  Each quantized operand's root mean square error is below a tenth (NVFP4) or a thirtieth (MXFP8) of its
values', a result passes two of them and the rows' bf16 rounding: the error's norm stays below a fifth of the result's
(a cosine above 0.98)."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NV = bsq.FMT_NVFP4 | bsq.FMT_A_ROWSCALED


def cosine(a, b):
    a, b = a.double().cpu().flatten(), b.detach().double().cpu().flatten()
    return float(a @ b / (a.norm() * b.norm()))


def stacked(quantize, w):
    q = [quantize(w[e]) for e in range(w.shape[0])]
    return {n: torch.stack([t[n] for t in q]) for n in q[0]}


@pytest.mark.parametrize("T,k,E,H,F,drop", [(300, 2, 8, 512, 384, False), (65, 4, 16, 256, 288, True)])
def test_forward_and_backward(T, k, E, H, F, drop):
    g = torch.Generator().manual_seed(T)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)   # noqa: E731
    x, w, dout = normal(T, H), normal(E, F, H) * H ** -0.5, normal(T, F)
    top = (torch.rand((T, E), generator=g) + torch.rand(E, generator=g)).topk(k, 1)
    experts, gate = top.indices.to(DEV), top.values.softmax(1).to(DEV)
    if drop:
        experts[torch.rand((T, k), generator=g).to(DEV) < 0.1] = -1
    o = bsq.moe_sort(experts, E, 32)
    p, src, offs = o["positions"], o["source"], o["offsets"]

    # forward: row-scaled NVFP4 tokens times per-expert NVFP4 weights
    qw = stacked(lambda m: bsq.nvfp4_quantize(m), w)
    qx = bsq.moe_gather_nvfp4_rowscaled(x, p, src)
    product = lambda q: bsq.blockscaled_grouped_gemm(   # noqa: E731
        NV, bsq.GROUP_M, offs, q["codes"], q["scales"], q["s_enc"], qw["row_codes"], qw["row_scales"],
        qw["s_enc"][:, 0].contiguous(), out=torch.zeros((src.numel(), F), dtype=torch.bfloat16, device=DEV))
    ys = product(qx)
    y = bsq.moe_combine(ys, p, gate)
    xs_plain = torch.cat([x, x.new_zeros((1, H))])[torch.where(src < 0, T, src // k)]
    assert torch.equal(product(bsq.nvfp4_quantize_rowscaled(xs_plain)), ys)

    # backward: MXFP8 towards the tokens, and along them towards the weights
    dys, dgate = bsq.moe_combine_backward(dout, ys, p, src, gate)
    wt = stacked(lambda m: bsq.mxfp8_quantize(m, bsq.COL), w)
    qd = bsq.mxfp8_quantize(dys, bsq.ROW | bsq.COL)
    dxs = bsq.blockscaled_grouped_gemm(bsq.FMT_MXFP8, bsq.GROUP_M, offs, qd["row_codes"], qd["row_scales"], None,
                                       wt["col_codes"], wt["col_scales"], None,
                                       out=torch.zeros((src.numel(), H), dtype=torch.bfloat16, device=DEV))
    dx = bsq.moe_combine(dxs, p)
    xs = bsq.moe_gather(x, p, src)
    assert torch.equal(xs, xs_plain)
    qc = bsq.mxfp8_quantize(xs, bsq.COL)
    dw = bsq.blockscaled_grouped_gemm(bsq.FMT_MXFP8, bsq.GROUP_K, offs, qd["col_codes"], qd["col_scales"], None,
                                      qc["col_codes"], qc["col_scales"], None, out_dtype=torch.float32)

    # the layer in fp32
    xr, wr, gr = (t.float().cpu().requires_grad_() for t in (x, w, gate))
    every = torch.einsum("th,efh->tef", xr, wr)
    e = experts.cpu()
    rows = every.gather(1, e.clamp(min=0).unsqueeze(2).expand(-1, -1, F))
    want = (torch.where((e >= 0).unsqueeze(2), rows, torch.zeros(())) * gr.unsqueeze(2)).sum(1)
    want.backward(dout.float().cpu())
    for got, ref, name in ((y, want, "y"), (dx, xr.grad, "dx"), (dw, wr.grad, "dw"), (dgate, gr.grad, "dgate")):
        assert cosine(got, ref) > 0.98, name
    assert (dgate[experts < 0] == 0).all()


def test_adapters_beside_shared_weights_both_ways():
    """nvfp4_lora_matvec, and nvfp4_matvec with lora_add on its fp32 output: the same sums, joined in another order."""
    M, N, K, r, L = 24, 520, 1024, 16, 6
    g = torch.Generator().manual_seed(1)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)   # noqa: E731
    x, a, b = normal(M, K), normal(L, r, K) * K ** -0.5, normal(L, N, r) * r ** -0.5
    q = bsq.nvfp4_quantize(normal(N, K) * K ** -0.5)
    w = (q["row_codes"], q["row_scales"], q["s_enc"][:1])
    ad = torch.randint(-1, L, (M,), generator=g).to(torch.int32).to(DEV)
    s = torch.rand(L, generator=g).to(DEV)
    one = bsq.nvfp4_lora_matvec(x, *w, ad, a, b, s, out_dtype=torch.float32)
    two = bsq.lora_add(bsq.nvfp4_matvec(x, *w, out_dtype=torch.float32), x, ad, a, b, s)
    # at most 3 r + 2 roundings of the up product's sum of magnitudes and two of the result on either side
    up = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for i in range(L):
        at = ad == i
        up[at] = ((x[at].double() @ a[i].double().t()).abs() @ b[i].double().abs().t()) * s[i].double()
    assert ((one - two).abs().double() <= 2.0 ** -24 * ((6 * r + 4) * up + 4 * two.abs().double())).all()
