"""Tensors of the caller that a call writes count as changed: autograd, which may have saved one for a backward pass, then
refuses that pass, as it does after torch's own operators in place, instead of computing with what the tensor holds now."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
M, N, K, L, R = 6, 64, 64, 2, 8


def rand(*shape, seed=1, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def lora():
    ad = torch.tensor([0, 1, -1, 1, 0, 0], dtype=torch.int32, device=DEV)
    return rand(M, K, seed=2), ad, rand(L, R, K, seed=3), rand(L, N, R, seed=4)


def nvfp4(rows, seed):
    q = bsq.nvfp4_quantize(rand(rows, K, seed=seed))
    return q["row_codes"], q["row_scales"], q["s_enc"][:1]


def routed():
    o = bsq.moe_sort(torch.tensor([[0, 1], [1, 2], [2, 0], [0, 2], [1, 0], [2, 1]], device=DEV), 3)
    return o["positions"], o["source"]


def writers():
    """(name, the tensors it is given to write, the call) of every entry point that writes tensors of the caller."""
    x, ad, a, b = lora()
    p, s = routed()
    new = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    y, o, wide = new(M, N), new(M, N), new(M, 2 * N)
    yield "lora_add in place", [y], lambda: bsq.lora_add(y, x, ad, a, b)
    yield "lora_add", [o], lambda: bsq.lora_add(y, x, ad, a, b, out=o)
    yield "lora_add to a slice", [wide], lambda: bsq.lora_add(wide[:, 3:3 + N], x, ad, a, b)
    yield "nvfp4_lora_matvec", [o], lambda: bsq.nvfp4_lora_matvec(x, *nvfp4(N, 5), ad, a, b, out=o)
    rows, tokens = new(s.numel(), K), new(M, K)
    yield "moe_gather", [rows], lambda: bsq.moe_gather(x, p, s, out=rows)
    yield "moe_combine", [tokens], lambda: bsq.moe_combine(rows, p, out=tokens)
    yield "nvfp4_matvec", [o], lambda: bsq.nvfp4_matvec(x, *nvfp4(N, 5), out=o)
    yield "nvfp4_gated_matvec", [o], lambda: bsq.nvfp4_gated_matvec(bsq.ACT_SILU, x, *nvfp4(N, 5), *nvfp4(N, 6), out=o)
    gu = new(M, 2 * N)
    yield "blockscaled_gated_gemm", [o, gu], lambda: bsq.blockscaled_gated_gemm(
        bsq.FMT_NVFP4, bsq.ACT_SILU, *nvfp4(M, 7), *nvfp4(N, 5), *nvfp4(N, 6), save_gate_up=True, out=o, gate_up=gu)
    yield "blockscaled_gated_gemm_backward", [gu], lambda: bsq.blockscaled_gated_gemm_backward(
        bsq.FMT_NVFP4, bsq.ACT_SILU, *nvfp4(M, 7), *nvfp4(N, 5), gu, out=gu)
    yield "blockscaled_gemm", [o], lambda: bsq.blockscaled_gemm(bsq.FMT_NVFP4, *nvfp4(M, 7), *nvfp4(N, 5), out=o)
    offs = torch.tensor([0, M], dtype=torch.int64, device=DEV)
    yield "blockscaled_grouped_gemm", [o], lambda: bsq.blockscaled_grouped_gemm(
        bsq.FMT_NVFP4, bsq.GROUP_M, offs, *nvfp4(M, 7), *nvfp4(N, 5), out=o)
    g, h = [rand(33, seed=8), rand(5, 7, seed=9, dtype=torch.float32)], [rand(33), rand(5, 7, dtype=torch.float32)]
    yield "clip_grad_norm in place", g, lambda: bsq.clip_grad_norm(g, 1.0)
    yield "clip_grad_norm", h, lambda: bsq.clip_grad_norm(g, 1.0, out=h)
    sumsq = bsq.grad_sumsq(g)
    yield "grad_clip in place", g, lambda: bsq.grad_clip(g, sumsq, 1.0)
    yield "grad_clip", h, lambda: bsq.grad_clip(g, sumsq, 1.0, out=h)


def test_written_tensors_count_as_changed():
    for name, written, call in writers():
        before = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, before)), name


def test_only_what_is_written_counts_as_changed():
    x, ad, a, b = lora()
    y, o = rand(M, N), rand(M, N)
    tensors = [x, ad, a, b, y]
    before = [t._version for t in tensors]
    bsq.lora_add(y, x, ad, a, b, out=o)
    g, h = [rand(9)], [rand(9)]
    version = g[0]._version
    bsq.clip_grad_norm(g, 0.5, out=h)
    assert [t._version for t in tensors] == before and g[0]._version == version
    version = y._version
    with pytest.raises(bsq.BsqError):   # rank 4: refused, nothing written
        bsq.lora_add(y, x, ad, a[:, :4].contiguous(), b[:, :, :4].contiguous())
    assert y._version == version


def test_a_saved_output_is_not_used_after_an_adapter_changed_it():
    x, ad, a, b = lora()
    w = rand(N, K).float().requires_grad_()
    y = x.float() @ w.t()
    loss = (y * y).sum()   # y is saved for the backward pass
    bsq.lora_add(y, x, ad, a, b)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    y = x.float() @ w.t()
    bsq.lora_add(y, x, ad, a, b)
    (y * y).sum().backward()   # saved afterwards: the gradient of the changed y
    want = (2 * y.detach().double()).t() @ x.double()
    # a sum over M tokens in fp32, of products that round once; 2 y is exact
    tol = (M + 2) * 2.0 ** -24 * ((2 * y.detach().double().abs()).t() @ x.double().abs())
    assert ((w.grad.double() - want).abs() <= tol).all()


def test_without_autograd():
    x, ad, a, b = lora()
    want = bsq.lora_add(rand(M, N), x, ad, a, b)
    with torch.inference_mode():
        y = rand(M, N)
        assert bsq.lora_add(y, x, ad, a, b) is y and torch.equal(y, want)
    out = bsq.lora_add(y, x, ad, a, b, out=torch.empty_like(want))
    bsq.lora_add(y, x, ad, a, b)   # a tensor that has no version, written outside of inference mode too
    assert torch.equal(y, out)
