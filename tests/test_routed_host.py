"""Refusals of the experts' and adapters' C entry points, on the host: every invalid argument is answered with its
documented status before any HIP call; and the binding's own checks on tensors that are not on a GPU."""
import pytest
import torch

import block_scaled_precision_nvfp4_amd as bsq

FAKE = 0x10000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(bsq.LIB_PATH):
        from block_scaled_precision_nvfp4_amd import build
        build.build()
    return bsq.lib()


def call(L, name, defaults, kw):
    a = dict(defaults)
    for k in kw:
        assert k in a
    a.update(kw)
    return getattr(L, name)(*a.values(), None)


SORT = dict(experts=FAKE, id_bytes=8, slots=64, E=8, align=32, rows=312 // 32 * 32, offsets=FAKE, positions=FAKE,
            source=FAKE, ws=FAKE)
SORT["rows"] = (64 + 8 * 31) // 32 * 32


@pytest.mark.parametrize("kw,status", [
    (dict(id_bytes=2), 3), (dict(slots=-1), 2), (dict(slots=(1 << 25) + 1), 2), (dict(E=0), 2), (dict(E=1025), 2),
    (dict(align=0), 3), (dict(align=24), 3), (dict(align=512), 3), (dict(rows=SORT["rows"] - 1), 2), (dict(rows=1 << 31), 2),
    (dict(experts=None), 1), (dict(offsets=None), 1), (dict(positions=None), 1), (dict(source=None), 1), (dict(ws=None, slots=8192, rows=1 << 20), 1),
    (dict(experts=FAKE + 4), 6), (dict(offsets=FAKE + 4), 6), (dict(positions=FAKE + 2), 6), (dict(source=FAKE + 1), 6),
    (dict(ws=FAKE + 8), 6)])
def test_sort_refusals(L, kw, status):
    assert call(L, "moe_sort", SORT, kw) == status
    assert b"moe_sort" in L.bsq_last_error()


def test_sort_sizes(L):
    assert L.moe_sort_rows(10, 4, 1) == 10
    assert L.moe_sort_rows(10, 4, 32) == 128       # (10 + 4 * 31) rounded down
    assert L.moe_sort_rows(2, 100, 32) == 64       # two slots fill two groups at most
    assert L.moe_sort_rows(0, 4, 32) == 0
    for bad in ((-1, 4, 1), (1, 0, 1), (1, 1025, 1), (1, 4, 3), (1, 4, 0), ((1 << 25) + 1, 4, 1)):
        assert L.moe_sort_rows(*bad) == -1
    assert L.moe_sort_workspace_bytes(-1, 4) == -1 and L.moe_sort_workspace_bytes(4, 0) == -1
    assert L.moe_sort_workspace_bytes(1 << 25, 1024) > 0


GATHER = dict(T=4, k=2, H=64, x=FAKE, ldx=64, positions=FAKE, source=FAKE, rows=8, out=FAKE)
SIZES = [(dict(T=-1), 2), (dict(k=-1), 2), (dict(H=-32), 2), (dict(rows=-1), 2), (dict(H=68, ldx=72), 2), (dict(k=65), 2),
         (dict(rows=1 << 31), 2), (dict(T=(1 << 23) + 1), 2), (dict(T=1 << 23, H=4096), 2), (dict(positions=None), 1),
         (dict(positions=FAKE + 2), 6)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(x=None), 1), (dict(source=None), 1), (dict(out=None), 1), (dict(ldx=56), 2), (dict(ldx=68), 2), (dict(x=FAKE + 8), 6),
    (dict(out=FAKE + 8), 6), (dict(source=FAKE + 2), 6)])
def test_gather_refusals(L, kw, status):
    assert call(L, "moe_gather", GATHER, kw) == status
    two = dict(GATHER, scales=FAKE)
    assert call(L, "moe_gather_mxfp8", two, kw) == status
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=FAKE), kw) == status


def test_quantized_gather_refusals(L):
    two = dict(GATHER, scales=FAKE)
    assert call(L, "moe_gather_mxfp8", two, dict(H=48)) == 2
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=FAKE), dict(H=56)) == 2
    assert call(L, "moe_gather_mxfp8", two, dict(scales=None)) == 1
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=None), {}) == 1
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=FAKE + 2), {}) == 6
    assert call(L, "moe_gather_mxfp8", two, dict(scales=FAKE + 4)) == 6


COMBINE = dict(T=4, k=2, H=64, y=FAKE, y_dtype=0, rows=8, positions=FAKE, weights=FAKE, out=FAKE, out_dtype=0)
BACKWARD = dict(T=4, k=2, H=64, dout=FAKE, y=FAKE, y_dtype=0, rows=8, positions=FAKE, source=FAKE, weights=FAKE, dy=FAKE,
                dw=FAKE)


@pytest.mark.parametrize("kw,status", [(k, s) for k, s in SIZES if "ldx" not in k])
def test_combine_sizes(L, kw, status):
    assert call(L, "moe_combine", COMBINE, kw) == status
    assert call(L, "moe_combine_backward", BACKWARD, kw) == status


@pytest.mark.parametrize("kw,status", [(dict(y_dtype=2), 3), (dict(out_dtype=-1), 3), (dict(y=None), 1), (dict(out=None), 1),
                                       (dict(y=FAKE + 8), 6), (dict(out=FAKE + 4), 6), (dict(weights=FAKE + 2), 6)])
def test_combine_refusals(L, kw, status):
    assert call(L, "moe_combine", COMBINE, kw) == status


@pytest.mark.parametrize("kw,status", [(dict(y_dtype=2), 3)] + [(dict([(n, None)]), 1) for n in
                                       ("dout", "y", "source", "weights", "dy", "dw")] +
                         [(dict([(n, FAKE + 2)]), 6) for n in ("dout", "y", "source", "weights", "dy", "dw")])
def test_combine_backward_refusals(L, kw, status):
    assert call(L, "moe_combine_backward", BACKWARD, kw) == status


def test_empty_combinations_need_no_buffers(L):
    assert call(L, "moe_combine", COMBINE, dict(T=0, out=None, y=None)) == 0
    assert call(L, "moe_combine", COMBINE, dict(H=0, out=None)) == 0
    assert call(L, "moe_gather", GATHER, dict(rows=0, out=None, source=None)) == 0
    assert call(L, "moe_combine_backward", BACKWARD, dict(T=0, rows=0, dy=None, y=None, source=None)) == 0


ADD = dict(M=4, N=64, K=64, r=16, n=2, x=FAKE, ldx=64, adapters=FAKE, a=FAKE, b=FAKE, scales=FAKE, y=FAKE, ldy=64,
           out=FAKE, ldo=64, dtype=0, ws=FAKE)
MATVEC = dict(flags=0, M=4, N=64, K=64, x=FAKE, ldx=64, c=FAKE, s=FAKE, e=FAKE, r=16, n=2, adapters=FAKE, a=FAKE, b=FAKE,
              scales=FAKE, y=FAKE, dtype=0, ws=FAKE)
ADAPTERS = [(dict(n=-1), 2), (dict(n=(1 << 24) + 1), 2), (dict(r=0), 2), (dict(r=12), 2), (dict(r=264), 2),
            (dict(adapters=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(ws=None), 1), (dict(a=FAKE + 8), 6),
            (dict(b=FAKE + 8), 6), (dict(ws=FAKE + 4), 6), (dict(adapters=FAKE + 2), 6), (dict(scales=FAKE + 2), 6),
            (dict(M=-1), 2), (dict(N=-1), 2), (dict(K=-8), 2), (dict(K=1 << 24, ldx=1 << 24), 2),
            (dict(M=(1 << 20) + 1), 2), (dict(N=(1 << 27) + 1, ), 2), (dict(dtype=2), 3), (dict(x=None), 1), (dict(y=None), 1),
            (dict(ldx=56), 2), (dict(ldx=68), 2), (dict(x=FAKE + 8), 6)]


@pytest.mark.parametrize("kw,status", ADAPTERS)
def test_lora_refusals(L, kw, status):
    assert call(L, "lora_add", ADD, kw) == status
    assert call(L, "nvfp4_lora_matvec", MATVEC, kw) == status


@pytest.mark.parametrize("kw,status", [(dict(K=60), 2), (dict(out=None), 1), (dict(ldy=60), 2), (dict(ldo=60), 2),
                                       (dict(ldy=72, ldo=80), 3), (dict(M=1 << 20, N=1 << 17, ldy=1 << 17, ldo=1 << 17), 2),
                                       (dict(y=FAKE + 1), 6), (dict(out=FAKE + 1), 6), (dict(dtype=1, out=FAKE + 2), 6)])
def test_lora_add_refusals(L, kw, status):
    assert call(L, "lora_add", ADD, kw) == status


@pytest.mark.parametrize("kw,status", [(dict(K=72, ldx=72), 2), (dict(flags=0x10), 3), (dict(c=None), 1), (dict(e=None), 1),
                                       (dict(y=FAKE + 2), 6), (dict(M=1 << 20, N=1 << 17), 2)])
def test_nvfp4_lora_refusals(L, kw, status):
    assert call(L, "nvfp4_lora_matvec", MATVEC, kw) == status


def test_lora_workspace(L):
    assert L.lora_workspace_bytes(16, 16) >= 16 * 16 * 4
    for bad in ((-1, 16), ((1 << 20) + 1, 16), (4, 0), (4, 12), (4, 264)):
        assert L.lora_workspace_bytes(*bad) == -1
        assert L.nvfp4_lora_workspace_bytes(bad[0], 64, bad[1], 0) == -1
    assert L.nvfp4_lora_workspace_bytes(16, 100, 16, 0) >= L.lora_workspace_bytes(16, 16) + 6400
    assert L.nvfp4_lora_workspace_bytes(16, 100, 16, 1) >= L.lora_workspace_bytes(16, 16)
    assert L.nvfp4_lora_workspace_bytes(16, -1, 16, 0) == -1 and L.nvfp4_lora_workspace_bytes(16, 64, 16, 2) == -1
    assert call(L, "lora_add", ADD, dict(M=0, y=None, out=None, ws=None)) == 0
    assert call(L, "nvfp4_lora_matvec", MATVEC, dict(N=0, y=None, ws=None)) == 0


def test_binding_wants_device_tensors():
    i32, f32, bf = torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), torch.zeros((2, 8), dtype=torch.bfloat16)
    src = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        bsq.moe_sort(i32, 4)
    with pytest.raises(TypeError):
        bsq.moe_sort(f32, 4)
    for f in (bsq.moe_gather, bsq.moe_gather_mxfp8, bsq.moe_gather_nvfp4_rowscaled):
        with pytest.raises(TypeError):
            f(bf, i32, src)
    with pytest.raises(TypeError):
        bsq.moe_combine(bf, i32, f32)
    with pytest.raises(TypeError):
        bsq.moe_combine(i32, i32, f32)
    with pytest.raises(TypeError):
        bsq.moe_combine_backward(bf, bf, i32, src, f32)
    with pytest.raises(TypeError):
        bsq.lora_add(bf, bf, src, bf, bf)
    with pytest.raises(TypeError):
        bsq.nvfp4_lora_matvec(bf, bf, bf, f32, src, bf, bf)


def test_a_gather_of_width_zero_still_writes_the_rows_scales(L):
    two = dict(GATHER, scales=None, x=None, source=None, out=None, H=0, ldx=0)
    assert call(L, "moe_gather_mxfp8", two, {}) == 0
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=None), {}) == 1
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=FAKE + 2), {}) == 6
    assert call(L, "moe_gather_nvfp4_rowscaled", dict(two, s_enc=None), dict(rows=0)) == 0
