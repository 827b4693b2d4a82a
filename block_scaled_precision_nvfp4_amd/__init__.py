"""Python binding of libbsq: block-scaled (NVFP4 / MXFP8) quantization and GEMM on MI355X.

Thin ctypes marshalling over the C ABI in include/bsq.h: every step of the computation
runs in the library's HIP kernels.  PyTorch only provides device memory (output
tensors are allocated with torch.empty) and the current HIP stream.  The functions
have the names of the C entry points and are not recorded by autograd: results have no
history, and a tensor of the caller that a call writes counts as changed.  Importing works without a GPU; calling a
compute function needs libbsq.so (built by ``python -m
block_scaled_precision_nvfp4_amd.build``) and fails loudly if it is missing.
"""
from __future__ import annotations

import ctypes as C
import os
from array import array
from operator import attrgetter
from typing import Dict, Optional, Sequence

import torch

ROW, COL = 1, 2
MX_SLAB = 4   # OR'ed into an MXFP8 cast's direction: codes in the slab layout
RNE, SR = 0, 1
FMT_NVFP4, FMT_MXFP8 = 0, 1
FMT_A_ROWSCALED, FMT_B_ROWSCALED = 0x10, 0x20
FMT_MX_SLAB_A, FMT_MX_SLAB_B = 0x40, 0x80   # OR'ed into FMT_MXFP8: that operand's codes in the slab layout
FMT_MX_SLAB = FMT_MX_SLAB_A | FMT_MX_SLAB_B
GROUP_M, GROUP_K = 1, 2
OUT_BF16, OUT_F32 = 0, 1
ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2   # BSQ_ACT_*
NVFP4_QUANTIZE_WORKSPACE_BYTES = 8192   # BSQ_NVFP4_QUANTIZE_WORKSPACE_BYTES

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsq.so")

_ERRORS = {1: "null pointer", 2: "shape", 3: "argument", 4: "unsupported", 5: "HIP", 6: "alignment"}


class BsqError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s failed (%s error %d): %s" % (fn, _ERRORS.get(status, "?"), status, msg))
        self.status = status


_lib = None


def lib():
    """Load libbsq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libbsq.so not found at %s; build it with "
                               "`python -m block_scaled_precision_nvfp4_amd.build`" % LIB_PATH)
        L = C.CDLL(LIB_PATH)
        vp, i64, i32, u32, u64 = C.c_void_p, C.c_int64, C.c_int, C.c_uint32, C.c_uint64
        L.nvfp4_quantize.argtypes = [vp, i64, i64, i32, i32, u64, u32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_noalloc.argtypes = [vp, i64, i64, i32, i32, u64, u32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_fprop_wgrad.argtypes = [vp, i64, i64, i32, u64, u32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.nvfp4_col_mxfp8_row_quantize.argtypes = [vp, i64, i64, i32, u64, u32, vp, vp, vp, vp, vp, vp, i32,
                                                   vp, vp, vp]
        L.nvfp4_quantize_rowscaled.argtypes = [vp, i64, i64, i32, u64, u32, vp, vp, vp, vp, vp, vp]
        L.nvfp4_dequantize.argtypes = [vp, vp, vp, i64, i64, vp, vp]
        L.mxfp8_quantize.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp]
        L.mxfp8_requantize_nvfp4.argtypes = [vp, vp, vp, i64, i64, i32, vp, vp, vp, vp, vp]
        L.rht_apply.argtypes = [vp, i64, i64, i32, vp, vp, vp]
        L.blockscaled_gemm.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        L.blockscaled_grouped_gemm.argtypes = [i32, i32, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        L.nvfp4_linear_workspace_bytes.argtypes = [i64, i64, i64]
        L.nvfp4_linear_workspace_bytes.restype = C.c_int64
        L.nvfp4_linear_saved_bytes.argtypes = [i64, i64]
        L.nvfp4_linear_saved_bytes.restype = C.c_int64
        L.nvfp4_linear_forward.argtypes = [vp, vp, i64, i64, i64, u64, vp, vp, vp, vp, vp]
        L.nvfp4_linear_backward.argtypes = [vp, vp, vp, i64, i64, i64, u64, vp, vp, vp, vp, vp]
        L.nvfp4_matvec.argtypes = [i32, i64, i64, i64, vp, i64, vp, vp, vp, vp, i32, vp]
        L.nvfp4_gated_matvec.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.blockscaled_gated_gemm.argtypes = [i32, i32, i64, i64, i64] + [vp] * 12
        L.blockscaled_gated_gemm_backward.argtypes = [i32, i32, i64, i64, i64] + [vp] * 9
        L.grad_workspace_bytes.argtypes = [i64]
        L.grad_workspace_bytes.restype = C.c_int64
        L.grad_sumsq.argtypes = [vp, vp, vp, i64, vp, vp, vp]
        L.grad_clip.argtypes = [vp, vp, vp, vp, i64, vp, C.c_double, vp, vp]
        L.clip_grad_norm.argtypes = [vp, vp, vp, vp, i64, C.c_double, vp, vp, vp]
        L.moe_sort_rows.argtypes = [i64, i64, i64]
        L.moe_sort_rows.restype = C.c_int64
        L.moe_sort_workspace_bytes.argtypes = [i64, i64]
        L.moe_sort_workspace_bytes.restype = C.c_int64
        L.moe_sort.argtypes = [vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.moe_gather.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp]
        L.moe_gather_nvfp4_rowscaled.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, vp, vp]
        L.moe_gather_mxfp8.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, vp]
        L.moe_combine.argtypes = [i64, i64, i64, vp, i32, i64, vp, vp, vp, i32, vp]
        L.moe_combine_backward.argtypes = [i64, i64, i64, vp, vp, i32, i64, vp, vp, vp, vp, vp, vp]
        L.lora_workspace_bytes.argtypes = [i64, i64]
        L.lora_workspace_bytes.restype = C.c_int64
        L.nvfp4_lora_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.nvfp4_lora_workspace_bytes.restype = C.c_int64
        L.lora_add.argtypes = [i64, i64, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, i32, vp, vp]
        L.nvfp4_lora_matvec.argtypes = [i32, i64, i64, i64, vp, i64, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp]
        for f in ("moe_sort", "moe_gather", "moe_gather_nvfp4_rowscaled", "moe_gather_mxfp8", "moe_combine",
                  "moe_combine_backward", "lora_add", "nvfp4_lora_matvec", "nvfp4_matvec", "nvfp4_gated_matvec", "blockscaled_gated_gemm", "blockscaled_gated_gemm_backward",
                  "grad_sumsq", "grad_clip", "clip_grad_norm", "nvfp4_linear_forward", "nvfp4_linear_backward", "nvfp4_quantize",
                  "nvfp4_quantize_noalloc",
                  "nvfp4_col_mxfp8_row_quantize", "nvfp4_quantize_fprop_wgrad", "nvfp4_quantize_rowscaled",
                  "nvfp4_dequantize", "mxfp8_quantize", "mxfp8_requantize_nvfp4", "rht_apply",
                  "blockscaled_gemm", "blockscaled_grouped_gemm", "bsq_version"):
            getattr(L, f).restype = C.c_int
        L.bsq_last_error.argtypes = []
        L.bsq_last_error.restype = C.c_char_p
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise BsqError(fn, status, lib().bsq_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without the Stream object around it, where this torch has that (1 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _dev_tensor(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA/HIP tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _workspace(ws: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    """The caller's scratch tensor (checked for size and device), or a new one."""
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != torch.device(device):
        raise TypeError("workspace must be a device tensor on %s" % (device,))
    if not ws.is_contiguous() or ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace must be contiguous and hold at least %d bytes" % nbytes)
    return ws


def _written(*tensors: Optional[torch.Tensor]):
    """Tensors of the caller that a call has written count as changed (their version counters), as after torch's own operators
    in place: a backward pass that saved one says so instead of using what it holds now.  The kernels write through
    pointers, which torch does not see.  None stands for a tensor that the call made itself."""
    given = [t for t in tensors if t is not None]
    if given:
        torch.autograd.graph.increment_version(given)


def _signs(rht_signs, device):
    if rht_signs is None:
        return None
    s = rht_signs
    if not isinstance(s, torch.Tensor):
        s = torch.tensor(s, dtype=torch.int8)
    s = s.to(device=device, dtype=torch.int8).contiguous()
    if s.numel() != 16:
        raise ValueError("rht_signs must have 16 entries")
    return s


def nvfp4_quantize(x: torch.Tensor, direction: int = ROW, rounding: int = RNE, sr_seed: int = 0,
                   sr_stream: int = 0, rht_signs=None, workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """NVFP4-quantize a bf16 [rows, cols] device tensor.  Returns the requested directions'
    ``{row,col}_codes`` / ``{row,col}_scales`` (uint8) and ``amax`` / ``s_enc`` (float32[2],
    index 0 rowwise, 1 columnwise), all on x's device.  ``workspace`` (a device tensor of at
    least NVFP4_QUANTIZE_WORKSPACE_BYTES bytes) is the call's scratch; one is allocated when
    none is given."""
    _dev_tensor(x, torch.bfloat16, "x")
    R, Cc = x.shape
    dev = x.device
    out: Dict[str, torch.Tensor] = {}
    u8 = dict(dtype=torch.uint8, device=dev)
    if direction & ROW:
        out["row_codes"] = torch.empty((R, Cc // 2), **u8)
        out["row_scales"] = torch.empty((R, Cc // 16), **u8)
    if direction & COL:
        out["col_codes"] = torch.empty((Cc, R // 2), **u8)
        out["col_scales"] = torch.empty((Cc, R // 16), **u8)
    out["amax"] = torch.empty(2, dtype=torch.float32, device=dev)
    out["s_enc"] = torch.empty(2, dtype=torch.float32, device=dev)
    ws = _workspace(workspace, NVFP4_QUANTIZE_WORKSPACE_BYTES, dev)
    sg = _signs(rht_signs, dev)
    _check("nvfp4_quantize", lib().nvfp4_quantize(
        x.data_ptr(), R, Cc, direction, rounding, sr_seed & (2 ** 64 - 1), sr_stream, _ptr(sg),
        _ptr(out.get("row_codes")), _ptr(out.get("row_scales")), _ptr(out.get("col_codes")),
        _ptr(out.get("col_scales")), out["amax"].data_ptr(), out["s_enc"].data_ptr(), ws.data_ptr(), _stream(dev)))
    return out


def nvfp4_quantize_fprop_wgrad(x: torch.Tensor, rounding: int = RNE, sr_seed: int = 0, sr_stream: int = 0,
                               rht_signs=None, workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """One pass over a bf16 [rows, cols] activation that writes its rowwise forward operand (RNE,
    no transform: ``row_codes``, ``row_scales``) and its columnwise wgrad operand (the given
    rounding and transform: ``col_codes``, ``col_scales``); ``amax`` / ``s_enc`` as for
    ``nvfp4_quantize`` (index 0 rowwise, 1 columnwise)."""
    _dev_tensor(x, torch.bfloat16, "x")
    R, Cc = x.shape
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    out = {"row_codes": torch.empty((R, Cc // 2), **u8), "row_scales": torch.empty((R, Cc // 16), **u8),
           "col_codes": torch.empty((Cc, R // 2), **u8), "col_scales": torch.empty((Cc, R // 16), **u8),
           "amax": torch.empty(2, dtype=torch.float32, device=dev),
           "s_enc": torch.empty(2, dtype=torch.float32, device=dev)}
    ws = _workspace(workspace, NVFP4_QUANTIZE_WORKSPACE_BYTES, dev)
    sg = _signs(rht_signs, dev)
    _check("nvfp4_quantize_fprop_wgrad", lib().nvfp4_quantize_fprop_wgrad(
        x.data_ptr(), R, Cc, rounding, sr_seed & (2 ** 64 - 1), sr_stream, _ptr(sg), out["row_codes"].data_ptr(),
        out["row_scales"].data_ptr(), out["col_codes"].data_ptr(), out["col_scales"].data_ptr(),
        out["amax"].data_ptr(), out["s_enc"].data_ptr(), ws.data_ptr(), _stream(dev)))
    return out


def nvfp4_col_mxfp8_row_quantize(x: torch.Tensor, rounding: int = RNE, sr_seed: int = 0, sr_stream: int = 0,
                                 rht_signs=None, mx_slab: bool = False,
                                 workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """One pass over a bf16 [rows, cols] device tensor that writes NVFP4 columnwise (as
    ``nvfp4_quantize(x, COL, ...)``: ``col_codes``, ``col_scales``, ``amax``, ``s_enc``) and
    MXFP8 rowwise (as ``mxfp8_quantize(x, ROW | (MX_SLAB if mx_slab else 0))``:
    ``mx_row_codes``, ``mx_row_scales``).  RHT and SR apply to the NVFP4 part only."""
    _dev_tensor(x, torch.bfloat16, "x")
    R, Cc = x.shape
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    out = {"col_codes": torch.empty((Cc, R // 2), **u8), "col_scales": torch.empty((Cc, R // 16), **u8),
           "amax": torch.empty(2, dtype=torch.float32, device=dev),
           "s_enc": torch.empty(2, dtype=torch.float32, device=dev),
           "mx_row_codes": torch.empty((R, Cc), **u8), "mx_row_scales": torch.empty((R, Cc // 32), **u8)}
    ws = _workspace(workspace, NVFP4_QUANTIZE_WORKSPACE_BYTES, dev)
    sg = _signs(rht_signs, dev)
    _check("nvfp4_col_mxfp8_row_quantize", lib().nvfp4_col_mxfp8_row_quantize(
        x.data_ptr(), R, Cc, rounding, sr_seed & (2 ** 64 - 1), sr_stream, _ptr(sg), out["col_codes"].data_ptr(),
        out["col_scales"].data_ptr(), out["amax"].data_ptr(), out["s_enc"].data_ptr(), ws.data_ptr(),
        MX_SLAB if mx_slab else 0, out["mx_row_codes"].data_ptr(), out["mx_row_scales"].data_ptr(),
        _stream(dev)))
    return out


def nvfp4_quantize_rowscaled(x: torch.Tensor, rounding: int = RNE, sr_seed: int = 0, sr_stream: int = 0,
                             rht_signs=None) -> Dict[str, torch.Tensor]:
    """Rowwise NVFP4 with one outer scale per row.  Returns ``codes`` [rows, cols/2],
    ``scales`` [rows, cols/16] (uint8), ``amax`` and ``s_enc`` (float32[rows])."""
    _dev_tensor(x, torch.bfloat16, "x")
    R, Cc = x.shape
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    out = {"codes": torch.empty((R, Cc // 2), **u8), "scales": torch.empty((R, Cc // 16), **u8),
           "amax": torch.empty(R, dtype=torch.float32, device=dev),
           "s_enc": torch.empty(R, dtype=torch.float32, device=dev)}
    sg = _signs(rht_signs, dev)
    _check("nvfp4_quantize_rowscaled", lib().nvfp4_quantize_rowscaled(
        x.data_ptr(), R, Cc, rounding, sr_seed & (2 ** 64 - 1), sr_stream, _ptr(sg), out["codes"].data_ptr(),
        out["scales"].data_ptr(), out["amax"].data_ptr(), out["s_enc"].data_ptr(), _stream(dev)))
    return out


def nvfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, s_enc: torch.Tensor) -> torch.Tensor:
    """bf16 [rows, cols] value of NVFP4 codes [rows, cols/2] with scales [rows, cols/16] and
    tensor scale ``s_enc`` (a 1-element float32 device tensor)."""
    _dev_tensor(codes, torch.uint8, "codes")
    _dev_tensor(scales, torch.uint8, "scales")
    _dev_tensor(s_enc, torch.float32, "s_enc")
    rows, half = codes.shape
    out = torch.empty((rows, half * 2), dtype=torch.bfloat16, device=codes.device)
    _check("nvfp4_dequantize", lib().nvfp4_dequantize(codes.data_ptr(), scales.data_ptr(), s_enc.data_ptr(),
                                                      rows, half * 2, out.data_ptr(), _stream(codes.device)))
    return out


def mxfp8_quantize(x: torch.Tensor, direction: int = ROW) -> Dict[str, torch.Tensor]:
    """MXFP8-cast a bf16 [rows, cols] device tensor (E4M3 codes, E8M0 scale per 32)."""
    _dev_tensor(x, torch.bfloat16, "x")
    R, Cc = x.shape
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    out: Dict[str, torch.Tensor] = {}
    if direction & ROW:
        out["row_codes"] = torch.empty((R, Cc), **u8)
        out["row_scales"] = torch.empty((R, Cc // 32), **u8)
    if direction & COL:
        out["col_codes"] = torch.empty((Cc, R), **u8)
        out["col_scales"] = torch.empty((Cc, R // 32), **u8)
    _check("mxfp8_quantize", lib().mxfp8_quantize(
        x.data_ptr(), R, Cc, direction, _ptr(out.get("row_codes")), _ptr(out.get("row_scales")),
        _ptr(out.get("col_codes")), _ptr(out.get("col_scales")), _stream(dev)))
    return out


def mxfp8_requantize_nvfp4(codes: torch.Tensor, scales: torch.Tensor, s_enc: torch.Tensor,
                           direction: int = COL) -> Dict[str, torch.Tensor]:
    """MXFP8 cast of the rowwise-dequantized value of an NVFP4 rowwise tensor (``codes``
    [rows, cols/2], ``scales`` [rows, cols/16], 1-element float32 ``s_enc``), without the
    bf16 intermediate; bit-identical to ``mxfp8_quantize(nvfp4_dequantize(...))``."""
    _dev_tensor(codes, torch.uint8, "codes")
    _dev_tensor(scales, torch.uint8, "scales")
    _dev_tensor(s_enc, torch.float32, "s_enc")
    R, Cc = codes.shape[0], codes.shape[1] * 2
    if tuple(scales.shape) != (R, Cc // 16):
        raise ValueError("scales must be [rows, cols/16]")
    dev = codes.device
    u8 = dict(dtype=torch.uint8, device=dev)
    out: Dict[str, torch.Tensor] = {}
    if direction & ROW:
        out["row_codes"] = torch.empty((R, Cc), **u8)
        out["row_scales"] = torch.empty((R, Cc // 32), **u8)
    if direction & COL:
        out["col_codes"] = torch.empty((Cc, R), **u8)
        out["col_scales"] = torch.empty((Cc, R // 32), **u8)
    _check("mxfp8_requantize_nvfp4", lib().mxfp8_requantize_nvfp4(
        codes.data_ptr(), scales.data_ptr(), s_enc.data_ptr(), R, Cc, direction, _ptr(out.get("row_codes")),
        _ptr(out.get("row_scales")), _ptr(out.get("col_codes")), _ptr(out.get("col_scales")), _stream(dev)))
    return out


def rht_apply(x: torch.Tensor, axis: int, rht_signs) -> torch.Tensor:
    """float32 16-point random Hadamard transform of a bf16 tensor along ``axis``."""
    _dev_tensor(x, torch.bfloat16, "x")
    R, Cc = x.shape
    sg = _signs(rht_signs, x.device)
    out = torch.empty((R, Cc), dtype=torch.float32, device=x.device)
    _check("rht_apply", lib().rht_apply(x.data_ptr(), R, Cc, axis, sg.data_ptr(), out.data_ptr(),
                                        _stream(x.device)))
    return out


def blockscaled_gemm(fmt: int, a_codes: torch.Tensor, a_scales: torch.Tensor, a_s_enc: Optional[torch.Tensor],
                     b_codes: torch.Tensor, b_scales: torch.Tensor, b_s_enc: Optional[torch.Tensor],
                     out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C[M, N] = A[M, K] B[N, K]^T on NVFP4 (fmt 0) or MXFP8 (fmt 1) operands, fp32 accumulate.
    ``fmt`` may carry FMT_A_ROWSCALED / FMT_B_ROWSCALED (NVFP4): that operand's ``s_enc`` then
    holds one float per row."""
    _dev_tensor(a_codes, torch.uint8, "a_codes")
    _dev_tensor(b_codes, torch.uint8, "b_codes")
    _dev_tensor(a_scales, torch.uint8, "a_scales")
    _dev_tensor(b_scales, torch.uint8, "b_scales")
    M, N = a_codes.shape[0], b_codes.shape[0]
    base = fmt & ~(FMT_A_ROWSCALED | FMT_B_ROWSCALED)
    K = a_codes.shape[1] * (2 if base == FMT_NVFP4 else 1)
    for flag, t, n, name in ((FMT_A_ROWSCALED, a_s_enc, M, "a_s_enc"), (FMT_B_ROWSCALED, b_s_enc, N, "b_s_enc")):
        if base == FMT_NVFP4 and t is not None:
            _dev_tensor(t, torch.float32, name)
            want = n if fmt & flag else 1
            if t.numel() < want:
                raise ValueError("%s has %d entries, needs %d" % (name, t.numel(), want))
    if b_codes.shape[1] != a_codes.shape[1]:
        raise ValueError("operands disagree on K")
    c_dtype = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}[out_dtype]
    if out is None:
        c = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    else:
        c = _dev_tensor(out, out_dtype, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (M, N)))
    _check("blockscaled_gemm", lib().blockscaled_gemm(
        fmt, M, N, K, a_codes.data_ptr(), a_scales.data_ptr(), _ptr(a_s_enc), b_codes.data_ptr(),
        b_scales.data_ptr(), _ptr(b_s_enc), c.data_ptr(), c_dtype, _stream(a_codes.device)))
    _written(out)
    return c


def blockscaled_grouped_gemm(fmt: int, mode: int, offsets: torch.Tensor, a_codes: torch.Tensor,
                             a_scales: torch.Tensor, a_s_enc: Optional[torch.Tensor], b_codes: torch.Tensor,
                             b_scales: torch.Tensor, b_s_enc: Optional[torch.Tensor],
                             out_dtype: torch.dtype = torch.bfloat16,
                             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One block-scaled GEMM per group; ``offsets`` is an int64 device tensor of groups + 1
    boundaries.  GROUP_M: A [M, K] (rows grouped), B [groups, N, K] (codes as [groups, N,
    K/2] or [groups * N, K/2] for NVFP4), C [M, N] (rows outside every group untouched).
    GROUP_K: A [M, K] and B [N, K] grouped along K, C [groups, M, N]."""
    _dev_tensor(offsets, torch.int64, "offsets")
    for t, nm in ((a_codes, "a_codes"), (b_codes, "b_codes"), (a_scales, "a_scales"), (b_scales, "b_scales")):
        _dev_tensor(t, torch.uint8, nm)
    for t, nm in ((a_s_enc, "a_s_enc"), (b_s_enc, "b_s_enc")):
        if t is not None:
            _dev_tensor(t, torch.float32, nm)
    G = offsets.numel() - 1
    if G < 0:
        raise ValueError("offsets needs groups + 1 entries")
    base = fmt & ~(FMT_A_ROWSCALED | FMT_B_ROWSCALED)
    epb = 2 if base == FMT_NVFP4 else 1
    M, K = a_codes.shape[0], a_codes.shape[-1] * epb
    if mode == GROUP_M:
        N = b_codes.shape[-2] if b_codes.dim() == 3 else (b_codes.shape[0] // G if G else 0)
        shape = (M, N)
    else:
        N = b_codes.shape[0]
        shape = (G, M, N)
    if b_codes.shape[-1] * epb != K:
        raise ValueError("operands disagree on K")
    c_dtype = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}[out_dtype]
    if out is None:
        c = torch.empty(shape, dtype=out_dtype, device=a_codes.device)
    else:
        c = _dev_tensor(out, out_dtype, "out")
        if tuple(out.shape) != shape:
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), shape))
    _check("blockscaled_grouped_gemm", lib().blockscaled_grouped_gemm(
        fmt, mode, G, offsets.data_ptr(), M, N, K, a_codes.data_ptr(), a_scales.data_ptr(), _ptr(a_s_enc),
        b_codes.data_ptr(), b_scales.data_ptr(), _ptr(b_s_enc), c.data_ptr(), c_dtype, _stream(a_codes.device)))
    _written(out)
    return c


def nvfp4_linear_forward(x: torch.Tensor, w: torch.Tensor, sr_seed: int, rht_signs,
                         workspace: Optional[torch.Tensor] = None):
    """NVFP4 linear forward: returns (y [T, N] bf16, saved) where ``saved`` (a uint8 device
    tensor) holds the quantized activation that nvfp4_linear_backward needs."""
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(w, torch.bfloat16, "w")
    T, K = x.shape
    N = w.shape[0]
    dev = x.device
    L = lib()
    saved = torch.empty(L.nvfp4_linear_saved_bytes(T, K), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = torch.empty(L.nvfp4_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device=dev)
    y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    sg = _signs(rht_signs, dev)
    _check("nvfp4_linear_forward", L.nvfp4_linear_forward(
        x.data_ptr(), w.data_ptr(), T, K, N, sr_seed & (2 ** 64 - 1), sg.data_ptr(), saved.data_ptr(),
        workspace.data_ptr(), y.data_ptr(), _stream(dev)))
    return y, saved


def nvfp4_linear_backward(dy: torch.Tensor, w: torch.Tensor, saved: torch.Tensor, sr_seed: int, rht_signs,
                          workspace: Optional[torch.Tensor] = None):
    """NVFP4 linear backward: returns (dx [T, K] bf16, dw [N, K] fp32)."""
    _dev_tensor(dy, torch.bfloat16, "dy")
    _dev_tensor(w, torch.bfloat16, "w")
    _dev_tensor(saved, torch.uint8, "saved")
    T, N = dy.shape
    K = w.shape[1]
    dev = dy.device
    L = lib()
    if saved.numel() < L.nvfp4_linear_saved_bytes(T, K):
        raise ValueError("saved buffer is too small for this layer")
    if workspace is None:
        workspace = torch.empty(L.nvfp4_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device=dev)
    dx = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
    dw = torch.empty((N, K), dtype=torch.float32, device=dev)
    sg = _signs(rht_signs, dev)
    _check("nvfp4_linear_backward", L.nvfp4_linear_backward(
        dy.data_ptr(), w.data_ptr(), saved.data_ptr(), T, K, N, sr_seed & (2 ** 64 - 1), sg.data_ptr(),
        workspace.data_ptr(), dx.data_ptr(), dw.data_ptr(), _stream(dev)))
    return dx, dw


# ---------------------------------------------------------------- a few tokens on NVFP4 weights

def _tokens(x: torch.Tensor):
    """x [M, K] bf16 on the device, its elements of a token adjacent; returns (M, K, elements between tokens)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA/HIP tensor")
    if x.dtype != torch.bfloat16:
        raise TypeError("x must have dtype torch.bfloat16, got %s" % x.dtype)
    if x.dim() != 2:
        raise ValueError("x must be [tokens, K]")
    M, K = x.shape
    if K > 1 and x.stride(1) != 1:
        raise ValueError("x must have adjacent elements along K")
    return M, K, x.stride(0) if M > 1 else -(-K // 8) * 8


def _weights(codes: torch.Tensor, scales: torch.Tensor, s_enc: torch.Tensor, K: int, name: str, dev):
    """An NVFP4 weight's checks against K; returns (rows, whether its scale is per row)."""
    _dev_tensor(codes, torch.uint8, name + "_codes")
    _dev_tensor(scales, torch.uint8, name + "_scales")
    _dev_tensor(s_enc, torch.float32, name + "_s_enc")
    N = codes.shape[0]
    if codes.dim() != 2 or codes.shape[1] * 2 != K:
        raise ValueError("%s_codes must be [rows, K/2] with K = %d, got %s" % (name, K, tuple(codes.shape)))
    if tuple(scales.shape) != (N, K // 16):
        raise ValueError("%s_scales must be [rows, K/16], got %s" % (name, tuple(scales.shape)))
    n = s_enc.numel()
    if n != 1 and n != N:
        raise ValueError("%s_s_enc must hold 1 value or one per row, got %d" % (name, n))
    if codes.device != dev or scales.device != dev or s_enc.device != dev:
        raise ValueError("%s and x must be on one device" % name)
    return N, n != 1


def nvfp4_matvec(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, w_s_enc: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] (bf16, a few tokens; tokens may be strided) times NVFP4 weights [N, K] transposed: y [M, N] in
    ``out_dtype`` (bf16 or float32).  ``w_s_enc`` holds the weight's tensor scale, or one per row."""
    M, K, ldx = _tokens(x)
    dev = x.device
    N, rows = _weights(w_codes, w_scales, w_s_enc, K, "w", dev)
    y_dtype = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}[out_dtype]
    y = _output(out, (M, N), out_dtype, dev)
    _check("nvfp4_matvec", lib().nvfp4_matvec(
        FMT_B_ROWSCALED if rows else 0, M, N, K, x.data_ptr(), ldx, w_codes.data_ptr(), w_scales.data_ptr(),
        w_s_enc.data_ptr(), y.data_ptr(), y_dtype, _stream(dev)))
    _written(out)
    return y


def nvfp4_gated_matvec(act: int, x: torch.Tensor, gate_codes: torch.Tensor, gate_scales: torch.Tensor,
                       gate_s_enc: torch.Tensor, up_codes: torch.Tensor, up_scales: torch.Tensor,
                       up_s_enc: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(x Wg^T) * (x Wu^T) for a few bf16 tokens x [M, K] and NVFP4 weights [F, K], in one kernel: h [M, F]
    bf16.  ``act`` is ACT_SILU, ACT_GELU or ACT_GELU_TANH; both s_enc hold one tensor scale, or one per row."""
    M, K, ldx = _tokens(x)
    dev = x.device
    F, rows = _weights(gate_codes, gate_scales, gate_s_enc, K, "gate", dev)
    Fu, urows = _weights(up_codes, up_scales, up_s_enc, K, "up", dev)
    if Fu != F or urows != rows:
        raise ValueError("gate and up must agree in rows and in the kind of their tensor scales")
    h = _output(out, (M, F), torch.bfloat16, dev)
    _check("nvfp4_gated_matvec", lib().nvfp4_gated_matvec(
        FMT_B_ROWSCALED if rows else 0, act, M, F, K, x.data_ptr(), ldx, gate_codes.data_ptr(),
        gate_scales.data_ptr(), gate_s_enc.data_ptr(), up_codes.data_ptr(), up_scales.data_ptr(),
        up_s_enc.data_ptr(), h.data_ptr(), _stream(dev)))
    _written(out)
    return h


# ---------------------------------------------------------------- the gated block's products

def _operand(fmt: int, rowscaled: int, codes: torch.Tensor, scales: torch.Tensor, s_enc: Optional[torch.Tensor],
             name: str, dev):
    """A quantized operand's checks; returns (rows, K)."""
    _dev_tensor(codes, torch.uint8, name + "_codes")
    _dev_tensor(scales, torch.uint8, name + "_scales")
    nv = (fmt & 0xF) == FMT_NVFP4
    if codes.dim() != 2:
        raise ValueError("%s_codes must have two dimensions" % name)
    rows, K = codes.shape[0], codes.shape[1] * (2 if nv else 1)
    if tuple(scales.shape) != (rows, K // (16 if nv else 32)):
        raise ValueError("%s_scales has shape %s for codes %s" % (name, tuple(scales.shape), tuple(codes.shape)))
    if codes.device != dev or scales.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))
    if nv:
        _dev_tensor(s_enc, torch.float32, name + "_s_enc")
        want = rows if fmt & rowscaled else 1
        if s_enc.numel() != want or s_enc.device != dev:
            raise ValueError("%s_s_enc must hold %d values on %s" % (name, want, dev))
    return rows, K


def blockscaled_gated_gemm(fmt: int, act: int, a_codes: torch.Tensor, a_scales: torch.Tensor,
                           a_s_enc: Optional[torch.Tensor], gate_codes: torch.Tensor, gate_scales: torch.Tensor,
                           gate_s_enc: Optional[torch.Tensor], up_codes: torch.Tensor, up_scales: torch.Tensor,
                           up_s_enc: Optional[torch.Tensor], save_gate_up: bool = False,
                           out: Optional[torch.Tensor] = None, gate_up: Optional[torch.Tensor] = None):
    """h = act(A Wg^T) * (A Wu^T) on NVFP4 or MXFP8 operands (``fmt`` and its flags as for ``blockscaled_gemm``; the
    ``_B`` flags apply to both weights): h [M, F] bf16, or with ``save_gate_up`` (h, gate_up) where gate_up
    [M, 2F] bf16 holds both projections for ``blockscaled_gated_gemm_backward``.  ``out`` and ``gate_up`` are
    tensors to write to; new ones are made when none are given."""
    _dev_tensor(a_codes, torch.uint8, "a_codes")
    dev = a_codes.device
    M, K = _operand(fmt, FMT_A_ROWSCALED, a_codes, a_scales, a_s_enc, "a", dev)
    gate = _operand(fmt, FMT_B_ROWSCALED, gate_codes, gate_scales, gate_s_enc, "gate", dev)
    up = _operand(fmt, FMT_B_ROWSCALED, up_codes, up_scales, up_s_enc, "up", dev)
    if gate != up or gate[1] != K:
        raise ValueError("operands disagree: a [%d, %d], gate %s, up %s" % (M, K, list(gate), list(up)))
    F = gate[0]
    h, gu = _output(out, (M, F), torch.bfloat16, dev), None
    if save_gate_up:
        gu = _output(gate_up, (M, 2 * F), torch.bfloat16, dev)
    elif gate_up is not None:
        raise ValueError("gate_up is written with save_gate_up only")
    _check("blockscaled_gated_gemm", lib().blockscaled_gated_gemm(
        fmt, act, M, F, K, a_codes.data_ptr(), a_scales.data_ptr(), _ptr(a_s_enc), gate_codes.data_ptr(),
        gate_scales.data_ptr(), _ptr(gate_s_enc), up_codes.data_ptr(), up_scales.data_ptr(), _ptr(up_s_enc),
        h.data_ptr(), _ptr(gu), _stream(dev)))
    _written(out, gate_up)
    return (h, gu) if save_gate_up else h


def blockscaled_gated_gemm_backward(fmt: int, act: int, dy_codes: torch.Tensor, dy_scales: torch.Tensor,
                                    dy_s_enc: Optional[torch.Tensor], w_codes: torch.Tensor, w_scales: torch.Tensor,
                                    w_s_enc: Optional[torch.Tensor], gate_up: torch.Tensor,
                                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient [M, 2F] bf16 of ``blockscaled_gated_gemm``'s gate_up from the output gradient dY [M, K] and the
    down projection's weight [F, K] (both along the block's output): dh = dY Wd^T, d_gate = dh u act'(g),
    d_up = dh act(g).  ``out`` may be ``gate_up`` itself."""
    _dev_tensor(dy_codes, torch.uint8, "dy_codes")
    dev = dy_codes.device
    M, K = _operand(fmt, FMT_A_ROWSCALED, dy_codes, dy_scales, dy_s_enc, "dy", dev)
    F, Kw = _operand(fmt, FMT_B_ROWSCALED, w_codes, w_scales, w_s_enc, "w", dev)
    if Kw != K:
        raise ValueError("operands disagree on K: dy %d, w %d" % (K, Kw))
    _dev_tensor(gate_up, torch.bfloat16, "gate_up")
    if tuple(gate_up.shape) != (M, 2 * F) or gate_up.device != dev:
        raise ValueError("gate_up must be [%d, %d] on %s, got %s" % (M, 2 * F, dev, tuple(gate_up.shape)))
    d = _output(out, (M, 2 * F), torch.bfloat16, dev)
    _check("blockscaled_gated_gemm_backward", lib().blockscaled_gated_gemm_backward(
        fmt, act, M, F, K, dy_codes.data_ptr(), dy_scales.data_ptr(), _ptr(dy_s_enc), w_codes.data_ptr(),
        w_scales.data_ptr(), _ptr(w_s_enc), gate_up.data_ptr(), d.data_ptr(), _stream(dev)))
    _written(out)
    return d


def _output(out: Optional[torch.Tensor], shape, dtype, dev) -> torch.Tensor:
    """The caller's output tensor (checked), or a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _dev_tensor(out, dtype, "out")
    if tuple(out.shape) != shape:
        raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), shape))
    if out.device != dev:
        raise ValueError("out must be on %s" % (dev,))
    return out


# ---------------------------------------------------------------- gradient clipping

_GRAD_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_dtype_of = attrgetter("dtype")


def _list_check(tensors: list, name: str, dev):
    """Explains what is wrong with a list of gradients (only called when something is)."""
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s %d must be a tensor" % (name, i))
        if not t.is_cuda or t.device != dev:
            raise ValueError("%s %d must be on %s, a GPU" % (name, i, dev))
        if t.dtype not in _GRAD_DTYPES:
            raise TypeError("%s %d must be bfloat16 or float32, got %s" % (name, i, t.dtype))
        if not t.is_contiguous():
            raise ValueError("%s %d must be contiguous" % (name, i))


class _GradList:
    """A list of gradients (and outputs) as the C ABI's host arrays.  Models have hundreds of them, so each
    property is taken over the whole list at once."""

    def __init__(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None):
        grads = list(grads)
        if not grads:
            raise ValueError("the list of gradients is empty")
        dev = getattr(grads[0], "device", None)
        self.ptrs, self.numels, self.dtypes = self._arrays(grads, "gradient", dev)
        self.outs = None
        if out is not None:
            out = list(out)
            if len(out) != len(grads):
                raise ValueError("out has %d tensors for %d gradients" % (len(out), len(grads)))
            self.outs, numels, dtypes = self._arrays(out, "out", dev)
            if numels != self.numels or dtypes != self.dtypes:
                i = next(i for i in range(len(out)) if numels[i] != self.numels[i] or dtypes[i] != self.dtypes[i])
                raise ValueError("out[%d] must have its gradient's type and number of elements" % i)
        self.n, self.device, self.written = len(grads), dev, grads if out is None else out

    @staticmethod
    def _arrays(tensors: list, name: str, dev):
        try:
            kinds = array("i", map(_GRAD_DTYPES.__getitem__, map(_dtype_of, tensors)))
            good = (dev.type == "cuda" and set(map(torch.Tensor.get_device, tensors)) == {dev.index}
                    and all(map(torch.Tensor.is_contiguous, tensors)))
        except (AttributeError, KeyError, TypeError):
            good = False
        if not good:
            _list_check(tensors, name, dev)
        return array("Q", map(torch.Tensor.data_ptr, tensors)), array("q", map(torch.Tensor.numel, tensors)), kinds

    def args(self, outs: bool = True):
        at = lambda a: None if a is None else a.buffer_info()[0]   # noqa: E731
        return (at(self.ptrs), *((at(self.outs),) if outs else ()), at(self.numels), at(self.dtypes), self.n)

    def workspace(self, workspace: Optional[torch.Tensor]) -> torch.Tensor:
        return _workspace(workspace, lib().grad_workspace_bytes(self.n), self.device)


def grad_sumsq(grads: Sequence[torch.Tensor], workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The sum of squares over all gradients (contiguous bf16 and float32 tensors) as a float64[1] device tensor; ranks
    that hold different gradients add theirs up before ``grad_clip``."""
    g = _GradList(grads)
    ws = g.workspace(workspace)
    sumsq = torch.empty(1, dtype=torch.float64, device=g.device)
    _check("grad_sumsq", lib().grad_sumsq(*g.args(False), sumsq.data_ptr(), ws.data_ptr(), _stream(g.device)))
    return sumsq


def grad_clip(grads: Sequence[torch.Tensor], sumsq: torch.Tensor, max_norm: float,
              out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (sqrt(sumsq) + 1e-6)), in place or into ``out`` (tensors of the
    gradients' types and sizes); returns the norm as a float32[1] device tensor."""
    g = _GradList(grads, out)
    _dev_tensor(sumsq, torch.float64, "sumsq")
    if sumsq.numel() != 1 or sumsq.device != g.device:
        raise ValueError("sumsq must hold one value on %s" % (g.device,))
    norm = torch.empty(1, dtype=torch.float32, device=g.device)
    _check("grad_clip", lib().grad_clip(*g.args(), sumsq.data_ptr(), max_norm, norm.data_ptr(), _stream(g.device)))
    torch.autograd.graph.increment_version(g.written)   # as _written
    return norm


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradients' global 2-norm (float32[1], on the device), and the gradients scaled so that it does not
    exceed ``max_norm``, in place or into ``out``.  The tensors are contiguous bf16 or float32.  ``workspace``: at least grad_workspace_bytes(len(grads))
    bytes of scratch; one is allocated when none is given."""
    g = _GradList(grads, out)
    ws = g.workspace(workspace)
    norm = torch.empty(1, dtype=torch.float32, device=g.device)
    _check("clip_grad_norm", lib().clip_grad_norm(*g.args(), max_norm, norm.data_ptr(), ws.data_ptr(),
                                                  _stream(g.device)))
    torch.autograd.graph.increment_version(g.written)   # as _written
    return norm


# ---------------------------------------------------------------- tokens and their experts

_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # the former without its Python around it


def _call(fn: str, dev, *args):
    """The C entry point on dev's current stream, which may belong to another device than the current one."""
    f = getattr(lib(), fn)
    if dev.index == _get_device():
        _check(fn, f(*args, _stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(fn, f(*args, _stream(dev)))


_TYPES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def _type(dtype: torch.dtype, name: str) -> int:
    if dtype not in _TYPES:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, dtype))
    return _TYPES[dtype]


def _on(t: torch.Tensor, dev, name: str):
    if t.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))


def _rows(x: torch.Tensor, dtype, name: str):
    """x [rows, columns] of a type with adjacent elements in a row; returns (rows, columns, elements between rows)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("%s must be a CUDA/HIP tensor" % name)
    if dtype is not None and x.dtype != dtype:
        raise TypeError("%s must have dtype %s, got %s" % (name, dtype, x.dtype))
    if x.dim() != 2:
        raise ValueError("%s must have two dimensions" % name)
    R, C_ = x.shape
    if C_ > 1 and x.stride(1) != 1:
        raise ValueError("%s must have adjacent elements in a row" % name)
    return R, C_, x.stride(0) if R > 1 else -(-C_ // 8) * 8


def _slots(positions: torch.Tensor, T: int, dev) -> int:
    """positions [T, k]; returns k."""
    _dev_tensor(positions, torch.int32, "positions")
    _on(positions, dev, "positions")
    if positions.dim() != 2 or positions.shape[0] != T:
        raise ValueError("positions must be [%d, k], got %s" % (T, tuple(positions.shape)))
    return positions.shape[1]


def _source(source: torch.Tensor, dev) -> int:
    _dev_tensor(source, torch.int32, "source")
    _on(source, dev, "source")
    if source.dim() != 1:
        raise ValueError("source must have one dimension")
    return source.shape[0]


def moe_sort(experts: torch.Tensor, num_experts: int, align: int = 1,
             workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """The order of token slots by expert for ``blockscaled_grouped_gemm``.  ``experts`` [T, k] (int32 or int64) holds each
    slot's expert; slots with ids outside [0, num_experts) are dropped.  Returns ``offsets`` (int64
    [num_experts + 1], each group starting at a multiple of ``align``; GROUP_K needs 32), ``positions`` (int32 [T, k], a
    slot's row or -1) and ``source`` (int32 [rows], a row's slot t k + j or -1), where rows holds any choice of
    experts.  ``workspace``: lib().moe_sort_workspace_bytes(T k, num_experts) bytes of scratch; one is allocated when
    none is given."""
    if not isinstance(experts, torch.Tensor) or experts.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts must be an int32 or int64 tensor")
    _dev_tensor(experts, experts.dtype, "experts")
    if experts.dim() != 2:
        raise ValueError("experts must be [tokens, k]")
    dev, n, L = experts.device, experts.numel(), lib()
    rows, need = L.moe_sort_rows(n, num_experts, align), L.moe_sort_workspace_bytes(n, num_experts)
    ws = _workspace(workspace, need, dev) if need > 0 or workspace is not None else None   # few slots need none
    offsets = torch.empty(max(num_experts, 0) + 1, dtype=torch.int64, device=dev)
    positions = torch.empty_like(experts, dtype=torch.int32)
    source = torch.empty(max(rows, 0), dtype=torch.int32, device=dev)
    _call("moe_sort", dev, experts.data_ptr(), experts.element_size(), n, num_experts, align, rows, offsets.data_ptr(),
          positions.data_ptr(), source.data_ptr(), _ptr(ws))
    return {"offsets": offsets, "positions": positions, "source": source}


def moe_gather(x: torch.Tensor, positions: torch.Tensor, source: torch.Tensor,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Tokens x [T, H] (bf16; rows may be strided) in the order of ``moe_sort``: [rows, H] bf16, zeros in rows without a
    token.  Its gradient is ``moe_combine(d, positions)``."""
    T, H, ldx = _rows(x, torch.bfloat16, "x")
    dev = x.device
    k, R = _slots(positions, T, dev), _source(source, dev)
    xs = _output(out, (R, H), torch.bfloat16, dev)
    _call("moe_gather", dev, T, k, H, x.data_ptr(), ldx, positions.data_ptr(), source.data_ptr(), R, xs.data_ptr())
    _written(out)
    return xs


def moe_gather_nvfp4_rowscaled(x: torch.Tensor, positions: torch.Tensor, source: torch.Tensor) -> Dict[str, torch.Tensor]:
    """``nvfp4_quantize_rowscaled(moe_gather(x, positions, source))`` without the copy in between: ``codes`` [rows, H/2],
    ``scales`` [rows, H/16] (uint8) and ``s_enc`` (float32[rows])."""
    T, H, ldx = _rows(x, torch.bfloat16, "x")
    dev = x.device
    k, R = _slots(positions, T, dev), _source(source, dev)
    u8 = dict(dtype=torch.uint8, device=dev)
    out = {"codes": torch.empty((R, H // 2), **u8), "scales": torch.empty((R, H // 16), **u8),
           "s_enc": torch.empty(R, dtype=torch.float32, device=dev)}
    _call("moe_gather_nvfp4_rowscaled", dev, T, k, H, x.data_ptr(), ldx, positions.data_ptr(), source.data_ptr(), R,
          out["codes"].data_ptr(), out["scales"].data_ptr(), out["s_enc"].data_ptr())
    return out


def moe_gather_mxfp8(x: torch.Tensor, positions: torch.Tensor, source: torch.Tensor) -> Dict[str, torch.Tensor]:
    """``mxfp8_quantize(moe_gather(x, positions, source))`` without the copy in between: ``row_codes`` [rows, H],
    ``row_scales`` [rows, H/32] (uint8); equal for finite values.  A value that is not finite becomes the NaN code under
    the scale byte 247, where the cast's codes of its block depend on the blocks beside it."""
    T, H, ldx = _rows(x, torch.bfloat16, "x")
    dev = x.device
    k, R = _slots(positions, T, dev), _source(source, dev)
    u8 = dict(dtype=torch.uint8, device=dev)
    out = {"row_codes": torch.empty((R, H), **u8), "row_scales": torch.empty((R, H // 32), **u8)}
    _call("moe_gather_mxfp8", dev, T, k, H, x.data_ptr(), ldx, positions.data_ptr(), source.data_ptr(), R,
          out["row_codes"].data_ptr(), out["row_scales"].data_ptr())
    return out


def _slot_weights(weights: Optional[torch.Tensor], positions: torch.Tensor):
    if weights is None:
        return
    _dev_tensor(weights, torch.float32, "weights")
    if weights.shape != positions.shape or weights.device != positions.device:
        raise ValueError("weights must be %s on %s" % (tuple(positions.shape), positions.device))


def moe_combine(y: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts' rows y [rows, H] (bf16 or float32) back to their tokens: out[t] = sum_j weights[t, j] y[positions[t, j]]
    (fp32, rounded once) as [T, H] of ``out_dtype`` (bf16 or float32).  ``weights`` [T, k] float32, or None for ones.  Its
    gradients: ``moe_combine_backward``, without weights ``moe_gather(dout, ...)``; both take dout in bf16."""
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a tensor")
    yt = _type(y.dtype, "y")
    _dev_tensor(y, y.dtype, "y")
    if y.dim() != 2:
        raise ValueError("y must be [rows, H]")
    dev, (R, H) = y.device, y.shape
    if not isinstance(positions, torch.Tensor) or positions.dim() != 2:
        raise ValueError("positions must be [tokens, k]")
    T = positions.shape[0]
    k = _slots(positions, T, dev)
    _slot_weights(weights, positions)
    ot = _type(out_dtype, "out_dtype")
    sums = _output(out, (T, H), out_dtype, dev)
    _call("moe_combine", dev, T, k, H, y.data_ptr(), yt, R, positions.data_ptr(), _ptr(weights), sums.data_ptr(), ot)
    _written(out)
    return sums


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, positions: torch.Tensor, source: torch.Tensor,
                         weights: torch.Tensor):
    """The gradients of ``moe_combine`` for dout [T, H] (bf16): (dy [rows, H] of y's type, zeros in rows without a token;
    dweights [T, k] float32, 0 for dropped slots)."""
    _dev_tensor(dout, torch.bfloat16, "dout")
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a tensor")
    yt = _type(y.dtype, "y")
    _dev_tensor(y, y.dtype, "y")
    if dout.dim() != 2 or y.dim() != 2 or dout.shape[1] != y.shape[1]:
        raise ValueError("dout must be [T, H] and y [rows, H], got %s and %s" % (tuple(dout.shape), tuple(y.shape)))
    dev, (T, H) = dout.device, dout.shape
    _on(y, dev, "y")
    k, R = _slots(positions, T, dev), _source(source, dev)
    if y.shape[0] != R:
        raise ValueError("y has %d rows, source %d" % (y.shape[0], R))
    _slot_weights(weights, positions)
    if weights is None:
        raise TypeError("weights must be a tensor")
    dy = torch.empty_like(y)
    dw = torch.empty_like(weights)
    _call("moe_combine_backward", dev, T, k, H, dout.data_ptr(), y.data_ptr(), yt, R, positions.data_ptr(),
          source.data_ptr(), weights.data_ptr(), dy.data_ptr(), dw.data_ptr())
    return dy, dw


# ---------------------------------------------------------------- low-rank adapters

def _adapters(adapters: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor, scales: Optional[torch.Tensor], M: int,
              N: int, K: int, dev):
    """The adapters' checks; returns (rank, number of adapters)."""
    _dev_tensor(adapters, torch.int32, "adapters")
    _dev_tensor(lora_a, torch.bfloat16, "lora_a")
    _dev_tensor(lora_b, torch.bfloat16, "lora_b")
    if tuple(adapters.shape) != (M,):
        raise ValueError("adapters must hold one id per token, got %s" % (tuple(adapters.shape),))
    if lora_a.dim() != 3 or lora_a.shape[2] != K:
        raise ValueError("lora_a must be [adapters, rank, %d], got %s" % (K, tuple(lora_a.shape)))
    n, r = lora_a.shape[0], lora_a.shape[1]
    if tuple(lora_b.shape) != (n, N, r):
        raise ValueError("lora_b must be [%d, %d, %d], got %s" % (n, N, r, tuple(lora_b.shape)))
    if scales is not None:
        _dev_tensor(scales, torch.float32, "scales")
        if scales.numel() != n:
            raise ValueError("scales must hold one value per adapter")
    for t in (adapters, lora_a, lora_b, scales):
        if t is not None and t.device != dev:
            raise ValueError("the adapters and x must be on one device")
    return r, n


def lora_add(y: torch.Tensor, x: torch.Tensor, adapters: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
             scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each token's low-rank adapter beside a projection's output y [M, N] (bf16 or float32; rows may be strided): y[m] +
    scales[a] (x[m] A_a^T) B_a^T with a = adapters[m] (int32; ids outside the adapters: none), x [M, K] bf16 (rows may be
    strided), lora_a [adapters, rank, K] and lora_b [adapters, N, rank] bf16, scales float32 or None for ones.
    Written to y itself, or to ``out`` [M, N]; like every call, without autograd's knowledge but for the tensor's version, so
    that a y which a backward pass has saved is refused there.  Its gradient towards x is the same call on dy [M, N],
    ``lora_add(zeros [M, K], dy, adapters, B^T [adapters, rank, N], A^T [adapters, K, rank], scales)``, where N has to be a
    multiple of 8 as K does here (zero columns fill dy and B^T up).  ``workspace``: lib().lora_workspace_bytes(M, rank) bytes; one is
    allocated when none is given."""
    M, K, ldx = _rows(x, torch.bfloat16, "x")
    dev = x.device
    My, N, ldy = _rows(y, None, "y")
    yt = _type(y.dtype, "y")
    if My != M or y.device != dev:
        raise ValueError("y must have x's %d tokens, on its device" % M)
    r, n = _adapters(adapters, lora_a, lora_b, scales, M, N, K, dev)
    if out is None:
        out, ldo = y, ldy
    else:
        Mo, No, ldo = _rows(out, y.dtype, "out")
        if (Mo, No) != (M, N) or out.device != dev:
            raise ValueError("out must be %s on %s" % ((M, N), dev))
    ws = _workspace(workspace, max(lib().lora_workspace_bytes(M, r), 0), dev)
    _call("lora_add", dev, M, N, K, r, n, x.data_ptr(), ldx, adapters.data_ptr(), lora_a.data_ptr(), lora_b.data_ptr(),
          _ptr(scales), y.data_ptr(), ldy, out.data_ptr(), ldo, yt, ws.data_ptr())
    _written(out)
    return out


def nvfp4_lora_matvec(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, w_s_enc: torch.Tensor,
                      adapters: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                      scales: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``nvfp4_matvec`` with each token's low-rank adapter added before the one rounding of y [M, N]; the adapters as for
    ``lora_add``.  ``workspace``: lib().nvfp4_lora_workspace_bytes(M, N, rank, OUT_BF16 or OUT_F32) bytes; one is
    allocated when none is given."""
    M, K, ldx = _tokens(x)
    dev = x.device
    N, rows = _weights(w_codes, w_scales, w_s_enc, K, "w", dev)
    r, n = _adapters(adapters, lora_a, lora_b, scales, M, N, K, dev)
    y_dtype = _type(out_dtype, "out_dtype")
    y = _output(out, (M, N), out_dtype, dev)
    ws = _workspace(workspace, max(lib().nvfp4_lora_workspace_bytes(M, N, r, y_dtype), 0), dev)
    _call("nvfp4_lora_matvec", dev, FMT_B_ROWSCALED if rows else 0, M, N, K, x.data_ptr(), ldx, w_codes.data_ptr(),
          w_scales.data_ptr(), w_s_enc.data_ptr(), r, n, adapters.data_ptr(), lora_a.data_ptr(), lora_b.data_ptr(),
          _ptr(scales), y.data_ptr(), y_dtype, ws.data_ptr())
    _written(out)
    return y
