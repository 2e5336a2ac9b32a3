"""Python binding of libnvfp4 (NVFP4 quantize / dequantize / prepack / GEMM for MI355X, gfx950).

Thin ctypes layer over the C ABI in ``include/nvfp4.h``: it allocates outputs and workspaces with
PyTorch (device memory and streams only), passes raw device pointers and the current HIP stream,
and turns a non-zero status into an exception.  Every step of the computation runs in the HIP
kernels of ``libnvfp4.so``; there is no fallback.  The function names mirror the C entry points.
"""
from __future__ import annotations

import ctypes
import os
from enum import IntEnum
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")


class Status(IntEnum):
    OK = 0
    ERR_NULL = 1
    ERR_SHAPE = 2
    ERR_STRIDE = 3
    ERR_ALIGN = 4
    ERR_DTYPE = 5
    ERR_MODE = 6
    ERR_WORKSPACE = 7
    ERR_HIP = 8
    ERR_DEVICE = 9
    ERR_PRECONDITION = 10


F32, BF16 = 0, 1
W4A4, W4A16 = 0, 1
SCALE_DYNAMIC, SCALE_STATIC = 0, 1

EXPORTED = (
    "nvfp4_status_string", "nvfp4_abi_version",
    "nvfp4_quantize_workspace_bytes", "nvfp4_quantize",
    "nvfp4_dequantize", "nvfp4_fake_quantize",
    "nvfp4_prepacked_bytes", "nvfp4_prepack_weight", "nvfp4_unpack_weight",
    "nvfp4_gemm_workspace_bytes", "nvfp4_gemm_workspace_bytes_ld", "nvfp4_gemm",
    "nvfp4_gemm_requant_workspace_bytes", "nvfp4_gemm_requant_workspace_bytes_ld", "nvfp4_gemm_requant",
    "nvfp4_quantize_bs", "nvfp4_dequantize_bs", "nvfp4_fake_quantize_bs", "nvfp4_prepack_weight_bs",
    "nvfp4_unpack_weight_bs", "nvfp4_gemm_bs", "nvfp4_gemm_requant_bs",
    "nvfp4_mx_quantize", "nvfp4_mx_dequantize", "nvfp4_mx_gemm",
    "nvfp4_quantize_noalloc", "nvfp4_set_debug_checks",
    "nvfp4_mx8_quantize", "nvfp4_rmsnorm", "nvfp4_rmsnorm_backward_workspace_bytes", "nvfp4_rmsnorm_backward",
    "nvfp4_mx_gemm_w4a8", "nvfp4_rope_axes",
)

_lib = None
_vp, _i64, _sz, _i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = Status(status)
        super().__init__(f"{call}: {self.status.name} ({lib().nvfp4_status_string(status).decode()})")


def lib():
    """The loaded libnvfp4 (ctypes.CDLL).  Raises if the HIP library has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libnvfp4.so not found at {LIB_PATH}; build it with "
                           "`python nvfp4_quantized_gemm_amd/build.py` (or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_status_string.argtypes = [_i]
    L.nvfp4_abi_version.restype = _i
    L.nvfp4_abi_version.argtypes = []
    L.nvfp4_set_debug_checks.restype = _i
    L.nvfp4_set_debug_checks.argtypes = [_i]
    L.nvfp4_quantize_workspace_bytes.restype = _sz
    L.nvfp4_quantize_workspace_bytes.argtypes = [_i64, _i64]
    L.nvfp4_quantize.restype = _i
    L.nvfp4_quantize.argtypes = [_vp, _i, _i64, _i64, _i64, _vp, _vp, _vp, _i, _vp, _sz, _vp]
    L.nvfp4_fake_quantize.restype = _i
    L.nvfp4_fake_quantize.argtypes = [_vp, _i, _i64, _i64, _i64, _vp, _i, _i64, _vp, _i, _vp, _sz, _vp]
    L.nvfp4_dequantize.restype = _i
    L.nvfp4_dequantize.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, _i, _i64, _vp]
    L.nvfp4_prepacked_bytes.restype = _sz
    L.nvfp4_prepacked_bytes.argtypes = [_i64, _i64]
    L.nvfp4_prepack_weight.restype = _i
    L.nvfp4_prepack_weight.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp]
    L.nvfp4_unpack_weight.restype = _i
    L.nvfp4_unpack_weight.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp]
    L.nvfp4_gemm_workspace_bytes.restype = _sz
    L.nvfp4_gemm_workspace_bytes.argtypes = [_i, _i64, _i64, _i64]
    L.nvfp4_gemm_workspace_bytes_ld.restype = _sz
    L.nvfp4_gemm_workspace_bytes_ld.argtypes = [_i, _i64, _i64, _i64, _i64]
    L.nvfp4_gemm.restype = _i
    L.nvfp4_gemm.argtypes = [_i, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i, _i64, _vp, _sz, _vp]
    L.nvfp4_gemm_requant_workspace_bytes.restype = _sz
    L.nvfp4_gemm_requant_workspace_bytes.argtypes = [_i, _i64, _i64, _i64]
    L.nvfp4_gemm_requant_workspace_bytes_ld.restype = _sz
    L.nvfp4_gemm_requant_workspace_bytes_ld.argtypes = [_i, _i64, _i64, _i64, _i64]
    L.nvfp4_gemm_requant.restype = _i
    L.nvfp4_gemm_requant.argtypes = [_i, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i, _vp, _vp, _vp,
                                     _vp, _i64, _vp, _sz, _vp]
    L.nvfp4_quantize_bs.restype = _i
    L.nvfp4_quantize_bs.argtypes = [_vp, _i, _i64, _i64, _i64, _i, _vp, _vp, _vp, _i, _vp, _sz, _vp]
    L.nvfp4_fake_quantize_bs.restype = _i
    L.nvfp4_fake_quantize_bs.argtypes = [_vp, _i, _i64, _i64, _i64, _i, _vp, _i, _i64, _vp, _i, _vp, _sz, _vp]
    L.nvfp4_dequantize_bs.restype = _i
    L.nvfp4_dequantize_bs.argtypes = [_vp, _vp, _vp, _i64, _i64, _i, _vp, _i, _i64, _vp]
    L.nvfp4_prepack_weight_bs.restype = _i
    L.nvfp4_prepack_weight_bs.argtypes = [_vp, _vp, _i64, _i64, _i, _vp, _vp]
    L.nvfp4_unpack_weight_bs.restype = _i
    L.nvfp4_unpack_weight_bs.argtypes = [_vp, _i64, _i64, _i, _vp, _vp, _vp]
    L.nvfp4_gemm_bs.restype = _i
    L.nvfp4_gemm_bs.argtypes = [_i, _vp, _vp, _vp, _i, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i, _i64, _vp, _sz, _vp]
    L.nvfp4_gemm_requant_bs.restype = _i
    L.nvfp4_gemm_requant_bs.argtypes = [_i, _vp, _vp, _vp, _i, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i, _vp, _vp,
                                        _vp, _vp, _i64, _vp, _sz, _vp]
    L.nvfp4_mx_quantize.restype = _i
    L.nvfp4_mx_quantize.argtypes = [_vp, _i, _i64, _i64, _i64, _vp, _vp, _vp]
    L.nvfp4_mx_dequantize.restype = _i
    L.nvfp4_mx_dequantize.argtypes = [_vp, _vp, _i64, _i64, _vp, _i, _i64, _vp]
    L.nvfp4_mx_gemm.restype = _i
    L.nvfp4_quantize_noalloc.restype = _i
    L.nvfp4_quantize_noalloc.argtypes = [_vp, _i, _i64, _i64, _i64, _i, _vp, _vp, _vp, _i, _vp]
    L.nvfp4_mx_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i, _i64, _vp]
    L.nvfp4_mx8_quantize.restype = _i
    L.nvfp4_mx8_quantize.argtypes = [_vp, _i, _i64, _i64, _i64, _vp, _vp, _vp]
    L.nvfp4_rmsnorm.restype = _i
    L.nvfp4_rmsnorm.argtypes = [_vp, _i64, _vp, _i64, _i, _i64, _i64, _vp, _i, ctypes.c_float, _vp, _i64, _vp, _vp,
                                _vp, _i, _i64, _i, _vp, _vp]
    L.nvfp4_rmsnorm_backward_workspace_bytes.restype = _sz
    L.nvfp4_rmsnorm_backward_workspace_bytes.argtypes = [_i64, _i64]
    L.nvfp4_rmsnorm_backward.restype = _i
    L.nvfp4_rmsnorm_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _i, _i64, _i64, _vp, _i, _vp, _vp, _i64,
                                         _vp, _vp, _sz, _vp]
    L.nvfp4_mx_gemm_w4a8.restype = _i
    L.nvfp4_mx_gemm_w4a8.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i, _i64, _vp]
    L.nvfp4_rope_axes.restype = _i
    L.nvfp4_rope_axes.argtypes = [_vp, _i, _i64, _i64, _i64, _i64, _i64, _vp, _i, _vp, _vp, _i, _i, _vp, _i64, _i64,
                                  _vp]
    _lib = L
    return L


def _check(status: int, call: str):
    if status != 0:
        raise NVFP4Error(status, call)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {dt}; libnvfp4 takes float32 or bfloat16")


def nvfp4_set_debug_checks(enable: bool) -> bool:
    """Turn the library's device-data precondition scans on or off for every later call; returns
    the previous setting.  When on, a call whose inputs hold a non-finite value, a NaN scale byte
    or an invalid tensor scale raises NVFP4Error(ERR_PRECONDITION) and launches nothing; every call
    then waits on its stream.  The initial setting comes from the NVFP4_DEBUG environment variable."""
    return bool(lib().nvfp4_set_debug_checks(1 if enable else 0))


def _rows(t: torch.Tensor, name: str):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit stride along K")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.shape[0], t.shape[1], t.stride(0)


# ---- quantize / dequantize ----------------------------------------------------------------------

def nvfp4_quantize_workspace_bytes(M: int, K: int) -> int:
    return int(lib().nvfp4_quantize_workspace_bytes(M, K))


def nvfp4_quantize(x: torch.Tensor, tensor_scale: torch.Tensor | None = None, *, static: bool | None = None,
                   packed=None, scales=None, workspace=None, block_size: int = 16, stream=None):
    """Quantize x [M, K] (fp32 or bf16, device).

    static=False (the default when tensor_scale is None): dynamic scale, computed on the device and
    written to tensor_scale (allocated when None).  static=True (the default when tensor_scale is
    given): tensor_scale holds the caller's S.  block_size: values per scale byte (16, 32 or 64).
    Returns (packed u8 [M, K/2], scales u8 [M, K/block_size], S f32 [1])."""
    M, K, ld = _rows(x, "x")
    dev = x.device
    if packed is None:
        packed = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((M, max(K // block_size, 0)), dtype=torch.uint8, device=dev)
    if static is None:
        static = tensor_scale is not None
    dynamic = not static
    if tensor_scale is None:
        if static:
            raise ValueError("static quantization needs tensor_scale")
        tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    S = tensor_scale
    ws_bytes = 0
    if dynamic:
        ws_bytes = nvfp4_quantize_workspace_bytes(M, K)
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().nvfp4_quantize_bs(_ptr(x), _dtype_code(x.dtype), M, K, ld, block_size, _ptr(packed), _ptr(scales),
                                 _ptr(S), SCALE_DYNAMIC if dynamic else SCALE_STATIC, _ptr(workspace), ws_bytes,
                                 _stream(stream))
    _check(st, "nvfp4_quantize_bs")
    return packed, scales, S


def nvfp4_quantize_noalloc(x: torch.Tensor, tensor_scale: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                           *, static: bool = False, block_size: int = 16, stream=None):
    """nvfp4_quantize into caller-given outputs with no workspace: the dynamic pass uses the library's
    own device scratch, so neither this call nor the library allocates anything.  tensor_scale is
    written (dynamic) or read (static).  Calls that overlap on one GPU race (they share the scratch)."""
    M, K, ld = _rows(x, "x")
    st = lib().nvfp4_quantize_noalloc(_ptr(x), _dtype_code(x.dtype), M, K, ld, block_size, _ptr(packed),
                                      _ptr(scales), _ptr(tensor_scale), SCALE_STATIC if static else SCALE_DYNAMIC,
                                      _stream(stream))
    _check(st, "nvfp4_quantize_noalloc")
    return packed, scales, tensor_scale


def _block_of(K: int, scales: torch.Tensor) -> int:
    """Block size of a canonical scale tensor [rows, K / block_size]."""
    n = scales.shape[1] if scales.dim() == 2 else 0
    return K // n if n else 16


def nvfp4_dequantize(packed: torch.Tensor, scales: torch.Tensor, tensor_scale: torch.Tensor,
                     dtype: torch.dtype = torch.float32, *, out=None, stream=None) -> torch.Tensor:
    """y = dequantize(packed, scales, S); the block size is read from the shape of scales."""
    M, K = packed.shape[0], packed.shape[1] * 2
    if out is None:
        out = torch.empty((M, K), dtype=dtype, device=packed.device)
    _, _, ld = _rows(out, "out")
    st = lib().nvfp4_dequantize_bs(_ptr(packed), _ptr(scales), _ptr(tensor_scale), M, K, _block_of(K, scales),
                                   _ptr(out), _dtype_code(out.dtype), ld, _stream(stream))
    _check(st, "nvfp4_dequantize_bs")
    return out


def nvfp4_fake_quantize(x: torch.Tensor, tensor_scale: torch.Tensor | None = None, *, static: bool | None = None,
                        out_dtype: torch.dtype | None = None, out=None, workspace=None, block_size: int = 16,
                        stream=None):
    """y = dequantize(quantize(x)) in one pass (x [M, K] fp32 or bf16 on the device).  Scale
    arguments as for nvfp4_quantize.  Returns (y, S)."""
    M, K, ld = _rows(x, "x")
    dev = x.device
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype or x.dtype, device=dev)
    _, _, ld_y = _rows(out, "out")
    if static is None:
        static = tensor_scale is not None
    if tensor_scale is None:
        if static:
            raise ValueError("static quantization needs tensor_scale")
        tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    ws_bytes = 0
    if not static:
        ws_bytes = nvfp4_quantize_workspace_bytes(M, K)
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().nvfp4_fake_quantize_bs(_ptr(x), _dtype_code(x.dtype), M, K, ld, block_size, _ptr(out),
                                      _dtype_code(out.dtype), ld_y, _ptr(tensor_scale),
                                      SCALE_STATIC if static else SCALE_DYNAMIC, _ptr(workspace), ws_bytes,
                                      _stream(stream))
    _check(st, "nvfp4_fake_quantize_bs")
    return out, tensor_scale


class FakeQuantizeSTE(torch.autograd.Function):
    """Quantization-aware-training op: forward is NVFP4 fake quantization (nvfp4_fake_quantize, output
    in x's dtype), backward is the straight-through estimator, i.e. the incoming gradient unchanged."""

    @staticmethod
    def forward(ctx, x, tensor_scale=None, block_size=16):
        y, _ = nvfp4_fake_quantize(x.contiguous(), tensor_scale, block_size=block_size)
        return y

    @staticmethod
    def backward(ctx, grad_out):
        return grad_out, None, None


def fake_quantize_ste(x: torch.Tensor, tensor_scale: torch.Tensor | None = None, block_size: int = 16) -> torch.Tensor:
    """NVFP4 fake quantization with a straight-through gradient (dynamic scale when tensor_scale is
    None, else the given static scale; block_size values per scale byte: 16, 32 or 64)."""
    return FakeQuantizeSTE.apply(x, tensor_scale, block_size)


# ---- weight prepack -------------------------------------------------------------------------------

def nvfp4_prepacked_bytes(N: int, K: int) -> int:
    return int(lib().nvfp4_prepacked_bytes(N, K))


def nvfp4_prepack_weight(packed: torch.Tensor, scales: torch.Tensor, *, out=None, stream=None) -> torch.Tensor:
    N, K = packed.shape[0], packed.shape[1] * 2
    nbytes = nvfp4_prepacked_bytes(N, K)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=packed.device)
    st = lib().nvfp4_prepack_weight_bs(_ptr(packed), _ptr(scales), N, K, _block_of(K, scales), _ptr(out),
                                       _stream(stream))
    _check(st, "nvfp4_prepack_weight_bs")
    return out


def nvfp4_unpack_weight(prepacked: torch.Tensor, N: int, K: int, *, block_size: int = 16, stream=None):
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=prepacked.device)
    scales = torch.empty((N, K // block_size), dtype=torch.uint8, device=prepacked.device)
    st = lib().nvfp4_unpack_weight_bs(_ptr(prepacked), N, K, block_size, _ptr(packed), _ptr(scales),
                                      _stream(stream))
    _check(st, "nvfp4_unpack_weight_bs")
    return packed, scales


# ---- GEMM -------------------------------------------------------------------------------------------

def nvfp4_gemm_workspace_bytes(mode: int, M: int, N: int, K: int, lda: int | None = None) -> int:
    """Workspace bytes of nvfp4_gemm for an activation with row pitch lda (elements; K when None)."""
    return int(lib().nvfp4_gemm_workspace_bytes_ld(mode, M, N, K, K if lda is None else lda))


def _activation_pitch(mode: int, a: torch.Tensor, a_scales, a_block_size):
    """(lda in elements, W4A4 activation block size) of a GEMM's A operand.  W4A4: a is packed codes
    [M, K/2] (a row-strided view is allowed: lda = 2 * its row stride) and a_scales the matching
    [M, K/block] view of [M, lda/block] bytes; the block size is a_block_size, else lda over the scale
    tensor's row stride.  W4A16: a is bf16 [M, K] with unit stride along K."""
    if mode != W4A4:
        _, _, lda = _rows(a, "a")
        return lda, 16
    lda = a.stride(0) * 2
    if a_block_size is not None:
        return lda, int(a_block_size)
    if a_scales is not None and a_scales.dim() == 2 and a_scales.shape[0] >= 1 and a_scales.stride(0) > 0:
        return lda, lda // a_scales.stride(0)
    return lda, _block_of(lda, a_scales)


def nvfp4_gemm(mode: int, a: torch.Tensor, a_scales, a_tensor_scale, b_prepacked: torch.Tensor,
               b_tensor_scale: torch.Tensor, N: int, K: int, out_dtype: torch.dtype = torch.bfloat16, *,
               out=None, workspace=None, a_block_size: int | None = None, stream=None) -> torch.Tensor:
    """Y = A B^T.  W4A4: a = packed u8 [M, K/2] with a_scales u8 [M, K/block] and a_tensor_scale
    (from nvfp4_quantize; both may be row-strided views of wider rows; the block size is
    a_block_size, else read from the scales' layout).  W4A16: a = bf16 [M, K], a_scales =
    a_tensor_scale = None."""
    M = a.shape[0]
    lda, ablk = _activation_pitch(mode, a, a_scales, a_block_size)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    ldc = out.stride(0)
    ws_need = nvfp4_gemm_workspace_bytes(mode, M, N, K, lda)
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=a.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().nvfp4_gemm_bs(mode, _ptr(a), _ptr(a_scales), _ptr(a_tensor_scale), ablk, _ptr(b_prepacked),
                             _ptr(b_tensor_scale), M, N, K, lda, _ptr(out), _dtype_code(out.dtype), ldc,
                             _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "nvfp4_gemm_bs")
    return out


ACT_NONE, ACT_GELU_TANH = 0, 1


def nvfp4_gemm_requant_workspace_bytes(mode: int, M: int, N: int, K: int, lda: int | None = None) -> int:
    """Workspace bytes of nvfp4_gemm_requant for an activation with row pitch lda (K when None)."""
    return int(lib().nvfp4_gemm_requant_workspace_bytes_ld(mode, M, N, K, K if lda is None else lda))


def nvfp4_gemm_requant(mode: int, a: torch.Tensor, a_scales, a_tensor_scale, b_prepacked: torch.Tensor,
                       b_tensor_scale: torch.Tensor, N: int, K: int, out_tensor_scale: torch.Tensor, *,
                       bias=None, act: int = ACT_NONE, packed=None, scales=None, y=None, workspace=None,
                       a_block_size: int | None = None, stream=None):
    """NVFP4 output of A B^T (+ bias) (-> act) under the static out_tensor_scale (device fp32 [1]).
    Operands as nvfp4_gemm.  Returns (packed u8 [M, N/2], scales u8 [M, N/16]); when y (fp32 [M, >= N])
    is given it also receives the fp32 values that were quantized."""
    M = a.shape[0]
    lda, ablk = _activation_pitch(mode, a, a_scales, a_block_size)
    if packed is None:
        packed = torch.empty((M, N // 2), dtype=torch.uint8, device=a.device)
    if scales is None:
        scales = torch.empty((M, N // 16), dtype=torch.uint8, device=a.device)
    ldy = 0 if y is None else y.stride(0)
    ws_need = nvfp4_gemm_requant_workspace_bytes(mode, M, N, K, lda)
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=a.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().nvfp4_gemm_requant_bs(mode, _ptr(a), _ptr(a_scales), _ptr(a_tensor_scale), ablk, _ptr(b_prepacked),
                                     _ptr(b_tensor_scale), M, N, K, lda, _ptr(bias), act, _ptr(out_tensor_scale),
                                     _ptr(packed), _ptr(scales), _ptr(y), ldy, _ptr(workspace), ws_bytes,
                                     _stream(stream))
    _check(st, "nvfp4_gemm_requant_bs")
    return packed, scales


# ---- MXFP4 (32-value blocks, E8M0 scales, no tensor scale) ------------------------------------

def nvfp4_mx_quantize(x: torch.Tensor, *, packed=None, scales=None, stream=None):
    """MXFP4-quantize x [M, K] (fp32 or bf16, K % 32 == 0).  Returns (packed u8 [M, K/2], scales u8 [M, K/32])."""
    M, K, ld = _rows(x, "x")
    if packed is None:
        packed = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((M, max(K // 32, 0)), dtype=torch.uint8, device=x.device)
    _check(lib().nvfp4_mx_quantize(_ptr(x), _dtype_code(x.dtype), M, K, ld, _ptr(packed), _ptr(scales), _stream(stream)),
           "nvfp4_mx_quantize")
    return packed, scales


def nvfp4_mx_dequantize(packed: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float32, *, out=None,
                        stream=None) -> torch.Tensor:
    M, K = packed.shape[0], packed.shape[1] * 2
    if out is None:
        out = torch.empty((M, K), dtype=dtype, device=packed.device)
    _, _, ld = _rows(out, "out")
    _check(lib().nvfp4_mx_dequantize(_ptr(packed), _ptr(scales), M, K, _ptr(out), _dtype_code(out.dtype), ld,
                                     _stream(stream)), "nvfp4_mx_dequantize")
    return out


def nvfp4_mx_gemm(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                  out_dtype: torch.dtype = torch.bfloat16, *, out=None, stream=None) -> torch.Tensor:
    """Y = A B^T with A [M, K] and B [N, K] both canonical MXFP4 (packed codes + E8M0 scales)."""
    M, K = a.shape[0], a.shape[1] * 2
    N = b.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check(lib().nvfp4_mx_gemm(_ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales), M, N, K, _ptr(out),
                               _dtype_code(out.dtype), out.stride(0), _stream(stream)), "nvfp4_mx_gemm")
    return out


# ---- the 8-bit activation path: MXFP8, RMS norm, W4A8, rotary positions --------------------------

ROPE_PAIRS, ROPE_HALVES = 0, 1


_u8, _f32 = torch.uint8, torch.float32


# The checks below run on every call, also where the call is one token's and takes as long as its launch, so
# they are few and plain: get_device() and `is` instead of comparing device and type objects, one condition
# for all operands of a kind, and the explanation only once something is wrong.

def _launch_device(ref: torch.Tensor) -> int:
    """Index of ref's device, which must be the current one (the library launches there)."""
    i = ref.get_device()
    if i < 0:
        raise ValueError("the operands must be device tensors")
    if i != torch._C._cuda_getDevice():
        raise ValueError(f"the operands are on {ref.device}, which is not the current device")
    return i


# Raw handle of the current stream of a device (current_stream() without making an object).  The calls below
# that take a stream run as under ``with torch.cuda.stream(stream)``: what they allocate is that stream's.
# None on a torch without device bindings, where no operand gets as far.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _written(t: torch.Tensor, name: str):
    """Mark a caller's tensor as written, for autograd, which cannot see stores through an address; refuse one whose
    gradient is being recorded, as the call records none (torch's own out= does the same)."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} is written in place and requires a gradient, which this call does not record")
    torch.autograd.graph.increment_version(t)


def _dense(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """Address of a dense tensor of the given shape (a tuple), type and device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _pitch(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """Row pitch (elements) of a matrix of the given shape, type and device with unit stride along K."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return shape[1]
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along K")
    return ld if shape[0] > 1 else shape[1]


def _weight(weight, K: int, dev: int):
    """(address, dtype code) of an optional weight vector."""
    if weight is None:
        return 0, 0
    return _dense(weight, "weight", (K,), weight.dtype, dev), _dtype_code(weight.dtype)


def nvfp4_mx8_quantize(x: torch.Tensor, *, codes=None, scales=None, stream=None):
    """MXFP8-quantize x [M, K] (fp32 or bf16, K % 32 == 0).  Returns (codes u8 [M, K], scales u8 [M, K/32]):
    E4M3 codes (``codes.view(torch.float8_e4m3fn)`` reads them) under one E8M0 byte per 32 values."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return nvfp4_mx8_quantize(x, codes=codes, scales=scales)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    dev = _launch_device(x)
    ld = K if x.is_contiguous() else _pitch(x, "x", x.shape, x.dtype, dev)
    if codes is None:
        codes = torch.empty(M, K, dtype=_u8, device=x.device)
    else:
        _dense(codes, "codes", (M, K), _u8, dev)
        _written(codes, "codes")
    if scales is None:
        scales = torch.empty(M, K // 32, dtype=_u8, device=x.device)
    else:
        _dense(scales, "scales", (M, K // 32), _u8, dev)
        _written(scales, "scales")
    st = lib().nvfp4_mx8_quantize(x.data_ptr(), _dtype_code(x.dtype), M, K, ld, codes.data_ptr(), scales.data_ptr(),
                                  _current_stream(dev))
    if st:
        raise NVFP4Error(st, "nvfp4_mx8_quantize")
    return codes, scales


class RMSNormOutput(NamedTuple):
    """What nvfp4_rmsnorm wrote; None for what was not asked for."""
    h: torch.Tensor | None
    codes: torch.Tensor | None
    scales: torch.Tensor | None
    y: torch.Tensor | None
    inv_rms: torch.Tensor | None


def nvfp4_rmsnorm(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                  eps: float = 1e-6, *, mx8: bool = True, y_dtype: torch.dtype | None = None,
                  fake_quantize: bool = False, save_inv_rms: bool = False, h=None, stream=None) -> RMSNormOutput:
    """y = rmsnorm(x + residual) * weight of [M, K] tensors (fp32 or bf16, K % 32 == 0, K <= 32768).

    mx8: write y as MXFP8 (codes, scales), the activation of nvfp4_mx_gemm_w4a8.  y_dtype: also write y
    itself (fp32 or bf16); with fake_quantize the values its MXFP8 codes stand for.  With a residual, h
    is the sum, rounded to x's type (into the given h, which may be x or residual, or a new tensor);
    without one it is written only into a given h.  save_inv_rms: keep what the backward pass needs."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return nvfp4_rmsnorm(x, residual, weight, eps, mx8=mx8, y_dtype=y_dtype, fake_quantize=fake_quantize,
                                 save_inv_rms=save_inv_rms, h=h)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    shape, dtype, device = x.shape, x.dtype, x.device
    M, K = shape
    dev = _launch_device(x)
    ld_x = K if x.is_contiguous() else _pitch(x, "x", shape, dtype, dev)
    p_r = ld_r = p_h = ld_h = p_w = w_code = p_c = p_s = p_y = y_code = p_i = 0
    codes = scales = y = inv_rms = None
    if residual is not None:
        ld_r, p_r = _pitch(residual, "residual", shape, dtype, dev), residual.data_ptr()
        if h is None:
            h = torch.empty(M, K, dtype=dtype, device=device)
            ld_h, p_h = K, h.data_ptr()
    if h is not None and not p_h:
        ld_h, p_h = _pitch(h, "h", shape, dtype, dev), h.data_ptr()
        _written(h, "h")
    if weight is not None:
        p_w, w_code = _weight(weight, K, dev)
    if mx8:
        codes = torch.empty(M, K, dtype=_u8, device=device)
        scales = torch.empty(M, K // 32, dtype=_u8, device=device)
        p_c, p_s = codes.data_ptr(), scales.data_ptr()
    if y_dtype is not None:
        y = torch.empty(M, K, dtype=y_dtype, device=device)
        p_y, y_code = y.data_ptr(), _dtype_code(y_dtype)
    elif fake_quantize:
        raise ValueError("fake_quantize needs y_dtype")
    if save_inv_rms:
        inv_rms = torch.empty(M, dtype=_f32, device=device)
        p_i = inv_rms.data_ptr()
    st = lib().nvfp4_rmsnorm(x.data_ptr(), ld_x, p_r, ld_r, _dtype_code(dtype), M, K, p_w, w_code, eps, p_h, ld_h, p_c,
                             p_s, p_y, y_code, K, 1 if fake_quantize else 0, p_i, _current_stream(dev))
    if st:
        raise NVFP4Error(st, "nvfp4_rmsnorm")
    return RMSNormOutput(h, codes, scales, y, inv_rms)


def nvfp4_rmsnorm_backward_workspace_bytes(M: int, K: int) -> int:
    return int(lib().nvfp4_rmsnorm_backward_workspace_bytes(M, K))


def nvfp4_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, inv_rms: torch.Tensor, weight: torch.Tensor | None = None,
                           dh: torch.Tensor | None = None, *, dweight: bool = True, dx=None, workspace=None,
                           stream=None):
    """Gradients of nvfp4_rmsnorm from dy (gradient of y), the forward's h (x where there was no residual)
    and inv_rms, and dh (gradient of h, or None).  Returns (dx, dw): dx [M, K] in h's type is the gradient
    of x and of residual; dw fp32 [K] is weight's (None with dweight=False)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return nvfp4_rmsnorm_backward(dy, h, inv_rms, weight, dh, dweight=dweight, dx=dx, workspace=workspace)
    if h.dim() != 2:
        raise ValueError("h must be 2-D")
    shape, dtype, device = h.shape, h.dtype, h.device
    M, K = shape
    dev = _launch_device(h)
    ld_h = K if h.is_contiguous() else _pitch(h, "h", shape, dtype, dev)
    ld_dy = _pitch(dy, "dy", shape, dtype, dev)
    p_dh = ld_dh = p_dw = p_ws = ws_bytes = 0
    if dh is not None:
        ld_dh, p_dh = _pitch(dh, "dh", shape, dtype, dev), dh.data_ptr()
    p_i = _dense(inv_rms, "inv_rms", (M,), _f32, dev)
    p_w, w_code = _weight(weight, K, dev)
    if dx is None:
        dx, ld_dx = torch.empty(M, K, dtype=dtype, device=device), K
    else:
        ld_dx = _pitch(dx, "dx", shape, dtype, dev)
        _written(dx, "dx")
    L = lib()
    dw = None
    if dweight:
        dw = torch.empty(K, dtype=_f32, device=device)
        if workspace is None:
            ws_bytes = L.nvfp4_rmsnorm_backward_workspace_bytes(M, K)
            workspace = torch.empty(ws_bytes, dtype=_u8, device=device)
        elif workspace.get_device() != dev:
            raise ValueError(f"workspace is on {workspace.device}, not on {device}")
        else:
            ws_bytes = workspace.numel() * workspace.element_size()
        p_dw, p_ws = dw.data_ptr(), workspace.data_ptr()
    st = L.nvfp4_rmsnorm_backward(dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, p_dh, ld_dh, _dtype_code(dtype), M, K, p_w,
                                  w_code, p_i, dx.data_ptr(), ld_dx, p_dw, p_ws, ws_bytes, _current_stream(dev))
    if st:
        raise NVFP4Error(st, "nvfp4_rmsnorm_backward")
    return dx, dw


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, fake_quantize):
        ctx.set_materialize_grads(False)
        x2 = _rows_of(x)
        if weight is not None and not (weight.is_contiguous() and weight.data_ptr() % 16 == 0):
            weight = weight.clone(memory_format=torch.contiguous_format)  # a slice of a flat buffer, an expanded scalar
        out = nvfp4_rmsnorm(x2, None if residual is None else _rows_of(residual), weight, eps, mx8=False,
                            y_dtype=x.dtype, fake_quantize=fake_quantize, save_inv_rms=True)
        ctx.save_for_backward(x2 if residual is None else out.h, out.inv_rms, weight)
        ctx.shape = x.shape
        ctx.has_residual = residual is not None
        return out.y.view(x.shape), None if residual is None else out.h.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, inv_rms, weight = ctx.saved_tensors
        want_dw = weight is not None and ctx.needs_input_grad[2]
        if dy is None:  # y is not used: only the sum's gradient goes through
            return dh, dh if ctx.has_residual else None, torch.zeros_like(weight) if want_dw else None, None, None
        dx, dw = nvfp4_rmsnorm_backward(_rows_of(dy), h, inv_rms, weight, None if dh is None else _rows_of(dh),
                                        dweight=want_dw)
        dx = dx.view(ctx.shape)
        return dx, dx if ctx.has_residual else None, dw.to(weight.dtype) if want_dw else None, None, None


def _rows_of(t: torch.Tensor) -> torch.Tensor:
    """t [..., K] as a matrix of rows of K that the kernels take (copied only where its layout needs it: a gradient
    that autograd has expanded, rows that overlap, memory off 16 bytes)."""
    m = t.reshape(-1, t.shape[-1])
    rows, K = m.shape
    pitched = m.stride(1) == 1 and (rows <= 1 or (m.stride(0) >= K and m.stride(0) * t.element_size() % 16 == 0))
    # clone, not contiguous(): that returns a dense tensor as it is, wherever it lies
    return m if pitched and m.data_ptr() % 16 == 0 else m.clone(memory_format=torch.contiguous_format)


def rmsnorm(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
            eps: float = 1e-6, fake_quantize: bool = False):
    """Differentiable RMS norm with the residual's addition over the last dimension: (y, h) with h the sum
    (None without a residual), of tensors in any strides.  fake_quantize: y holds the values of its MXFP8 codes,
    with a straight-through gradient (quantization-aware training)."""
    return _RMSNorm.apply(x, residual, weight, eps, fake_quantize)


def nvfp4_mx_gemm_w4a8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                       out_dtype: torch.dtype = torch.bfloat16, *, out=None, stream=None) -> torch.Tensor:
    """Y = A B^T with A [M, K] MXFP8 (codes u8 [M, K], scales u8 [M, K/32]) and B [N, K] MXFP4 (packed u8
    [N, K/2], scales u8 [N, K/32]); all dense.  out: a tensor [M, N] (fp32 or bf16, unit stride along N)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return nvfp4_mx_gemm_w4a8(a, a_scales, b, b_scales, out_dtype, out=out)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    dev = _launch_device(a)
    if not (a.dtype is _u8 and a.is_contiguous()
            and b.dtype is _u8 and b.is_contiguous() and b.shape[1] == K // 2 and b.get_device() == dev
            and a_scales.dtype is _u8 and a_scales.is_contiguous() and a_scales.shape == (M, K // 32)
            and b_scales.dtype is _u8 and b_scales.is_contiguous() and b_scales.shape == (N, K // 32)
            and a_scales.get_device() == dev and b_scales.get_device() == dev):
        _dense(a, "a", (M, K), _u8, dev)
        _dense(a_scales, "a_scales", (M, K // 32), _u8, dev)
        _dense(b, "b", (N, K // 2), _u8, dev)
        _dense(b_scales, "b_scales", (N, K // 32), _u8, dev)
    if out is None:
        out, ldc = torch.empty(M, N, dtype=out_dtype, device=a.device), N
    else:
        ldc = _pitch(out, "out", (M, N), out.dtype, dev)
        _written(out, "out")
    st = lib().nvfp4_mx_gemm_w4a8(a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(), M, N, K,
                                  out.data_ptr(), _dtype_code(out.dtype), ldc, _current_stream(dev))
    if st:
        raise NVFP4Error(st, "nvfp4_mx_gemm_w4a8")
    return out


def rope_inv_freq(axis_dims, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Frequencies of nvfp4_rope_axes: theta^(-2 i / d) for the pairs i of each axis' d elements, fp32."""
    parts = [float(theta) ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in axis_dims if d > 0]
    return torch.cat(parts).float().to(device) if parts else torch.empty(0, device=device)


def nvfp4_rope_axes(x: torch.Tensor, positions: torch.Tensor, axis_dims, inv_freq: torch.Tensor, *,
                    layout: int = ROPE_PAIRS, inverse: bool = False, out=None, stream=None) -> torch.Tensor:
    """Rotary positions with several axes of x [T, H, D] (fp32 or bf16; token and head strides free, unit
    stride along D).  positions fp32 [T, axes]; axis_dims: how many leading elements of a head each axis
    turns; inv_freq fp32, one per pair (rope_inv_freq).  inverse: turn back (the gradient).  out: a
    tensor [T, H, D], x itself to turn in place, or None for a new dense one."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return nvfp4_rope_axes(x, positions, axis_dims, inv_freq, layout=layout, inverse=inverse, out=out)
    if x.dim() != 3:
        raise ValueError("x must be [T, H, D]")
    T, H, D = x.shape
    dev = _launch_device(x)
    n = len(axis_dims)
    p_pos = _dense(positions, "positions", (T, n), _f32, dev)
    p_f = _dense(inv_freq, "inv_freq", (sum(axis_dims) // 2,), _f32, dev)
    xt, xh, xd = x.stride()
    if out is None:
        out = torch.empty(T, H, D, dtype=x.dtype, device=x.device)
        yt, yh, yd = H * D, D, 1
    elif out.shape != x.shape or out.dtype is not x.dtype or out.get_device() != dev:
        raise ValueError("out must have x's shape, type and device")
    else:
        yt, yh, yd = out.stride()
        _written(out, "out")
    if xd != 1 or yd != 1:
        raise ValueError("x and out must have unit stride along D")
    if T == 1:  # the pitch of a single token or head is never used, whatever it is
        xt = yt = 0
    if H == 1:
        xh = yh = 0
    st = lib().nvfp4_rope_axes(x.data_ptr(), _dtype_code(x.dtype), T, H, D, xt, xh, p_pos, n,
                               (ctypes.c_int32 * n)(*axis_dims), p_f, layout, 1 if inverse else 0, out.data_ptr(), yt, yh,
                               _current_stream(dev))
    if st:
        raise NVFP4Error(st, "nvfp4_rope_axes")
    return out


def _heads_of(t: torch.Tensor) -> torch.Tensor:
    """t [T, H, D] in a layout that the rotation reads (copied only where its own needs it)."""
    es = t.element_size()
    taken = t.dim() != 3 or (t.stride(2) == 1 and t.data_ptr() % 16 == 0
                             and t.stride(0) * es % 16 == 0 and t.stride(1) * es % 16 == 0)
    return t if taken else t.clone(memory_format=torch.contiguous_format)


class _RopeAxes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, axis_dims, inv_freq, layout):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = (axis_dims, layout)
        return nvfp4_rope_axes(_heads_of(x), positions, axis_dims, inv_freq, layout=layout)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        positions, inv_freq = ctx.saved_tensors
        axis_dims, layout = ctx.how
        dx = nvfp4_rope_axes(_heads_of(dy), positions, axis_dims, inv_freq, layout=layout, inverse=True)
        return dx, None, None, None, None


def rope_axes(x: torch.Tensor, positions: torch.Tensor, axis_dims, inv_freq: torch.Tensor,
              layout: int = ROPE_PAIRS) -> torch.Tensor:
    """Differentiable nvfp4_rope_axes of x in any strides (the gradient of x is the inverse rotation)."""
    return _RopeAxes.apply(x, positions, tuple(axis_dims), inv_freq, layout)


__all__ = [
    "Status", "NVFP4Error", "lib", "LIB_PATH", "EXPORTED", "F32", "BF16", "W4A4", "W4A16",
    "SCALE_DYNAMIC", "SCALE_STATIC", "nvfp4_set_debug_checks",
    "nvfp4_quantize_workspace_bytes", "nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_dequantize",
    "nvfp4_fake_quantize",
    "FakeQuantizeSTE", "fake_quantize_ste",
    "nvfp4_prepacked_bytes", "nvfp4_prepack_weight", "nvfp4_unpack_weight",
    "nvfp4_gemm_workspace_bytes", "nvfp4_gemm",
    "ACT_NONE", "ACT_GELU_TANH", "nvfp4_gemm_requant_workspace_bytes", "nvfp4_gemm_requant",
    "nvfp4_mx_quantize", "nvfp4_mx_dequantize", "nvfp4_mx_gemm",
    "nvfp4_mx8_quantize", "RMSNormOutput", "nvfp4_rmsnorm", "nvfp4_rmsnorm_backward_workspace_bytes",
    "nvfp4_rmsnorm_backward", "rmsnorm", "nvfp4_mx_gemm_w4a8",
    "ROPE_PAIRS", "ROPE_HALVES", "rope_inv_freq", "nvfp4_rope_axes", "rope_axes",
]
