"""Python binding of libfh, the NVFP4 quantized linear layer for B200 (sm_100a).

Argument marshalling only: every function below has the name of the C entry
point it calls (include/fh.h), checks that the torch tensors it is given have
the dtype, device and contiguity the C ABI expects, passes their device
pointers and the current CUDA stream, and raises FHError on a non-zero status.
All arithmetic runs in the CUDA kernels of libfh.so.  There is no fallback:
importing this package fails if libfh.so has not been built
(``python nvfp4_quantized_linear_fh_b200/build.py``).

The layer is the NVFP4 linear layer of FastH3's diffusion transformer (FastH3
thread digest, farwalk.ai, tweets 5/8 and 6/8; FastH3 Trim, comfyui-wiki news,
"What the ComfyUI repack contains").
"""
from __future__ import annotations

import ctypes
import os
from operator import index as _index

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfh.so")

FH_OK = 0
FH_ERR_INVALID_ARG = 1
FH_ERR_UNSUPPORTED_SHAPE = 2
FH_ERR_CUDA = 3
FH_ERR_TIMEOUT = 4
FH_ERR_NO_DEVICE = 5

FH_SCALES_ROWMAJOR = 0
FH_SCALES_MMA_TILED = 1

# Bits of fh_kv_pages_update's status word.
FH_KV_NO_PAGES = 1
FH_KV_TABLE_FULL = 2
FH_KV_BAD_LENGTH = 4
FH_KV_STACK_OVERFLOW = 8
FH_KV_SLOTS_FULL = 16
FH_KV_MAX_BATCH = 8192


class FHError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libfh status {status}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python nvfp4_quantized_linear_fh_b200/build.py` "
                      "(the NVFP4 layer has no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)
_c = ctypes
_P = _c.c_void_p
_I64 = _c.c_int64
_SIG = {
    "fh_version": (_c.c_int, []),
    "fh_last_error": (_c.c_char_p, []),
    "fh_scale_from_amax": (_c.c_float, [_c.c_float]),
    "fh_scales_bytes": (_c.c_size_t, [_I64, _I64, _c.c_int]),
    "fh_amax": (_c.c_int, [_P, _I64, _I64, _I64, _P, _P]),
    "fh_quantize_act": (_c.c_int, [_P, _I64, _I64, _I64, _c.c_float, _P, _P, _P, _c.c_int, _P]),
    "fh_gelu_quantize_act": (_c.c_int, [_P, _I64, _I64, _I64, _c.c_float, _P, _P, _P, _P]),
    "fh_nvfp4_linear": (_c.c_int, [_P, _P, _c.c_float, _P, _P, _c.c_float, _P, _P, _I64, _I64, _I64, _P]),
    "fh_nvfp4_linear_gelu_quant": (_c.c_int, [_P, _P, _c.c_float, _P, _P, _c.c_float, _P, _c.c_float, _P, _P, _P,
                                              _I64, _I64, _I64, _P]),
    "fh_scales_to_rowmajor": (_c.c_int, [_P, _P, _I64, _I64, _P]),
    "fh_nvfp4_linear_fused_quant": (_c.c_int, [_P, _I64, _I64, _I64, _c.c_float, _P, _P, _c.c_float, _P, _P, _I64,
                                               _P, _P, _P, _P, _P]),
    "fh_nvfp4_linear_fused_quant_sync_bytes": (_c.c_size_t, [_I64]),
    "fh_nvfp4_linear_host": (_c.c_int, [_P, _I64, _I64, _c.c_float, _P, _P, _c.c_float, _P, _I64, _P, _P, _I64, _P,
                                        _c.c_size_t, _P]),
    "fh_nvfp4_linear_host_workspace_bytes": (_c.c_size_t, [_I64, _I64, _I64]),
    "fh_nvfp4_linear_host_noalloc": (_c.c_int, [_P, _I64, _I64, _c.c_float, _P, _P, _c.c_float, _P, _I64, _P, _P,
                                                _P]),
    "fh_gelu_bf16": (_c.c_int, [_P, _P, _I64, _P]),
    "fh_quantize_int8_rows": (_c.c_int, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "fh_int8_attention_scores": (_c.c_int, [_P, _P, _P, _P, _c.c_float, _P, _I64, _I64, _I64, _I64, _P]),
    "fh_adaln_modulation": (_c.c_int, [_P, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P]),
    "fh_kv_pages_update": (_c.c_int, [_P, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _P, _P]),
    "fh_kv_cache_write": (_c.c_int, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "fh_kv_cache_read": (_c.c_int, [_P, _P, _I64, _P, _P, _I64, _I64, _P]),
    "fh_kv_attention": (_c.c_int, [_P, _P, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _c.c_float, _c.c_int, _I64,
                                   _I64, _I64, _P, _I64, _P, _P, _c.c_size_t, _P]),
    "fh_kv_attention_workspace_bytes": (_c.c_size_t, [_I64, _I64, _I64, _I64, _I64]),
    "fh_device_status": (_c.c_int, [_P]),
    "fh_selftest_mma_rate": (_c.c_int, [_c.c_int32, _c.c_int32, _c.POINTER(_c.c_int32), _P]),
    "fh_selftest_bounded_wait": (_c.c_int, [_c.c_uint32, _P]),
}
for _name, (_res, _args) in _SIG.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib():
    """The loaded ctypes library (for tests that call the C ABI directly)."""
    return _lib


def _check(status: int):
    if status != FH_OK:
        raise FHError(status, _lib.fh_last_error().decode())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _P(stream.cuda_stream)


def _ptr(t):
    return None if t is None else _P(t.data_ptr())


def _need(t, dtypes, what, ndim=None):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must have dtype in {dtypes}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{what} must have {ndim} dimensions")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8,)


# --- host entry points --------------------------------------------------------

def fh_version() -> int:
    return _lib.fh_version()


def fh_last_error() -> str:
    return _lib.fh_last_error().decode()


def fh_scale_from_amax(amax: float) -> float:
    return _lib.fh_scale_from_amax(float(amax))


def fh_scales_bytes(rows: int, K: int, layout: int = FH_SCALES_MMA_TILED) -> int:
    return _lib.fh_scales_bytes(rows, K, layout)


# --- device entry points ------------------------------------------------------

def fh_amax(x: torch.Tensor, amax: torch.Tensor, stream=None) -> None:
    """amax[0] = max(amax[0], max |x|) for BF16 x [rows, cols] (row stride x.stride(0))."""
    _need(x, _BF16, "x", 2)
    _need(amax, (torch.float32,), "amax")
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    _check(_lib.fh_amax(_ptr(x), x.shape[0], x.shape[1], x.stride(0), _ptr(amax), _stream(stream)))


def fh_quantize_act(x: torch.Tensor, global_scale: float, codes: torch.Tensor, scales: torch.Tensor,
                    clip_count: torch.Tensor | None = None, scale_layout: int = FH_SCALES_MMA_TILED,
                    stream=None) -> None:
    """NVFP4-quantize BF16 x [M, K] into codes [M, K/2] and scales (see include/fh.h)."""
    _need(x, _BF16, "x", 2)
    _need(codes, _U8, "codes")
    _need(scales, _U8, "scales")
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    M, K = x.shape
    if codes.numel() < M * (K // 2) or not codes.is_contiguous():
        raise ValueError("codes must be contiguous with M*K/2 bytes")
    need = fh_scales_bytes(M, K, scale_layout)
    if scales.numel() < need or not scales.is_contiguous():
        raise ValueError(f"scales must be contiguous with {need} bytes")
    if clip_count is not None:
        _need(clip_count, (torch.int64, torch.uint64), "clip_count")
    _check(_lib.fh_quantize_act(_ptr(x), M, K, x.stride(0), float(global_scale), _ptr(codes), _ptr(scales),
                                _ptr(clip_count), scale_layout, _stream(stream)))


def fh_gelu_quantize_act(x: torch.Tensor, global_scale: float, codes: torch.Tensor, scales: torch.Tensor,
                         clip_count: torch.Tensor | None = None, stream=None) -> None:
    """NVFP4 codes and tensor-core-layout scales of GELU(x) for BF16 x [M, K] (row stride x.stride(0))."""
    _need(x, _BF16, "x", 2)
    if x.stride(1) != 1:
        raise ValueError("x must be row-major (unit column stride)")
    _need(codes, _U8, "codes", 2)
    _need(scales, _U8, "scales")
    M, K = x.shape
    if tuple(codes.shape) != (M, K // 2) or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous [M, K/2] uint8 tensor")
    if scales.numel() < fh_scales_bytes(M, K):
        raise ValueError("scales too small for the tensor-core scale layout")
    if clip_count is not None and (clip_count.dtype != torch.int64 or clip_count.device.type != "cuda"):
        raise TypeError("clip_count must be a CUDA int64 tensor")
    _check(_lib.fh_gelu_quantize_act(_ptr(x), M, K, x.stride(0), float(global_scale), _ptr(codes), _ptr(scales),
                                     _ptr(clip_count), _stream(stream)))


def fh_nvfp4_linear(a_codes: torch.Tensor, a_scales: torch.Tensor, a_gscale: float,
                    w_codes: torch.Tensor, w_scales: torch.Tensor, w_gscale: float,
                    bias: torch.Tensor | None, y: torch.Tensor, stream=None) -> None:
    """y[M, N] = bf16(a_g * w_g * A . W^T + bias) on the tcgen05 tensor cores."""
    for t, n in ((a_codes, "a_codes"), (w_codes, "w_codes")):
        _need(t, _U8, n, 2)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scales, _U8, "a_scales")
    _need(w_scales, _U8, "w_scales")
    _need(y, _BF16, "y", 2)
    M, K = a_codes.shape[0], a_codes.shape[1] * 2
    N = w_codes.shape[0]
    if w_codes.shape[1] * 2 != K or tuple(y.shape) != (M, N) or not y.is_contiguous():
        raise ValueError("shape mismatch: a_codes [M, K/2], w_codes [N, K/2], y [M, N] contiguous")
    if a_scales.numel() < fh_scales_bytes(M, K) or w_scales.numel() < fh_scales_bytes(N, K):
        raise ValueError("scale arrays too small for the tensor-core scale layout")
    if bias is not None:
        _need(bias, _BF16, "bias")
        if bias.numel() != N or not bias.is_contiguous():
            raise ValueError("bias must be contiguous with N elements")
    _check(_lib.fh_nvfp4_linear(_ptr(a_codes), _ptr(a_scales), float(a_gscale), _ptr(w_codes), _ptr(w_scales),
                                float(w_gscale), _ptr(bias), _ptr(y), M, N, K, _stream(stream)))


def fh_nvfp4_linear_gelu_quant(a_codes: torch.Tensor, a_scales: torch.Tensor, a_gscale: float,
                               w_codes: torch.Tensor, w_scales: torch.Tensor, w_gscale: float,
                               bias: torch.Tensor | None, out_gscale: float, out_codes: torch.Tensor,
                               out_scales: torch.Tensor, out_clip: torch.Tensor | None = None, stream=None) -> None:
    """NVFP4 input of the next layer, GELU(bf16(a_g * w_g * A . W^T + bias)) quantized with out_gscale,
    written as out_codes [M, N/2] and tensor-core-layout out_scales; out_clip (int64, 1 element) += clips."""
    for t, n in ((a_codes, "a_codes"), (w_codes, "w_codes"), (out_codes, "out_codes")):
        _need(t, _U8, n, 2)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scales, _U8, "a_scales")
    _need(w_scales, _U8, "w_scales")
    _need(out_scales, _U8, "out_scales")
    M, K = a_codes.shape[0], a_codes.shape[1] * 2
    N = w_codes.shape[0]
    if w_codes.shape[1] * 2 != K or tuple(out_codes.shape) != (M, N // 2):
        raise ValueError("shape mismatch: a_codes [M, K/2], w_codes [N, K/2], out_codes [M, N/2]")
    if (a_scales.numel() < fh_scales_bytes(M, K) or w_scales.numel() < fh_scales_bytes(N, K)
            or out_scales.numel() < fh_scales_bytes(M, N)):
        raise ValueError("scale arrays too small for the tensor-core scale layout")
    if bias is not None:
        _need(bias, _BF16, "bias")
        if bias.numel() != N or not bias.is_contiguous():
            raise ValueError("bias must be contiguous with N elements")
    if out_clip is not None and (out_clip.dtype != torch.int64 or out_clip.device.type != "cuda"):
        raise TypeError("out_clip must be a CUDA int64 tensor")
    _check(_lib.fh_nvfp4_linear_gelu_quant(_ptr(a_codes), _ptr(a_scales), float(a_gscale), _ptr(w_codes),
                                           _ptr(w_scales), float(w_gscale), _ptr(bias), float(out_gscale),
                                           _ptr(out_codes), _ptr(out_scales), _ptr(out_clip), M, N, K,
                                           _stream(stream)))


def fh_nvfp4_linear_fused_quant_sync_bytes(M: int) -> int:
    return _lib.fh_nvfp4_linear_fused_quant_sync_bytes(M)


def empty_fused_sync(M: int, device="cuda") -> torch.Tensor:
    """A zeroed sync buffer for fh_nvfp4_linear_fused_quant (each call leaves it zero again)."""
    return torch.zeros(max(1, fh_nvfp4_linear_fused_quant_sync_bytes(M) // 4), dtype=torch.int32, device=device)


def fh_nvfp4_linear_fused_quant(x: torch.Tensor, a_gscale: float, w_codes: torch.Tensor, w_scales: torch.Tensor,
                                w_gscale: float, bias: torch.Tensor | None, y: torch.Tensor, a_codes: torch.Tensor,
                                a_scales: torch.Tensor, clip: torch.Tensor | None, sync: torch.Tensor,
                                stream=None) -> None:
    """y [M, N] = the NVFP4 layer on BF16 x [M, K] with the quantization in the same kernel; also writes x's
    codes and tensor-core-layout scales into a_codes / a_scales (see include/fh.h).  sync: empty_fused_sync(M)."""
    _need(x, _BF16, "x", 2)
    _need(w_codes, _U8, "w_codes", 2)
    _need(w_scales, _U8, "w_scales")
    _need(y, _BF16, "y", 2)
    _need(a_codes, _U8, "a_codes", 2)
    _need(a_scales, _U8, "a_scales")
    _need(sync, (torch.int32, torch.uint32), "sync")
    if x.stride(1) != 1 or not (y.is_contiguous() and a_codes.is_contiguous() and w_codes.is_contiguous()):
        raise ValueError("x rows must be contiguous; y, a_codes, w_codes contiguous")
    M, K = x.shape
    N = w_codes.shape[0]
    if w_codes.shape[1] * 2 != K or tuple(y.shape) != (M, N) or tuple(a_codes.shape) != (M, K // 2):
        raise ValueError("shape mismatch: x [M, K], w_codes [N, K/2], y [M, N], a_codes [M, K/2]")
    if a_scales.numel() < fh_scales_bytes(M, K, FH_SCALES_MMA_TILED):
        raise ValueError("a_scales too small")
    if sync.numel() * 4 < fh_nvfp4_linear_fused_quant_sync_bytes(M):
        raise ValueError("sync too small")
    if bias is not None:
        _need(bias, _BF16, "bias")
    if clip is not None and (clip.dtype != torch.int64 or clip.device.type != "cuda"):
        raise TypeError("clip must be a CUDA int64 tensor")
    _check(_lib.fh_nvfp4_linear_fused_quant(_ptr(x), M, K, x.stride(0), float(a_gscale), _ptr(w_codes),
                                            _ptr(w_scales), float(w_gscale), _ptr(bias), _ptr(y), N, _ptr(a_codes),
                                            _ptr(a_scales), _ptr(clip), _ptr(sync), _stream(stream)))


def fh_nvfp4_linear_host_workspace_bytes(K: int, N: int, chunk_rows: int = 4096) -> int:
    return _lib.fh_nvfp4_linear_host_workspace_bytes(K, N, chunk_rows)


def fh_nvfp4_linear_host(x_host: torch.Tensor, a_gscale: float, w_codes: torch.Tensor, w_scales: torch.Tensor,
                         w_gscale: float, bias: torch.Tensor | None, y_host: torch.Tensor,
                         clip: torch.Tensor | None = None, chunk_rows: int = 4096,
                         workspace: torch.Tensor | None = None, stream=None) -> None:
    """y_host [M, N] = the NVFP4 layer on x_host [M, K]: host BF16 tensors (pin them for overlap), weights on the
    device; chunked upload, quantize, GEMM and download overlap (see include/fh.h).  Ordered on the stream:
    synchronize before reading y_host.  workspace: CUDA uint8 of fh_nvfp4_linear_host_workspace_bytes bytes, or
    None to allocate one for this call."""
    for t, n in ((x_host, "x_host"), (y_host, "y_host")):
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu" or t.dtype not in _BF16 or t.dim() != 2:
            raise TypeError(f"{n} must be a 2-D BF16 CPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(w_codes, _U8, "w_codes", 2)
    _need(w_scales, _U8, "w_scales")
    M, K = x_host.shape
    N = w_codes.shape[0]
    if w_codes.shape[1] * 2 != K or tuple(y_host.shape) != (M, N):
        raise ValueError("shape mismatch: x_host [M, K], w_codes [N, K/2], y_host [M, N]")
    if bias is not None:
        _need(bias, _BF16, "bias")
    if clip is not None and (clip.dtype != torch.int64 or clip.device.type != "cuda"):
        raise TypeError("clip must be a CUDA int64 tensor")
    need = fh_nvfp4_linear_host_workspace_bytes(K, N, chunk_rows)
    own = workspace is None
    if own:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=w_codes.device)
    _need(workspace, _U8, "workspace")
    torch_stream = torch.cuda.current_stream(w_codes.device) if stream is None else stream
    _check(_lib.fh_nvfp4_linear_host(_P(x_host.data_ptr()), M, K, float(a_gscale), _ptr(w_codes), _ptr(w_scales),
                                     float(w_gscale), _ptr(bias), N, _P(y_host.data_ptr()), _ptr(clip), chunk_rows,
                                     _ptr(workspace), workspace.numel(), _stream(torch_stream)))
    if own:
        # The call's work on `stream` still uses the workspace after this returns:
        # the caching allocator must not hand the block to other streams before
        # that work has finished.
        workspace.record_stream(torch_stream)


def fh_nvfp4_linear_host_noalloc(x_host: torch.Tensor, a_gscale: float, w_codes: torch.Tensor,
                                 w_scales: torch.Tensor, w_gscale: float, bias: torch.Tensor | None,
                                 y_host: torch.Tensor, clip: torch.Tensor | None = None, stream=None) -> None:
    """fh_nvfp4_linear_host without a workspace: the chunks are staged in the library's static device scratch
    array (see include/fh.h), so nothing is allocated on the device.  Calls sharing a device must not overlap on
    the GPU.  Ordered on the stream: synchronize before reading y_host."""
    for t, n in ((x_host, "x_host"), (y_host, "y_host")):
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu" or t.dtype not in _BF16 or t.dim() != 2:
            raise TypeError(f"{n} must be a 2-D BF16 CPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(w_codes, _U8, "w_codes", 2)
    _need(w_scales, _U8, "w_scales")
    M, K = x_host.shape
    N = w_codes.shape[0]
    if w_codes.shape[1] * 2 != K or tuple(y_host.shape) != (M, N):
        raise ValueError("shape mismatch: x_host [M, K], w_codes [N, K/2], y_host [M, N]")
    if bias is not None:
        _need(bias, _BF16, "bias")
    if clip is not None and (clip.dtype != torch.int64 or clip.device.type != "cuda"):
        raise TypeError("clip must be a CUDA int64 tensor")
    _check(_lib.fh_nvfp4_linear_host_noalloc(_P(x_host.data_ptr()), M, K, float(a_gscale), _ptr(w_codes),
                                             _ptr(w_scales), float(w_gscale), _ptr(bias), N, _P(y_host.data_ptr()),
                                             _ptr(clip), _stream(stream)))


def fh_scales_to_rowmajor(tiled: torch.Tensor, rowmajor: torch.Tensor, rows: int, K: int, stream=None) -> None:
    _need(tiled, _U8, "tiled")
    _need(rowmajor, _U8, "rowmajor")
    if rowmajor.numel() < rows * (K // 16) or tiled.numel() < fh_scales_bytes(rows, K):
        raise ValueError("buffer too small")
    _check(_lib.fh_scales_to_rowmajor(_ptr(tiled), _ptr(rowmajor), rows, K, _stream(stream)))


def fh_gelu_bf16(x: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    _need(x, _BF16, "x")
    _need(y, _BF16, "y")
    if x.numel() != y.numel() or not x.is_contiguous() or not y.is_contiguous():
        raise ValueError("x and y must be contiguous with the same number of elements")
    _check(_lib.fh_gelu_bf16(_ptr(x), _ptr(y), x.numel(), _stream(stream)))


def fh_quantize_int8_rows(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Per-row symmetric INT8: BF16 x [rows, d] (row stride x.stride(0)) -> q int8 [rows, d], scales FP32 [rows]."""
    _need(x, _BF16, "x", 2)
    _need(q, (torch.int8,), "q", 2)
    _need(scales, (torch.float32,), "scales", 1)
    rows, d = x.shape
    if x.stride(1) != 1 or not q.is_contiguous() or not scales.is_contiguous():
        raise ValueError("x needs unit column stride; q and scales must be contiguous")
    if tuple(q.shape) != (rows, d) or scales.numel() != rows:
        raise ValueError("shape mismatch: q [rows, d], scales [rows]")
    _check(_lib.fh_quantize_int8_rows(_ptr(x), rows, d, x.stride(0), _ptr(q), _ptr(scales), _stream(stream)))


def fh_int8_attention_scores(q: torch.Tensor, q_scales: torch.Tensor, k: torch.Tensor, k_scales: torch.Tensor,
                             sm_scale: float, s: torch.Tensor, stream=None) -> None:
    """S [heads, tq, tk] FP32 = (acc * (s_q * sm_scale)) * s_k for INT8 q [heads, tq, d], k [heads, tk, d]."""
    _need(q, (torch.int8,), "q", 3)
    _need(k, (torch.int8,), "k", 3)
    _need(q_scales, (torch.float32,), "q_scales")
    _need(k_scales, (torch.float32,), "k_scales")
    _need(s, (torch.float32,), "s", 3)
    for t, n in ((q, "q"), (k, "k"), (q_scales, "q_scales"), (k_scales, "k_scales"), (s, "s")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    heads, tq, d = q.shape
    tk = k.shape[1]
    if (k.shape[0] != heads or k.shape[2] != d or tuple(s.shape) != (heads, tq, tk)
            or q_scales.numel() != heads * tq or k_scales.numel() != heads * tk):
        raise ValueError("shape mismatch: q [H, tq, d], k [H, tk, d], scales [H, t], s [H, tq, tk]")
    _check(_lib.fh_int8_attention_scores(_ptr(q), _ptr(q_scales), _ptr(k), _ptr(k_scales), float(sm_scale),
                                         _ptr(s), heads, tq, tk, d, _stream(stream)))


def fh_adaln_modulation(temb: torch.Tensor, basis: torch.Tensor, proj: torch.Tensor, bias: torch.Tensor | None,
                        code: torch.Tensor, mod: torch.Tensor, stream=None) -> None:
    """code [bt, r] = temb [bt, d] . basis^T (basis [r, d] FP16); mod [blocks, bt, n] = proj [blocks, n, r] . code^T
    + bias [blocks, n], all FP32 results."""
    _need(temb, _BF16, "temb", 2)
    _need(basis, (torch.float16,), "basis", 2)
    _need(proj, (torch.float16,), "proj", 3)
    _need(code, (torch.float32,), "code", 2)
    _need(mod, (torch.float32,), "mod", 3)
    if bias is not None:
        _need(bias, (torch.float16,), "bias", 2)
    for t, nm in ((temb, "temb"), (basis, "basis"), (proj, "proj"), (code, "code"), (mod, "mod"), (bias, "bias")):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    bt, d = temb.shape
    r = basis.shape[0]
    blocks, n = proj.shape[0], proj.shape[1]
    if (basis.shape[1] != d or proj.shape[2] != r or tuple(code.shape) != (bt, r)
            or tuple(mod.shape) != (blocks, bt, n) or (bias is not None and tuple(bias.shape) != (blocks, n))):
        raise ValueError("shape mismatch: temb [bt, d], basis [r, d], proj [blocks, n, r], bias [blocks, n], "
                         "code [bt, r], mod [blocks, bt, n]")
    _check(_lib.fh_adaln_modulation(_ptr(temb), bt, d, _ptr(basis), r, _ptr(proj), _ptr(bias), blocks, n,
                                    _ptr(code), _ptr(mod), _stream(stream)))


# --- the paged NVFP4 key/value cache -------------------------------------------------

class _CKVCache(_c.Structure):
    """fh_kv_cache of include/fh.h."""
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("num_pages", _I64),
                ("page_size", _I64), ("kv_heads", _I64), ("head_dim", _I64), ("k_gscale", _c.c_float),
                ("v_gscale", _c.c_float)]


class KVCache:
    """One attention layer's keys and values in pages of NVFP4 tokens (fh_kv_cache in include/fh.h): uint8 codes
    [pages, kv_heads, page_size, head_dim / 2] and E4M3 scales [pages, kv_heads, page_size, head_dim / 16] of each,
    contiguous on one device, and their FP32 scales.  Holds the tensors; empty_kv_cache makes new ones.  Its
    attributes are fixed: calls read the C struct that was filled from them."""

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                 k_gscale: float, v_gscale: float):
        shape = None
        for t, n, per in ((k_codes, "k_codes", 2), (k_scales, "k_scales", 16), (v_codes, "v_codes", 2),
                          (v_scales, "v_scales", 16)):
            _need(t, _U8, n, 4)
            s = (*t.shape[:3], t.shape[3] * per)
            if (shape is not None and s != shape) or not t.is_contiguous() or t.device != k_codes.device:
                raise ValueError("k_codes and v_codes [pages, kv_heads, page_size, head_dim / 2], k_scales and "
                                 "v_scales [pages, kv_heads, page_size, head_dim / 16], contiguous on one device")
            shape = s
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = shape
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_gscale, self.v_gscale = float(k_gscale), float(v_gscale)
        self.device, self.index = k_codes.device, k_codes.get_device()
        self._c = _CKVCache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                            self.num_pages, self.page_size, self.kv_heads, self.head_dim, self.k_gscale,
                            self.v_gscale)
        self._ref = _P(_c.addressof(self._c))

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"KVCache.{name} is fixed; make another KVCache of the tensors")
        super().__setattr__(name, value)


def empty_kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, k_gscale: float, v_gscale: float,
                   device="cuda") -> KVCache:
    """A cache of num_pages uninitialised pages."""
    def new(per):
        return torch.empty((num_pages, kv_heads, page_size, head_dim // per), dtype=torch.uint8, device=device)
    return KVCache(new(2), new(16), new(2), new(16), k_gscale, v_gscale)


# The cache's calls run once a layer and token, some for a few microseconds: their checks are written for few
# attribute reads.  A device is compared by its index (0.06 us; by its type 0.21) and the stream is read as the raw
# handle (0.07 us; 1.3 through torch.cuda.current_stream, 3.4 by _stream).

def _need_all(index, dtype, names, *tensors):
    """Contiguous tensors of one dtype on CUDA device `index`."""
    for t in tensors:
        if type(t) is not torch.Tensor and not isinstance(t, torch.Tensor) or t.dtype is not dtype:
            raise TypeError(f"{names} must be tensors of {dtype}")
        if t.get_device() != index:
            raise ValueError(f"{names} must be on cuda:{index}")
        if not t.is_contiguous():
            raise ValueError(f"{names} must be contiguous")


def _need_current(index):
    """The library launches on the current device."""
    if index < 0:
        raise TypeError("tensors must be CUDA tensors")
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on cuda:{index}, which is not the current device")


def _raw_stream(stream, index):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def fh_kv_pages_update(held: torch.Tensor, target: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                       free_count: torch.Tensor, free_count_out: torch.Tensor, lens: torch.Tensor,
                       q_starts: torch.Tensor, slots: torch.Tensor, status: torch.Tensor, page_size: int,
                       stream=None) -> None:
    """Block tables, free stack, lens, q_starts and slots of a step in which request b goes from held[b] to target[b]
    cached tokens (see include/fh.h).  int32: held, target, lens [batch], block_table [batch, max_pages], free_pages
    [capacity], q_starts [batch + 1], free_count, free_count_out, status [1]; int64 slots.  lens may be held or
    target, free_count_out may be free_count."""
    if not isinstance(held, torch.Tensor):
        raise TypeError("held must be a tensor")
    index = held.get_device()
    _need_current(index)
    _need_all(index, torch.int32, "held, target, block_table, free_pages, free_count, free_count_out, lens, q_starts, "
              "status", held, target, block_table, free_pages, free_count, free_count_out, lens, q_starts, status)
    _need_all(index, torch.int64, "slots", slots)
    n = held.numel()
    if (target.numel() != n or lens.numel() != n or q_starts.numel() != n + 1 or block_table.dim() != 2
            or block_table.shape[0] != n or free_count.numel() != 1 or free_count_out.numel() != 1
            or status.numel() != 1):
        raise ValueError("shape mismatch: held, target, lens [batch], q_starts [batch + 1], block_table [batch, "
                         "max_pages], free_count, free_count_out, status [1]")
    _check(_lib.fh_kv_pages_update(held.data_ptr(), target.data_ptr(), n, _index(page_size), block_table.data_ptr(),
                                   block_table.shape[1], free_pages.data_ptr(), free_pages.numel(),
                                   free_count.data_ptr(), free_count_out.data_ptr(), lens.data_ptr(),
                                   q_starts.data_ptr(), slots.data_ptr(), slots.numel(), status.data_ptr(),
                                   _raw_stream(stream, index)))


def _kv_rows(cache, t, tokens, what):
    """The token stride of BF16 rows [tokens, kv_heads, head_dim] of the cache's heads."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _BF16:
        raise TypeError(f"{what} must be a BF16 tensor")
    if t.get_device() != cache.index:
        raise ValueError(f"{what} must be on cuda:{cache.index}")
    if t.shape != (tokens, cache.kv_heads, cache.head_dim):
        raise ValueError(f"{what} must have the shape [tokens, kv_heads, head_dim] of slots and cache")
    return _row_stride(t, what)


def _row_stride(t, what):
    """The token stride of [tokens, heads, d] rows, whose heads must lie one after the other."""
    tokens, heads, d = t.shape
    s = t.stride()
    if s[2] != 1 or (s[1] != d and heads > 1):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return s[0] if tokens > 1 else heads * d


def fh_kv_cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                      clip_count: torch.Tensor | None = None, stream=None) -> None:
    """Quantize BF16 k, v [tokens, kv_heads, head_dim] (any token stride) into the cache's slots (int64 [tokens];
    negative: left out; distinct); clip_count (int64, 1 element) += elements beyond the scales' range."""
    index = cache.index
    _need_current(index)
    _need_all(index, torch.int64, "slots", slots)
    n = slots.numel()
    ldk, ldv = _kv_rows(cache, k, n, "k"), _kv_rows(cache, v, n, "v")
    if clip_count is not None:
        _need_all(index, torch.int64, "clip_count", clip_count)
        if clip_count.numel() < 1:
            raise ValueError("clip_count must have an element")
    _check(_lib.fh_kv_cache_write(cache._ref, k.data_ptr(), v.data_ptr(), n, ldk, ldv, slots.data_ptr(),
                                  None if clip_count is None else clip_count.data_ptr(), _raw_stream(stream, index)))


def fh_kv_cache_read(cache: KVCache, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """BF16 k, v [tokens, kv_heads, head_dim] = the cached values of slots (int64 [tokens]; rows of negative ones are
    left as they were)."""
    index = cache.index
    _need_current(index)
    _need_all(index, torch.int64, "slots", slots)
    n = slots.numel()
    ldk, ldv = _kv_rows(cache, k, n, "k"), _kv_rows(cache, v, n, "v")
    _check(_lib.fh_kv_cache_read(cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), ldk, ldv,
                                 _raw_stream(stream, index)))


def fh_kv_attention_workspace_bytes(total_q: int, batch: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return _lib.fh_kv_attention_workspace_bytes(total_q, batch, q_heads, kv_heads, head_dim)


def empty_kv_attention_workspace(total_q: int, batch: int, q_heads: int, kv_heads: int, head_dim: int,
                                 device="cuda") -> torch.Tensor:
    """A zeroed workspace for fh_kv_attention of at most these sizes (each call leaves its counters zero again)."""
    need = fh_kv_attention_workspace_bytes(total_q, batch, q_heads, kv_heads, head_dim)
    if need == 0:
        raise ValueError("sizes that fh_kv_attention does not support")
    return torch.zeros(need, dtype=torch.uint8, device=device)


def fh_kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lens: torch.Tensor,
                    q_starts: torch.Tensor, sm_scale: float, out: torch.Tensor, workspace: torch.Tensor, *,
                    causal: bool = True, window: int = 0, max_q: int | None = None, max_kv: int | None = None,
                    lse: torch.Tensor | None = None, stream=None) -> None:
    """out [total_q, q_heads, head_dim] = attention of BF16 q (same shape; any token strides) over the cache, for
    requests with query rows q_starts[b] .. q_starts[b + 1] - 1 and lens[b] cached tokens in the pages of block_table
    [batch, max_pages] (int32 all; see include/fh.h).  workspace: empty_kv_attention_workspace(...).  max_q, max_kv:
    upper bounds of a request's queries and cached tokens, which choose the kernel.  lse: FP32 [total_q, q_heads]."""
    index = cache.index
    _need_current(index)
    for t, what in ((q, "q"), (out, "out")):
        if not isinstance(t, torch.Tensor) or t.dtype not in _BF16:
            raise TypeError(f"{what} must be a BF16 tensor")
    _need_all(index, torch.int32, "block_table, lens, q_starts", block_table, lens, q_starts)
    _need_all(index, torch.uint8, "workspace", workspace)
    shape = q.shape
    n = lens.numel()
    if (len(shape) != 3 or shape[2] != cache.head_dim or out.shape != shape or q.get_device() != index
            or out.get_device() != index or q_starts.numel() != n + 1 or block_table.dim() != 2
            or block_table.shape[0] != n):
        raise ValueError("shape mismatch: q, out [total_q, q_heads, head_dim], lens [batch], q_starts [batch + 1], "
                         "block_table [batch, max_pages], on the cache's device")
    total_q, heads, _ = shape
    if lse is not None:
        _need_all(index, torch.float32, "lse", lse)
        if lse.shape != (total_q, heads):
            raise ValueError("lse must be [total_q, q_heads]")
    max_pages = block_table.shape[1]
    _check(_lib.fh_kv_attention(cache._ref, q.data_ptr(), total_q, heads, _row_stride(q, "q"), block_table.data_ptr(),
                                max_pages, lens.data_ptr(), q_starts.data_ptr(), n, float(sm_scale), 1 if causal else 0,
                                _index(window), total_q if max_q is None else _index(max_q),
                                max_pages * cache.page_size if max_kv is None else _index(max_kv), out.data_ptr(),
                                _row_stride(out, "out"), None if lse is None else lse.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _raw_stream(stream, index)))


def fh_selftest_bounded_wait(limit_us: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test (see include/fh.h); fh_device_status then reports the timeout."""
    _check(_lib.fh_selftest_bounded_wait(int(limit_us), _stream(stream)))


def fh_selftest_mma_rate(iters: int, with_scale_copies: bool = False, stream=None) -> int:
    """Enqueue the FP4 tensor-rate probe (see include/fh.h); returns the number of CTA pairs.
    Each pair performs iters * 2 * 256 * 256 * 256 FLOP."""
    pairs = _c.c_int32(0)
    _check(_lib.fh_selftest_mma_rate(int(iters), 1 if with_scale_copies else 0, _c.byref(pairs), _stream(stream)))
    return pairs.value


def fh_device_status(stream=None) -> None:
    """Synchronize and raise FHError(FH_ERR_TIMEOUT) if a kernel gave up on a bounded wait."""
    _check(_lib.fh_device_status(_stream(stream)))


# --- allocation helpers (marshalling only) ----------------------------------------

def empty_quantized(rows: int, K: int, device="cuda", layout: int = FH_SCALES_MMA_TILED):
    """Uninitialised (codes [rows, K/2], scales) buffers for fh_quantize_act."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=device)
    scales = torch.empty(max(fh_scales_bytes(rows, K, layout), 1), dtype=torch.uint8, device=device)
    return codes, scales
