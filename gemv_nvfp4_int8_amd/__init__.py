"""Python binding of libqproj, the gfx950 quantized dense projection library.

Argument marshalling only: each function takes torch tensors (device memory
owned by the caller), checks their dtypes and shapes so that no kernel can
be handed a buffer smaller than it will touch, and calls the C entry point of
the same name with raw pointers, sizes and torch's current HIP stream.
Every step of the computation runs in the library's HIP kernels; there is no
fallback.  If ``libqproj.so`` has not been built, the first call into the
library raises ImportError (build it with ``__graft_entry__.build()`` or
``python -m gemv_nvfp4_int8_amd._build``).

The operations and their rounding rules are documented in include/qproj.h,
(the operators around the projections) include/qproj_layer.h and (rotary
positions, paged cache, attention and log probabilities)
include/qproj_decoder.h.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqproj.so")

QP_OK = 0
QP_ERR_NULL = -1
QP_ERR_SHAPE = -2
QP_ERR_RANGE = -3
QP_ERR_FORMAT = -4
QP_ERR_HIP = -5
QP_ERR_ALIGN = -6
QP_ERR_ALLOC = -7
QP_ERR_SCRATCH = -8

QP_FP8_PER_ROW = 0
QP_FP8_BLOCK128 = 1
QP_FP8_SINGLE_SCALE = 2
QP_BF16 = 3
QP_NVFP4 = 4

QP_ACT_FP8_ROW = 0
QP_ACT_FP8_BLOCK128 = 1
QP_ACT_INT8_BLOCK32 = 2
QP_ACT_BF16 = 16

QP_BLOCKSCALE_TILES_128 = 1
QP_BLOCKSCALE_TILES_256 = 2
QP_BLOCKSCALE_TILES_256_QUARTERS = 3
QP_BLOCKSCALE_KSPLIT = 256

QP_KV_BF16 = 0
QP_KV_FP8_ROW = 1

QP_ROPE_HALF = 0
QP_ROPE_INTERLEAVED = 1

QP_ROPE_PLAIN = 0
QP_ROPE_LINEAR = 1
QP_ROPE_BASE = 2
QP_ROPE_WAVELENGTH = 3
QP_ROPE_RAMP = 4

QP_LOGITS_BF16 = 0
QP_LOGITS_F32 = 1
QP_LOGPROBS_MAX_TOP = 32

QP_TILES_BANDED = 0
QP_TILES_MFAST = 1
QP_TILES_NFAST = 2


class QProjError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libqproj.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"libqproj.so not found at {LIB_PATH}: the HIP library must be "
                "built (python -m gemv_nvfp4_int8_amd._build) -- there is no "
                "fallback path")
        L = ctypes.CDLL(LIB_PATH)
        P, U, F, I = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_float, ctypes.c_int
        D, Q = ctypes.c_double, ctypes.c_uint64
        PP = ctypes.POINTER(ctypes.c_void_p)
        sig = {
            "requant_w_nvfp4_int8": [P, P, F, P, P, U, U, P],
            "requant_a_bf16_int8": [P, P, P, U, U, P],
            "int8_gemm_blockscaled": [P, P, P, P, P, U, U, U, P],
            "int8_gemm_blockscaled_f16ops": [P, P, P, P, P, U, U, U, P],
            "int8_w4a8_prefill": [P, P, P, P, P, P, U, U, U, P],
            "int8_w4a8_prefill_noalloc": [P, P, P, P, U, U, U, P],
            "qproj_encode_test": [I, P, P, U, P],
            "int8_gemm_block_partials": [P, P, P, U, U, U, P],
            "quantize_bf16_nvfp4": [P, P, P, F, U, U, P],
            "w4a4_gemm": [P, P, P, P, P, F, F, U, U, U, P],
            "w4a4_gemm_tiles": [P, P, P, P, P, F, F, U, U, U, I, P],
            "requant_w_blockfp8_rowwise": [I, P, P, P, P, PP, PP, U, U, P],
            "quant_rowwise_fp8": [P, P, P, U, U, P],
            "fp8_gemm_rowscale": [P, P, P, P, P, U, U, U, P],
            "fp8_rowwise_proj": [I, P, P, P, P, P, P, P, P, U, U, U, P],
            "fp8_gemv_rowscale": [P, P, P, P, U, U, U, P],
            "fp8_gemv_blockscale": [P, P, P, P, U, U, U, P],
            "w4a16_gemv": [P, P, P, F, P, U, U, U, P],
            "rmsnorm_residual_quant": [P, P, P, F, I, P, P, P, U, U, P],
            "silu_mul_quant": [P, I, P, P, U, U, P],
            "fp8_gemm_blockscale": [P, P, P, P, P, U, U, U, P],
            "fp8_gemm_blockscale_kernel": [U, U, U],
            "moe_fp8_blockscale": [P, P, P, P, P, P, P, ctypes.c_uint64, P, U, U, U, U, U, I, P],
            "rope_inv_freq": [P, U, D, I, D, D, D, U],
            "qk_norm_rope_cache": [P, P, P, F, P, P, F, I, U, P, I, P, P, P, P, P, U, U, U, U, U, U, P],
            "paged_attention": [P, I, P, P, P, P, P, P, P, F, U, P, Q, P, U, U, U, U, U, U, U, U, U, P],
            "token_logprobs": [P, I, P, P, P, P, P, P, Q, U, U, U, P],
            "qproj_cache_create": [PP],
            "qproj_cache_destroy": [P],
            "qproj_cache_evict": [P, P],
            "qproj_cache_stats": [P, ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)],
            "requant_w_blockfp8_rowwise_cached": [P, I, P, P, U, U, PP, PP, P],
            "requant_w_nvfp4_int8_cached": [P, P, P, F, U, U, PP, PP, P],
            "fp8_rowwise_proj_cached": [P, I, P, P, P, P, P, P, U, U, U, P],
            "int8_w4a8_prefill_cached": [P, P, P, P, F, P, P, P, U, U, U, P],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.qproj_launch_count.restype = ctypes.c_uint64
        L.qproj_launch_count.argtypes = []
        L.qproj_status_string.restype = ctypes.c_char_p
        L.qproj_status_string.argtypes = [ctypes.c_int]
        L.qproj_noalloc_scratch_bytes.restype = ctypes.c_uint64
        L.qproj_noalloc_scratch_bytes.argtypes = []
        L.moe_fp8_blockscale_workspace.restype = ctypes.c_uint64
        L.moe_fp8_blockscale_workspace.argtypes = [U, U, U]
        L.paged_attention_workspace.restype = ctypes.c_uint64
        L.paged_attention_workspace.argtypes = [U, U, U, U, U, U]
        L.token_logprobs_workspace.restype = ctypes.c_uint64
        L.token_logprobs_workspace.argtypes = [U, U, U]
        L.qproj_abi_version.restype = ctypes.c_int
        L.qproj_abi_version.argtypes = []
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().qproj_status_string(int(status)).decode()


def launch_count() -> int:
    return int(lib().qproj_launch_count())


def abi_version() -> int:
    return int(lib().qproj_abi_version())


# ------------------------------------------------------------------ helpers
# torch's current stream of the current device, as a raw handle.  The
# private accessor costs ~0.1 us against ~2.7 us for building a Stream object
# (per-call overhead matters: a narrow GEMV runs in a few microseconds).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor):
    return t.data_ptr()


def _need(t: torch.Tensor, name: str, dtypes, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


def _ptr_or_null(t):
    return None if t is None else t.data_ptr()


def _one_device(*tensors):
    """The one device index of the tensors given (None is passed over)."""
    devices = {t.get_device() for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError(f"tensors on several devices: {sorted(devices)}")
    return devices.pop()


def _need_on(device, t, name, dtypes, shape=None):
    """_need of a tensor on `device` (no shape: the caller has taken it from the tensor)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.get_device() != device:
        raise ValueError(f"{name}: on device {t.get_device()}, not {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


def _outside_u32(name):
    """Raised where whole numbers, or-ed, pass 32 bits: the library would take them
    modulo 2^32."""
    return ValueError(f"{name}: a whole number outside 0..2^32-1")


def _current(device):
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"tensors on device {device}, which is not the current one")


def _check(fn: str, status: int):
    if status != QP_OK:
        raise QProjError(fn, status)


BF16 = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") \
    else (torch.bfloat16, torch.int16)
U8 = (torch.uint8, torch.float8_e4m3fn)
I8 = (torch.int8,)
F32 = (torch.float32,)
I32 = (torch.int32,)


# --------------------------------------------------------------- entry points
def requant_w_nvfp4_int8(w_packed, w_e4m3, scale2, w_i8, w_scale, stream=None):
    n, kh = w_packed.shape
    k = 2 * kh
    _need(w_packed, "w_packed", U8, (n, kh))
    _need(w_e4m3, "w_e4m3", U8, (n, k // 16))
    _need(w_i8, "w_i8", I8, (n, k))
    _need(w_scale, "w_scale", F32, (n, k // 32))
    _check("requant_w_nvfp4_int8", lib().requant_w_nvfp4_int8(
        _ptr(w_packed), _ptr(w_e4m3), float(scale2), _ptr(w_i8), _ptr(w_scale),
        n, k, _stream(stream)))


def requant_a_bf16_int8(a, a_i8, a_scale, stream=None):
    m, k = a.shape
    _need(a, "a", BF16, (m, k))
    _need(a_i8, "a_i8", I8, (m, k))
    _need(a_scale, "a_scale", F32, (m, k // 32))
    _check("requant_a_bf16_int8", lib().requant_a_bf16_int8(
        _ptr(a), _ptr(a_i8), _ptr(a_scale), m, k, _stream(stream)))


def int8_gemm_blockscaled(a_i8, w_i8, a_scale, w_scale, out, stream=None):
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _need(a_i8, "a_i8", I8, (m, k))
    _need(w_i8, "w_i8", I8, (n, k))
    _need(a_scale, "a_scale", F32, (m, k // 32))
    _need(w_scale, "w_scale", F32, (n, k // 32))
    _need(out, "out", BF16, (m, n))
    _check("int8_gemm_blockscaled", lib().int8_gemm_blockscaled(
        _ptr(a_i8), _ptr(w_i8), _ptr(a_scale), _ptr(w_scale), _ptr(out),
        m, n, k, _stream(stream)))


def int8_gemm_blockscaled_f16ops(a_i8, w_i8, a_scale, w_scale, out, stream=None):
    """The operand-route ablation of int8_gemm_blockscaled (FP16 MFMA on
    converted operands; bit-identical output; k % 128 == 0)."""
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _need(a_i8, "a_i8", I8, (m, k))
    _need(w_i8, "w_i8", I8, (n, k))
    _need(a_scale, "a_scale", F32, (m, k // 32))
    _need(w_scale, "w_scale", F32, (n, k // 32))
    _need(out, "out", BF16, (m, n))
    _check("int8_gemm_blockscaled_f16ops", lib().int8_gemm_blockscaled_f16ops(
        _ptr(a_i8), _ptr(w_i8), _ptr(a_scale), _ptr(w_scale), _ptr(out),
        m, n, k, _stream(stream)))


def int8_w4a8_prefill(a_bf16, w_i8, w_scale, a_i8_scratch, a_scale_scratch,
                      out, stream=None):
    m, k = a_bf16.shape
    n = w_i8.shape[0]
    _need(a_bf16, "a_bf16", BF16, (m, k))
    _need(w_i8, "w_i8", I8, (n, k))
    _need(w_scale, "w_scale", F32, (n, k // 32))
    _need(a_i8_scratch, "a_i8_scratch", I8, (m, k))
    _need(a_scale_scratch, "a_scale_scratch", F32, (m, k // 32))
    _need(out, "out", BF16, (m, n))
    _check("int8_w4a8_prefill", lib().int8_w4a8_prefill(
        _ptr(a_bf16), _ptr(w_i8), _ptr(w_scale), _ptr(a_i8_scratch),
        _ptr(a_scale_scratch), _ptr(out), m, n, k, _stream(stream)))


QP_ENC_E4M3_NOSAT, QP_ENC_E2M1_NOSAT, QP_ENC_INT8 = 0, 1, 2
QP_ENC_E4M3, QP_ENC_E2M1, QP_ENC_E4M3_SCALE = 3, 4, 5


def encode_test(kind, y, out, stream=None):
    """Test export: the kernels' device encoder `kind` on float32 values y
    (a 1-D tensor, length a multiple of 8), one code byte per value in out."""
    n = y.numel()
    _need(y, "y", F32, (n,))
    _need(out, "out", U8, (n,))
    _check("qproj_encode_test", lib().qproj_encode_test(int(kind), _ptr(y), _ptr(out), n,
                                                        _stream(stream)))


def noalloc_scratch_bytes() -> int:
    return int(lib().qproj_noalloc_scratch_bytes())


def int8_w4a8_prefill_noalloc(a_bf16, w_i8, w_scale, out, stream=None):
    """int8_w4a8_prefill with the activation scratch held inside the library
    (a fixed per-GPU array): allocates nothing; calls on one GPU must not
    overlap."""
    m, k = a_bf16.shape
    n = w_i8.shape[0]
    _need(a_bf16, "a_bf16", BF16, (m, k))
    _need(w_i8, "w_i8", I8, (n, k))
    _need(w_scale, "w_scale", F32, (n, k // 32))
    _need(out, "out", BF16, (m, n))
    _check("int8_w4a8_prefill_noalloc", lib().int8_w4a8_prefill_noalloc(
        _ptr(a_bf16), _ptr(w_i8), _ptr(w_scale), _ptr(out), m, n, k, _stream(stream)))


def int8_gemm_block_partials(a_i8, w_i8, p, stream=None):
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _need(a_i8, "a_i8", I8, (m, k))
    _need(w_i8, "w_i8", I8, (n, k))
    _need(p, "p", I32, (m, n, k // 32))
    _check("int8_gemm_block_partials", lib().int8_gemm_block_partials(
        _ptr(a_i8), _ptr(w_i8), _ptr(p), m, n, k, _stream(stream)))


def quantize_bf16_nvfp4(x, packed, scale, scale2=1.0, stream=None):
    rows, k = x.shape
    _need(x, "x", BF16, (rows, k))
    _need(packed, "packed", U8, (rows, k // 2))
    _need(scale, "scale", U8, (rows, k // 16))
    _check("quantize_bf16_nvfp4", lib().quantize_bf16_nvfp4(
        _ptr(x), _ptr(packed), _ptr(scale), float(scale2), rows, k,
        _stream(stream)))


def w4a4_gemm(a_packed, a_scale, w_packed, w_scale, out, scale_a2, scale_w2,
              stream=None, tile_order=None):
    """tile_order: None (w4a4_gemm) or one of QP_TILES_* (w4a4_gemm_tiles)."""
    m, kh = a_packed.shape
    n = w_packed.shape[0]
    k = 2 * kh
    _need(a_packed, "a_packed", U8, (m, kh))
    _need(a_scale, "a_scale", U8, (m, k // 16))
    _need(w_packed, "w_packed", U8, (n, kh))
    _need(w_scale, "w_scale", U8, (n, k // 16))
    _need(out, "out", BF16, (m, n))
    if tile_order is None:
        _check("w4a4_gemm", lib().w4a4_gemm(
            _ptr(a_packed), _ptr(a_scale), _ptr(w_packed), _ptr(w_scale), _ptr(out),
            float(scale_a2), float(scale_w2), m, n, k, _stream(stream)))
    else:
        _check("w4a4_gemm_tiles", lib().w4a4_gemm_tiles(
            _ptr(a_packed), _ptr(a_scale), _ptr(w_packed), _ptr(w_scale), _ptr(out),
            float(scale_a2), float(scale_w2), m, n, k, int(tile_order), _stream(stream)))


def requant_w_blockfp8_rowwise(fmt, w, scale, w_out=None, scale_out=None,
                               stream=None):
    """Returns the (weight_ptr, scale_ptr) pair the row-wise GEMM should read:
    the inputs' own pointers for QP_FP8_PER_ROW, w_out / scale_out after the
    requant for QP_FP8_BLOCK128."""
    n, k = w.shape
    _need(w, "w", U8, (n, k))
    if fmt == QP_FP8_BLOCK128:
        _need(scale, "scale", F32, (n // 128, k // 128))
        _need(w_out, "w_out", U8, (n, k))
        _need(scale_out, "scale_out", F32, (n,))
    elif fmt == QP_FP8_PER_ROW:
        _need(scale, "scale", F32, (n,))
    wres, sres = ctypes.c_void_p(), ctypes.c_void_p()
    _check("requant_w_blockfp8_rowwise", lib().requant_w_blockfp8_rowwise(
        int(fmt), _ptr(w), _ptr(scale),
        _ptr(w_out) if w_out is not None else None,
        _ptr(scale_out) if scale_out is not None else None,
        ctypes.byref(wres), ctypes.byref(sres), n, k, _stream(stream)))
    return wres.value, sres.value


def quant_rowwise_fp8(x, q, scale, stream=None):
    rows, k = x.shape
    _need(x, "x", BF16, (rows, k))
    _need(q, "q", U8, (rows, k))
    _need(scale, "scale", F32, (rows,))
    _check("quant_rowwise_fp8", lib().quant_rowwise_fp8(
        _ptr(x), _ptr(q), _ptr(scale), rows, k, _stream(stream)))


def fp8_gemm_rowscale(a, a_scale, w, w_scale, out, stream=None):
    m, k = a.shape
    n = w.shape[0]
    _need(a, "a", U8, (m, k))
    _need(a_scale, "a_scale", F32, (m,))
    _need(w, "w", U8, (n, k))
    _need(w_scale, "w_scale", F32, (n,))
    _need(out, "out", BF16, (m, n))
    _check("fp8_gemm_rowscale", lib().fp8_gemm_rowscale(
        _ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(out), m, n, k,
        _stream(stream)))


def fp8_rowwise_proj(fmt, w, w_scale, w_rowwise, w_rowwise_scale, act, act_q,
                     act_scale, out, stream=None):
    n, k = w.shape
    m = act.shape[0]
    _need(w, "w", U8, (n, k))
    _need(act, "act", BF16, (m, k))
    _need(act_q, "act_q", U8, (m, k))
    _need(act_scale, "act_scale", F32, (m,))
    _need(out, "out", BF16, (m, n))
    if fmt == QP_FP8_BLOCK128:
        _need(w_scale, "w_scale", F32, (n // 128, k // 128))
        _need(w_rowwise, "w_rowwise", U8, (n, k))
        _need(w_rowwise_scale, "w_rowwise_scale", F32, (n,))
    else:
        _need(w_scale, "w_scale", F32, (n,))
    _check("fp8_rowwise_proj", lib().fp8_rowwise_proj(
        int(fmt), _ptr(w), _ptr(w_scale),
        _ptr(w_rowwise) if w_rowwise is not None else None,
        _ptr(w_rowwise_scale) if w_rowwise_scale is not None else None,
        _ptr(act), _ptr(act_q), _ptr(act_scale), _ptr(out), m, n, k,
        _stream(stream)))


def fp8_gemv_rowscale(x, w, row_scale, out, stream=None):
    m, k = x.shape
    n = w.shape[0]
    _need(x, "x", BF16, (m, k))
    _need(w, "w", U8, (n, k))
    _need(row_scale, "row_scale", F32, (n,))
    _need(out, "out", BF16, (m, n))
    _check("fp8_gemv_rowscale", lib().fp8_gemv_rowscale(
        _ptr(x), _ptr(w), _ptr(row_scale), _ptr(out), m, n, k, _stream(stream)))


def fp8_gemv_blockscale(x, w, block_scale, out, stream=None):
    m, k = x.shape
    n = w.shape[0]
    _need(x, "x", BF16, (m, k))
    _need(w, "w", U8, (n, k))
    _need(block_scale, "block_scale", F32, (n // 128, k // 128))
    _need(out, "out", BF16, (m, n))
    _check("fp8_gemv_blockscale", lib().fp8_gemv_blockscale(
        _ptr(x), _ptr(w), _ptr(block_scale), _ptr(out), m, n, k, _stream(stream)))


def w4a16_gemv(x, w_packed, w_e4m3, scale2, out, stream=None):
    m, k = x.shape
    n = w_packed.shape[0]
    _need(x, "x", BF16, (m, k))
    _need(w_packed, "w_packed", U8, (n, k // 2))
    _need(w_e4m3, "w_e4m3", U8, (n, k // 16))
    _need(out, "out", BF16, (m, n))
    _check("w4a16_gemv", lib().w4a16_gemv(
        _ptr(x), _ptr(w_packed), _ptr(w_e4m3), float(scale2), _ptr(out), m, n, k,
        _stream(stream)))


def _need_act(q, scale, fmt, rows, k):
    """Check the output pair of an activation format (qp_act_format)."""
    if fmt == QP_ACT_FP8_BLOCK128:
        _need(q, "q", U8, (rows, k))
        _need(scale, "scale", F32, (rows, (k + 127) // 128))
    elif fmt == QP_ACT_FP8_ROW:
        _need(q, "q", U8, (rows, k))
        flat = isinstance(scale, torch.Tensor) and scale.dim() == 1
        _need(scale, "scale", F32, (rows,) if flat else (rows, 1))
    elif fmt == QP_ACT_INT8_BLOCK32:
        _need(q, "q", I8, (rows, k))
        _need(scale, "scale", F32, (rows, k // 32))
    elif fmt == QP_ACT_BF16:
        _need(q, "q", BF16, (rows, k))
        if scale is not None:
            raise ValueError("scale: QP_ACT_BF16 has none")


def rmsnorm_residual_quant(x, residual, weight, eps, fmt, q, scale, residual_out=None,
                           stream=None):
    """q, scale = the form `fmt` (QP_ACT_*) of the RMS norm of
    h = bf16(x + residual), which is written to residual_out (it may be
    residual itself).  residual None: h = x, and no residual_out.
    QP_ACT_BF16: q is BF16 and scale None."""
    rows, k = x.shape
    _need(x, "x", BF16, (rows, k))
    _need(weight, "weight", BF16, (k,))
    _need_act(q, scale, fmt, rows, k)
    if residual is not None:
        _need(residual, "residual", BF16, (rows, k))
    if residual_out is not None:
        _need(residual_out, "residual_out", BF16, (rows, k))
    _check("rmsnorm_residual_quant", lib().rmsnorm_residual_quant(
        _ptr(x), None if residual is None else _ptr(residual), _ptr(weight), float(eps),
        int(fmt), _ptr(q), None if scale is None else _ptr(scale), None if residual_out is None else _ptr(residual_out),
        rows, k, _stream(stream)))


def silu_mul_quant(gate_up, fmt, q, scale, stream=None):
    """q, scale = the form `fmt` (QP_ACT_*) of silu(gate) * up, where a row of
    gate_up holds its gate values and then its up values.  QP_ACT_BF16: q is
    BF16 and scale None."""
    rows, k2 = gate_up.shape
    k = k2 // 2
    _need(gate_up, "gate_up", BF16, (rows, 2 * k))
    _need_act(q, scale, fmt, rows, k)
    _check("silu_mul_quant", lib().silu_mul_quant(
        _ptr(gate_up), int(fmt), _ptr(q), None if scale is None else _ptr(scale), rows, k,
        _stream(stream)))


def fp8_gemm_blockscale(a, a_scale, w, block_scale, out, stream=None):
    """Block-scaled FP8 GEMM: a with one scale per 128 of a row
    (QP_ACT_FP8_BLOCK128), w with one per 128 x 128 block."""
    m, k = a.shape
    n = w.shape[0]
    kb = (k + 127) // 128
    _need(a, "a", U8, (m, k))
    _need(a_scale, "a_scale", F32, (m, kb))
    _need(w, "w", U8, (n, k))
    _need(block_scale, "block_scale", F32, ((n + 127) // 128, kb))
    _need(out, "out", BF16, (m, n))
    _check("fp8_gemm_blockscale", lib().fp8_gemm_blockscale(
        _ptr(a), _ptr(a_scale), _ptr(w), _ptr(block_scale), _ptr(out), m, n, k,
        _stream(stream)))


def fp8_gemm_blockscale_kernel(m, n, k) -> int:
    """The kernel fp8_gemm_blockscale runs for a shape: QP_BLOCKSCALE_TILES_*, or
    QP_BLOCKSCALE_KSPLIT + 16s of rows of A + 8 * 16s of rows of W (+ 64: W past
    the caches) of a workgroup."""
    kernel = lib().fp8_gemm_blockscale_kernel(m, n, k)
    if kernel < 0:
        raise QProjError("fp8_gemm_blockscale_kernel", kernel)
    return kernel


def moe_fp8_blockscale_workspace(t, topk, i) -> int:
    """Bytes of scratch moe_fp8_blockscale needs for t tokens, topk experts a
    token and an intermediate size i."""
    return int(lib().moe_fp8_blockscale_workspace(t, topk, i))


def moe_fp8_blockscale(x, router_logits, w13, s13, w2, s2, topk, renormalize, workspace, out,
                       stream=None):
    """A mixture-of-experts layer for up to 16 tokens: routing, gate and up
    products, activation, down product and the weighted sum."""
    t, h = x.shape
    e, i2, _ = w13.shape
    i = i2 // 2
    _need(x, "x", BF16, (t, h))
    _need(router_logits, "router_logits", F32, (t, e))
    _need(w13, "w13", U8, (e, 2 * i, h))
    _need(s13, "s13", F32, (e, 2 * i // 128, h // 128))
    _need(w2, "w2", U8, (e, h, i))
    _need(s2, "s2", F32, (e, h // 128, i // 128))
    _need(out, "out", BF16, (t, h))
    _need(workspace, "workspace", (torch.uint8,), (workspace.numel(),))
    _check("moe_fp8_blockscale", lib().moe_fp8_blockscale(
        _ptr(x), _ptr(router_logits), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
        _ptr(workspace), workspace.numel(), _ptr(out), t, e, int(topk), h, i, int(renormalize),
        _stream(stream)))


def rope_inv_freq(rot, base, scaling=QP_ROPE_PLAIN, factor=1.0, low=0.0, high=0.0, original=0):
    """The rotary frequencies [rot/2] (F32, a host tensor) of base^(-2i/rot),
    scaled (QP_ROPE_*) for contexts `factor` times the model's `original` one."""
    if (int(rot) | int(scaling) | int(original)) >> 32:
        raise _outside_u32("rope_inv_freq")
    out = torch.empty(int(rot) // 2, dtype=torch.float32)
    _check("rope_inv_freq", lib().rope_inv_freq(
        _ptr(out), int(rot), float(base), int(scaling), float(factor), float(low), float(high),
        int(original)))
    return out


class KVCache:
    """A paged cache in the caller's tensors: k and v [pages, kv_heads,
    page_size, d], BF16, or E4M3 with F32 scales [pages, kv_heads, page_size].
    The tensors stay the caller's and are kept referenced; each call takes the
    memory that they then have, and refuses other shapes than those given here."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.pages, self.kv_heads, self.page_size, self.d = k.shape
        if (self.pages | self.kv_heads | self.page_size | self.d) >> 32:
            raise _outside_u32("KVCache")
        self.fmt = QP_KV_BF16 if k.dtype in BF16 else QP_KV_FP8_ROW
        dtypes = BF16 if self.fmt == QP_KV_BF16 else U8
        self._parts = [("k", k, dtypes, k.shape), ("v", v, dtypes, k.shape)]
        if self.fmt == QP_KV_FP8_ROW:
            self._parts += [("k_scale", k_scale, F32, k.shape[:3]), ("v_scale", v_scale, F32, k.shape[:3])]
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a BF16 cache has no scales")
        for name, t, kind, shape in self._parts:
            _need(t, name, kind, shape)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = _one_device(k, v, k_scale, v_scale)
        self._known = None

    def _args(self):
        now = (self.fmt, *[t.data_ptr() for _, t, _, _ in self._parts], None, None)[:5]
        known = now == self._known
        for name, t, kind, shape in self._parts:
            # in other memory all is checked, in the same what may have changed in place
            if not known or t.shape != shape or not t.is_contiguous():
                _need_on(self.device, t, name, kind, shape)
        self._known = now
        return now


def qk_norm_rope_cache(qkv, q_norm, k_norm, eps, positions, inv_freq, rope_scale, layout, slots, cache,
                       q_out, stream=None):
    """Norms of queries and keys for each head (q_norm and k_norm None: none),
    the first 2 * len(inv_freq) entries of each turned by position * inv_freq
    (layout QP_ROPE_HALF or QP_ROPE_INTERLEAVED; inv_freq None: not turned),
    the queries written to q_out [t, q_heads, d], keys and values to the
    KVCache at their slots (page * page_size + offset; -1: to none)."""
    t, q_heads, d = q_out.shape
    kv = cache.kv_heads
    if d != cache.d:
        raise ValueError(f"q_out: head size {d}, the cache's is {cache.d}")
    half = 0 if inv_freq is None else inv_freq.numel()
    if (t | q_heads | 2 * half | int(layout)) >> 32:
        raise _outside_u32("qk_norm_rope_cache")
    device = cache.device
    _need_on(device, qkv, "qkv", BF16, (t, (q_heads + 2 * kv) * d))
    _need_on(device, q_out, "q_out", BF16)
    _need_on(device, positions, "positions", I32, (t,))
    _need_on(device, slots, "slots", I32, (t,))
    if inv_freq is not None:
        _need_on(device, inv_freq, "inv_freq", F32, (half,))
    if q_norm is not None:
        _need_on(device, q_norm, "q_norm", BF16, (d,))
    if k_norm is not None:
        _need_on(device, k_norm, "k_norm", BF16, (d,))
    _current(device)
    _check("qk_norm_rope_cache", lib().qk_norm_rope_cache(
        _ptr(qkv), _ptr_or_null(q_norm), _ptr_or_null(k_norm), float(eps), _ptr(positions),
        _ptr_or_null(inv_freq), float(rope_scale), int(layout), 2 * half, _ptr(slots), *cache._args(),
        _ptr(q_out), t, q_heads, kv, d, cache.pages, cache.page_size, _stream(stream)))


def paged_attention_workspace(t, seqs, max_q, q_heads, kv_heads, d) -> int:
    """Bytes of scratch paged_attention needs for t rows of seqs sequences with
    at most max_q rows each; 0 for a shape that it refuses."""
    if (t | seqs | max_q | q_heads | kv_heads | d) >> 32:
        return 0
    return int(lib().paged_attention_workspace(t, seqs, max_q, q_heads, kv_heads, d))


def paged_attention(q, cache, page_table, q_start, kv_len, max_q, scale, window, workspace, out,
                    stream=None):
    """Attention of the rows q_start[s]..q_start[s+1]-1 of q [t, q_heads, d],
    the last of sequence s's kv_len[s] positions, over that sequence's pages
    page_table[s] of the KVCache; window 0: over all positions up to the
    row's own, else over the last `window` of them."""
    t, q_heads, d = q.shape
    seqs, width = page_table.shape
    if d != cache.d:
        raise ValueError(f"q: head size {d}, the cache's is {cache.d}")
    if (t | q_heads | seqs | width | int(max_q) | int(window)) >> 32:
        raise _outside_u32("paged_attention")
    device = cache.device
    _need_on(device, q, "q", BF16)
    _need_on(device, out, "out", BF16, (t, q_heads, d))
    _need_on(device, page_table, "page_table", I32)
    _need_on(device, q_start, "q_start", I32, (seqs + 1,))
    _need_on(device, kv_len, "kv_len", I32, (seqs,))
    room = workspace.numel()
    _need_on(device, workspace, "workspace", (torch.uint8,), (room,))
    _current(device)
    _check("paged_attention", lib().paged_attention(
        _ptr(q), *cache._args(), _ptr(page_table), _ptr(q_start), _ptr(kv_len), float(scale), int(window),
        _ptr(workspace), room, _ptr(out), t, seqs, int(max_q), q_heads, cache.kv_heads, d,
        cache.pages, cache.page_size, width, _stream(stream)))


def token_logprobs_workspace(rows, vocab, top) -> int:
    """Bytes of scratch token_logprobs needs; 0 for a shape that it refuses."""
    if (rows | vocab | top) >> 32:
        return 0
    return int(lib().token_logprobs_workspace(rows, vocab, top))


def token_logprobs(logits, targets, logprob, entropy, top_ids, top_logprobs, workspace, stream=None):
    """Log probabilities of `targets` [rows] under logits [rows, vocab] (BF16 or
    F32) into logprob [rows], the entropy into entropy [rows], the most probable
    tokens and their log probabilities into top_ids and top_logprobs
    [rows, top].  Targets with logprob, entropy, and the last two may be None."""
    rows, vocab = logits.shape
    asked = top_ids is not None or top_logprobs is not None
    top = top_ids.shape[-1] if asked and isinstance(top_ids, torch.Tensor) else 0
    if (rows | vocab | top) >> 32:
        raise _outside_u32("token_logprobs")
    f32 = isinstance(logits, torch.Tensor) and logits.dtype == torch.float32
    _need(logits, "logits", F32 if f32 else BF16, (rows, vocab))
    device = logits.get_device()
    if targets is not None:
        _need_on(device, targets, "targets", I32, (rows,))
    if logprob is not None:
        _need_on(device, logprob, "logprob", F32, (rows,))
    if entropy is not None:
        _need_on(device, entropy, "entropy", F32, (rows,))
    if asked:
        _need_on(device, top_ids, "top_ids", I32, (rows, top))
        _need_on(device, top_logprobs, "top_logprobs", F32, (rows, top))
    _need_on(device, workspace, "workspace", (torch.uint8,), (workspace.numel(),))
    _current(device)
    _check("token_logprobs", lib().token_logprobs(
        _ptr(logits), QP_LOGITS_F32 if f32 else QP_LOGITS_BF16, _ptr_or_null(targets),
        _ptr_or_null(logprob), _ptr_or_null(entropy), _ptr_or_null(top_ids) if top else None,
        _ptr_or_null(top_logprobs) if top else None, _ptr(workspace), workspace.numel(), rows, vocab,
        top, _stream(stream)))


class DerivedWeights:
    """A derived-weight cache (the library's qp_cache): weights requantised on
    first use and kept, keyed by the source weight's device address
    (dispatch_proj_rowwise.rs, requant_weight_rowwise_fp8_cached and its
    DerivedWeights cache).  The cache owns the derived device buffers; the
    requant methods return their device addresses as ints.  close() (or
    garbage collection) frees them: no kernel reading one may be pending."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check("qproj_cache_create", lib().qproj_cache_create(ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().qproj_cache_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self):
        """(entries, bytes) held by the cache."""
        e, b = ctypes.c_uint64(), ctypes.c_uint64()
        _check("qproj_cache_stats", lib().qproj_cache_stats(self._h, ctypes.byref(e), ctypes.byref(b)))
        return int(e.value), int(b.value)

    def evict(self, w):
        _check("qproj_cache_evict", lib().qproj_cache_evict(self._h, _ptr(w)))

    def requant_w_blockfp8_rowwise(self, fmt, w, scale, stream=None):
        """Row-wise FP8 copy of a block-scaled weight (passthrough for
        QP_FP8_PER_ROW): returns (weight address, scale address)."""
        n, k = w.shape
        _need(w, "w", U8, (n, k))
        if fmt == QP_FP8_BLOCK128:
            _need(scale, "scale", F32, (n // 128, k // 128))
        wq, sq = ctypes.c_void_p(), ctypes.c_void_p()
        _check("requant_w_blockfp8_rowwise_cached", lib().requant_w_blockfp8_rowwise_cached(
            self._h, int(fmt), _ptr(w), _ptr(scale), n, k, ctypes.byref(wq), ctypes.byref(sq),
            _stream(stream)))
        return wq.value, sq.value

    def requant_w_nvfp4_int8(self, w_packed, w_e4m3, scale2, stream=None):
        """int8 copy [n,k] and F32 per-32 scales [n,k/32] of an NVFP4 weight:
        returns (weight address, scale address)."""
        n, kh = w_packed.shape
        k = 2 * kh
        _need(w_packed, "w_packed", U8, (n, k // 2))
        _need(w_e4m3, "w_e4m3", U8, (n, k // 16))
        wq, sq = ctypes.c_void_p(), ctypes.c_void_p()
        _check("requant_w_nvfp4_int8_cached", lib().requant_w_nvfp4_int8_cached(
            self._h, _ptr(w_packed), _ptr(w_e4m3), float(scale2), n, k, ctypes.byref(wq),
            ctypes.byref(sq), _stream(stream)))
        return wq.value, sq.value

    def fp8_rowwise_proj(self, fmt, w, w_scale, act, act_q, act_scale, out, stream=None):
        m, k = act.shape
        n = w.shape[0]
        _need(w, "w", U8, (n, k))
        _need(w_scale, "w_scale", F32, (n,) if fmt == QP_FP8_PER_ROW else (n // 128, k // 128))
        _need(act, "act", BF16, (m, k))
        _need(act_q, "act_q", U8, (m, k))
        _need(act_scale, "act_scale", F32, (m,))
        _need(out, "out", BF16, (m, n))
        _check("fp8_rowwise_proj_cached", lib().fp8_rowwise_proj_cached(
            self._h, int(fmt), _ptr(w), _ptr(w_scale), _ptr(act), _ptr(act_q), _ptr(act_scale),
            _ptr(out), m, n, k, _stream(stream)))

    def int8_w4a8_prefill(self, a, w_packed, w_e4m3, scale2, a_i8, a_scale, out, stream=None):
        m, k = a.shape
        n = w_packed.shape[0]
        _need(a, "a", BF16, (m, k))
        _need(w_packed, "w_packed", U8, (n, k // 2))
        _need(w_e4m3, "w_e4m3", U8, (n, k // 16))
        _need(a_i8, "a_i8", I8, (m, k))
        _need(a_scale, "a_scale", F32, (m, k // 32))
        _need(out, "out", BF16, (m, n))
        _check("int8_w4a8_prefill_cached", lib().int8_w4a8_prefill_cached(
            self._h, _ptr(a), _ptr(w_packed), _ptr(w_e4m3), float(scale2), _ptr(a_i8),
            _ptr(a_scale), _ptr(out), m, n, k, _stream(stream)))


__all__ = [
    "requant_w_nvfp4_int8", "requant_a_bf16_int8", "int8_gemm_blockscaled",
    "int8_w4a8_prefill", "int8_gemm_block_partials", "quantize_bf16_nvfp4",
    "w4a4_gemm", "requant_w_blockfp8_rowwise", "quant_rowwise_fp8",
    "fp8_gemm_rowscale", "fp8_rowwise_proj", "fp8_gemv_rowscale",
    "fp8_gemv_blockscale", "w4a16_gemv", "rmsnorm_residual_quant",
    "silu_mul_quant", "fp8_gemm_blockscale", "fp8_gemm_blockscale_kernel",
    "moe_fp8_blockscale", "moe_fp8_blockscale_workspace", "rope_inv_freq",
    "KVCache", "qk_norm_rope_cache", "paged_attention",
    "paged_attention_workspace", "token_logprobs", "token_logprobs_workspace",
    "DerivedWeights",
    "launch_count", "status_string", "abi_version", "lib", "QProjError",
]
