"""Thin Python binding of libw4a8.so (C ABI in include/w4a8.h).

Argument marshalling only: torch tensors (device memory) become raw pointers,
the current torch stream becomes the hipStream_t, and a non-OK status raises.
Every step of the computation runs in the library's HIP kernels; there is no
fallback.  Importing this module loads the library and raises ImportError if
it has not been built (``python -m w4a8_quantized_gemm_quantize_amd.build_lib``
or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a8.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libw4a8.so is not built ({LIB_PATH}); run build_lib.py first")

_lib = ctypes.CDLL(LIB_PATH)

OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_HIP, ERR_NONFINITE = range(7)
F32, BF16, I32 = 0, 1, 2
GROUP = 64
N_TILE = 16
K_MAX = 150976
LQQ_K_MAX = 133120

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SIGS = {
    "w4a8_abi_version": ([], ctypes.c_int32),
    "w4a8_pack_layout_version": ([], ctypes.c_int32),
    "w4a8_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "quantize_act_blockwise": ([_P, _I64, _I64, _I32, _P, _P, _P], ctypes.c_int),
    "dequantize_act_blockwise": ([_P, _P, _I64, _I64, _I32, _P, ctypes.c_int, _P], ctypes.c_int),
    "pack_w4_grouped": ([_P, _I64, _I64, _I32, _P, _P, _P, _P], ctypes.c_int),
    "unpack_w4_grouped": ([_P, _P, _I64, _I64, _I32, _P, _P, _P], ctypes.c_int),
    "w4a8_gemm": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_int, _P],
                  ctypes.c_int),
    "w4a8_gemm_workspace_bytes": ([_I64, _I64, _I64], ctypes.c_size_t),
    "w4a8_gemm_ws": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_int, _P,
                      ctypes.c_size_t, _P], ctypes.c_int),
    "w4a8_gemm_bf16act_workspace_bytes": ([_I64, _I64], ctypes.c_size_t),
    "w4a8_gemm_bf16act": ([_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_int, _P,
                           ctypes.c_size_t, _P], ctypes.c_int),
    "pack_w4_lqq": ([_P, _I64, _I64, _I32, _P, _P, _P, _P], ctypes.c_int),
    "unpack_w4_lqq": ([_P, _P, _I64, _I64, _I32, _P, _P, _P, _P], ctypes.c_int),
    "w4a8_gemm_lqq": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_int, _P],
                      ctypes.c_int),
    "w4a8_gemm_lqq_bf16act": ([_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_int, _P,
                               ctypes.c_size_t, _P], ctypes.c_int),
    "pack_w8_channel": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "unpack_w8_channel": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "w8a8_gemm": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_int, _P], ctypes.c_int),
    "w8a8_gemm_bf16act": ([_P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_int, _P, ctypes.c_size_t,
                           _P], ctypes.c_int),
    "w4a8_gemm_blockact": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _P, ctypes.c_int,
                            _P], ctypes.c_int),
    "dequant_add_requant": ([_P, _P, _P, ctypes.c_int, _I64, _I64, _I32, _P, _P, _P, _P],
                            ctypes.c_int),
    "w4a8_probe_mfma_i8": ([_I64, _I32, _P, _P, _P], ctypes.c_int),
    "w4a8_moe_route": ([_P, ctypes.c_int, _I64, _P, _I64, _I32, _I32, ctypes.c_int, _I32, _I32,
                        _I32, _I32, ctypes.c_float, _P, _P, _P], ctypes.c_int),
    "w4a8_moe_ffn_workspace_bytes": ([_I64, _I32, _I32, _I64, _I64, ctypes.c_int],
                                     ctypes.c_size_t),
    "w4a8_moe_ffn": ([_P] * 9 + [_I64, _I32, _I32, _I64, _I64, _I32, _P, ctypes.c_int, _P,
                                 ctypes.c_size_t, _P], ctypes.c_int),
    "w4a8_lora_workspace_bytes": ([_I64, _I32, _I32, _I64], ctypes.c_size_t),
    "w4a8_lora_add": ([_P, _I64, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _P, _I64, _P,
                       _I64, ctypes.c_int, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "w4a8_qk_norm_rope": ([_P, _I64, _P, _I64, ctypes.c_int, _P, _P, ctypes.c_float, _P, _P, _I64,
                           _I32, _I32, _I64, _I32, _I32, _I32, _P, _I64, _P, _I64, ctypes.c_int,
                           _P], ctypes.c_int),
    "w4a8_kv8_write": ([_P, _I64, _P, _I64, ctypes.c_int, _P, _I64, _I32, _P, _P, _I64, _I64, _I32,
                        _I32, _I32, _I64, _P, _P, _P], ctypes.c_int),
    "w4a8_kv8_read": ([_P, _P, _P, _I64, _I32, _P, _P, _I64, _I64, _I32, _I32, _I32, _I64, _P, _I64,
                       _P, _I64, ctypes.c_int, _P], ctypes.c_int),
    "w4a8_attn_kv8_workspace_bytes": ([_I64, _I64, _I32, _I64, _I32, _I32, _I32, _I32, _I32],
                                      ctypes.c_size_t),
    "w4a8_attn_kv8": ([_P, _I64, _P, _P, _P, _I64, _I32, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                       _I32, _I64, _I32, _I32, ctypes.c_float, _P, _I64, _P, _P, ctypes.c_size_t,
                       _P], ctypes.c_int),
    "w4a8_gemm_bf16act_noalloc": ([_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_int, _P],
                                  ctypes.c_int),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)


class W4A8Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def abi_version() -> int:
    return int(_lib.w4a8_abi_version())


def pack_layout_version() -> int:
    return int(_lib.w4a8_pack_layout_version())


def status_string(status: int) -> str:
    return _lib.w4a8_status_string(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object (0.2 us instead of
# 2.7 us, half of a small call's host time), where this torch has the functions.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _raw_device is not None:
        return _raw_stream(_raw_device())
    return torch.cuda.current_stream().cuda_stream


def _empty(stream, shape, dtype, device):
    """A new tensor for a call enqueued on `stream`.  Allocated under that stream,
    so torch's caching allocator does not hand the memory to work on another
    stream while the call's kernels may still use it (a workspace the binding
    creates is released when the call returns, before its kernels finish)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(fn, status):
    if status != OK:
        raise W4A8Error(fn, status)


def _dev(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")


class W4A8SizeError(W4A8Error):
    """A tensor argument holds fewer elements than the call's sizes need (raised
    before anything is launched; status W4A8_ERR_SHAPE)."""

    def __init__(self, fn: str, name: str, have: int, need: int):
        self.status = ERR_SHAPE
        RuntimeError.__init__(self, f"{fn}: {name} holds {have} elements, the call needs {need}")


_U8 = (torch.uint8, torch.int8)
_I16 = (torch.int16,)
_F32 = (torch.float32,)


def _sized(fn, t, dtypes, need, name):
    """The library takes raw pointers and cannot see buffer sizes: check that a
    tensor argument is a contiguous CUDA tensor of one of `dtypes` holding at
    least `need` elements.  None passes through (the library rejects a missing
    pointer itself)."""
    if t is None:
        return
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{fn}: {name} must be a contiguous CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} must be of dtype {' or '.join(map(str, dtypes))}, "
                         f"not {t.dtype}")
    if t.numel() < need:
        raise W4A8SizeError(fn, name, t.numel(), need)


def _per(total: int, block: int) -> int:
    return total // block if block > 0 else 0


def _gemm_args(fn, m, n, k, a_scale, w_packed, w_bytes_per_elem, params, param_dtypes,
               group, ch_scale, out):
    """Sizes of the GEMM operands: a_scale [m], weights n k w_bytes_per_elem bytes,
    group parameters [n, k / group] (if the format has them), ch_scale [n], out [m, n]."""
    _sized(fn, a_scale, _F32, m, "a_scale")
    _sized(fn, w_packed, _U8, (n * k * w_bytes_per_elem) // 2, "w_packed")
    if param_dtypes is not None:
        _sized(fn, params, param_dtypes, n * _per(k, group), "group parameters")
    _sized(fn, ch_scale, _F32, n, "ch_scale")
    _sized(fn, out, tuple(_OUT), m * n, "out")


# ------------------------------------------------------------ activations --

def quantize_act_blockwise(x: torch.Tensor, block: int, q=None, scales=None, stream=None):
    """x bf16 [rows, cols] -> (q int8 [rows, cols], scales f32 [rows, cols // block])."""
    _dev(x, torch.bfloat16, "x")
    rows, cols = x.shape
    if q is None:
        q = _empty(stream, (rows, cols), dtype=torch.int8, device=x.device)
    if scales is None:
        scales = _empty(stream, (rows, cols // block if block > 0 else 0), dtype=torch.float32,
                             device=x.device)
    _sized("quantize_act_blockwise", q, (torch.int8,), rows * cols, "q")
    _sized("quantize_act_blockwise", scales, _F32, rows * _per(cols, block), "scales")
    _check("quantize_act_blockwise",
           _lib.quantize_act_blockwise(_ptr(x), rows, cols, block, _ptr(q), _ptr(scales),
                                       _stream(stream)))
    return q, scales


def dequantize_act_blockwise(q: torch.Tensor, scales: torch.Tensor, block: int,
                             out_dtype=torch.float32, out=None, stream=None):
    """-> x_hat [rows, cols] as float32 or bfloat16."""
    _dev(q, torch.int8, "q")
    _dev(scales, torch.float32, "scales")
    rows, cols = q.shape
    code = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        out = _empty(stream, (rows, cols), dtype=out_dtype, device=q.device)
    _sized("dequantize_act_blockwise", scales, _F32, rows * _per(cols, block), "scales")
    _sized("dequantize_act_blockwise", out, (out_dtype,), rows * cols, "out")
    _check("dequantize_act_blockwise",
           _lib.dequantize_act_blockwise(_ptr(q), _ptr(scales), rows, cols, block, _ptr(out),
                                         code, _stream(stream)))
    return out


# ---------------------------------------------------------------- weights --

def pack_w4_grouped(w: torch.Tensor, group: int = GROUP, stream=None):
    """w bf16 [n, k] -> (w_packed uint8 [n*k/2], grp_scale uint8 [n*k/group], ch_scale f32 [n])."""
    _dev(w, torch.bfloat16, "w")
    n, k = w.shape
    dev = w.device
    w_packed = _empty(stream, (n * k // 2,), dtype=torch.uint8, device=dev)
    grp_scale = _empty(stream, (n * (k // group) if group > 0 else 0,), dtype=torch.uint8,
                            device=dev)
    ch_scale = _empty(stream, (n,), dtype=torch.float32, device=dev)
    _check("pack_w4_grouped",
           _lib.pack_w4_grouped(_ptr(w), n, k, group, _ptr(w_packed), _ptr(grp_scale),
                                _ptr(ch_scale), _stream(stream)))
    return w_packed, grp_scale, ch_scale


def unpack_w4_grouped(w_packed, grp_scale, n: int, k: int, group: int = GROUP, stream=None):
    """Test hook: packed layout -> (q int8 [n, k], s_g uint8 [n, k/group]) canonical."""
    dev = w_packed.device
    q = _empty(stream, (n, k), dtype=torch.int8, device=dev)
    s_g = _empty(stream, (n, k // group), dtype=torch.uint8, device=dev)
    _sized("unpack_w4_grouped", w_packed, _U8, n * k // 2, "w_packed")
    _sized("unpack_w4_grouped", grp_scale, _U8, n * _per(k, group), "grp_scale")
    _check("unpack_w4_grouped",
           _lib.unpack_w4_grouped(_ptr(w_packed), _ptr(grp_scale), n, k, group, _ptr(q),
                                  _ptr(s_g), _stream(stream)))
    return q, s_g


# ------------------------------------------------------------------- GEMM --

_OUT = {torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32}


def w4a8_gemm(a_q, a_scale, w_packed, grp_scale, ch_scale, n: int, out_dtype=torch.bfloat16,
              group: int = GROUP, out=None, stream=None):
    """a_q int8 [m, k], a_scale f32 [m] -> out [m, n] (float32, bfloat16 or raw int32 acc)."""
    _dev(a_q, torch.int8, "a_q")
    m, k = a_q.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a_q.device)
    _gemm_args("w4a8_gemm", m, n, k, a_scale, w_packed, 1, grp_scale, _U8, group, ch_scale, out)
    _check("w4a8_gemm",
           _lib.w4a8_gemm(_ptr(a_q), _ptr(a_scale), _ptr(w_packed), _ptr(grp_scale),
                          _ptr(ch_scale), m, n, k, group, _ptr(out), _OUT[out.dtype],
                          _stream(stream)))
    return out


def gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    """Split-K scratch of w4a8_gemm_ws for an m x n x k product (0: not split)."""
    return int(_lib.w4a8_gemm_workspace_bytes(m, n, k))


def w4a8_gemm_ws(a_q, a_scale, w_packed, grp_scale, ch_scale, n: int,
                 out_dtype=torch.bfloat16, group: int = GROUP, out=None, workspace=None,
                 stream=None):
    """w4a8_gemm with a caller workspace that lets batches whose output tiles would
    not fill the GPU (5 <= m <= 64 where a split pays, or m > 64 with few tiles) split K
    (same result)."""
    _dev(a_q, torch.int8, "a_q")
    m, k = a_q.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a_q.device)
    need = gemm_workspace_bytes(m, n, k)
    if workspace is None and need > 0:
        workspace = _empty(stream, (need,), dtype=torch.uint8, device=a_q.device)
    _gemm_args("w4a8_gemm_ws", m, n, k, a_scale, w_packed, 1, grp_scale, _U8, group, ch_scale,
               out)
    _sized("w4a8_gemm_ws", workspace, _U8, 0, "workspace")
    _check("w4a8_gemm_ws",
           _lib.w4a8_gemm_ws(_ptr(a_q), _ptr(a_scale), _ptr(w_packed), _ptr(grp_scale),
                             _ptr(ch_scale), m, n, k, group, _ptr(out), _OUT[out.dtype],
                             _ptr(workspace), 0 if workspace is None else workspace.numel(),
                             _stream(stream)))
    return out


def workspace_bytes(m: int, k: int, n: int = None) -> int:
    """Workspace of the fused entry points: codes and scales, plus (given n) the
    split-K partials that let batches whose output tiles would not fill the GPU
    split K."""
    base = int(_lib.w4a8_gemm_bf16act_workspace_bytes(m, k))
    return base + (gemm_workspace_bytes(m, n, k) if n is not None else 0)


def w4a8_gemm_bf16act(a, w_packed, grp_scale, ch_scale, n: int, out_dtype=torch.bfloat16,
                      group: int = GROUP, out=None, workspace=None, stream=None):
    """a bf16 [m, k] -> out [m, n]; per-token quantization into `workspace` then the GEMM."""
    _dev(a, torch.bfloat16, "a")
    m, k = a.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a.device)
    need = workspace_bytes(m, k, n)
    if workspace is None:
        workspace = _empty(stream, (max(need, 16),), dtype=torch.uint8, device=a.device)
    _gemm_args("w4a8_gemm_bf16act", m, n, k, None, w_packed, 1, grp_scale, _U8, group, ch_scale,
               out)
    _sized("w4a8_gemm_bf16act", workspace, _U8, 0, "workspace")
    _check("w4a8_gemm_bf16act",
           _lib.w4a8_gemm_bf16act(_ptr(a), _ptr(w_packed), _ptr(grp_scale), _ptr(ch_scale), m,
                                  n, k, group, _ptr(out), _OUT[out.dtype], _ptr(workspace),
                                  workspace.numel(), _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def w4a8_gemm_bf16act_noalloc(a, w_packed, grp_scale, ch_scale, n: int, out,
                              group: int = GROUP, stream=None):
    """w4a8_gemm_bf16act with the library's static device workspace: the caller
    passes `out` ([m, n] float32, bfloat16 or int32) and nothing is allocated.
    Calls that overlap on one GPU share that workspace and race."""
    _dev(a, torch.bfloat16, "a")
    m, k = a.shape
    _gemm_args("w4a8_gemm_bf16act_noalloc", m, n, k, None, w_packed, 1, grp_scale, _U8, group,
               ch_scale, out)
    _check("w4a8_gemm_bf16act_noalloc",
           _lib.w4a8_gemm_bf16act_noalloc(_ptr(a), _ptr(w_packed), _ptr(grp_scale),
                                          _ptr(ch_scale), m, n, k, group, _ptr(out),
                                          _OUT[out.dtype], _stream(stream)))
    return out


def workspace_views(workspace, m: int, k: int):
    """(a_q [m, k] int8, a_scale [m] f32) views of a w4a8_gemm_bf16act workspace."""
    off = (m * k + 255) // 256 * 256
    a_q = workspace[: m * k].view(torch.int8).view(m, k)
    a_s = workspace[off: off + 4 * m].view(torch.float32)
    return a_q, a_s


# ------------------------------------------------------------ LQQ weights --

def pack_w4_lqq(w: torch.Tensor, group: int = GROUP, stream=None):
    """w bf16 [n, k] -> (w_packed uint8 [n*k/2], grp_param int16 [n*k/group] holding
    uint16 s | (128 + min) << 8, ch_scale f32 [n])."""
    _dev(w, torch.bfloat16, "w")
    n, k = w.shape
    dev = w.device
    w_packed = _empty(stream, (n * k // 2,), dtype=torch.uint8, device=dev)
    grp_param = _empty(stream, (n * (k // group) if group > 0 else 0,), dtype=torch.int16,
                            device=dev)
    ch_scale = _empty(stream, (n,), dtype=torch.float32, device=dev)
    _check("pack_w4_lqq",
           _lib.pack_w4_lqq(_ptr(w), n, k, group, _ptr(w_packed), _ptr(grp_param),
                            _ptr(ch_scale), _stream(stream)))
    return w_packed, grp_param, ch_scale


def unpack_w4_lqq(w_packed, grp_param, n: int, k: int, group: int = GROUP, stream=None):
    """Test hook -> (q_u4 uint8 [n, k], s_u8 uint8 [n, k/group], w_min int8 [n, k/group])."""
    dev = w_packed.device
    q = _empty(stream, (n, k), dtype=torch.uint8, device=dev)
    s_u8 = _empty(stream, (n, k // group), dtype=torch.uint8, device=dev)
    w_min = _empty(stream, (n, k // group), dtype=torch.int8, device=dev)
    _sized("unpack_w4_lqq", w_packed, _U8, n * k // 2, "w_packed")
    _sized("unpack_w4_lqq", grp_param, _I16, n * _per(k, group), "grp_param")
    _check("unpack_w4_lqq",
           _lib.unpack_w4_lqq(_ptr(w_packed), _ptr(grp_param), n, k, group, _ptr(q),
                              _ptr(s_u8), _ptr(w_min), _stream(stream)))
    return q, s_u8, w_min


def w4a8_gemm_lqq(a_q, a_scale, w_packed, grp_param, ch_scale, n: int,
                  out_dtype=torch.bfloat16, group: int = GROUP, out=None, stream=None):
    _dev(a_q, torch.int8, "a_q")
    m, k = a_q.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a_q.device)
    _gemm_args("w4a8_gemm_lqq", m, n, k, a_scale, w_packed, 1, grp_param, _I16, group,
               ch_scale, out)
    _check("w4a8_gemm_lqq",
           _lib.w4a8_gemm_lqq(_ptr(a_q), _ptr(a_scale), _ptr(w_packed), _ptr(grp_param),
                              _ptr(ch_scale), m, n, k, group, _ptr(out), _OUT[out.dtype],
                              _stream(stream)))
    return out


def w4a8_gemm_lqq_bf16act(a, w_packed, grp_param, ch_scale, n: int, out_dtype=torch.bfloat16,
                          group: int = GROUP, out=None, workspace=None, stream=None):
    _dev(a, torch.bfloat16, "a")
    m, k = a.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a.device)
    if workspace is None:
        workspace = _empty(stream, (max(workspace_bytes(m, k, n), 16),), dtype=torch.uint8,
                                device=a.device)
    _gemm_args("w4a8_gemm_lqq_bf16act", m, n, k, None, w_packed, 1, grp_param, _I16, group,
               ch_scale, out)
    _sized("w4a8_gemm_lqq_bf16act", workspace, _U8, 0, "workspace")
    _check("w4a8_gemm_lqq_bf16act",
           _lib.w4a8_gemm_lqq_bf16act(_ptr(a), _ptr(w_packed), _ptr(grp_param), _ptr(ch_scale),
                                      m, n, k, group, _ptr(out), _OUT[out.dtype],
                                      _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


# ------------------------------------------------------------------ W8A8 --

def pack_w8_channel(w: torch.Tensor, stream=None):
    """w bf16 [n, k] -> (w_packed int8 [n*k] tiled layout, ch_scale f32 [n])."""
    _dev(w, torch.bfloat16, "w")
    n, k = w.shape
    w_packed = _empty(stream, (n * k,), dtype=torch.int8, device=w.device)
    ch_scale = _empty(stream, (n,), dtype=torch.float32, device=w.device)
    _check("pack_w8_channel",
           _lib.pack_w8_channel(_ptr(w), n, k, _ptr(w_packed), _ptr(ch_scale), _stream(stream)))
    return w_packed, ch_scale


def unpack_w8_channel(w_packed, n: int, k: int, stream=None):
    q8 = _empty(stream, (n, k), dtype=torch.int8, device=w_packed.device)
    _sized("unpack_w8_channel", w_packed, _U8, n * k, "w_packed")
    _check("unpack_w8_channel",
           _lib.unpack_w8_channel(_ptr(w_packed), n, k, _ptr(q8), _stream(stream)))
    return q8


def w8a8_gemm(a_q, a_scale, w_packed, ch_scale, n: int, out_dtype=torch.bfloat16, out=None,
              stream=None):
    _dev(a_q, torch.int8, "a_q")
    m, k = a_q.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a_q.device)
    _gemm_args("w8a8_gemm", m, n, k, a_scale, w_packed, 2, None, None, GROUP, ch_scale, out)
    _check("w8a8_gemm",
           _lib.w8a8_gemm(_ptr(a_q), _ptr(a_scale), _ptr(w_packed), _ptr(ch_scale), m, n, k,
                          _ptr(out), _OUT[out.dtype], _stream(stream)))
    return out


def w8a8_gemm_bf16act(a, w_packed, ch_scale, n: int, out_dtype=torch.bfloat16, out=None,
                      workspace=None, stream=None):
    _dev(a, torch.bfloat16, "a")
    m, k = a.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a.device)
    if workspace is None:
        workspace = _empty(stream, (max(workspace_bytes(m, k, n), 16),), dtype=torch.uint8,
                                device=a.device)
    _gemm_args("w8a8_gemm_bf16act", m, n, k, None, w_packed, 2, None, None, GROUP, ch_scale, out)
    _sized("w8a8_gemm_bf16act", workspace, _U8, 0, "workspace")
    _check("w8a8_gemm_bf16act",
           _lib.w8a8_gemm_bf16act(_ptr(a), _ptr(w_packed), _ptr(ch_scale), m, n, k, _ptr(out),
                                  _OUT[out.dtype], _ptr(workspace), workspace.numel(),
                                  _stream(stream)))
    return out


# ------------------------------------------ per-block activation scales GEMM --

def w4a8_gemm_blockact(a_q, a_scale, w_packed, grp_scale, ch_scale, n: int, block: int,
                       out_dtype=torch.bfloat16, group: int = GROUP, out=None, stream=None):
    """a_q int8 [m, k], a_scale f32 [m, k / block] -> out [m, n] (float32 or bfloat16)."""
    _dev(a_q, torch.int8, "a_q")
    _dev(a_scale, torch.float32, "a_scale")
    m, k = a_q.shape
    if out is None:
        out = _empty(stream, (m, n), dtype=out_dtype, device=a_q.device)
    _gemm_args("w4a8_gemm_blockact", 0, n, k, None, w_packed, 1, grp_scale, _U8, group,
               ch_scale, out)
    _sized("w4a8_gemm_blockact", a_scale, _F32, m * _per(k, block), "a_scale")
    _sized("w4a8_gemm_blockact", out, tuple(_OUT), m * n, "out")
    _check("w4a8_gemm_blockact",
           _lib.w4a8_gemm_blockact(_ptr(a_q), _ptr(a_scale), _ptr(w_packed), _ptr(grp_scale),
                                   _ptr(ch_scale), m, n, k, group, block, _ptr(out),
                                   _OUT[out.dtype], _stream(stream)))
    return out


# ---------------------------------------------------- EQuARX receive step --

def dequant_add_requant(q_in, s_in, x, block: int, want_sum: bool = False, q_out=None,
                        s_out=None, sum_out=None, stream=None):
    """(q_in int8 [r, c], s_in f32 [r, c/block]) + x (float32 or bfloat16 [r, c])
    -> (q_out int8, s_out f32, sum f32 or None): requantized per block."""
    _dev(q_in, torch.int8, "q_in")
    _dev(s_in, torch.float32, "s_in")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be float32 or bfloat16")
    _dev(x, x.dtype, "x")
    rows, cols = q_in.shape
    dev = q_in.device
    if q_out is None:
        q_out = _empty(stream, (rows, cols), dtype=torch.int8, device=dev)
    if s_out is None:
        s_out = _empty(stream, (rows, cols // block if block > 0 else 0), dtype=torch.float32,
                            device=dev)
    if want_sum and sum_out is None:
        sum_out = _empty(stream, (rows, cols), dtype=torch.float32, device=dev)
    fn = "dequant_add_requant"
    _sized(fn, s_in, _F32, rows * _per(cols, block), "s_in")
    _sized(fn, x, (x.dtype,), rows * cols, "x")
    _sized(fn, q_out, (torch.int8,), rows * cols, "q_out")
    _sized(fn, s_out, _F32, rows * _per(cols, block), "s_out")
    _sized(fn, sum_out, _F32, rows * cols, "sum_out")
    _check("dequant_add_requant",
           _lib.dequant_add_requant(_ptr(q_in), _ptr(s_in), _ptr(x),
                                    BF16 if x.dtype == torch.bfloat16 else F32, rows, cols,
                                    block, _ptr(sum_out), _ptr(q_out), _ptr(s_out),
                                    _stream(stream)))
    return q_out, s_out, sum_out


# ------------------------------------------------ rows that choose weights --

_SCORES = {"softmax": 0, "sigmoid": 1}
_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}


def _rows(fn, t, dtypes, cols, name):
    """A 2-D CUDA tensor of one of `dtypes` and `cols` columns whose rows are
    contiguous; returns the elements from one row to the next."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{fn}: {name} must be a 2-D CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} must be of dtype {' or '.join(map(str, dtypes))}, "
                         f"not {t.dtype}")
    if t.size(1) != cols:
        raise W4A8SizeError(fn, f"a row of {name}", t.size(1), cols)
    if t.is_contiguous():
        return cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{fn}: rows of {name} must be contiguous")
    return t.stride(0) if t.size(0) > 1 else cols


def _addr(t):
    """A tensor's address; None (a null pointer, refused by the library where a tensor is
    needed) for None."""
    return None if t is None else t.data_ptr()


def _workspace(stream, need, device):
    """A call's workspace, as _empty; at least 16 bytes."""
    if stream is None:
        return torch.empty(need or 16, dtype=torch.uint8, device=device)
    return _empty(stream, (need or 16,), torch.uint8, device)


def moe_route(logits, top_k: int, bias=None, score: str = "softmax", groups: int = 1,
              topk_groups: int = 1, group_top: int = 2, renormalize: bool = True,
              scale: float = 1.0, ids=None, weights=None, stream=None):
    """logits float32 or bfloat16 [tokens, experts] (rows may be strided) ->
    (ids int32 [tokens, top_k], weights float32 [tokens, top_k]): the experts of each
    token, largest key first, -1 with weight 0 where none is left."""
    fn = "moe_route"
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError(f"{fn}: logits must be a 2-D CUDA tensor")
    if score not in _SCORES:
        raise ValueError(f"{fn}: score must be 'softmax' or 'sigmoid', not {score!r}")
    tokens, experts = logits.shape
    ld = _rows(fn, logits, _FLOATS, experts, "logits")
    # outputs made here fit by construction
    if ids is None:
        ids = _empty(stream, (tokens, top_k), torch.int32, logits.device)
    else:
        _sized(fn, ids, (torch.int32,), tokens * top_k, "ids")
    if weights is None:
        weights = _empty(stream, (tokens, top_k), torch.float32, logits.device)
    else:
        _sized(fn, weights, _F32, tokens * top_k, "weights")
    _sized(fn, bias, _F32, experts, "bias")
    status = _lib.w4a8_moe_route(
        logits.data_ptr(), _FLOATS[logits.dtype], ld, _addr(bias), tokens, experts, top_k,
        _SCORES[score], groups, topk_groups, group_top, 1 if renormalize else 0, scale,
        ids.data_ptr(), weights.data_ptr(), _stream(stream))
    if status:
        raise W4A8Error(fn, status)
    return ids, weights


@functools.lru_cache(maxsize=4096)
def _moe_bytes(*sizes):
    return int(_lib.w4a8_moe_ffn_workspace_bytes(*sizes))


def moe_ffn_workspace_bytes(tokens: int, experts: int, top_k: int, hidden: int, inter: int,
                            out_dtype=torch.bfloat16) -> int:
    return _moe_bytes(tokens, experts, top_k, hidden, inter, _FLOATS[out_dtype])


def w4a8_moe_ffn(x, ids, weights, w13, w2, inter: int, out_dtype=torch.bfloat16,
                 group: int = GROUP, out=None, workspace=None, stream=None):
    """Gated feed-forward layer of routed experts.

    x bf16 [tokens, hidden]; ids int32 and weights float32 [tokens, top_k] (moe_route's;
    an id outside the experts is an unused slot); w13 and w2 the (w_packed, grp_scale,
    ch_scale) of pack_w4_grouped for the stacked matrices [experts * 2 * inter, hidden]
    (per expert inter gate rows, then inter up rows) and [experts * hidden, inter]
    -> out [tokens, hidden] (bfloat16 or float32)."""
    fn = "w4a8_moe_ffn"
    _dev(x, torch.bfloat16, "x")
    _dev(ids, torch.int32, "ids")
    tokens, hidden = x.shape
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError(f"{fn}: ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    p13, g13, c13 = w13
    p2, g2, c2 = w2
    if c13 is None:                    # the number of experts is its size
        raise W4A8Error(fn, ERR_NULL)
    if inter <= 0 or c13.numel() % (2 * inter):
        raise W4A8SizeError(fn, "w13 ch_scale", c13.numel(), 2 * inter)
    experts = c13.numel() // (2 * inter)
    if out is not None:
        out_dtype = out.dtype
        _sized(fn, out, tuple(_FLOATS), tokens * hidden, "out")
    elif out_dtype not in _FLOATS:
        raise ValueError(f"{fn}: out_dtype must be float32 or bfloat16")
    else:
        out = _empty(stream, (tokens, hidden), out_dtype, x.device)
    code = _FLOATS[out_dtype]
    _sized(fn, weights, _F32, tokens * top_k, "weights")
    n13, n2 = experts * 2 * inter, experts * hidden
    _sized(fn, p13, _U8, n13 * hidden // 2, "w13 w_packed")
    _sized(fn, g13, _U8, n13 * _per(hidden, group), "w13 grp_scale")
    _sized(fn, c13, _F32, n13, "w13 ch_scale")
    _sized(fn, p2, _U8, n2 * inter // 2, "w2 w_packed")
    _sized(fn, g2, _U8, n2 * _per(inter, group), "w2 grp_scale")
    _sized(fn, c2, _F32, n2, "w2 ch_scale")
    if workspace is None:
        need = _moe_bytes(tokens, experts, top_k, hidden, inter, code)
        workspace = _workspace(stream, need, x.device)
    else:
        _sized(fn, workspace, _U8, 0, "workspace")
    status = _lib.w4a8_moe_ffn(
        x.data_ptr(), ids.data_ptr(), _addr(weights), _addr(p13), _addr(g13), c13.data_ptr(),
        _addr(p2), _addr(g2), _addr(c2), tokens, experts, top_k, hidden, inter, group,
        out.data_ptr(), code, workspace.data_ptr(), workspace.numel(), _stream(stream))
    if status:
        raise W4A8Error(fn, status)
    return out


@functools.lru_cache(maxsize=4096)
def lora_workspace_bytes(tokens: int, adapters: int, rank: int, k: int) -> int:
    return int(_lib.w4a8_lora_workspace_bytes(tokens, adapters, rank, k))


def lora_add(x, a, b, ids, y, scale=None, out=None, workspace=None, stream=None):
    """out = y + scale[l] * ((x a[l]^T) b[l]^T) with l = ids[t] for each row t (outside the
    adapters: out = y).  x bf16 [tokens, k] and y, out [tokens, n] (both bfloat16 or both
    float32) may have strided rows; a bf16 [adapters, rank, k], b bf16 [adapters, n, rank],
    ids int32 [tokens], scale float32 [adapters] or None.  out may be y and may share memory
    with x."""
    fn = "lora_add"
    _dev(a, torch.bfloat16, "a")
    _dev(b, torch.bfloat16, "b")
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError(f"{fn}: a must be [adapters, rank, k] and b [adapters, n, rank]")
    adapters, rank, k = a.shape
    of_b, n, rank_b = b.shape
    if of_b != adapters or rank_b != rank:
        raise ValueError(f"{fn}: a must be [adapters, rank, k] and b [adapters, n, rank]")
    ldx = _rows(fn, x, (torch.bfloat16,), k, "x")
    ldy = _rows(fn, y, _FLOATS, n, "y")
    tokens = x.size(0)
    if y.size(0) != tokens:
        raise W4A8SizeError(fn, "y (rows)", y.size(0), tokens)
    if out is None:
        if stream is None and ldy == n:
            out = torch.empty_like(y)
        else:
            out = _empty(stream, (tokens, n), y.dtype, y.device)
        ldo = n
    else:
        ldo = _rows(fn, out, (y.dtype,), n, "out")
        if out.shape[0] != tokens:
            raise W4A8SizeError(fn, "out (rows)", out.shape[0], tokens)
    _sized(fn, ids, (torch.int32,), tokens, "ids")
    _sized(fn, scale, _F32, adapters, "scale")
    if workspace is None:
        need = lora_workspace_bytes(tokens, adapters, rank, k)
        workspace = _workspace(stream, need, x.device)
    else:
        _sized(fn, workspace, _U8, 0, "workspace")
    status = _lib.w4a8_lora_add(
        x.data_ptr(), ldx, a.data_ptr(), b.data_ptr(), _addr(scale), _addr(ids), tokens, adapters,
        rank, k, n, y.data_ptr(), ldy, out.data_ptr(), ldo, _FLOATS[y.dtype],
        workspace.data_ptr(), workspace.numel(), _stream(stream))
    if status:
        raise W4A8Error(fn, status)
    return out


# --------------------------------------- attention over an 8-bit cache --

_Tensor = torch.Tensor


def _misplaced(fn, t, name, dev):
    """What is wrong with a tensor argument that is not on the current device."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor")
    raise ValueError(f"{fn}: {name} is on {t.device}, the current device is cuda:{dev}")


def _device_of(fn, t, name):
    """The index of a tensor's device, which has to be the current one: launches go there."""
    if not isinstance(t, _Tensor) or t.get_device() < 0:
        _misplaced(fn, t, name, -1)
    dev = _raw_device() if _raw_device is not None else torch.cuda.current_device()
    if t.get_device() != dev:
        _misplaced(fn, t, name, dev)
    return dev


def _new(stream, like, dtype, *sizes):
    """A new tensor on the device of `like`, for a call enqueued on `stream` (as _empty; sizes
    one by one are 0.4 us faster than as a tuple)."""
    if stream is not None:
        return _empty(stream, sizes, dtype, like.device)
    if dtype is like.dtype:
        return like.new_empty(*sizes)
    return torch.empty(*sizes, dtype=dtype, device=like.device)


def _heads(fn, t, dtypes, name, dev, rows=None, heads=None, dim=None):
    """A tensor [rows, heads, head_dim] on the current device `dev` of one of `dtypes` (of
    these sizes where given) whose rows are contiguous; returns its sizes and the elements
    from one row to the next."""
    if not isinstance(t, _Tensor) or t.get_device() != dev:
        _misplaced(fn, t, name, dev)
    if t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} must be of dtype {' or '.join(map(str, dtypes))}, "
                         f"not {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{fn}: {name} must be [rows, heads, head_dim]")
    r, h, d = t.shape
    if (rows is not None and r != rows) or (heads is not None and h != heads) or \
            (dim is not None and d != dim):
        for have, need, what in ((r, rows, "rows"), (h, heads, "heads"), (d, dim, "head_dim")):
            if need is not None and have != need:
                raise W4A8SizeError(fn, f"{name} ({what})", have, need)
    if t.is_contiguous():
        return r, h, d, h * d
    sr, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{fn}: rows of {name} must be contiguous")
    return r, h, d, sr if r > 1 else h * d


def _flat(fn, t, dtype, need, name, dev):
    """A contiguous tensor of `dtype` on the current device `dev` with at least `need`
    elements."""
    if not isinstance(t, _Tensor) or t.get_device() != dev:
        _misplaced(fn, t, name, dev)
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous {dtype} tensor")
    if t.numel() < need:
        raise W4A8SizeError(fn, name, t.numel(), need)


def qk_norm_rope(q, k, cos_sin=None, positions=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, out_dtype=None, q_out=None,
                 k_out=None, stream=None):
    """RMS norms per head and the rotation by position of q [tokens, q_heads, head_dim] and k
    [tokens, kv_heads, head_dim] (both float32 or both bfloat16; rows may be strided, e.g.
    columns of a fused projection) -> (q_out, k_out), out_dtype (default: the inputs').

    q_weight and k_weight float32 [head_dim], None: not normed; cos_sin float32 [max_pos,
    rot] (rot / 2 cosines, then rot / 2 sines; None: no rotation) and positions int32
    [tokens]; a row whose position is outside the table is left as it was.  Pairs are rot / 2
    apart, or neighbours where interleaved.  q_out and k_out may be q and k."""
    fn = "qk_norm_rope"
    dev = _device_of(fn, q, "q")
    tokens, q_heads, dim, ldq = _heads(fn, q, _FLOATS, "q", dev)
    _, kv_heads, _, ldk = _heads(fn, k, (q.dtype,), "k", dev, tokens, None, dim)
    if out_dtype is None:
        out_dtype = (q_out if q_out is not None else k_out if k_out is not None else q).dtype
    if out_dtype not in _FLOATS:
        raise ValueError(f"{fn}: out_dtype must be float32 or bfloat16")
    if q_out is None:
        q_out, ldqo = _new(stream, q, out_dtype, tokens, q_heads, dim), q_heads * dim
    else:
        ldqo = _heads(fn, q_out, (out_dtype,), "q_out", dev, tokens, q_heads, dim)[3]
    if k_out is None:
        k_out, ldko = _new(stream, q, out_dtype, tokens, kv_heads, dim), kv_heads * dim
    else:
        ldko = _heads(fn, k_out, (out_dtype,), "k_out", dev, tokens, kv_heads, dim)[3]
    if q_weight is not None:
        _flat(fn, q_weight, torch.float32, dim, "q_weight", dev)
    if k_weight is not None:
        _flat(fn, k_weight, torch.float32, dim, "k_weight", dev)
    max_pos = rot = 0
    if cos_sin is not None:
        _flat(fn, cos_sin, torch.float32, 0, "cos_sin", dev)
        if cos_sin.dim() != 2:
            raise ValueError(f"{fn}: cos_sin must be [max_pos, rot]")
        max_pos, rot = cos_sin.shape
        if positions is not None:            # the library refuses a missing one itself
            _flat(fn, positions, torch.int32, tokens, "positions", dev)
    else:
        positions = None
    status = _lib.w4a8_qk_norm_rope(
        q.data_ptr(), ldq, k.data_ptr(), ldk, _FLOATS[q.dtype], _addr(q_weight), _addr(k_weight),
        eps, _addr(cos_sin), _addr(positions), max_pos, rot, 1 if interleaved else 0, tokens,
        q_heads, kv_heads, dim, q_out.data_ptr(), ldqo, k_out.data_ptr(), ldko,
        _FLOATS[out_dtype], _stream(stream))
    if status:
        raise W4A8Error(fn, status)
    return q_out, k_out


def kv8_cache(pages: int, kv_heads: int, head_dim: int, page: int, device="cuda"):
    """An empty paged 8-bit cache: (kv uint8 [pages, kv_heads, 2, page, head_dim], opaque
    inside; kv_scale float32 [pages, kv_heads, 2])."""
    kv = torch.zeros((pages, kv_heads, 2, page, head_dim), dtype=torch.uint8, device=device)
    return kv, torch.zeros((pages, kv_heads, 2), dtype=torch.float32, device=device)


def _kv_args(fn, kv, kv_scale, block_table, lens, row_start, dev):
    """Checks what the calls on the cache share; (the cache's sizes, ldb, blocks, seqs)."""
    _flat(fn, kv, torch.uint8, 0, "kv", dev)
    if kv.dim() != 5 or kv.size(2) != 2:
        raise ValueError(f"{fn}: kv must be [pages, kv_heads, 2, page, head_dim]")
    pages, kv_heads, _, page, dim = kv.shape
    _flat(fn, kv_scale, torch.float32, pages * kv_heads * 2, "kv_scale", dev)
    _flat(fn, lens, torch.int32, 0, "lens", dev)
    if lens.dim() != 1:
        raise ValueError(f"{fn}: lens must be [seqs]")
    seqs = lens.size(0)
    if not isinstance(block_table, _Tensor) or block_table.get_device() != dev:
        _misplaced(fn, block_table, "block_table", dev)
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError(f"{fn}: block_table must be int32 [seqs, blocks]")
    have, blocks = block_table.shape
    if have != seqs:
        raise W4A8SizeError(fn, "block_table (rows)", have, seqs)
    ldb = blocks
    if not block_table.is_contiguous():
        ldb, step = block_table.stride()
        if blocks > 1 and step != 1:
            raise ValueError(f"{fn}: rows of block_table must be contiguous")
        if seqs <= 1:
            ldb = blocks
    if row_start is not None:
        _flat(fn, row_start, torch.int32, seqs + 1, "row_start", dev)
    # the library counts them in 32 bits, and refuses the most that these hold
    return (pages, kv_heads, page, dim), ldb, min(blocks, 0x7fffffff), seqs


def kv8_write(k, v, kv, kv_scale, block_table, lens, row_start=None, stream=None):
    """Quantizes new rows k and v [rows, kv_heads, head_dim] (both float32 or both bfloat16,
    rows may be strided) into the cache: sequence s's rows row_start[s] .. row_start[s + 1] - 1
    (row_start None: its one row s) are its last tokens, lens int32 [seqs] counts all of them,
    block_table int32 [seqs, blocks] names the page of each run of `page` tokens (-1: none).
    One scale per page and head: older codes of a page are taken over to a scale that grew."""
    fn = "kv8_write"
    dev = _device_of(fn, kv, "kv")
    (pages, kv_heads, page, dim), ldb, blocks, seqs = _kv_args(fn, kv, kv_scale, block_table, lens,
                                                               row_start, dev)
    rows, _, _, ldk = _heads(fn, k, _FLOATS, "k", dev, None, kv_heads, dim)
    ldv = _heads(fn, v, (k.dtype,), "v", dev, rows, kv_heads, dim)[3]
    status = _lib.w4a8_kv8_write(
        k.data_ptr(), ldk, v.data_ptr(), ldv, _FLOATS[k.dtype], block_table.data_ptr(), ldb, blocks,
        lens.data_ptr(), _addr(row_start), seqs, rows, kv_heads, dim, page, pages, kv.data_ptr(),
        kv_scale.data_ptr(), _stream(stream))
    if status:
        raise W4A8Error(fn, status)


def kv8_read(kv, kv_scale, block_table, lens, row_start=None, tokens=None,
             out_dtype=torch.bfloat16, k=None, v=None, stream=None):
    """The last row_start[s + 1] - row_start[s] tokens of each sequence out of the cache
    (row_start None: the last one) -> (k, v) [tokens, kv_heads, head_dim], float32 or bfloat16;
    `tokens` is row_start's last entry.  Tokens without a page read as zeros, rows of no
    token are left as they were."""
    fn = "kv8_read"
    dev = _device_of(fn, kv, "kv")
    (pages, kv_heads, page, dim), ldb, blocks, seqs = _kv_args(fn, kv, kv_scale, block_table, lens,
                                                               row_start, dev)
    if tokens is None:
        if row_start is None:
            tokens = seqs
        elif k is not None:
            tokens = k.size(0)
        else:
            raise ValueError(f"{fn}: tokens (or k and v) must be given with row_start")
    if k is not None:
        out_dtype = k.dtype
    elif v is not None:
        out_dtype = v.dtype
    if out_dtype not in _FLOATS:
        raise ValueError(f"{fn}: out_dtype must be float32 or bfloat16")
    if k is None:
        k, ldk = _new(stream, kv, out_dtype, tokens, kv_heads, dim), kv_heads * dim
    else:
        ldk = _heads(fn, k, (out_dtype,), "k", dev, tokens, kv_heads, dim)[3]
    if v is None:
        v, ldv = _new(stream, kv, out_dtype, tokens, kv_heads, dim), kv_heads * dim
    else:
        ldv = _heads(fn, v, (out_dtype,), "v", dev, tokens, kv_heads, dim)[3]
    status = _lib.w4a8_kv8_read(
        kv.data_ptr(), kv_scale.data_ptr(), block_table.data_ptr(), ldb, blocks, lens.data_ptr(),
        _addr(row_start), seqs, tokens, kv_heads, dim, page, pages, k.data_ptr(), ldk, v.data_ptr(),
        ldv, _FLOATS[out_dtype], _stream(stream))
    if status:
        raise W4A8Error(fn, status)
    return k, v


@functools.lru_cache(maxsize=4096)
def attn_kv8_workspace_bytes(rows: int, seqs: int, ragged: bool, max_rows: int, blocks: int,
                             q_heads: int, kv_heads: int, head_dim: int, page: int) -> int:
    """Workspace of attn_kv8 for `rows` query rows of `seqs` sequences (at most max_rows each,
    `ragged`: with row_start) whose block tables hold `blocks` pages; 0: none."""
    if max(blocks, q_heads, kv_heads, head_dim, page) > 0x7fffffff:
        return 0                             # refused
    return int(_lib.w4a8_attn_kv8_workspace_bytes(rows, seqs, 1 if ragged else 0, max_rows, blocks,
                                                  q_heads, kv_heads, head_dim, page))


def attn_kv8(q, kv, kv_scale, block_table, lens, row_start=None, max_rows=None,
             causal: bool = True, window: int = 0, scale=None, want_lse: bool = False, out=None,
             lse=None, workspace=None, stream=None):
    """Attention of q bfloat16 [rows, q_heads, head_dim] (rows may be strided) over the cache
    -> out bfloat16 [rows, q_heads, head_dim], and with want_lse (or lse given) also the
    logarithm of the softmax's sum, float32 [rows, q_heads].

    Sequence s's rows row_start[s] .. row_start[s + 1] - 1 (None: its one row s) are its last
    tokens; they must be in the cache already (kv8_write).  max_rows bounds a sequence's rows
    (default: all rows).  scale defaults to head_dim ** -0.5; window > 0: only the last
    `window` tokens up to the row's own.  A row that sees nothing gives 0 and -inf."""
    fn = "attn_kv8"
    dev = _device_of(fn, kv, "kv")
    (pages, kv_heads, page, dim), ldb, blocks, seqs = _kv_args(fn, kv, kv_scale, block_table, lens,
                                                               row_start, dev)
    rows, q_heads, _, ldq = _heads(fn, q, (torch.bfloat16,), "q", dev, None, None, dim)
    if max_rows is None:
        max_rows = 1 if row_start is None else max(rows, 1)
    if out is None:
        out, ldo = _new(stream, q, torch.bfloat16, rows, q_heads, dim), q_heads * dim
    else:
        ldo = _heads(fn, out, (torch.bfloat16,), "out", dev, rows, q_heads, dim)[3]
    if lse is not None:
        _flat(fn, lse, torch.float32, rows * q_heads, "lse", dev)
    elif want_lse:
        lse = _new(stream, kv_scale, torch.float32, rows, q_heads)
    if workspace is None:
        need = attn_kv8_workspace_bytes(rows, seqs, row_start is not None, max_rows, blocks,
                                        q_heads, kv_heads, dim, page)
        if need:
            workspace = _workspace(stream, need, q.device)
    else:
        _flat(fn, workspace, torch.uint8, 0, "workspace", dev)
    if not 0 <= window <= 1 << 30:           # refused, also where 32 bits would not hold it
        window = -1 if window < 0 else 0x7fffffff
    status = _lib.w4a8_attn_kv8(
        q.data_ptr(), ldq, kv.data_ptr(), kv_scale.data_ptr(), block_table.data_ptr(), ldb, blocks,
        lens.data_ptr(), _addr(row_start), seqs, rows, max_rows, q_heads, kv_heads, dim, page, pages,
        1 if causal else 0, window, dim ** -0.5 if scale is None else scale, out.data_ptr(), ldo,
        _addr(lse), _addr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(stream))
    if status:
        raise W4A8Error(fn, status)
    return out if lse is None else (out, lse)


# -------------------------------------------------------- measurement aid --

def probe_mfma_i8(workgroups: int, iters: int, device=None, stream=None):
    """Int8 matrix-core reference loop: returns (ops, sink, clocks) where ops is
    the int8 operation count of the launch and clocks (after the stream is
    synchronized) holds [shader clock ticks, 100 MHz real-time ticks]."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    sink = _empty(stream, (workgroups * 512,), dtype=torch.int32, device=dev)
    clocks = _empty(stream, (2,), dtype=torch.int64, device=dev)
    _check("w4a8_probe_mfma_i8",
           _lib.w4a8_probe_mfma_i8(workgroups, iters, _ptr(sink), _ptr(clocks), _stream(stream)))
    return workgroups * iters * 4194304, sink, clocks
