"""Python binding of libbitdelta.so (include/bitdelta.h).

Argument marshalling only: every step of compression and apply runs in the
HIP kernels of the native library.  PyTorch provides the device memory (tensor
storage) and the stream (the current HIP stream of the tensor's device).  The
``bd_*`` functions mirror the C entry points one to one; ``compress``,
``apply`` and ``reconstruct`` additionally allocate outputs and workspace with
torch.  If the native library is missing or cannot be loaded, every call
raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libbitdelta.so")

# enums of the C ABI
BD_OK, BD_ERR_INVALID_ARG, BD_ERR_SHAPE, BD_ERR_DTYPE, BD_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
BD_ERR_WORKSPACE, BD_ERR_DEVICE, BD_ERR_NONFINITE, BD_ERR_USER_ID, BD_ERR_BATCH = 5, 6, 7, 8, 9
BD_F32, BD_BF16, BD_F16 = 0, 1, 2
BD_SCALE_MATRIX, BD_SCALE_GROUP, BD_SCALE_ROW, BD_SCALE_COL = 0, 1, 2, 3
BD_MX4_TOKENS_BF16, BD_MX4_TOKENS_MX4 = 0, 1
MX4_TOKENS = {"bf16": BD_MX4_TOKENS_BF16, "mx4": BD_MX4_TOKENS_MX4}
MODE_NAMES = {"matrix": BD_SCALE_MATRIX, "group": BD_SCALE_GROUP, "row": BD_SCALE_ROW,
              "col": BD_SCALE_COL}


class bd_compress_params(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("clip_k", ctypes.c_float),
                ("scale_dtype", ctypes.c_int32)]


class BitDeltaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libbitdelta.so (after torch, so both share torch's HIP runtime)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not found: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        P = ctypes.POINTER(bd_compress_params)
        L.bd_abi_version.restype = ctypes.c_int
        L.bd_abi_version.argtypes = []
        L.bd_status_string.restype = ctypes.c_char_p
        L.bd_status_string.argtypes = [ctypes.c_int]
        L.bd_signs_bytes.restype = sz
        L.bd_signs_bytes.argtypes = [i64, i64]
        L.bd_scales_count.restype = i64
        L.bd_scales_count.argtypes = [P, i64, i64]
        L.bd_compress_workspace_bytes.restype = sz
        L.bd_compress_workspace_bytes.argtypes = [P, i64, i64]
        L.bd_apply_workspace_bytes.restype = sz
        L.bd_apply_workspace_bytes.argtypes = [P, i64, i32, i64, i64, ctypes.c_int, ctypes.c_int]
        L.bd_compress.restype = ctypes.c_int
        L.bd_compress.argtypes = [vp, vp, ctypes.c_int, i64, i64, P, vp, vp, vp, sz, vp]
        L.bd_quantize_base.restype = ctypes.c_int
        L.bd_quantize_base.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, vp]
        L.bd_apply_q8_workspace_bytes.restype = sz
        L.bd_apply_q8_workspace_bytes.argtypes = [P, i64, i32, i64, i64, ctypes.c_int,
                                                  ctypes.c_int]
        L.bd_apply_q8.restype = ctypes.c_int
        L.bd_apply_q8.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, i64, vp, vp, P, i32, vp, vp,
                                  ctypes.c_int, vp, sz, vp]
        L.bd_select_axis_workspace_bytes.restype = sz
        L.bd_select_axis_workspace_bytes.argtypes = [i64, i64, ctypes.c_float]
        L.bd_select_axis.restype = ctypes.c_int
        L.bd_select_axis.argtypes = [vp, vp, ctypes.c_int, i64, i64, ctypes.c_float, vp, vp, vp,
                                     sz, vp]
        L.bd_reconstruct.restype = ctypes.c_int
        L.bd_reconstruct.argtypes = [vp, vp, P, i64, i64, vp, ctypes.c_int, vp, ctypes.c_int, vp]
        L.bd_apply.restype = ctypes.c_int
        L.bd_apply.argtypes = [vp, ctypes.c_int, i64, i64, vp, i64, vp, vp, P, i32, vp, vp,
                               ctypes.c_int, vp, sz, vp]
        L.bd_apply_noalloc.restype = ctypes.c_int
        L.bd_apply_noalloc.argtypes = [vp, ctypes.c_int, i64, i64, vp, i64, vp, vp, P, i32, vp, vp,
                                       ctypes.c_int, vp, vp]
        L.bd_apply_paged_workspace_bytes.restype = sz
        L.bd_apply_paged_workspace_bytes.argtypes = [P, i64, i32, i64, i64, ctypes.c_int,
                                                     ctypes.c_int]
        L.bd_apply_paged.restype = ctypes.c_int
        L.bd_apply_paged.argtypes = [vp, ctypes.c_int, i64, i64, vp, i64, vp, vp, ctypes.c_uint64,
                                     ctypes.c_uint64, i32, P, vp, i32, vp, vp, ctypes.c_int, vp, sz,
                                     vp]
        L.bd_device_status.restype = ctypes.c_int
        L.bd_device_status.argtypes = [vp, vp]
        L.bd_batch_workspace_bytes.restype = sz
        L.bd_batch_workspace_bytes.argtypes = [i64, i32, i64, ctypes.c_int]
        L.bd_batch_prepare.restype = ctypes.c_int
        L.bd_batch_prepare.argtypes = [vp, ctypes.c_int, i64, i64, vp, i32, vp, sz, vp]
        L.bd_base_gemm.restype = ctypes.c_int
        L.bd_base_gemm.argtypes = [vp, ctypes.c_int, i64, i64, vp, i64, vp, vp]
        L.bd_delta_apply.restype = ctypes.c_int
        L.bd_delta_apply.argtypes = [vp, sz, vp, ctypes.c_int, i64, i64, i32, i64, vp, vp, P, vp,
                                     vp]
        L.bd_batch_encode.restype = ctypes.c_int
        L.bd_batch_encode.argtypes = [vp, sz, vp, ctypes.c_int, i64, i64, i32, vp, P, vp]
        L.bd_delta_apply_encoded.restype = ctypes.c_int
        L.bd_delta_apply_encoded.argtypes = [vp, sz, ctypes.c_int, i64, i64, i32, i64, vp, vp, P,
                                             vp, vp]
        L.bd_base_gemm_n_workspace_bytes.restype = sz
        L.bd_base_gemm_n_workspace_bytes.argtypes = [ctypes.c_int, i64, i64, i32, vp]
        L.bd_base_gemm_n.restype = ctypes.c_int
        L.bd_base_gemm_n.argtypes = [vp, ctypes.c_int, i64, i64, i32, vp, vp, vp, vp, sz, vp]
        L.bd_base_gemm_q8_n.restype = ctypes.c_int
        L.bd_base_gemm_q8_n.argtypes = [vp, ctypes.c_int, i64, i64, i32, vp, vp, vp, vp, vp, sz,
                                        vp]
        L.bd_delta_apply_encoded_n.restype = ctypes.c_int
        L.bd_delta_apply_encoded_n.argtypes = [vp, sz, ctypes.c_int, i64, i64, i32, i32, vp, vp,
                                               vp, P, vp, vp]
        L.bd_decode_prepare.restype = ctypes.c_int
        L.bd_decode_prepare.argtypes = [vp, ctypes.c_int, i64, i64, vp, i32, vp, P, vp, sz, vp]
        L.bd_decode_apply.restype = ctypes.c_int
        L.bd_decode_apply.argtypes = [vp, ctypes.c_int, i64, i64, vp, i64, vp, vp, P, i32, vp,
                                      ctypes.c_int, vp, sz, vp]
        L.bd_mx4_scale_stride.restype = sz
        L.bd_mx4_scale_stride.argtypes = [i64]
        L.bd_quantize_mx4.restype = ctypes.c_int
        L.bd_quantize_mx4.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, vp, vp]
        L.bd_dequantize_mx4.restype = ctypes.c_int
        L.bd_dequantize_mx4.argtypes = [vp, vp, i64, i64, vp, ctypes.c_int, vp]
        for f in (L.bd_base_gemm_mx4_n_workspace_bytes, L.bd_base_gemm_mx4x4_n_workspace_bytes):
            f.restype = sz
            f.argtypes = [i64, i64, i32, vp]
        L.bd_base_gemm_mx4_n.restype = ctypes.c_int
        L.bd_base_gemm_mx4_n.argtypes = [vp, ctypes.c_int, i64, i64, i32, vp, vp, vp, vp, vp, sz,
                                         vp]
        L.bd_base_gemm_mx4x4_n.restype = ctypes.c_int
        L.bd_base_gemm_mx4x4_n.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp]
        L.bd_apply_mx4_workspace_bytes.restype = sz
        L.bd_apply_mx4_workspace_bytes.argtypes = [P, i64, i32, i64, i64, ctypes.c_int,
                                                   ctypes.c_int, ctypes.c_int]
        L.bd_apply_mx4.restype = ctypes.c_int
        L.bd_apply_mx4.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, i64, vp, vp, P, i32, vp, vp,
                                   ctypes.c_int, ctypes.c_int, vp, sz, vp]
        L.bd_fp8_scale_stride.restype = sz
        L.bd_fp8_scale_stride.argtypes = [i64]
        L.bd_quantize_fp8.restype = ctypes.c_int
        L.bd_quantize_fp8.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, vp, vp]
        L.bd_quantize_fp8_tokens.restype = ctypes.c_int
        L.bd_quantize_fp8_tokens.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, vp]
        L.bd_dequantize_fp8.restype = ctypes.c_int
        L.bd_dequantize_fp8.argtypes = [vp, vp, i64, i64, vp, ctypes.c_int, vp]
        L.bd_rmsnorm_fp8.restype = ctypes.c_int
        L.bd_rmsnorm_fp8.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, ctypes.c_int, i64, i64,
                                     ctypes.c_float, vp, vp, vp, vp, vp]
        L.bd_base_gemm_fp8_n_workspace_bytes.restype = sz
        L.bd_base_gemm_fp8_n_workspace_bytes.argtypes = [i64, i64, i32, vp]
        L.bd_base_gemm_fp8_n.restype = ctypes.c_int
        L.bd_base_gemm_fp8_n.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, ctypes.c_int, vp, sz,
                                         vp]
        L.bd_apply_fp8_workspace_bytes.restype = sz
        L.bd_apply_fp8_workspace_bytes.argtypes = [P, i64, i32, i64, i64, ctypes.c_int, ctypes.c_int]
        L.bd_apply_fp8.restype = ctypes.c_int
        L.bd_apply_fp8.argtypes = [vp, ctypes.c_int, i64, i64, vp, vp, vp, vp, i64, vp, vp, P, i32, vp,
                                   vp, ctypes.c_int, vp, sz, vp]
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().bd_status_string(int(s)).decode()


def params(mode="matrix", group_size: int = 128, clip_k: float = 0.0,
           scale_dtype: int = BD_F32, bits: int = 1) -> bd_compress_params:
    m = MODE_NAMES[mode] if isinstance(mode, str) else int(mode)
    return bd_compress_params(bits, m, group_size, clip_k, scale_dtype)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: Optional[torch.Tensor] = None, stream=None):
    if stream is not None:
        return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))
    dev = t.device if t is not None else torch.device("cuda")
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BD_BF16
    if t.dtype == torch.float32:
        return BD_F32
    if t.dtype == torch.float16:
        return BD_F16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _torch_dtype(code: int):
    return {BD_F32: torch.float32, BD_BF16: torch.bfloat16, BD_F16: torch.float16}[code]


def _check(st: int, where: str):
    if st != BD_OK:
        raise BitDeltaError(st, where)


# Argument checks done before any pointer reaches the library: the C ABI takes raw
# device pointers, so a host tensor, a strided view, int64 user ids or a scales bank
# too small for the scale mode would otherwise be read as something else on the GPU.

def _dev(t, name: str, dtypes=None, shape=None, device=None, optional: bool = False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ids(user_ids, T, device):
    _dev(user_ids, "user_ids", (torch.int32,), (T,), device)


def _bank(signs_bank, scales_bank, p, n_users, d_out, d_in, device):
    _dev(signs_bank, "signs_bank", (torch.int64,), (n_users, d_out, d_in // 64), device)
    _scales(scales_bank, p, n_users, d_out, d_in, device)


def _scales(scales_bank, p, n_users, d_out, d_in, device, optional=False):
    if scales_bank is not None and isinstance(scales_bank, torch.Tensor):
        need = n_users * max(bd_scales_count(p, d_out, d_in), 0)
        if scales_bank.numel() < need:
            raise ValueError(f"scales_bank holds {scales_bank.numel()} values, the scale mode "
                             f"needs {need} ({n_users} users)")
    _dev(scales_bank, "scales_bank", (scales_dtype(p),), None, device, optional)


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------------ queries

def bd_signs_bytes(d_out: int, d_in: int) -> int:
    return int(lib().bd_signs_bytes(d_out, d_in))


def bd_scales_count(p: bd_compress_params, d_out: int, d_in: int) -> int:
    return int(lib().bd_scales_count(ctypes.byref(p), d_out, d_in))


def bd_compress_workspace_bytes(p: bd_compress_params, d_out: int, d_in: int) -> int:
    return int(lib().bd_compress_workspace_bytes(ctypes.byref(p), d_out, d_in))


def bd_select_axis_workspace_bytes(d_out: int, d_in: int, clip_k: float = 0.0) -> int:
    return int(lib().bd_select_axis_workspace_bytes(d_out, d_in, float(clip_k)))


def bd_apply_workspace_bytes(p: bd_compress_params, T: int, n_users: int, d_out: int, d_in: int,
                             x_dtype: int, y_dtype: int) -> int:
    return int(lib().bd_apply_workspace_bytes(ctypes.byref(p), T, n_users, d_out, d_in, x_dtype,
                                              y_dtype))


# -------------------------------------------------------------- entry points

def bd_compress(w_fine, w_base, p, signs_out, scales_out, workspace, stream=None) -> int:
    _dev(w_fine, "w_fine", (torch.float32, torch.bfloat16))
    d_out, d_in = w_fine.shape
    dev = w_fine.device
    _dev(w_base, "w_base", (w_fine.dtype,), (d_out, d_in), dev, optional=True)
    _dev(signs_out, "signs_out", (torch.int64,), (d_out, d_in // 64), dev)
    _scales(scales_out, p, 1, d_out, d_in, dev)
    _dev(workspace, "workspace", None, None, dev)
    return int(lib().bd_compress(_ptr(w_fine), _ptr(w_base), _dtype_code(w_fine), d_out, d_in,
                                 ctypes.byref(p), _ptr(signs_out), _ptr(scales_out),
                                 _ptr(workspace), _nbytes(workspace), _stream(w_fine, stream)))


def bd_reconstruct(signs, scales, p, d_out, d_in, w_base, out, stream=None) -> int:
    _dev(signs, "signs", (torch.int64,), (d_out, d_in // 64))
    dev = signs.device
    _scales(scales, p, 1, d_out, d_in, dev)
    _dev(w_base, "w_base", (torch.float32, torch.bfloat16), (d_out, d_in), dev, optional=True)
    _dev(out, "out", (torch.float32, torch.bfloat16), (d_out, d_in), dev)
    return int(lib().bd_reconstruct(_ptr(signs), _ptr(scales), ctypes.byref(p), d_out, d_in,
                                    _ptr(w_base), _dtype_code(w_base) if w_base is not None else 0,
                                    _ptr(out), _dtype_code(out), _stream(out, stream)))


def _apply_args(x, w_base_rows, signs_bank, scales_bank, p, n_users, user_ids, y, workspace,
                wdtypes=None):
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    dev = x.device
    d_out = w_base_rows.shape[0]
    _dev(w_base_rows, "w_base", wdtypes or (x.dtype,), (d_out, d_in), dev)
    _bank(signs_bank, scales_bank, p, n_users, d_out, d_in, dev)
    _ids(user_ids, T, dev)
    _dev(y, "y", (torch.float32, torch.bfloat16), (T, d_out), dev)
    _dev(workspace, "workspace", None, None, dev)
    return T, d_in, d_out


def bd_apply(x, w_base, signs_bank, scales_bank, p, n_users, user_ids, y, workspace,
             stream=None) -> int:
    T, d_in, d_out = _apply_args(x, w_base, signs_bank, scales_bank, p, n_users, user_ids, y,
                                 workspace)
    return int(lib().bd_apply(_ptr(x), _dtype_code(x), T, d_in, _ptr(w_base), d_out,
                              _ptr(signs_bank), _ptr(scales_bank), ctypes.byref(p), int(n_users),
                              _ptr(user_ids), _ptr(y), _dtype_code(y), _ptr(workspace),
                              _nbytes(workspace), _stream(x, stream)))


def bd_apply_noalloc(x, w_base, signs_bank, scales_bank, p, n_users, user_ids, y, status=None,
                     stream=None) -> int:
    """bd_apply without a workspace (the library's scratch; see include/bitdelta.h);
    status: optional int32[1] device tensor that receives the call's status word."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    dev = x.device
    d_out = w_base.shape[0]
    _dev(w_base, "w_base", (x.dtype,), (d_out, d_in), dev)
    _bank(signs_bank, scales_bank, p, n_users, d_out, d_in, dev)
    _ids(user_ids, T, dev)
    _dev(y, "y", (torch.float32, torch.bfloat16), (T, d_out), dev)
    _dev(status, "status", (torch.int32,), (1,), dev, optional=True)
    return int(lib().bd_apply_noalloc(_ptr(x), _dtype_code(x), T, d_in, _ptr(w_base), d_out,
                                      _ptr(signs_bank), _ptr(scales_bank), ctypes.byref(p),
                                      int(n_users), _ptr(user_ids), _ptr(y), _dtype_code(y),
                                      _ptr(status), _stream(x, stream)))


def bd_apply_paged_workspace_bytes(p, T: int, n_slots: int, d_out: int, d_in: int,
                                   x_dtype: int, y_dtype: int) -> int:
    return int(lib().bd_apply_paged_workspace_bytes(ctypes.byref(p), T, n_slots, d_out, d_in,
                                                    x_dtype, y_dtype))


def bd_apply_paged(x, w_base, signs_pool, scales_pool, signs_stride: int, scales_stride: int,
                   n_slots: int, p, slot_of_user, user_ids, y, workspace, stream=None) -> int:
    """bd_apply over banks in a pool of slots (include/bitdelta.h).  signs_pool and
    scales_pool: uint8 views that start at slot 0's signs / scales of this matrix and
    reach the last slot's; strides in bytes (0: dense [n_slots][...] banks of the bank
    dtypes instead); slot_of_user: int32[n_users] device table."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    dev = x.device
    d_out = w_base.shape[0]
    _dev(w_base, "w_base", (x.dtype,), (d_out, d_in), dev)
    n_sc = bd_scales_count(p, d_out, d_in)
    esz = 2 if p.scale_dtype == BD_F16 else 4
    for t, name, stride, need in ((signs_pool, "signs_pool", signs_stride, d_out * d_in // 8),
                                  (scales_pool, "scales_pool", scales_stride, n_sc * esz)):
        _dev(t, name, None, None, dev)
        span = (n_slots - 1) * (stride or need) + need if n_slots > 0 else 0
        if _nbytes(t) < span:
            raise ValueError(f"{name} holds {_nbytes(t)} bytes, {n_slots} slots need {span}")
    _dev(slot_of_user, "slot_of_user", (torch.int32,), None, dev)
    if slot_of_user.dim() != 1:
        raise ValueError("slot_of_user must be one-dimensional")
    _ids(user_ids, T, dev)
    _dev(y, "y", (torch.float32, torch.bfloat16), (T, d_out), dev)
    _dev(workspace, "workspace", None, None, dev)
    return int(lib().bd_apply_paged(_ptr(x), _dtype_code(x), T, d_in, _ptr(w_base), d_out,
                                    _ptr(signs_pool), _ptr(scales_pool), int(signs_stride),
                                    int(scales_stride), int(n_slots), ctypes.byref(p),
                                    _ptr(slot_of_user), slot_of_user.numel(), _ptr(user_ids),
                                    _ptr(y), _dtype_code(y), _ptr(workspace), _nbytes(workspace),
                                    _stream(x, stream)))


def bd_device_status(workspace, stream=None) -> int:
    _dev(workspace, "workspace")
    return int(lib().bd_device_status(_ptr(workspace), _stream(workspace, stream)))


def bd_batch_workspace_bytes(T: int, n_users: int, d_in: int, x_dtype: int) -> int:
    return int(lib().bd_batch_workspace_bytes(T, n_users, d_in, x_dtype))


def bd_batch_prepare(x, user_ids, n_users, batch, stream=None) -> int:
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    _ids(user_ids, T, x.device)
    _dev(batch, "batch", None, None, x.device)
    return int(lib().bd_batch_prepare(_ptr(x), _dtype_code(x), T, d_in, _ptr(user_ids),
                                      int(n_users), _ptr(batch), _nbytes(batch),
                                      _stream(x, stream)))


def bd_base_gemm(x, w_base, y, stream=None) -> int:
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    _dev(w_base, "w_base", (x.dtype,), (w_base.shape[0], d_in), x.device)
    _dev(y, "y", (torch.float32,), (T, w_base.shape[0]), x.device)
    return int(lib().bd_base_gemm(_ptr(x), _dtype_code(x), T, d_in, _ptr(w_base),
                                  w_base.shape[0], _ptr(y), _stream(x, stream)))


def bd_delta_apply(batch, x, n_users, signs_bank, scales_bank, p, y, stream=None) -> int:
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    dev = x.device
    _dev(y, "y", (torch.float32,), None, dev)
    if y.dim() != 2 or y.shape[0] != T:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected ({T}, d_out)")
    d_out = y.shape[1]
    _bank(signs_bank, scales_bank, p, n_users, d_out, d_in, dev)
    _dev(batch, "batch", None, None, dev)
    return int(lib().bd_delta_apply(_ptr(batch), _nbytes(batch), _ptr(x), _dtype_code(x), T, d_in,
                                    int(n_users), d_out, _ptr(signs_bank), _ptr(scales_bank),
                                    ctypes.byref(p), _ptr(y), _stream(y, stream)))


def bd_batch_encode(batch, x, n_users, scales_bank, p, stream=None) -> int:
    _dev(x, "x", (torch.bfloat16,))
    T, d_in = x.shape
    dev = x.device
    _dev(batch, "batch", None, None, dev)
    if p.mode == BD_SCALE_COL:
        _scales(scales_bank, p, n_users, 1, d_in, dev)
    else:
        _dev(scales_bank, "scales_bank", None, None, dev, optional=True)
    return int(lib().bd_batch_encode(_ptr(batch), _nbytes(batch), _ptr(x), _dtype_code(x), T,
                                     d_in, int(n_users), _ptr(scales_bank), ctypes.byref(p),
                                     _stream(x, stream)))


def bd_delta_apply_encoded(batch, T, d_in, n_users, signs_bank, scales_bank, p, y,
                           stream=None) -> int:
    _dev(y, "y", (torch.float32,))
    dev = y.device
    if y.dim() != 2 or y.shape[0] != T:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected ({T}, d_out)")
    d_out = y.shape[1]
    _bank(signs_bank, scales_bank, p, n_users, d_out, d_in, dev)
    _dev(batch, "batch", None, None, dev)
    return int(lib().bd_delta_apply_encoded(_ptr(batch), _nbytes(batch), BD_BF16, int(T),
                                            int(d_in), int(n_users), d_out, _ptr(signs_bank),
                                            _ptr(scales_bank), ctypes.byref(p), _ptr(y),
                                            _stream(y, stream)))


def _ptr_array(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def bd_base_gemm_n_workspace_bytes(x_dtype: int, T: int, d_in: int, d_outs) -> int:
    arr = (ctypes.c_int64 * len(d_outs))(*[int(d) for d in d_outs])
    return int(lib().bd_base_gemm_n_workspace_bytes(x_dtype, T, d_in, len(d_outs), arr))


def bd_base_gemm_n(x, w_bases, ys, workspace=None, stream=None) -> int:
    """Base products of up to 4 matrices that read x, in one launch (K split in ordered
    parts through `workspace` where that fills the chip better; None: no split)."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    if not 1 <= len(w_bases) <= 4 or len(ys) != len(w_bases):
        raise ValueError("1..4 matrices, one output each")
    for w, y in zip(w_bases, ys):
        _dev(w, "w_base", (x.dtype,), (w.shape[0], d_in), x.device)
        _dev(y, "y", (torch.float32,), (T, w.shape[0]), x.device)
    _dev(workspace, "workspace", None, None, x.device, optional=True)
    d_outs = (ctypes.c_int64 * len(ys))(*[w.shape[0] for w in w_bases])
    return int(lib().bd_base_gemm_n(_ptr(x), _dtype_code(x), T, d_in, len(ys),
                                    _ptr_array(w_bases), d_outs, _ptr_array(ys), _ptr(workspace),
                                    0 if workspace is None else _nbytes(workspace),
                                    _stream(x, stream)))


def bd_base_gemm_q8_n(x, wqs, wscales, ys, workspace=None, stream=None) -> int:
    """bd_base_gemm_n on INT8 base rows (quantize_base): up to 4 matrices that read x, in
    one launch; `workspace` as for bd_base_gemm_n (sized by its query, None: no split)."""
    _dev(x, "x", (torch.bfloat16,))
    T, d_in = x.shape
    if not 1 <= len(wqs) <= 4 or len(ys) != len(wqs) or len(wscales) != len(wqs):
        raise ValueError("1..4 matrices, one scale vector and one output each")
    for w, sc, y in zip(wqs, wscales, ys):
        _dev(w, "wq", (torch.int8,), (w.shape[0], d_in), x.device)
        _dev(sc, "wscales", (torch.float32,), (w.shape[0],), x.device)
        _dev(y, "y", (torch.float32,), (T, w.shape[0]), x.device)
    _dev(workspace, "workspace", None, None, x.device, optional=True)
    d_outs = (ctypes.c_int64 * len(ys))(*[w.shape[0] for w in wqs])
    return int(lib().bd_base_gemm_q8_n(_ptr(x), _dtype_code(x), T, d_in, len(ys), _ptr_array(wqs),
                                       _ptr_array(wscales), d_outs, _ptr_array(ys), _ptr(workspace),
                                       0 if workspace is None else _nbytes(workspace),
                                       _stream(x, stream)))


def bd_delta_apply_encoded_n(batch, T, d_in, n_users, signs_banks, scales_banks, p, ys,
                             stream=None) -> int:
    """Delta products of up to 4 matrices on one encoded batch, in one launch."""
    if not 1 <= len(ys) <= 4 or len(signs_banks) != len(ys) or len(scales_banks) != len(ys):
        raise ValueError("1..4 matrices, one bank and one output each")
    dev = ys[0].device if isinstance(ys[0], torch.Tensor) else None
    for sb, sc, y in zip(signs_banks, scales_banks, ys):
        _dev(y, "y", (torch.float32,), None, dev)
        if y.dim() != 2 or y.shape[0] != T:
            raise ValueError(f"y has shape {tuple(y.shape)}, expected ({T}, d_out)")
        _bank(sb, sc, p, n_users, y.shape[1], d_in, dev)
    _dev(batch, "batch", None, None, dev)
    d_outs = (ctypes.c_int64 * len(ys))(*[y.shape[1] for y in ys])
    return int(lib().bd_delta_apply_encoded_n(_ptr(batch), _nbytes(batch), BD_BF16, int(T),
                                              int(d_in), int(n_users), len(ys), d_outs,
                                              _ptr_array(signs_banks), _ptr_array(scales_banks),
                                              ctypes.byref(p), _ptr_array(ys),
                                              _stream(ys[0], stream)))


def bd_decode_prepare(x, user_ids, n_users, scales_bank, p, workspace, stream=None) -> int:
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    dev = x.device
    _ids(user_ids, T, dev)
    if p.mode == BD_SCALE_COL:
        _scales(scales_bank, p, n_users, 1, d_in, dev)
    else:
        _dev(scales_bank, "scales_bank", None, None, dev, optional=True)
    _dev(workspace, "workspace", None, None, dev)
    return int(lib().bd_decode_prepare(_ptr(x), _dtype_code(x), T, d_in, _ptr(user_ids),
                                       int(n_users), _ptr(scales_bank), ctypes.byref(p),
                                       _ptr(workspace), _nbytes(workspace), _stream(x, stream)))


def bd_decode_apply(x, w_base, signs_bank, scales_bank, p, n_users, y, workspace,
                    stream=None) -> int:
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, d_in = x.shape
    dev = x.device
    d_out = w_base.shape[0]
    _dev(w_base, "w_base", (x.dtype,), (d_out, d_in), dev)
    _bank(signs_bank, scales_bank, p, n_users, d_out, d_in, dev)
    _dev(y, "y", (torch.float32, torch.bfloat16), (T, d_out), dev)
    _dev(workspace, "workspace", None, None, dev)
    return int(lib().bd_decode_apply(_ptr(x), _dtype_code(x), T, d_in, _ptr(w_base),
                                     d_out, _ptr(signs_bank), _ptr(scales_bank),
                                     ctypes.byref(p), int(n_users), _ptr(y), _dtype_code(y),
                                     _ptr(workspace), _nbytes(workspace), _stream(x, stream)))


# ------------------------------------------------------- allocating helpers

def workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns >= 256-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def scales_dtype(p: bd_compress_params):
    return torch.float16 if p.scale_dtype == BD_F16 else torch.float32


def compress(w_fine: torch.Tensor, w_base: Optional[torch.Tensor], p: bd_compress_params,
             signs_out=None, scales_out=None, ws=None, stream=None,
             check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    d_out, d_in = w_fine.shape
    dev = w_fine.device
    if signs_out is None:
        signs_out = torch.empty((d_out, d_in // 64), dtype=torch.int64, device=dev)
    n_sc = bd_scales_count(p, d_out, d_in)
    if n_sc < 0:
        raise BitDeltaError(BD_ERR_INVALID_ARG, "bd_scales_count")
    if scales_out is None:
        scales_out = torch.empty(n_sc, dtype=scales_dtype(p), device=dev)
    if ws is None:
        ws = workspace(bd_compress_workspace_bytes(p, d_out, d_in), dev)
    _check(bd_compress(w_fine, w_base, p, signs_out, scales_out, ws, stream), "bd_compress")
    if check:
        _check(bd_device_status(ws, stream), "bd_compress (device)")
    return signs_out, scales_out


def bd_select_axis(w_fine, w_base, clip_k, errors, axis, workspace, stream=None) -> int:
    _dev(w_fine, "w_fine", (torch.float32, torch.bfloat16))
    d_out, d_in = w_fine.shape
    dev = w_fine.device
    _dev(w_base, "w_base", (w_fine.dtype,), (d_out, d_in), dev, optional=True)
    _dev(errors, "errors", (torch.float64,), (2,), dev, optional=True)
    _dev(axis, "axis", (torch.int32,), (1,), dev, optional=True)
    _dev(workspace, "workspace", None, None, dev)
    return int(lib().bd_select_axis(_ptr(w_fine), _ptr(w_base), _dtype_code(w_fine), d_out, d_in,
                                    float(clip_k), _ptr(errors), _ptr(axis), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(w_fine, stream)))


def bd_quantize_base(w, q_out, scales_out, stream=None) -> int:
    _dev(w, "w", (torch.float32, torch.bfloat16))
    d_out, d_in = w.shape
    _dev(q_out, "q_out", (torch.int8,), (d_out, d_in), w.device)
    _dev(scales_out, "scales_out", (torch.float32,), (d_out,), w.device)
    return int(lib().bd_quantize_base(_ptr(w), _dtype_code(w), d_out, d_in, _ptr(q_out),
                                      _ptr(scales_out), _stream(w, stream)))


def bd_apply_q8(x, wq, wscales, signs_bank, scales_bank, p, n_users, user_ids, y, workspace,
                stream=None) -> int:
    T, d_in, d_out = _apply_args(x, wq, signs_bank, scales_bank, p, n_users, user_ids, y,
                                 workspace, wdtypes=(torch.int8,))
    _dev(wscales, "wscales", (torch.float32,), (d_out,), x.device)
    return int(lib().bd_apply_q8(_ptr(x), _dtype_code(x), T, d_in, _ptr(wq), _ptr(wscales), d_out,
                                 _ptr(signs_bank), _ptr(scales_bank), ctypes.byref(p),
                                 int(n_users), _ptr(user_ids), _ptr(y), _dtype_code(y),
                                 _ptr(workspace), _nbytes(workspace),
                                 _stream(x, stream)))


def quantize_base(w: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """INT8 rows and their fp32 scales (bd_quantize_base)."""
    d_out, d_in = w.shape
    q = torch.empty((d_out, d_in), dtype=torch.int8, device=w.device)
    s = torch.empty(d_out, dtype=torch.float32, device=w.device)
    _check(bd_quantize_base(w, q, s, stream), "bd_quantize_base")
    return q, s


def bd_apply_q8_workspace_bytes(p, T: int, n_users: int, d_out: int, d_in: int, x_dtype: int,
                                y_dtype: int) -> int:
    return int(lib().bd_apply_q8_workspace_bytes(ctypes.byref(p), T, n_users, d_out, d_in,
                                                 x_dtype, y_dtype))


def apply_q8(x, wq, wscales, signs_bank, scales_bank, p, user_ids, y_dtype=torch.float32,
             ws=None, stream=None, check: bool = False) -> torch.Tensor:
    T, d_in = x.shape
    d_out = wq.shape[0]
    U = signs_bank.shape[0]
    y = torch.empty((T, d_out), dtype=y_dtype, device=x.device)
    if ws is None:
        ws = workspace(bd_apply_q8_workspace_bytes(p, T, U, d_out, d_in, _dtype_code(x),
                                                   _dtype_code(y)), x.device)
    _check(bd_apply_q8(x, wq, wscales, signs_bank, scales_bank, p, U, user_ids, y, ws, stream),
           "bd_apply_q8")
    if check:
        _check(bd_device_status(ws, stream), "bd_apply_q8 (device)")
    return y


# -------------------------------------------------------- MX4 base weights
# (a matrix [rows][cols] is codes uint8 [rows][cols // 2] and scales uint8
# [rows][bd_mx4_scale_stride(cols)]; see include/bitdelta.h)

def bd_mx4_scale_stride(cols: int) -> int:
    return int(lib().bd_mx4_scale_stride(int(cols)))


# A decode step is a chain of launches of a few microseconds, so these calls check their
# tensors in one expression and leave the naming of what is wrong to _dev.

def _need(t, name, dtype, shape, idx):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == idx and idx >= 0
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        _dev(t, name, (dtype,), shape, torch.device("cuda", idx) if idx >= 0 else None)


def _run(f, idx, stream, *args) -> int:
    """f(*args, stream) with device idx current (the launches need it)."""
    raw = torch._C._cuda_getCurrentRawStream(idx) if stream is None else _stream(None, stream)
    if torch._C._cuda_getDevice() == idx:
        return f(*args, raw)
    with torch.cuda.device(idx):
        return f(*args, raw)


def _tokens_2d(x, name, dtypes):
    """(device index, rows, columns) of a two-dimensional tensor of one of dtypes."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda or x.dtype not in dtypes:
        _dev(x, name, dtypes)
        raise ValueError(f"{name} must be two-dimensional")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.get_device(), *x.shape


def _mx4(codes, scales, name: str, idx=None, cols: Optional[int] = None):
    """(device index, rows, cols) of an MX4 matrix after the checks of its two tensors."""
    if isinstance(codes, torch.Tensor) and (
            codes.dim() != 2 or (cols is not None and 2 * codes.shape[1] != cols)):
        raise ValueError(f"{name} codes have shape {tuple(codes.shape)}, expected (rows, "
                         f"{'cols' if cols is None else cols} / 2)")
    if idx is None:
        _dev(codes, name + " codes", (torch.uint8,))
        idx = codes.get_device()
    _need(codes, name + " codes", torch.uint8, None, idx)
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    _need(scales, name + " scales", torch.uint8, (rows, 16 * ((cols + 511) // 512)), idx)
    return idx, rows, cols


def bd_quantize_mx4(w, codes_out, scales_out, values_out=None, stream=None) -> int:
    idx, rows, cols = _tokens_2d(w, "w", (torch.float32, torch.bfloat16))
    _need(codes_out, "codes_out", torch.uint8, (rows, cols // 2), idx)
    _need(scales_out, "scales_out", torch.uint8, (rows, 16 * ((cols + 511) // 512)), idx)
    if values_out is not None:
        _need(values_out, "values_out", w.dtype, (rows, cols), idx)
    return _quantize_mx4(w, idx, rows, cols, codes_out, scales_out, values_out, stream)


def _quantize_mx4(w, idx, rows, cols, codes, scales, values, stream) -> int:
    return _run(lib().bd_quantize_mx4, idx, stream, w.data_ptr(), _dtype_code(w), rows, cols,
                codes.data_ptr(), scales.data_ptr(), None if values is None else values.data_ptr())


def bd_dequantize_mx4(codes, scales, out, stream=None) -> int:
    idx, rows, cols = _mx4(codes, scales, "base")
    _dev(out, "out", (torch.float32, torch.bfloat16), (rows, cols), codes.device)
    return _run(lib().bd_dequantize_mx4, idx, stream, codes.data_ptr(), scales.data_ptr(), rows,
                cols, out.data_ptr(), _dtype_code(out))


def _mx4_bases(bases, idx, d_in):
    """Row counts of 1..4 MX4 matrices on device idx, after their checks."""
    if not 1 <= len(bases) <= 4:
        raise ValueError("1..4 matrices")
    return [_mx4(codes, scales, "base", idx, d_in)[1] for codes, scales in bases]


def _mx4_outs(ys, T, rows, workspace, idx):
    if len(ys) != len(rows):
        raise ValueError("1..4 matrices, one output each")
    for y, n in zip(ys, rows):
        _need(y, "y", torch.float32, (T, n), idx)
    if workspace is not None:
        _dev(workspace, "workspace", None, None, ys[0].device)


# host arrays of 1..4 pointers and sizes (made once: their types cost as much as a call)
_PTRS = [None] + [ctypes.c_void_p * n for n in range(1, 5)]
_SIZES = [None] + [ctypes.c_int64 * n for n in range(1, 5)]


def _mx4_args(bases, sizes, ys, ws):
    P = _PTRS[len(ys)]
    return (len(ys), P(*[c.data_ptr() for c, _ in bases]), P(*[s.data_ptr() for _, s in bases]), sizes,
            P(*[y.data_ptr() for y in ys]), None if ws is None else ws.data_ptr(),
            0 if ws is None else _nbytes(ws))


def bd_base_gemm_mx4_n_workspace_bytes(T: int, d_in: int, d_outs) -> int:
    arr = (ctypes.c_int64 * len(d_outs))(*[int(d) for d in d_outs])
    return lib().bd_base_gemm_mx4_n_workspace_bytes(T, d_in, len(d_outs), arr)


def bd_base_gemm_mx4_n(x, bases, ys, workspace=None, stream=None) -> int:
    """Base products of bf16 tokens with up to 4 MX4 matrices; bases: (codes, scales) of
    each, ys: fp32 outputs, `workspace` sized by the query (None: no split of K)."""
    idx, T, d_in = _tokens_2d(x, "x", (torch.bfloat16,))
    rows = _mx4_bases(bases, idx, d_in)
    _mx4_outs(ys, T, rows, workspace, idx)
    return _run(lib().bd_base_gemm_mx4_n, idx, stream, x.data_ptr(), BD_BF16, T, d_in,
                *_mx4_args(bases, _SIZES[len(rows)](*rows), ys, workspace))


def bd_base_gemm_mx4x4_n_workspace_bytes(T: int, d_in: int, d_outs) -> int:
    arr = (ctypes.c_int64 * len(d_outs))(*[int(d) for d in d_outs])
    return lib().bd_base_gemm_mx4x4_n_workspace_bytes(T, d_in, len(d_outs), arr)


def bd_base_gemm_mx4x4_n(x_codes, x_scales, bases, ys, workspace=None, stream=None) -> int:
    """bd_base_gemm_mx4_n on MX4 tokens (codes and scales of bd_quantize_mx4)."""
    idx, T, d_in = _mx4(x_codes, x_scales, "token")
    rows = _mx4_bases(bases, idx, d_in)
    _mx4_outs(ys, T, rows, workspace, idx)
    return _run(lib().bd_base_gemm_mx4x4_n, idx, stream, x_codes.data_ptr(), x_scales.data_ptr(), T,
                d_in, *_mx4_args(bases, _SIZES[len(rows)](*rows), ys, workspace))


def _tokens(tokens) -> int:
    if isinstance(tokens, str):
        if tokens not in MX4_TOKENS:
            raise ValueError(f"tokens is {tokens!r}, expected one of {sorted(MX4_TOKENS)}")
        return MX4_TOKENS[tokens]
    return int(tokens)


def bd_apply_mx4_workspace_bytes(p, T: int, n_users: int, d_out: int, d_in: int, x_dtype: int,
                                 y_dtype: int, tokens="bf16") -> int:
    return lib().bd_apply_mx4_workspace_bytes(ctypes.byref(p), T, n_users, d_out, d_in, x_dtype,
                                              y_dtype, _tokens(tokens))


def _apply_mx4_checks(x, codes, scales, signs_bank, scales_bank, p, n_users, user_ids):
    idx, T, d_in = _tokens_2d(x, "x", (torch.bfloat16, torch.float32))
    _, d_out, _ = _mx4(codes, scales, "base", idx, d_in)
    _need(signs_bank, "signs_bank", torch.int64, (n_users, d_out, d_in // 64), idx)
    _scales(scales_bank, p, n_users, d_out, d_in, x.device)
    _need(user_ids, "user_ids", torch.int32, (T,), idx)
    return idx, T, d_in, d_out


def _apply_mx4(x, idx, T, d_in, d_out, codes, scales, signs_bank, scales_bank, p, n_users,
               user_ids, y, ws, tokens, stream) -> int:
    return _run(lib().bd_apply_mx4, idx, stream, x.data_ptr(), _dtype_code(x), T, d_in,
                codes.data_ptr(), scales.data_ptr(), d_out, signs_bank.data_ptr(),
                scales_bank.data_ptr(), ctypes.byref(p), int(n_users), user_ids.data_ptr(),
                y.data_ptr(), _dtype_code(y), tokens, ws.data_ptr(), _nbytes(ws))


def bd_apply_mx4(x, codes, scales, signs_bank, scales_bank, p, n_users, user_ids, y, workspace,
                 tokens="bf16", stream=None) -> int:
    """bd_apply on an MX4 base; tokens: "bf16" or "mx4", how the base product takes x."""
    idx, T, d_in, d_out = _apply_mx4_checks(x, codes, scales, signs_bank, scales_bank, p, n_users,
                                            user_ids)
    _dev(y, "y", (torch.float32, torch.bfloat16), (T, d_out), x.device)
    _dev(workspace, "workspace", None, None, x.device)
    return _apply_mx4(x, idx, T, d_in, d_out, codes, scales, signs_bank, scales_bank, p, n_users,
                      user_ids, y, workspace, _tokens(tokens), stream)


def _current(stream, t):
    """The context of a helper's call on `stream` (a stream or its handle): what the call
    allocates on t's device is that stream's, as under torch.cuda.stream."""
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(getattr(stream, "cuda_stream", stream))
        dev = t.device if isinstance(t, torch.Tensor) and t.is_cuda else None  # (checked by the call)
        # (ExternalStream takes a handle of 0 for none and picks a stream from its pool)
        stream = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def quantize_mx4(w: torch.Tensor, values: bool = False, stream=None):
    """(codes, scales) of w in MX4, and with `values` also what they stand for, in w's
    dtype (bd_quantize_mx4)."""
    if stream is not None:
        with _current(stream, w):
            return quantize_mx4(w, values)
    idx, rows, cols = _tokens_2d(w, "w", (torch.float32, torch.bfloat16))
    codes = w.new_empty((rows, cols // 2), dtype=torch.uint8)
    scales = w.new_empty((rows, 16 * ((cols + 511) // 512)), dtype=torch.uint8)
    out = torch.empty_like(w) if values else None
    _check(_quantize_mx4(w, idx, rows, cols, codes, scales, out, stream), "bd_quantize_mx4")
    return (codes, scales, out) if values else (codes, scales)


def dequantize_mx4(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.bfloat16,
                   stream=None) -> torch.Tensor:
    _, rows, cols = _mx4(codes, scales, "base")
    if stream is not None:
        with _current(stream, codes):
            return dequantize_mx4(codes, scales, out_dtype)
    out = torch.empty((rows, cols), dtype=out_dtype, device=codes.device)
    _check(bd_dequantize_mx4(codes, scales, out), "bd_dequantize_mx4")
    return out


def base_gemm_mx4(x: torch.Tensor, bases, ws=None, stream=None):
    """[x . W^T] in fp32 for 1..4 MX4 matrices (codes, scales) and bf16 tokens x."""
    if stream is not None:
        with _current(stream, x):
            return base_gemm_mx4(x, bases, ws)
    idx, T, d_in = _tokens_2d(x, "x", (torch.bfloat16,))
    rows = _mx4_bases(bases, idx, d_in)
    ys = [x.new_empty((T, n), dtype=torch.float32) for n in rows]
    sizes = _SIZES[len(rows)](*rows)
    if ws is None:
        need = lib().bd_base_gemm_mx4_n_workspace_bytes(T, d_in, len(rows), sizes)
        ws = workspace(need, x.device) if need > 0 else None
    else:
        _dev(ws, "workspace", None, None, x.device)
    _check(_run(lib().bd_base_gemm_mx4_n, idx, stream, x.data_ptr(), BD_BF16, T, d_in,
                *_mx4_args(bases, sizes, ys, ws)), "bd_base_gemm_mx4_n")
    return ys


def base_gemm_mx4x4(xq, bases, ws=None, stream=None):
    """base_gemm_mx4 on MX4 tokens xq = (codes, scales)."""
    x_codes, x_scales = xq
    if stream is not None:
        with _current(stream, x_codes):
            return base_gemm_mx4x4(xq, bases, ws)
    idx, T, d_in = _mx4(x_codes, x_scales, "token")
    rows = _mx4_bases(bases, idx, d_in)
    ys = [x_codes.new_empty((T, n), dtype=torch.float32) for n in rows]
    sizes = _SIZES[len(rows)](*rows)
    if ws is None:
        need = lib().bd_base_gemm_mx4x4_n_workspace_bytes(T, d_in, len(rows), sizes)
        ws = workspace(need, x_codes.device) if need > 0 else None
    else:
        _dev(ws, "workspace", None, None, x_codes.device)
    _check(_run(lib().bd_base_gemm_mx4x4_n, idx, stream, x_codes.data_ptr(), x_scales.data_ptr(), T,
                d_in, *_mx4_args(bases, sizes, ys, ws)), "bd_base_gemm_mx4x4_n")
    return ys


def apply_mx4(x, codes, scales, signs_bank, scales_bank, p, user_ids, y_dtype=torch.float32,
              tokens="bf16", ws=None, stream=None, check: bool = False) -> torch.Tensor:
    """bd_apply on an MX4 base (codes, scales); tokens: how the base product reads x,
    "bf16" as it is or "mx4" quantised within the call."""
    if stream is not None:
        with _current(stream, x):
            return apply_mx4(x, codes, scales, signs_bank, scales_bank, p, user_ids, y_dtype, tokens,
                             ws, None, check)
    U, tok = signs_bank.shape[0], _tokens(tokens)
    idx, T, d_in, d_out = _apply_mx4_checks(x, codes, scales, signs_bank, scales_bank, p, U, user_ids)
    y = x.new_empty((T, d_out), dtype=y_dtype)
    if ws is None:
        ws = workspace(bd_apply_mx4_workspace_bytes(p, T, U, d_out, d_in, _dtype_code(x),
                                                    _dtype_code(y), tok), x.device)
    else:
        _dev(ws, "workspace", None, None, x.device)
    _check(_apply_mx4(x, idx, T, d_in, d_out, codes, scales, signs_bank, scales_bank, p, U, user_ids,
                      y, ws, tok, stream), "bd_apply_mx4")
    if check:
        _check(bd_device_status(ws, stream), "bd_apply_mx4 (device)")
    return y


# -------------------------------------------------------- FP8 base weights
# (a weight [rows][cols] is codes float8_e4m3fn [rows][cols] and scales float32
# [ceil(rows / 128)][ceil(cols / 128)]; tokens [T][d_in] are codes float8_e4m3fn [T][d_in] and
# scale bytes uint8 [T][bd_fp8_scale_stride(d_in)]; see include/bitdelta.h)

_E4M3 = torch.float8_e4m3fn


def bd_fp8_scale_stride(cols: int) -> int:
    return int(lib().bd_fp8_scale_stride(int(cols)))


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _plain(t, dtype, idx) -> bool:
    """Whether t is a contiguous tensor of dtype on device idx (the whole check of most calls)."""
    return type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == idx and t.is_contiguous()


def _fp8(codes, scales, name: str, idx=None, cols: Optional[int] = None):
    """(device index, rows, cols) of an FP8 weight after the checks of its two tensors."""
    if idx is None and type(codes) is torch.Tensor and codes.is_cuda:
        idx = codes.get_device()
    if idx is not None and _plain(codes, _E4M3, idx) and _plain(scales, torch.float32, idx) and codes.dim() == 2:
        r, c = codes.shape
        if (cols is None or c == cols) and scales.shape == ((r + 127) // 128, (c + 127) // 128):
            return idx, r, c
    idx, r, c = _fp8_codes(codes, name, idx, cols)
    _need(scales, name + " scales", torch.float32, (_blocks(r), _blocks(c)), idx)
    return idx, r, c


def _fp8_tokens(codes, scales, idx=None, shape=None):
    """The same for tokens; shape: the (T, d_in) they must have."""
    if shape is not None and isinstance(codes, torch.Tensor) and codes.shape != shape:
        raise ValueError(f"token codes have shape {tuple(codes.shape)}, expected {tuple(shape)}")
    if idx is None and type(codes) is torch.Tensor and codes.is_cuda:
        idx = codes.get_device()
    if idx is not None and _plain(codes, _E4M3, idx) and _plain(scales, torch.uint8, idx) and codes.dim() == 2:
        r, c = codes.shape
        if scales.shape == (r, 4 * ((c + 511) // 512)):
            return idx, r, c
    idx, r, c = _fp8_codes(codes, "token", idx, None)
    _need(scales, "token scales", torch.uint8, (r, 4 * ((c + 511) // 512)), idx)
    return idx, r, c


def _fp8_codes(codes, name, idx, cols):
    if isinstance(codes, torch.Tensor) and (
            codes.dim() != 2 or (cols is not None and codes.shape[1] != cols)):
        raise ValueError(f"{name} codes have shape {tuple(codes.shape)}, expected (rows, "
                         f"{'cols' if cols is None else cols})")
    if idx is None:
        _dev(codes, name + " codes", (_E4M3,))
        idx = codes.get_device()
    _need(codes, name + " codes", _E4M3, None, idx)
    return idx, *codes.shape


def bd_quantize_fp8(w, codes_out, scales_out, values_out=None, stream=None) -> int:
    idx, rows, cols = _tokens_2d(w, "w", (torch.float32, torch.bfloat16))
    _need(codes_out, "codes_out", _E4M3, (rows, cols), idx)
    _need(scales_out, "scales_out", torch.float32, (_blocks(rows), _blocks(cols)), idx)
    if values_out is not None:
        _need(values_out, "values_out", w.dtype, (rows, cols), idx)
    return _run(lib().bd_quantize_fp8, idx, stream, w.data_ptr(), _dtype_code(w), rows, cols,
                codes_out.data_ptr(), scales_out.data_ptr(),
                None if values_out is None else values_out.data_ptr())


def bd_quantize_fp8_tokens(x, codes_out, scales_out, stream=None) -> int:
    idx, T, d_in = _tokens_2d(x, "x", (torch.float32, torch.bfloat16))
    _need(codes_out, "codes_out", _E4M3, (T, d_in), idx)
    _need(scales_out, "scales_out", torch.uint8, (T, 4 * ((d_in + 511) // 512)), idx)
    return _run(lib().bd_quantize_fp8_tokens, idx, stream, x.data_ptr(), _dtype_code(x), T, d_in,
                codes_out.data_ptr(), scales_out.data_ptr())


def bd_dequantize_fp8(codes, scales, out, stream=None) -> int:
    idx, rows, cols = _fp8(codes, scales, "base")
    _dev(out, "out", (torch.float32, torch.bfloat16), (rows, cols), codes.device)
    return _run(lib().bd_dequantize_fp8, idx, stream, codes.data_ptr(), scales.data_ptr(), rows, cols,
                out.data_ptr(), _dtype_code(out))


_NORM_DTYPES = (torch.float32, torch.bfloat16)


def _norm_in(h, weight, residual):
    idx, T, d = _tokens_2d(h, "h", _NORM_DTYPES)
    if not (_plain(weight, getattr(weight, "dtype", None), idx) and weight.dtype in _NORM_DTYPES
            and weight.shape == (d,)):
        _dev(weight, "weight", _NORM_DTYPES, (d,), h.device)
    if residual is not None and not (_plain(residual, getattr(residual, "dtype", None), idx)
                                     and residual.dtype in _NORM_DTYPES and residual.shape == (T, d)):
        _dev(residual, "residual", _NORM_DTYPES, (T, d), h.device)
    return idx, T, d


def _norm(idx, T, d, h, weight, eps, residual, h_out, x_out, codes, scales, stream) -> int:
    return _run(lib().bd_rmsnorm_fp8, idx, stream, h.data_ptr(), _dtype_code(h),
                None if residual is None else residual.data_ptr(),
                BD_F32 if residual is None else _dtype_code(residual), weight.data_ptr(),
                _dtype_code(weight), T, d, float(eps), None if h_out is None else h_out.data_ptr(),
                x_out.data_ptr(), codes.data_ptr(), scales.data_ptr())


def bd_rmsnorm_fp8(h, weight, eps, residual, h_out, x_out, codes_out, scales_out, stream=None) -> int:
    """RMS norm of h + residual (residual may be None; h_out may be h or, in h's dtype, the
    residual): the sum in h_out, the
    norm in bf16 in x_out and in FP8 in codes_out, scales_out."""
    idx, T, d = _norm_in(h, weight, residual)
    if residual is not None:
        _need(h_out, "h_out", h.dtype, (T, d), idx)
    _need(x_out, "x_out", torch.bfloat16, (T, d), idx)
    _need(codes_out, "codes_out", _E4M3, (T, d), idx)
    _need(scales_out, "scales_out", torch.uint8, (T, 4 * ((d + 511) // 512)), idx)
    return _norm(idx, T, d, h, weight, eps, residual, None if residual is None else h_out, x_out, codes_out,
                 scales_out, stream)


def _fp8_bases(bases, idx, d_in):
    """Row counts of 1..4 FP8 matrices on device idx, after their checks."""
    if not 1 <= len(bases) <= 4:
        raise ValueError("1..4 matrices")
    return [_fp8(codes, scales, "base", idx, d_in)[1] for codes, scales in bases]


def bd_base_gemm_fp8_n_workspace_bytes(T: int, d_in: int, d_outs) -> int:
    arr = (ctypes.c_int64 * len(d_outs))(*[int(d) for d in d_outs])
    return lib().bd_base_gemm_fp8_n_workspace_bytes(T, d_in, len(d_outs), arr)


def _fp8_args(bases, sizes, ys, ws):
    n, w, sc, d, y, *rest = _mx4_args(bases, sizes, ys, ws)
    return (n, w, sc, d, y, _dtype_code(ys[0]), *rest)


def bd_base_gemm_fp8_n(x_codes, x_scales, bases, ys, workspace=None, stream=None) -> int:
    """Base products of FP8 tokens with up to 4 FP8 matrices; bases: (codes, scales) of each,
    ys: outputs, all fp32 or all bf16, `workspace` sized by the query (None: no split of K)."""
    idx, T, d_in = _fp8_tokens(x_codes, x_scales)
    rows = _fp8_bases(bases, idx, d_in)
    if len(ys) != len(rows):
        raise ValueError("1..4 matrices, one output each")
    dt = torch.bfloat16 if isinstance(ys[0], torch.Tensor) and ys[0].dtype is torch.bfloat16 else torch.float32
    for y, n in zip(ys, rows):
        _need(y, "y", dt, (T, n), idx)
    if workspace is not None:
        _dev(workspace, "workspace", None, None, ys[0].device)
    return _run(lib().bd_base_gemm_fp8_n, idx, stream, x_codes.data_ptr(), x_scales.data_ptr(), T, d_in,
                *_fp8_args(bases, _SIZES[len(rows)](*rows), ys, workspace))


def bd_apply_fp8_workspace_bytes(p, T: int, n_users: int, d_out: int, d_in: int, x_dtype: int,
                                 y_dtype: int) -> int:
    return lib().bd_apply_fp8_workspace_bytes(ctypes.byref(p), T, n_users, d_out, d_in, x_dtype, y_dtype)


def _apply_fp8_checks(x, codes, scales, signs_bank, scales_bank, p, n_users, user_ids, xq):
    idx, T, d_in = _tokens_2d(x, "x", (torch.bfloat16, torch.float32))
    _, d_out, _ = _fp8(codes, scales, "base", idx, d_in)
    _need(signs_bank, "signs_bank", torch.int64, (n_users, d_out, d_in // 64), idx)
    _scales(scales_bank, p, n_users, d_out, d_in, x.device)
    _need(user_ids, "user_ids", torch.int32, (T,), idx)
    if xq is not None:
        _fp8_tokens(*xq, idx, (T, d_in))
    return idx, T, d_in, d_out


def _apply_fp8(x, idx, T, d_in, d_out, xq, codes, scales, signs_bank, scales_bank, p, n_users, user_ids, y,
               ws, stream) -> int:
    xc, xs = (None, None) if xq is None or T == 0 else (xq[0].data_ptr(), xq[1].data_ptr())
    return _run(lib().bd_apply_fp8, idx, stream, x.data_ptr(), _dtype_code(x), T, d_in, xc, xs,
                codes.data_ptr(), scales.data_ptr(), d_out, signs_bank.data_ptr(), scales_bank.data_ptr(),
                ctypes.byref(p), int(n_users), user_ids.data_ptr(), y.data_ptr(), _dtype_code(y),
                ws.data_ptr(), _nbytes(ws))


def bd_apply_fp8(x, codes, scales, signs_bank, scales_bank, p, n_users, user_ids, y, workspace, xq=None,
                 stream=None) -> int:
    """bd_apply on an FP8 base; xq: the tokens' FP8 form (codes, scales), or None: quantised
    within the call."""
    idx, T, d_in, d_out = _apply_fp8_checks(x, codes, scales, signs_bank, scales_bank, p, n_users,
                                            user_ids, xq)
    _dev(y, "y", (torch.float32, torch.bfloat16), (T, d_out), x.device)
    _dev(workspace, "workspace", None, None, x.device)
    return _apply_fp8(x, idx, T, d_in, d_out, xq, codes, scales, signs_bank, scales_bank, p, n_users,
                      user_ids, y, workspace, stream)


def quantize_fp8(w: torch.Tensor, values: bool = False, stream=None):
    """(codes, scales) of a weight in FP8, and with `values` also what they stand for, in w's
    dtype (bd_quantize_fp8)."""
    if stream is not None:
        with _current(stream, w):
            return quantize_fp8(w, values)
    idx, rows, cols = _tokens_2d(w, "w", (torch.float32, torch.bfloat16))
    codes = w.new_empty((rows, cols), dtype=_E4M3)
    scales = w.new_empty((_blocks(rows), _blocks(cols)), dtype=torch.float32)
    out = torch.empty_like(w) if values else None
    _check(_run(lib().bd_quantize_fp8, idx, None, w.data_ptr(), _dtype_code(w), rows, cols, codes.data_ptr(),
                scales.data_ptr(), None if out is None else out.data_ptr()), "bd_quantize_fp8")
    return (codes, scales, out) if values else (codes, scales)


def quantize_fp8_tokens(x: torch.Tensor, stream=None):
    """(codes, scale bytes) of a batch's tokens in FP8 (bd_quantize_fp8_tokens)."""
    if stream is not None:
        with _current(stream, x):
            return quantize_fp8_tokens(x)
    idx, T, d_in = _tokens_2d(x, "x", (torch.float32, torch.bfloat16))
    codes = x.new_empty((T, d_in), dtype=_E4M3)
    scales = x.new_empty((T, 4 * ((d_in + 511) // 512)), dtype=torch.uint8)
    _check(_run(lib().bd_quantize_fp8_tokens, idx, None, x.data_ptr(), _dtype_code(x), T, d_in,
                codes.data_ptr(), scales.data_ptr()), "bd_quantize_fp8_tokens")
    return codes, scales


def dequantize_fp8(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.bfloat16,
                   stream=None) -> torch.Tensor:
    idx, rows, cols = _fp8(codes, scales, "base")
    if stream is not None:
        with _current(stream, codes):
            return dequantize_fp8(codes, scales, out_dtype)
    out = codes.new_empty((rows, cols), dtype=out_dtype)
    _check(_run(lib().bd_dequantize_fp8, idx, None, codes.data_ptr(), scales.data_ptr(), rows, cols,
                out.data_ptr(), _dtype_code(out)), "bd_dequantize_fp8")
    return out


def rmsnorm_fp8(h: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                inplace: bool = False, stream=None):
    """RMS norm of h + residual (or of h): (the sum, in h itself with `inplace`; the norm in
    bf16; the norm in FP8 as (codes, scale bytes)) (bd_rmsnorm_fp8)."""
    if stream is not None:
        with _current(stream, h):
            return rmsnorm_fp8(h, weight, eps, residual, inplace)
    idx, T, d = _norm_in(h, weight, residual)
    h_out = h if residual is None or inplace else torch.empty_like(h)
    x = h.new_empty((T, d), dtype=torch.bfloat16)
    codes = h.new_empty((T, d), dtype=_E4M3)
    scales = h.new_empty((T, 4 * ((d + 511) // 512)), dtype=torch.uint8)
    _check(_norm(idx, T, d, h, weight, eps, residual, h_out, x, codes, scales, None), "bd_rmsnorm_fp8")
    return h_out, x, (codes, scales)


def base_gemm_fp8(xq, bases, y_dtype=torch.float32, ws=None, stream=None):
    """[x . W^T] in y_dtype (fp32, or bf16: the fp32 sums rounded once) for 1..4 FP8 matrices
    (codes, scales) and FP8 tokens xq = (codes, scale bytes)."""
    x_codes, x_scales = xq
    if stream is not None:
        with _current(stream, x_codes):
            return base_gemm_fp8(xq, bases, y_dtype, ws)
    idx, T, d_in = _fp8_tokens(x_codes, x_scales)
    rows = _fp8_bases(bases, idx, d_in)
    ys = [x_codes.new_empty((T, n), dtype=y_dtype) for n in rows]
    sizes = _SIZES[len(rows)](*rows)
    if ws is None:
        need = lib().bd_base_gemm_fp8_n_workspace_bytes(T, d_in, len(rows), sizes)
        ws = workspace(need, x_codes.device) if need > 0 else None
    else:
        _dev(ws, "workspace", None, None, x_codes.device)
    _check(_run(lib().bd_base_gemm_fp8_n, idx, None, x_codes.data_ptr(), x_scales.data_ptr(), T, d_in,
                *_fp8_args(bases, sizes, ys, ws)), "bd_base_gemm_fp8_n")
    return ys


def apply_fp8(x, codes, scales, signs_bank, scales_bank, p, user_ids, y_dtype=torch.float32, xq=None,
              ws=None, stream=None, check: bool = False) -> torch.Tensor:
    """bd_apply on an FP8 base (codes, scales); xq: the tokens' FP8 form (codes, scale bytes;
    from rmsnorm_fp8 or quantize_fp8_tokens), or None: quantised within the call."""
    if stream is not None:
        with _current(stream, x):
            return apply_fp8(x, codes, scales, signs_bank, scales_bank, p, user_ids, y_dtype, xq, ws, None,
                             check)
    U = signs_bank.shape[0]
    idx, T, d_in, d_out = _apply_fp8_checks(x, codes, scales, signs_bank, scales_bank, p, U, user_ids, xq)
    y = x.new_empty((T, d_out), dtype=y_dtype)
    if ws is None:
        ws = workspace(bd_apply_fp8_workspace_bytes(p, T, U, d_out, d_in, _dtype_code(x), _dtype_code(y)),
                       x.device)
    else:
        _dev(ws, "workspace", None, None, x.device)
    _check(_apply_fp8(x, idx, T, d_in, d_out, xq, codes, scales, signs_bank, scales_bank, p, U, user_ids, y,
                      ws, stream), "bd_apply_fp8")
    if check:
        _check(bd_device_status(ws, stream), "bd_apply_fp8 (device)")
    return y


def select_axis(w_fine: torch.Tensor, w_base: Optional[torch.Tensor], clip_k: float = 0.0,
                ws=None, stream=None, check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Returns (errors float64[2] = {ROW, COL}, axis int32[1]) on the device."""
    d_out, d_in = w_fine.shape
    dev = w_fine.device
    errors = torch.empty(2, dtype=torch.float64, device=dev)
    axis = torch.empty(1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(bd_select_axis_workspace_bytes(d_out, d_in, clip_k), dev)
    _check(bd_select_axis(w_fine, w_base, clip_k, errors, axis, ws, stream), "bd_select_axis")
    if check:
        _check(bd_device_status(ws, stream), "bd_select_axis (device)")
    return errors, axis


def reconstruct(signs, scales, p, d_out, d_in, w_base=None, out_dtype=torch.float32, stream=None):
    out = torch.empty((d_out, d_in), dtype=out_dtype, device=signs.device)
    _check(bd_reconstruct(signs, scales, p, d_out, d_in, w_base, out, stream), "bd_reconstruct")
    return out


def apply(x: torch.Tensor, w_base: torch.Tensor, signs_bank: torch.Tensor,
          scales_bank: torch.Tensor, p: bd_compress_params, user_ids: torch.Tensor,
          y: Optional[torch.Tensor] = None, y_dtype=torch.float32, ws=None, stream=None,
          check: bool = False) -> torch.Tensor:
    T, d_in = x.shape
    d_out = w_base.shape[0]
    n_users = signs_bank.shape[0]
    if y is None:
        y = torch.empty((T, d_out), dtype=y_dtype, device=x.device)
    if ws is None:
        ws = workspace(bd_apply_workspace_bytes(p, T, n_users, d_out, d_in, _dtype_code(x),
                                                _dtype_code(y)), x.device)
    _check(bd_apply(x, w_base, signs_bank, scales_bank, p, n_users, user_ids, y, ws, stream),
           "bd_apply")
    if check:
        _check(bd_device_status(ws, stream), "bd_apply (device)")
    return y
