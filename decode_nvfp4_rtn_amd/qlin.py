"""Thin Python binding over libqlin.so (include/qlin.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libqlin.so.  torch supplies device memory and the current stream.
Importing this module loads the library and raises ImportError when it has
not been built (``python -m decode_nvfp4_rtn_amd.build``); there is no
fallback implementation.

Function names match the C entry points.  Tensors must be contiguous and on
the GPU; outputs are allocated with torch unless passed in.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlin.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m decode_nvfp4_rtn_amd.build`")
_lib = ctypes.CDLL(LIB_PATH)

QL_OK, QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE, QL_EWORKSPACE, QL_EHIP, QL_EFORMAT = range(8)
QL_F32, QL_BF16 = 0, 1
QL_NVFP4, QL_INT4_G128, QL_LUT2, QL_INT4_SP24 = 0, 1, 2, 3
QL_STATIC_SCALE = 1
QL_KV_BF16, QL_KV_E4M3, QL_KV_NVFP4 = 0, 1, 2
QL_ROPE_INTERLEAVED = 1
QL_ROUTE_RENORMALIZE = 1
QL_ROWS_GATHER, QL_ROWS_SILU_MUL = 1, 2

_vp, _i64, _sz, _int, _uint = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint

_SIGS = {
    "ql_status_str": (ctypes.c_char_p, [_int]),
    "ql_version": (_int, []),
    "quantize_nvfp4_workspace": (_sz, [_i64, _i64]),
    "quantize_nvfp4": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _uint, _vp, _sz, _vp]),
    "quantize_nvfp4_noalloc": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _uint, _vp]),
    "quantize_int4_g128": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "quantize_int4_g128_sp24": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "fit_lut2_workspace": (_sz, [_i64, _i64]),
    "fit_lut2": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "repack_weights_bytes": (_sz, [_int, _i64, _i64]),
    "repack_weights": (_int, [_int, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "gemm_w4a4": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "gemm_w4a4_workspace": (_sz, [_i64, _i64, _i64]),
    "gemm_w4a4_ws": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _sz, _vp]),
    "gemm_w4a16": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "gemm_lut2": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "gemm_w4a16_workspace": (_sz, [_i64, _i64, _i64]),
    "gemm_lut2_workspace": (_sz, [_i64, _i64, _i64]),
    "gemm_w4a16_ws": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _sz, _vp]),
    "gemm_lut2_ws": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _sz, _vp]),
    "gemm_w4a16_sp24": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "gemm_w4a16_sp24_workspace": (_sz, [_i64, _i64, _i64]),
    "quantize_gemm_w4a4_workspace": (_sz, [_i64, _i64]),
    "quantize_gemm_w4a4": (_int, [_vp, _i64, _i64, _vp, _uint, _vp, _i64, _vp, _int, _vp, _sz,
                                  _vp]),
    "gemm_w4a16_sp24_ws": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _sz, _vp]),
    "kv_cache_bytes": (_sz, [_int, _i64, _i64, _i64, _i64]),
    "kv_append": (_int, [_vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _vp]),
    "kv_gather": (_int, [_vp, _vp, _i64, _vp, _vp, _int, _vp]),
    "qkv_norm_rope_append": (_int, [_vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, ctypes.c_float,
                                    _vp, _vp, _i64, _i64, _uint, _vp, _vp, _vp]),
    "kv_attention_workspace": (_sz, [_vp, _i64, _i64, _i64, _i64, _i64]),
    "kv_attention": (_int, [_vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _i64,
                            _i64, _vp, ctypes.c_float, _vp, _vp, _sz, _vp]),
    "kv_commit": (_int, [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _vp]),
    "group_rows_workspace": (_sz, [_i64, _i64]),
    "group_rows": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_workspace": (_sz, [_i64, _i64, _i64]),
    "moe_route": (_int, [_vp, _int, _i64, _i64, _i64, _i64, _uint, _vp, _vp, _vp, _vp, _vp, _vp,
                         _sz, _vp]),
    "moe_gemm_w4a16": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _uint, _vp,
                              _int, _vp]),
    "moe_gemm_w4a4": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64,
                             _uint, _vp, _int, _vp]),
    "moe_combine": (_int, [_vp, _int, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "lora_add_workspace": (_sz, [_i64, _i64, _i64, _i64]),
    "lora_add": (_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64,
                        _vp, _i64, _int, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class QlinError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {_lib.ql_status_str(status).decode()} (status {status})")


def _check(fn, status):
    if status != QL_OK:
        raise QlinError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _bytes(t, name, nbytes, dtype=None):
    """t is a contiguous GPU tensor (of dtype, if given) of at least nbytes bytes."""
    _dev(t, name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes; the call needs {nbytes}")
    return t


def _matrix(t, name, dtype):
    _dev(t, name)
    if t.dtype != dtype or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    return t.shape


def ql_status_str(status):
    return _lib.ql_status_str(status).decode()


def ql_version():
    return _lib.ql_version()


def quantize_nvfp4_workspace(rows, cols):
    return _lib.quantize_nvfp4_workspace(rows, cols)


def quantize_nvfp4(x, tensor_scale=None, codes=None, scales=None, workspace=None, stream=None,
                   ts_out=None):
    """NVFP4 round-to-nearest quantization of x [rows, cols] (fp32 or bf16).

    tensor_scale: None computes s_t from max|x| (written to ts_out, a 1-element
    fp32 GPU tensor, allocated when not given); a 1-element fp32 GPU tensor
    holding a calibrated s_t is used as is (QL_STATIC_SCALE).
    Returns (codes uint8 [rows, cols/2], scales uint8 [rows, cols/16], s_t fp32 [1]).
    """
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {x.dim()}-D")
    rows, cols = x.shape
    dt = {torch.float32: QL_F32, torch.bfloat16: QL_BF16}.get(x.dtype)
    if dt is None:
        raise ValueError("x must be float32 or bfloat16")
    dev = x.device
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    _bytes(codes, "codes", rows * (cols // 2), torch.uint8)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    _bytes(scales, "scales", rows * (cols // 16), torch.uint8)
    flags = 0
    if tensor_scale is None:
        ts = ts_out if ts_out is not None else torch.empty(1, dtype=torch.float32, device=dev)
        _bytes(ts, "ts_out", 4, torch.float32)
    else:
        ts = _bytes(tensor_scale, "tensor_scale", 4, torch.float32)
        flags = QL_STATIC_SCALE
    wsb = _lib.quantize_nvfp4_workspace(rows, cols)
    if workspace is None and not flags:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _bytes(workspace, "workspace", 0, torch.uint8)
    _check("quantize_nvfp4", _lib.quantize_nvfp4(
        _ptr(x), dt, rows, cols, _ptr(codes), _ptr(scales), _ptr(ts), flags,
        _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream)))
    return codes, scales, ts


def quantize_nvfp4_noalloc(x, codes, scales, tensor_scale, static_scale=False, stream=None):
    """quantize_nvfp4 without a workspace (the library keeps the partial maxima
    in a per-GPU array), for callers that cannot allocate: every output is the
    caller's.  tensor_scale (1-element fp32 GPU tensor) receives s_t, or holds
    a calibrated s_t when static_scale.  Calls that may overlap on one GPU
    (different streams without ordering) race on that array.
    Returns (codes, scales, tensor_scale)."""
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {x.dim()}-D")
    rows, cols = x.shape
    dt = {torch.float32: QL_F32, torch.bfloat16: QL_BF16}.get(x.dtype)
    if dt is None:
        raise ValueError("x must be float32 or bfloat16")
    _bytes(codes, "codes", rows * (cols // 2), torch.uint8)
    _bytes(scales, "scales", rows * (cols // 16), torch.uint8)
    _bytes(tensor_scale, "tensor_scale", 4, torch.float32)
    _check("quantize_nvfp4_noalloc", _lib.quantize_nvfp4_noalloc(
        _ptr(x), dt, rows, cols, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
        QL_STATIC_SCALE if static_scale else 0, _stream(stream)))
    return codes, scales, tensor_scale


def quantize_int4_g128(w, codes=None, scales=None, stream=None, sparse24=False):
    """Symmetric INT4 group-128 quantization of fp32 weights [n, k]; with
    sparse24, 2:4 magnitude pruning along k first (quantize_int4_g128_sp24).
    Returns (codes uint8 [n, k/2], scales int16 (bf16 bits) [n, k/128])."""
    n, k = _matrix(w, "w", torch.float32)
    if codes is None:
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    _bytes(codes, "codes", n * (k // 2), torch.uint8)
    if scales is None:
        scales = torch.empty((n, k // 128), dtype=torch.int16, device=w.device)
    _bytes(scales, "scales", n * (k // 128) * 2)
    name = "quantize_int4_g128_sp24" if sparse24 else "quantize_int4_g128"
    _check(name, getattr(_lib, name)(_ptr(w), n, k, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def fit_lut2_workspace(n, k):
    return _lib.fit_lut2_workspace(n, k)


def fit_lut2(w, idx=None, centroids=None, workspace=None, stream=None):
    """2-bit codebook fit of fp32 weights [n, k] (10 Lloyd iterations per row).
    Returns (idx uint8 [n, k/4], centroids int16 (bf16 bits) [n, 4])."""
    n, k = _matrix(w, "w", torch.float32)
    if idx is None:
        idx = torch.empty((n, k // 4), dtype=torch.uint8, device=w.device)
    _bytes(idx, "idx", n * (k // 4), torch.uint8)
    if centroids is None:
        centroids = torch.empty((n, 4), dtype=torch.int16, device=w.device)
    _bytes(centroids, "centroids", n * 8)
    wsb = _lib.fit_lut2_workspace(n, k)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=w.device)
    _bytes(workspace, "workspace", 0, torch.uint8)
    _check("fit_lut2", _lib.fit_lut2(_ptr(w), n, k, _ptr(idx), _ptr(centroids), _ptr(workspace),
                                     workspace.numel(), _stream(stream)))
    return idx, centroids


# Bytes of the canonical (codes, scales or codebook) inputs of repack_weights.
_CANONICAL_BYTES = {
    QL_NVFP4: lambda n, k: (n * (k // 2), n * (k // 16)),
    QL_INT4_G128: lambda n, k: (n * (k // 2), n * (k // 128) * 2),
    QL_INT4_SP24: lambda n, k: (n * (k // 2), n * (k // 128) * 2),
    QL_LUT2: lambda n, k: (n * (k // 4), n * 8),
}


def repack_weights_bytes(fmt, n, k):
    return _lib.repack_weights_bytes(fmt, n, k)


def repack_weights(fmt, n, k, codes, scales_or_lut, tensor_scale=None, packed=None, stream=None):
    """Repack canonical quantized weights into the kernel operand order.
    Returns the packed blob (uint8 GPU tensor)."""
    if fmt not in _CANONICAL_BYTES:
        raise ValueError(f"unknown weight format {fmt}")
    code_bytes, aux_bytes = _CANONICAL_BYTES[fmt](n, k)
    _bytes(codes, "codes", code_bytes, torch.uint8)
    _bytes(scales_or_lut, "scales_or_lut", aux_bytes)
    if fmt == QL_NVFP4:
        if tensor_scale is None:
            raise ValueError("an NVFP4 blob needs the weights' tensor_scale")
        _bytes(tensor_scale, "tensor_scale", 4, torch.float32)
    nbytes = _lib.repack_weights_bytes(fmt, n, k)
    if packed is None:
        packed = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    _bytes(packed, "packed", nbytes, torch.uint8)
    _check("repack_weights", _lib.repack_weights(
        fmt, n, k, _ptr(codes), _ptr(scales_or_lut), _ptr(tensor_scale), _ptr(packed),
        packed.numel(), _stream(stream)))
    return packed


def _out(y, m, n, dtype, dev):
    if y is None:
        y = torch.empty((m, n), dtype=dtype, device=dev)
    else:
        _dev(y, "y")
        if tuple(y.shape) != (m, n):
            raise ValueError(f"y must be [{m}, {n}], got {list(y.shape)}")
    dt = {torch.float32: QL_F32, torch.bfloat16: QL_BF16}.get(y.dtype)
    if dt is None:
        raise ValueError("y must be float32 or bfloat16")
    return y, dt


# Host-side shape and size checks (no device access, no synchronisation).
# Every buffer a kernel reads or writes must be at least as large as the call
# says; in particular a packed blob must hold repack_weights_bytes(fmt, n, k)
# bytes, so no kernel reads past it whatever its contents.

def _typed(t, name, dtype):
    _dev(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _rows(t, name, dtype, m, cols):
    _typed(t, name, dtype)
    if t.dim() != 2 or t.shape[1] != cols or t.shape[0] < m:
        raise ValueError(f"{name} must be [>= {m}, {cols}], got {list(t.shape)}")


def _blob(w_packed, fmt, n, k):
    _typed(w_packed, "w_packed", torch.uint8)
    need = _lib.repack_weights_bytes(fmt, n, k)
    if w_packed.numel() < need:
        raise ValueError(f"w_packed holds {w_packed.numel()} bytes; a format-{fmt} blob "
                         f"of [{n}, {k}] takes {need}")


def gemm_w4a4_workspace(m, n, k):
    return _lib.gemm_w4a4_workspace(m, n, k)


def gemm_w4a4(a_codes, a_scales, a_tensor_scale, w_packed, m, n, k, y=None,
              out_dtype=torch.float32, stream=None, workspace=None):
    """NVFP4 W4A4 prefill GEMM: Y [m, n] = dequant(A) dequant(W)^T.

    workspace: None calls gemm_w4a4 (no k split of the last round of tiles);
    a uint8 GPU tensor of at least gemm_w4a4_workspace(m, n, k) bytes calls
    gemm_w4a4_ws with it."""
    _rows(a_codes, "a_codes", torch.uint8, m, k // 2)
    _rows(a_scales, "a_scales", torch.uint8, m, k // 16)
    _typed(a_tensor_scale, "a_tensor_scale", torch.float32)
    if a_tensor_scale.numel() < 1:
        raise ValueError("a_tensor_scale must hold one value")
    _blob(w_packed, QL_NVFP4, n, k)
    y, dt = _out(y, m, n, out_dtype, a_codes.device)
    if workspace is not None:
        _typed(workspace, "workspace", torch.uint8)
    if workspace is None:
        _check("gemm_w4a4", _lib.gemm_w4a4(
            _ptr(a_codes), _ptr(a_scales), _ptr(a_tensor_scale), _ptr(w_packed), m, n, k,
            _ptr(y), dt, _stream(stream)))
    else:
        _check("gemm_w4a4_ws", _lib.gemm_w4a4_ws(
            _ptr(a_codes), _ptr(a_scales), _ptr(a_tensor_scale), _ptr(w_packed), m, n, k,
            _ptr(y), dt, _ptr(workspace), workspace.numel(), _stream(stream)))
    return y


def quantize_gemm_w4a4_workspace(m, k):
    return _lib.quantize_gemm_w4a4_workspace(m, k)


def quantize_gemm_w4a4(x, w_packed, n, y=None, out_dtype=torch.float32, tensor_scale=None,
                       ts_out=None, workspace=None, stream=None):
    """quantize_nvfp4(x) then gemm_w4a4 in one call whose GEMM quantizes the
    activation tiles as it loads them (x: bf16 [m, k]).

    tensor_scale: None computes s_t (written to ts_out, allocated when not
    given); a 1-element fp32 GPU tensor holding a calibrated s_t is used as is
    (QL_STATIC_SCALE: one launch).  workspace: the amax pass's partial maxima
    (quantize_gemm_w4a4_workspace(m, k) bytes), allocated when not given.
    Returns (y, s_t)."""
    _typed(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {x.dim()}-D")
    m, k = x.shape
    _blob(w_packed, QL_NVFP4, n, k)
    y, dt = _out(y, m, n, out_dtype, x.device)
    flags = 0
    if tensor_scale is None:
        ts = ts_out if ts_out is not None else torch.empty(1, dtype=torch.float32, device=x.device)
        _bytes(ts, "ts_out", 4, torch.float32)
        if workspace is None:
            workspace = torch.empty(max(16, _lib.quantize_gemm_w4a4_workspace(m, k)),
                                    dtype=torch.uint8, device=x.device)
    else:
        ts = _bytes(tensor_scale, "tensor_scale", 4, torch.float32)
        flags = QL_STATIC_SCALE
    if workspace is not None:
        _typed(workspace, "workspace", torch.uint8)
    _check("quantize_gemm_w4a4", _lib.quantize_gemm_w4a4(
        _ptr(x), m, k, _ptr(ts), flags, _ptr(w_packed), n, _ptr(y), dt, _ptr(workspace),
        0 if workspace is None else workspace.numel(), _stream(stream)))
    return y, ts


def gemm_w4a16_workspace(m, n, k):
    return _lib.gemm_w4a16_workspace(m, n, k)


def gemm_lut2_workspace(m, n, k):
    return _lib.gemm_lut2_workspace(m, n, k)


def gemm_w4a16_sp24_workspace(m, n, k):
    return _lib.gemm_w4a16_sp24_workspace(m, n, k)


def _decode(name, fmt, x, w_packed, n, k, y, out_dtype, stream, workspace):
    m = x.shape[0] if x.dim() == 2 else -1
    _rows(x, "x", torch.bfloat16, m, k)
    _blob(w_packed, fmt, n, k)
    y, dt = _out(y, m, n, out_dtype, x.device)
    if workspace is None:
        _check(name, getattr(_lib, name)(_ptr(x), _ptr(w_packed), m, n, k, _ptr(y), dt,
                                         _stream(stream)))
    else:
        _typed(workspace, "workspace", torch.uint8)
        _check(name + "_ws", getattr(_lib, name + "_ws")(
            _ptr(x), _ptr(w_packed), m, n, k, _ptr(y), dt, _ptr(workspace), workspace.numel(),
            _stream(stream)))
    return y


def gemm_w4a16(x, w_packed, n, k, y=None, out_dtype=torch.bfloat16, stream=None, workspace=None):
    """W4A16 decode GEMM: Y [m, n] = X bf16 [m, k] times INT4-g128 weights^T.

    workspace: None calls gemm_w4a16; a uint8 GPU tensor of at least
    gemm_w4a16_workspace(m, n, k) bytes calls gemm_w4a16_ws with it (k split
    over blocks for shapes with long k or few row tiles)."""
    return _decode("gemm_w4a16", QL_INT4_G128, x, w_packed, n, k, y, out_dtype, stream, workspace)


def gemm_lut2(x, w_packed, n, k, y=None, out_dtype=torch.bfloat16, stream=None, workspace=None):
    """LUT2 decode GEMM: Y [m, n] = X bf16 [m, k] times codebook weights^T.

    workspace: as gemm_w4a16 (gemm_lut2_workspace / gemm_lut2_ws)."""
    return _decode("gemm_lut2", QL_LUT2, x, w_packed, n, k, y, out_dtype, stream, workspace)


def gemm_w4a16_sp24(x, w_packed, n, k, y=None, out_dtype=torch.bfloat16, stream=None,
                    workspace=None):
    """2:4 sparse W4A16 decode GEMM: Y [m, n] = X bf16 [m, k] times 2:4 INT4 weights^T.

    workspace: as gemm_w4a16 (gemm_w4a16_sp24_workspace / gemm_w4a16_sp24_ws)."""
    return _decode("gemm_w4a16_sp24", QL_INT4_SP24, x, w_packed, n, k, y, out_dtype, stream,
                   workspace)


# ---------------------------------------------------------------------------
# Paged key/value cache (include/qlin.h describes formats and layout)
# ---------------------------------------------------------------------------

class _KVStruct(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", _i64), ("data", _vp), ("bytes", _sz)]


def kv_cache_bytes(fmt, n_pages, page_size, n_kv, head_dim):
    """Bytes of a cache; 0 for sizes or a format that are not supported."""
    return _lib.kv_cache_bytes(fmt, n_pages, page_size, n_kv, head_dim)


class KVCache:
    """One layer's paged cache of keys and values: a uint8 GPU tensor ``data``
    and what it holds.  fmt: QL_KV_BF16, QL_KV_E4M3 or QL_KV_NVFP4; page_size a
    power of two of 16..4096; head_dim 64, 128 or 256.  ``data`` is allocated
    when not given and needs no initialisation.  The calls take its address as
    it is here: the attributes cannot be assigned again."""

    def __init__(self, fmt, n_pages, page_size, n_kv, head_dim, data=None, device=None):
        nbytes = _lib.kv_cache_bytes(fmt, n_pages, page_size, n_kv, head_dim)
        if nbytes == 0:
            raise ValueError(f"no cache of format {fmt}: {n_pages} pages of {page_size} tokens, "
                             f"{n_kv} heads of {head_dim}")
        if data is None:
            data = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
        _bytes(data, "data", nbytes, torch.uint8)
        struct = _KVStruct(fmt, n_kv, head_dim, page_size, n_pages, data.data_ptr(), data.numel())
        self.__dict__.update(fmt=fmt, n_pages=n_pages, page_size=page_size, n_kv=n_kv,
                             head_dim=head_dim, data=data, device=data.device, _struct=struct,
                             _ref=ctypes.byref(struct))

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"KVCache.{name} is fixed: make another KVCache")
        super().__setattr__(name, value)


# The calls below are a few microseconds of GPU work each at decode sizes, so
# their Python side is kept short: integers for pointers, no per-call stream
# object (torch.cuda.current_stream() alone takes 2.8 us).

_XDT = {torch.float32: QL_F32, torch.bfloat16: QL_BF16}


def _queue(stream, dev):
    """Address of the stream a call on `dev` goes to."""
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _vector(t, name, dtype, dev, count):
    """Address of t, a contiguous [count] tensor of dtype on dev."""
    if t.device != dev or t.dtype != dtype or t.shape != (count,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{count}] tensor on {dev}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _heads(t, name, dev, heads, d):
    """Token stride of t [tokens, heads, d] on dev, a token's heads contiguous."""
    shape = t.shape
    if t.device != dev or len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be [tokens, {heads}, {d}] on {dev}, got {list(shape)} on "
                         f"{t.device}")
    if shape[0] == 0:
        return heads * d
    a, b, c = t.stride()
    if c != 1 or (heads > 1 and b != d):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return a if shape[0] > 1 else heads * d


def _new(shape, dtype, dev, stream):
    """A buffer for a call on `stream`: memory of that stream's own pool, so
    that work queued elsewhere on what the memory held before cannot meet it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _rows_out(t, name, shape, dtypes, dev):
    if t.device != dev or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor on {dev} of "
                         f"{' or '.join(map(str, dtypes))}, got {t.dtype} {list(t.shape)} on "
                         f"{t.device}")
    return t


def _table(t, dev, n_seqs):
    """Row stride and columns of a block table."""
    if t.device != dev or t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != n_seqs:
        raise ValueError(f"block_table must be an int32 [{n_seqs}, pages] tensor on {dev}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    rows, cols = t.stride()
    if t.shape[1] > 1 and cols != 1:
        raise ValueError("block_table: a sequence's row must be contiguous")
    return (rows if n_seqs > 1 else t.shape[1]), t.shape[1]


def _seqs(cu_q):
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be an int32 [n_seqs + 1] tensor")
    return cu_q.shape[0] - 1


def kv_append(cache, k, v, slots, stream=None):
    """Write k, v [tokens, n_kv, head_dim] (fp32 or bf16; slices of a fused qkv
    tensor will do) to their slots (int64 [tokens]; negative: skipped)."""
    dev = cache.device
    ks = _heads(k, "k", dev, cache.n_kv, cache.head_dim)
    vs = _heads(v, "v", dev, cache.n_kv, cache.head_dim)
    tokens = k.shape[0]
    dt = _XDT.get(k.dtype)
    if dt is None or v.dtype != k.dtype or v.shape[0] != tokens:
        raise ValueError("k and v must be float32 or bfloat16, of one type and length")
    at = _vector(slots, "slots", torch.int64, dev, tokens)
    st = _lib.kv_append(cache._ref, k.data_ptr(), v.data_ptr(), dt, tokens, ks, vs, at,
                        _queue(stream, dev))
    if st:
        raise QlinError("kv_append", st)


def kv_gather(cache, slots, k=None, v=None, out_dtype=torch.bfloat16, stream=None):
    """Read rows back: (k, v) [tokens, n_kv, head_dim] in out_dtype (fp32 or
    bf16); a slot outside the cache gives zeros."""
    dev = cache.device
    tokens = slots.shape[0] if slots.dim() == 1 else -1
    at = _vector(slots, "slots", torch.int64, dev, tokens)
    shape = (tokens, cache.n_kv, cache.head_dim)
    k = _new(shape, out_dtype, dev, stream) if k is None else _rows_out(k, "k", shape, _XDT, dev)
    if v is not None:
        _rows_out(v, "v", shape, _XDT, dev)
    else:       # the quicker of the two calls (1.2 us, and 1.7)
        v = torch.empty_like(k) if stream is None else _new(shape, k.dtype, dev, stream)
    dt = _XDT.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise ValueError("k and v must be float32 or bfloat16, of one type")
    st = _lib.kv_gather(cache._ref, at, tokens, k.data_ptr(), v.data_ptr(), dt,
                        _queue(stream, dev))
    if st:
        raise QlinError("kv_gather", st)
    return k, v


def qkv_norm_rope_append(cache, qkv, n_q, slots, positions=None, rope=None, q_weight=None,
                         k_weight=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """From a fused projection qkv [tokens, (n_q + 2 n_kv) * head_dim] (fp32 or
    bf16): RMS norm of each query and key head (weights fp32 [head_dim], None:
    no norm), rotation by the tokens' positions (rope fp32 [max_pos, rot]:
    cosines, then sines, of rot / 2 pairs; None: no rotation; pairs (i, i +
    rot / 2), or (2 i, 2 i + 1) if interleaved), and K and V written to slots
    (int64 [tokens]; negative: skipped).  Returns the queries, bf16
    [tokens, n_q, head_dim]."""
    dev, d = cache.device, cache.head_dim
    width = (n_q + 2 * cache.n_kv) * d
    dt = _XDT.get(qkv.dtype)
    if dt is None or qkv.device != dev or qkv.dim() != 2 or qkv.shape[1] != width:
        raise ValueError(f"qkv must be a float32 or bfloat16 [tokens, {width}] tensor on {dev}, "
                         f"got {qkv.dtype} {list(qkv.shape)} on {qkv.device}")
    tokens = qkv.shape[0]
    stride, inner = qkv.stride()
    if tokens and inner != 1:
        raise ValueError("qkv: a token's row must be contiguous")
    slot_at = _vector(slots, "slots", torch.int64, dev, tokens)
    max_pos = rot = 0
    pos_at = rope_at = None
    if rope is not None:
        if (rope.device != dev or rope.dtype != torch.float32 or rope.dim() != 2
                or not rope.is_contiguous()):
            raise ValueError(f"rope must be a contiguous float32 [max_pos, rot] tensor on {dev}")
        if positions is None:
            raise ValueError("a rotation needs positions")
        max_pos, rot = rope.shape
        rope_at = rope.data_ptr()
        pos_at = _vector(positions, "positions", torch.int32, dev, tokens)
    qw = None if q_weight is None else _vector(q_weight, "q_weight", torch.float32, dev, d)
    kw = None if k_weight is None else _vector(k_weight, "k_weight", torch.float32, dev, d)
    shape = (tokens, n_q, d)
    if q_out is None:
        q_out = _new(shape, torch.bfloat16, dev, stream)
    else:
        _rows_out(q_out, "q_out", shape, (torch.bfloat16,), dev)
    st = _lib.qkv_norm_rope_append(
        cache._ref, qkv.data_ptr(), dt, tokens, stride if tokens > 1 else width, n_q, qw, kw, eps,
        pos_at, rope_at, max_pos, rot, QL_ROPE_INTERLEAVED if interleaved else 0,
        q_out.data_ptr(), slot_at, _queue(stream, dev))
    if st:
        raise QlinError("qkv_norm_rope_append", st)
    return q_out


def kv_attention_workspace(cache, tokens, n_q, n_seqs, max_q, max_kv):
    return _lib.kv_attention_workspace(cache._ref, tokens, n_q, n_seqs, max_q, max_kv)


def kv_attention(cache, q, cu_q, kv_lens, block_table, max_q, max_kv, tree=None, scale=None,
                 y=None, workspace=None, stream=None):
    """Attention of each sequence's newest tokens over its cached context and
    themselves.

    q bf16 [tokens, n_q, head_dim], the sequences' tokens one after another;
    cu_q int32 [n_seqs + 1] where each starts; kv_lens int32 [n_seqs] the keys
    of each, the new tokens' own included (append them first); block_table
    int32 [n_seqs, pages].  tree: int64 [tokens], bit j of token i's set where
    it sees new token j of its sequence (at most 64); None: a causal chain, and
    with one token ordinary decoding.  max_q: at least every sequence's new
    tokens; max_kv: about the largest length.  scale: head_dim ** -0.5 when not
    given.  workspace: uint8 of kv_attention_workspace(...) bytes, allocated
    when not given.  Returns y bf16 [tokens, n_q, head_dim]."""
    dev, d = cache.device, cache.head_dim
    n_q = q.shape[1] if q.dim() == 3 else -1
    stride = _heads(q, "q", dev, n_q, d)
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16")
    tokens, n_seqs = q.shape[0], _seqs(cu_q)
    cu_at = _vector(cu_q, "cu_q", torch.int32, dev, n_seqs + 1)
    lens_at = _vector(kv_lens, "kv_lens", torch.int32, dev, n_seqs)
    tstride, cols = _table(block_table, dev, n_seqs)
    tree_at = None if tree is None else _vector(tree, "tree", torch.int64, dev, tokens)
    shape = (tokens, n_q, d)
    if y is None:
        y = _new(shape, torch.bfloat16, dev, stream)
    else:
        _rows_out(y, "y", shape, (torch.bfloat16,), dev)
    ws_at, have = None, 0
    if workspace is None:
        have = _lib.kv_attention_workspace(cache._ref, tokens, n_q, n_seqs, max_q, max_kv)
        if have:
            workspace = _new((have,), torch.uint8, dev, stream)
            ws_at = workspace.data_ptr()
    else:
        _bytes(workspace, "workspace", 0, torch.uint8)
        ws_at, have = workspace.data_ptr(), workspace.numel()
    st = _lib.kv_attention(
        cache._ref, q.data_ptr(), stride, tokens, n_q, n_seqs, cu_at, lens_at,
        block_table.data_ptr(), tstride, cols, max_q, max_kv, tree_at,
        d ** -0.5 if scale is None else scale, y.data_ptr(), ws_at, have, _queue(stream, dev))
    if st:
        raise QlinError("kv_attention", st)
    return y


def kv_commit(cache, cu_q, kv_lens, block_table, path, stream=None):
    """Move the rows of each sequence's accepted drafts right behind its
    context: path int32 [n_seqs, max_path <= 64], accepted draft indices, root
    first, padded with -1; cu_q, kv_lens and block_table as the verification's
    kv_attention call."""
    dev, n_seqs = cache.device, _seqs(cu_q)
    cu_at = _vector(cu_q, "cu_q", torch.int32, dev, n_seqs + 1)
    lens_at = _vector(kv_lens, "kv_lens", torch.int32, dev, n_seqs)
    tstride, cols = _table(block_table, dev, n_seqs)
    if (path.device != dev or path.dtype != torch.int32 or path.dim() != 2
            or path.shape[0] != n_seqs or not path.is_contiguous()):
        raise ValueError(f"path must be a contiguous int32 [{n_seqs}, max_path] tensor on {dev}, "
                         f"got {path.dtype} {list(path.shape)} on {path.device}")
    st = _lib.kv_commit(cache._ref, n_seqs, cu_at, lens_at, block_table.data_ptr(), tstride, cols,
                        path.data_ptr(), path.shape[1], _queue(stream, dev))
    if st:
        raise QlinError("kv_commit", st)


# ---------------------------------------------------------------------------
# Rows that choose their own weights: experts and adapters
# ---------------------------------------------------------------------------

class RowPlan:
    """The rows of a batch in the order of the weights they meet, as
    ``group_rows`` or ``moe_route`` makes it: int32 tensors ``order`` [rows] (the
    row at each place), ``where`` [tokens, top_k] (each row's place) and
    ``offsets`` [groups + 1] (where each group's run begins; rows of no group
    from offsets[groups] on).  ``tokens`` rows of ``top_k`` choices each.  The
    three are views of one allocation, made when asked for."""

    __slots__ = ("groups", "tokens", "top_k", "device", "_data", "_order", "_where", "_offsets")

    def __init__(self, groups, tokens, top_k, dev, stream=None):
        self.groups, self.tokens, self.top_k, self.device = groups, tokens, top_k, dev
        rows = tokens * top_k
        self._data = _new((2 * rows + groups + 1,), torch.int32, dev, stream)
        at = self._data.data_ptr()
        self._order, self._where, self._offsets = at, at + 4 * rows, at + 8 * rows

    @property
    def order(self):
        return self._data.as_strided((self.tokens * self.top_k,), (1,), 0)

    @property
    def where(self):
        return self._data.as_strided((self.tokens, self.top_k), (self.top_k, 1), self.tokens * self.top_k)

    @property
    def offsets(self):
        return self._data.as_strided((self.groups + 1,), (1,), 2 * self.tokens * self.top_k)


def _call(name, dev, *args):
    """An entry point's call with `dev` current: launches and launch plans go by
    the current device."""
    if torch._C._cuda_getDevice() == dev.index:
        st = getattr(_lib, name)(*args)
    else:
        with torch.cuda.device(dev):
            st = getattr(_lib, name)(*args)
    if st:
        raise QlinError(name, st)


def _whole(x, name):
    """x as an integer, or a refusal (a bool or a float is no count)."""
    if isinstance(x, bool) or not hasattr(x, "__index__"):
        raise ValueError(f"{name} must be a whole number, got {x!r}")
    return x.__index__()


def _workspace(workspace, need, dev, stream):
    """(address, bytes, what keeps it alive) of a call's workspace."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _new((need,), torch.uint8, dev, stream)
    elif workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    else:
        _bytes(workspace, "workspace", 0, torch.uint8)
    return workspace.data_ptr(), workspace.numel(), workspace


def _for_plan(plan, groups, tokens, top_k, dev, stream):
    if plan is None:
        return RowPlan(groups, tokens, top_k, dev, stream)
    if (plan.groups, plan.tokens, plan.top_k, plan.device) != (groups, tokens, top_k, dev):
        raise ValueError(f"plan is of {plan.tokens} x {plan.top_k} rows and {plan.groups} groups on "
                         f"{plan.device}; the call needs {tokens} x {top_k}, {groups}, {dev}")
    return plan


def group_rows(ids, groups, plan=None, workspace=None, stream=None):
    """The plan of given choices: ids int32 [rows] or [tokens, top_k], each the
    row's group (an adapter, an expert) or, outside of 0 .. groups - 1, none.
    plan: one of the same sizes to write (allocated when not given); workspace:
    uint8 of group_rows_workspace(rows, groups) bytes, allocated when not given."""
    if not ids.is_cuda or ids.dtype != torch.int32 or ids.dim() not in (1, 2) or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous int32 [rows] or [tokens, top_k] GPU tensor, got "
                         f"{ids.dtype} {list(ids.shape)} on {ids.device}")
    dev, groups = ids.device, _whole(groups, "groups")
    tokens, top_k = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
    if not 1 <= groups <= 1024 or not 1 <= top_k <= 64:
        raise ValueError(f"1 .. 1024 groups and 1 .. 64 choices to a token, got {groups} and {top_k}")
    plan = _for_plan(plan, groups, tokens, top_k, dev, stream)
    rows = tokens * top_k
    at, have, keep = _workspace(workspace, _lib.group_rows_workspace(rows, groups), dev, stream)
    _call("group_rows", dev, ids.data_ptr(), rows, groups, plan._order, plan._where,
          plan._offsets, at, have, _queue(stream, dev))
    return plan


def group_rows_workspace(rows, groups):
    return _lib.group_rows_workspace(rows, groups)


def moe_route(logits, top_k, renormalize=True, ids=None, weights=None, plan=None, workspace=None,
              stream=None):
    """A router's choice: logits [tokens, experts] (fp32 or bf16; a row's experts
    contiguous) -> (ids int32 [tokens, top_k], weights fp32 [tokens, top_k],
    plan).  The top_k largest, of equal ones the lowest expert; softmax weights
    over the chosen experts, or over all if not renormalize.  An expert at
    -infinity or NaN is not chosen: its place holds -1 and weight 0.  ids,
    weights, plan and workspace (uint8 of moe_route_workspace(...) bytes) are
    allocated when not given."""
    dt = _XDT.get(logits.dtype)
    if dt is None or not logits.is_cuda or logits.dim() != 2:
        raise ValueError(f"logits must be a float32 or bfloat16 [tokens, experts] GPU tensor, got "
                         f"{logits.dtype} {list(logits.shape)} on {logits.device}")
    dev, top_k = logits.device, _whole(top_k, "top_k")
    tokens, experts = logits.shape
    stride, inner = logits.stride()
    if experts > 1 and inner != 1:
        raise ValueError("logits: a token's experts must be contiguous")
    if not 1 <= top_k <= min(64, experts) or experts > 1024:
        raise ValueError(f"top_k of 1 .. min(64, experts) and at most 1024 experts, got {top_k} of {experts}")
    plan = _for_plan(plan, experts, tokens, top_k, dev, stream)
    shape = (tokens, top_k)
    ids = _new(shape, torch.int32, dev, stream) if ids is None else _rows_out(ids, "ids", shape, (torch.int32,), dev)
    weights = (_new(shape, torch.float32, dev, stream) if weights is None
               else _rows_out(weights, "weights", shape, (torch.float32,), dev))
    at, have, keep = _workspace(workspace, _lib.moe_route_workspace(tokens, experts, top_k), dev, stream)
    _call("moe_route", dev, logits.data_ptr(), dt, tokens, experts, stride if tokens > 1 else experts, top_k,
          QL_ROUTE_RENORMALIZE if renormalize else 0, ids.data_ptr(), weights.data_ptr(),
          plan._order, plan._where, plan._offsets, at, have,
          _queue(stream, dev))
    return ids, weights, plan


def moe_route_workspace(tokens, experts, top_k):
    return _lib.moe_route_workspace(tokens, experts, top_k)


def _experts(experts, plan, fmt, n, k):
    """Bytes between the blobs of a stack uint8 [experts, bytes]."""
    if (experts.device != plan.device or experts.dtype != torch.uint8 or experts.dim() != 2
            or experts.shape[0] != plan.groups):
        raise ValueError(f"experts must be a uint8 [{plan.groups}, bytes] tensor on {plan.device}, got "
                         f"{experts.dtype} {list(experts.shape)} on {experts.device}")
    step, inner = experts.stride()
    if inner != 1:
        raise ValueError("experts: a blob's bytes must be contiguous")
    if experts.shape[1] < _lib.repack_weights_bytes(fmt, n, k):
        raise ValueError(f"experts hold {experts.shape[1]} bytes each; a format-{fmt} blob of [{n}, {k}] takes "
                         f"{_lib.repack_weights_bytes(fmt, n, k)}")
    return step if plan.groups > 1 else experts.shape[1] // 16 * 16


def _operand(t, name, dtype, rows, cols, dev):
    """Address of t, a contiguous [rows, cols] tensor of dtype on dev."""
    if t.device != dev or t.dtype != dtype or t.shape != (rows, cols) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{rows}, {cols}] tensor on {dev}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _product(plan, n, k, gather, silu_mul, y, out_dtype, stream):
    """(n, k, rows of x, flags, y, its type) of an experts' product."""
    n, k = _whole(n, "n"), _whole(k, "k")
    if n < 1 or k < 1:
        raise ValueError(f"an expert's weights are [n, k] of 1 or more, got [{n}, {k}]")
    pairs = plan.tokens * plan.top_k
    shape = (pairs, n // 2 if silu_mul else n)
    y = _new(shape, out_dtype, plan.device, stream) if y is None else _rows_out(y, "y", shape, _XDT, plan.device)
    dt = _XDT.get(y.dtype)
    if dt is None:
        raise ValueError("y must be float32 or bfloat16")
    flags = (QL_ROWS_GATHER if gather else 0) | (QL_ROWS_SILU_MUL if silu_mul else 0)
    return n, k, plan.tokens if gather else pairs, flags, y, dt


def moe_gemm_w4a16(x, experts, plan, n, k, gather=True, silu_mul=False, y=None,
                   out_dtype=torch.bfloat16, stream=None):
    """The plan's rows times their experts' INT4 weights: y [pairs, n] in the
    plan's order.

    x bf16: [tokens, k], the plan's tokens (gather), or [pairs, k] in the plan's
    order.  experts: uint8 [experts, bytes], an INT4 blob of [n, k] each
    (``repack_weights(..., packed=experts[e])``).  silu_mul: the weights' first
    n / 2 rows are a gate, and y [pairs, n / 2] = silu(gate) * up.  Rows of y
    whose pair has no expert are zero."""
    n, k, rows, flags, y, dt = _product(plan, n, k, gather, silu_mul, y, out_dtype, stream)
    x_at = _operand(x, "x", torch.bfloat16, rows, k, plan.device)
    step = _experts(experts, plan, QL_INT4_G128, n, k)
    _call("moe_gemm_w4a16", plan.device, x_at, experts.data_ptr(), plan.groups, step, plan._order,
          plan._offsets, plan.tokens * plan.top_k, plan.top_k, n, k, flags,
          y.data_ptr(), dt, _queue(stream, plan.device))
    return y


def moe_gemm_w4a4(a_codes, a_scales, a_tensor_scale, experts, plan, n, k, gather=True, silu_mul=False,
                  y=None, out_dtype=torch.bfloat16, stream=None):
    """moe_gemm_w4a16 for NVFP4 weights and activations: a_codes, a_scales and
    a_tensor_scale are quantize_nvfp4's of x."""
    n, k, rows, flags, y, dt = _product(plan, n, k, gather, silu_mul, y, out_dtype, stream)
    dev = plan.device
    c_at = _operand(a_codes, "a_codes", torch.uint8, rows, k // 2, dev)
    s_at = _operand(a_scales, "a_scales", torch.uint8, rows, k // 16, dev)
    t_at = _vector(a_tensor_scale, "a_tensor_scale", torch.float32, dev, 1)
    step = _experts(experts, plan, QL_NVFP4, n, k)
    _call("moe_gemm_w4a4", dev, c_at, s_at, t_at, experts.data_ptr(), plan.groups, step, plan._order,
          plan._offsets, plan.tokens * plan.top_k, plan.top_k, n, k, flags,
          y.data_ptr(), dt, _queue(stream, dev))
    return y


def moe_combine(rows, plan, weights, out=None, out_dtype=torch.bfloat16, stream=None):
    """Back to the tokens: out[t] = sum_j weights[t, j] * rows[plan.where[t, j]],
    rows [pairs, n] (fp32 or bf16) in the plan's order, weights fp32 [tokens,
    top_k].  Pairs without an expert add nothing."""
    dev = plan.device
    if (rows.device != dev or rows.dtype not in _XDT or rows.dim() != 2 or not rows.is_contiguous()
            or rows.shape[0] != plan.tokens * plan.top_k):
        raise ValueError(f"rows must be a contiguous float32 or bfloat16 [{plan.tokens * plan.top_k}, n] tensor "
                         f"on {dev}, got {rows.dtype} {list(rows.shape)} on {rows.device}")
    n = rows.shape[1]
    w_at = _operand(weights, "weights", torch.float32, plan.tokens, plan.top_k, dev)
    shape = (plan.tokens, n)
    out = _new(shape, out_dtype, dev, stream) if out is None else _rows_out(out, "out", shape, _XDT, dev)
    dt = _XDT.get(out.dtype)
    if dt is None:
        raise ValueError("out must be float32 or bfloat16")
    _call("moe_combine", dev, rows.data_ptr(), _XDT[rows.dtype], plan._where, plan._offsets,
          plan.groups, w_at, plan.tokens, plan.top_k, n, out.data_ptr(), dt,
          _queue(stream, dev))
    return out


def _strided(t, name, dtypes, rows, dev):
    """Row stride and columns of t [rows, columns], a row's elements contiguous."""
    if t.device != dev or t.dtype not in dtypes or t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be a [{rows}, columns] tensor on {dev} of "
                         f"{' or '.join(map(str, dtypes))}, got {t.dtype} {list(t.shape)} on {t.device}")
    step, inner = t.stride()
    if t.shape[1] > 1 and inner != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    return (step if rows > 1 else t.shape[1]), t.shape[1]


def lora_add_workspace(rows, adapters, rank, k):
    return _lib.lora_add_workspace(rows, adapters, rank, k)


def lora_add(y, x, a, b, plan, scale=None, out=None, workspace=None, stream=None):
    """Low-rank adapters beside a projection: out[t] = y[t] + scale[i] * B_i (A_i
    x[t]), i the adapter of row t (plan: group_rows of the rows' adapters); rows
    without one: out = y.

    y [rows, n] (fp32 or bf16), x bf16 [rows, k]: a row's elements contiguous,
    rows any stride (a slice of a fused projection will do).  a bf16 [adapters,
    rank, k], b bf16 [adapters, n, rank], rank a multiple of 8 up to 128; scale
    fp32 [adapters] (None: 1).  out: like y, y itself when not given; it shares no
    memory with x, or with y in part (slices side by side of one buffer's rows will
    do)."""
    dev = plan.device
    if torch._C._cuda_getDevice() != dev.index:   # the workspace goes by the device too
        with torch.cuda.device(dev):
            return lora_add(y, x, a, b, plan, scale, out, workspace, stream)
    if plan.top_k != 1:
        raise ValueError(f"a row has one adapter; the plan has {plan.top_k} choices to a row")
    rows, adapters = plan.tokens, plan.groups
    ys, n = _strided(y, "y", _XDT, rows, dev)
    xs, k = _strided(x, "x", (torch.bfloat16,), rows, dev)
    if (a.device != dev or a.dtype != torch.bfloat16 or a.dim() != 3 or a.shape[0] != adapters
            or a.shape[2] != k or not a.is_contiguous()):
        raise ValueError(f"a must be a contiguous bfloat16 [{adapters}, rank, {k}] tensor on {dev}, got "
                         f"{a.dtype} {list(a.shape)} on {a.device}")
    rank = a.shape[1]
    if (b.device != dev or b.dtype != torch.bfloat16 or b.shape != (adapters, n, rank)
            or not b.is_contiguous()):
        raise ValueError(f"b must be a contiguous bfloat16 [{adapters}, {n}, {rank}] tensor on {dev}, got "
                         f"{b.dtype} {list(b.shape)} on {b.device}")
    s_at = None if scale is None else _vector(scale, "scale", torch.float32, dev, adapters)
    if out is None:
        out = y
    os_, cols = (ys, n) if out is y else _strided(out, "out", (y.dtype,), rows, dev)
    if cols != n:
        raise ValueError(f"out must be [{rows}, {n}], got {list(out.shape)}")
    at, have, keep = _workspace(workspace, _lib.lora_add_workspace(rows, adapters, rank, k), dev, stream)
    _call("lora_add", dev, y.data_ptr(), ys, x.data_ptr(), xs, a.data_ptr(), b.data_ptr(), s_at, adapters, rank,
          plan._order, plan._offsets, rows, n, k, out.data_ptr(), os_,
          _XDT[y.dtype], at, have, _queue(stream, dev))
    return out


def raw():
    """The ctypes handle of libqlin.so (for tests that call the C ABI directly)."""
    return _lib
