"""ctypes binding of libwush (argument marshalling only).

Every function here has the name of the C entry point it wraps and only
converts arguments (ints, floats, device pointers from torch tensors, the
current HIP stream) and turns a non-OK status into an exception.  All
computation happens inside libwush.so.  Importing this module fails loudly
when the library has not been built: there is no fallback path.
"""

import ctypes
import os

# torch ships its own HIP runtime.  Loading libwush.so first would map the
# system HIP/HSA runtime as well, and two runtimes in one process do not see
# each other's device state ("no ROCm-capable device" on launch, crashes in
# later copies).  Importing torch first makes libwush bind to the runtime torch
# already loaded (same soname).
import torch  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwush.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libwush.so not found at {LIB_PATH}; build it with "
        "`python -m aware_block_transforms_amd.build` (no CPU fallback exists)")

lib = ctypes.CDLL(LIB_PATH)

# enums (must match include/wush.h)
WUSH_OK, WUSH_E_ARG, WUSH_E_SHAPE, WUSH_E_NUMERIC, WUSH_E_HIP, WUSH_E_UNSUPPORTED = range(6)
FORMATS = {"mxfp4": 0, "nvfp4": 1, "int4": 2}
KINDS = {"identity": 0, "hadamard": 1, "wus": 2, "wush": 3}
DTYPES = {"f32": 0, "bf16": 1}
BLOCK = {"mxfp4": 32, "nvfp4": 16, "int4": 32}

_i, _f, _p, _sz = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_fp = ctypes.POINTER(ctypes.c_float)
_l = ctypes.c_int64

_SIGS = {
    "wush_format_block": ([_i], _i),
    "wush_block_moments": ([_i, _i, _i, _p, _p], _i),
    "wush_build_transforms": ([_i, _i, _i, _i, _p, _p, _p, _p], _i),
    "wush_transform_quant": ([_i, _i, _i, _i, _p, _p, _f, _p, _p, _p], _i),
    "wush_transform_apply": ([_i, _i, _i, _i, _p, _p, _p, _p], _i),
    "wush_build_shared": ([_i, _i, _i, _i, _p, _p, _i, _p, _p, _p], _i),
    "wush_mxfp4_planes_bytes": ([_i, _i], _sz),
    "wush_build_transforms_dev_ws_bytes": ([_i, _i], _sz),
    "wush_build_transforms_dev": ([_i, _i, _i, _i, _p, _p, _p, _p, _p, _sz, _p], _i),
    "wush_mxfp4_scale_planes": ([_i, _i, _p, _p, _p], _i),
    "wush_transform_quant_mx_planes": ([_i, _i, _i, _p, _p, _p, _p, _p], _i),
    "wush_w4a4_gemm_mx_planes": ([_i, _i, _i, _p, _p, _p, _p, _p, _p], _i),
    "wush_transform_quant_shared": ([_i, _i, _i, _i, _p, _p, _i, _p, _f, _p, _p, _p], _i),
    "wush_nvfp4_global_scale_shared": ([_i, _i, _i, _p, _p, _i, _p, _p, _p], _i),
    "wush_pack_weights_shared": ([_i, _i, _i, _p, _p, _i, _p, _p, _p, _p, _p], _i),
    "wush_nvfp4_global_scale": ([_i, _i, _i, _p, _p, _fp, _p], _i),
    "wush_pack_weights": ([_i, _i, _i, _p, _p, _p, _p, _fp, _p], _i),
    "wush_build_hd": ([_i, _i, _i, _p, _p, _p, _p], _i),
    "wush_block_moments_dev_ws_bytes": ([_i, _i, _i], _sz),
    "wush_block_moments_dev": ([_i, _i, _i, _i, _p, _p, _p, _sz, _p], _i),
    "wush_transform_quant_hd": ([_i, _i, _i, _i, _p, _p, _f, _p, _p, _p], _i),
    "wush_nvfp4_global_scale_hd": ([_i, _i, _i, _p, _p, _fp, _p], _i),
    "wush_pack_weights_hd": ([_i, _i, _i, _p, _p, _p, _p, _fp, _p], _i),
    "wush_w4a4_gemm_ws_bytes": ([_i, _i, _i, _i], _sz),
    "wush_w4a4_gemm": ([_i, _i, _i, _i, _p, _p, _f, _p, _p, _f, _p, _p, _sz, _p], _i),
    "wush_w4a4_gemm_noalloc_max_ws_bytes": ([], _sz),
    "wush_w4a4_gemm_noalloc": ([_i, _i, _i, _i, _p, _p, _f, _p, _p, _f, _p, _p], _i),
    "wush_layer_loss": ([_i, _i, _p, _p, _p, _p, _p], _i),
    "wush_loss_ws_bytes": ([_i, _i], _sz),
    "wush_had256_packed_bytes": ([_i, _i], _sz),
    "wush_had256_pack_weights": ([_i, _i, _p, _p, _p], _i),
    "wush_had256_gemv_ws_bytes": ([_i, _i], _sz),
    "wush_had256_gemv": ([_i, _i, _i, _p, _p, _p, _p, _sz, _p], _i),
    "wush_had256_rotate": ([_i, _i, _p, _p, _p], _i),
    "wush_block_norm": ([_i, _i, _i, _i, _i, _p, _p, _i, _p, _f, _p, _f, _p, _f, _p, _p, _p, _p, _p], _i),
    "wush_block_norm_bwd_ws_bytes": ([_i, _i], _sz),
    "wush_block_norm_bwd": ([_i, _i, _i, _i, _i, _p, _p, _p, _p, _i, _p, _f, _p, _f, _p, _p, _p, _p, _p, _p, _p, _p,
                             _p, _sz, _p], _i),
    "wush_act8_pack": ([_i, _i, _i, _p, _p, _p, _p], _i),
    "wush_act8_unpack": ([_i, _i, _i, _p, _p, _p, _p], _i),
    "wush_act8_swiglu": ([_i, _i, _i, _i, _p, _p, _l, _p, _p, _p, _p, _p, _p], _i),
    "wush_act8_swiglu_bwd": ([_i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _l, _p], _i),
    "wush_adapter_ws_bytes": ([_i, _i, _i, _i], _sz),
    "wush_adapter_forward": ([_i, _i, _i, _i, _i, _p, _l, _i, _p, _p, _i, _i, _p, _p, _p, _p, _p, _l, _p, _l, _p, _p,
                              _sz, _p], _i),
    "wush_adapter_backward_ws_bytes": ([_i, _i, _i, _i, _i, _i], _sz),
    "wush_adapter_backward": ([_i, _i, _i, _i, _i, _i, _p, _l, _p, _p, _l, _i, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p,
                               _l, _p, _l, _p, _p, _p, _sz, _p], _i),
    "wush_status_string": ([_i], ctypes.c_char_p),
    "wush_last_error": ([], ctypes.c_char_p),
    "wush_version": ([], ctypes.c_char_p),
}
for _name, (_args, _ret) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _ret

EXPORTED = tuple(_SIGS)


class WushError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        detail = lib.wush_last_error().decode()
        super().__init__(f"{where}: {lib.wush_status_string(status).decode()} ({status}): {detail}")


def _check(status, where):
    if status != WUSH_OK:
        raise WushError(status, where)


def _ptr(t):
    """Raw address of a torch tensor / numpy array (or None)."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def _stream(stream):
    if stream is not None:
        return stream
    # the current stream's handle without the Stream object around it (0.4 instead of 3 us), where this torch gives it:
    # the function is not part of its documented interface
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


# ----------------------------------------------------------------------------- host calls


def wush_block_moments(bs, X, Sx):
    """X: host float32 [n][d_in] (numpy or CPU tensor), Sx: host float32 [d_in/bs][bs][bs] out."""
    n, d_in = X.shape
    _check(lib.wush_block_moments(bs, n, d_in, _ptr(X), _ptr(Sx)), "wush_block_moments")


def wush_build_transforms(kind, bs, W, Sx, Tx, Tw):
    """Host arrays: W [d_out][d_in] f32, Sx [nblk][bs][bs] f32 (or None), Tx/Tw out."""
    k = KINDS[kind] if isinstance(kind, str) else int(kind)
    d_out, d_in = (W.shape if W is not None else (0, Tx.shape[0] * bs))
    _check(lib.wush_build_transforms(k, bs, d_in, d_out, _ptr(W), _ptr(Sx), _ptr(Tx), _ptr(Tw)),
           "wush_build_transforms")


def wush_build_hd(bs, W, Sx, dx, dw):
    """Host arrays: W [d_out][d_in] f32, Sx [nblk][bs][bs] f32; dx, dw out [d_in] f32."""
    d_out, d_in = W.shape
    _check(lib.wush_build_hd(bs, d_in, d_out, _ptr(W), _ptr(Sx), _ptr(dx), _ptr(dw)), "wush_build_hd")


# ----------------------------------------------------------------------------- device calls


def wush_transform_quant(fmt, X, Tx, codes, scales, g=0.0, stream=None):
    """X: device [n][d_in] float32 or bfloat16; Tx: device [nblk][bs][bs] f32 or None (identity)."""
    import torch
    n, d_in = X.shape
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("X must be float32 or bfloat16")
    _check(lib.wush_transform_quant(_fmt(fmt), xdt, n, d_in, _ptr(X), _ptr(Tx), float(g), _ptr(codes),
                                    _ptr(scales), _stream(stream)), "wush_transform_quant")


def wush_transform_apply(X, Tx, Y, stream=None):
    """Y = T x per block (fp32, the transform wush_transform_quant quantizes).  Tx: [nblk][bs][bs]."""
    import torch
    n, d_in = X.shape
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("X must be float32 or bfloat16")
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    _check(lib.wush_transform_apply(xdt, Tx.shape[-1], n, d_in, _ptr(X), _ptr(Tx), _ptr(Y), _stream(stream)),
           "wush_transform_apply")


def wush_build_shared(kind, W, Sx, bs, group, ngroups):
    """Host numpy: per-group (Tx, Tw) [ngroups][bs][bs] float32 from the groups' summed moments."""
    import numpy as np
    W = np.ascontiguousarray(W, dtype=np.float32)
    d_out, d_in = W.shape
    group = np.ascontiguousarray(group, dtype=np.int32)
    Sx = None if Sx is None else np.ascontiguousarray(Sx, dtype=np.float32)
    Tx = np.empty((ngroups, bs, bs), dtype=np.float32)
    Tw = np.empty_like(Tx)
    _check(lib.wush_build_shared(KINDS[kind], bs, d_in, d_out, W.ctypes.data,
                                 None if Sx is None else Sx.ctypes.data, int(ngroups), group.ctypes.data,
                                 Tx.ctypes.data, Tw.ctypes.data), "wush_build_shared")
    return Tx, Tw


def wush_transform_quant_shared(fmt, X, Tx, group, codes, scales, g=0.0, stream=None):
    """X: device [n][d_in] f32/bf16; Tx: device [ngroups][bs][bs] f32; group: device [nblk] int32."""
    import torch
    n, d_in = X.shape
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("X must be float32 or bfloat16")
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    _check(lib.wush_transform_quant_shared(_fmt(fmt), xdt, n, d_in, _ptr(X), _ptr(Tx), Tx.shape[0], _ptr(group),
                                           float(g), _ptr(codes), _ptr(scales), _stream(stream)),
           "wush_transform_quant_shared")


def wush_nvfp4_global_scale_shared(X, Tx, group, stream=None):
    import torch
    n, d_in = X.shape
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    g = ctypes.c_float(0.0)
    _check(lib.wush_nvfp4_global_scale_shared(xdt, n, d_in, _ptr(X), _ptr(Tx), Tx.shape[0], _ptr(group),
                                              ctypes.byref(g), _stream(stream)), "wush_nvfp4_global_scale_shared")
    return g.value


def wush_pack_weights_shared(fmt, W, Tw, group, codes, scales, stream=None):
    """W: device [d_out][d_in] f32.  Returns the NVFP4 tensor scale (1.0 for other formats)."""
    d_out, d_in = W.shape
    g = ctypes.c_float(0.0)
    _check(lib.wush_pack_weights_shared(_fmt(fmt), d_out, d_in, _ptr(W), _ptr(Tw), Tw.shape[0], _ptr(group),
                                        _ptr(codes), _ptr(scales), ctypes.byref(g), _stream(stream)),
           "wush_pack_weights_shared")
    return g.value


def wush_build_transforms_dev_ws_bytes(bs, d_in):
    return lib.wush_build_transforms_dev_ws_bytes(bs, d_in)


def wush_build_transforms_dev(kind, bs, W, Sx, Tx, Tw, ws=None, stream=None):
    """Device tensors: W [d_out][d_in] f32, Sx [nblk][bs][bs] f32 -> Tx, Tw [nblk][bs][bs] f32 (synchronises)."""
    import torch
    d_out, d_in = W.shape
    need = lib.wush_build_transforms_dev_ws_bytes(bs, d_in)
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=Tx.device)
    _check(lib.wush_build_transforms_dev(KINDS[kind], bs, d_in, d_out, _ptr(W), _ptr(Sx), _ptr(Tx), _ptr(Tw), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)), "wush_build_transforms_dev")


def wush_mxfp4_planes_bytes(rows, K):
    return lib.wush_mxfp4_planes_bytes(rows, K)


def wush_mxfp4_scale_planes(scales, planes, K, stream=None):
    """scales: device [rows][K/32] uint8 (row-major) -> planes: device uint8 of wush_mxfp4_planes_bytes."""
    _check(lib.wush_mxfp4_scale_planes(scales.shape[0], K, _ptr(scales), _ptr(planes), _stream(stream)),
           "wush_mxfp4_scale_planes")


def wush_transform_quant_mx_planes(X, Tx, codes, planes, stream=None):
    import torch
    n, d_in = X.shape
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("X must be float32 or bfloat16")
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    _check(lib.wush_transform_quant_mx_planes(xdt, n, d_in, _ptr(X), _ptr(Tx), _ptr(codes), _ptr(planes),
                                              _stream(stream)), "wush_transform_quant_mx_planes")


def wush_w4a4_gemm_mx_planes(a_codes, a_planes, b_codes, b_planes, Y, stream=None):
    M, N = Y.shape
    K = a_codes.shape[1] * 2
    _check(lib.wush_w4a4_gemm_mx_planes(M, N, K, _ptr(a_codes), _ptr(a_planes), _ptr(b_codes), _ptr(b_planes),
                                        _ptr(Y), _stream(stream)), "wush_w4a4_gemm_mx_planes")


def wush_nvfp4_global_scale(X, Tx, stream=None):
    import torch
    n, d_in = X.shape
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    g = ctypes.c_float(0.0)
    _check(lib.wush_nvfp4_global_scale(xdt, n, d_in, _ptr(X), _ptr(Tx), ctypes.byref(g), _stream(stream)),
           "wush_nvfp4_global_scale")
    return g.value


def wush_pack_weights(fmt, W, Tw, codes, scales, stream=None):
    """W: device [d_out][d_in] f32.  Returns the NVFP4 tensor scale (1.0 for other formats)."""
    d_out, d_in = W.shape
    g = ctypes.c_float(0.0)
    _check(lib.wush_pack_weights(_fmt(fmt), d_out, d_in, _ptr(W), _ptr(Tw), _ptr(codes), _ptr(scales),
                                 ctypes.byref(g), _stream(stream)), "wush_pack_weights")
    return g.value


def wush_block_moments_dev_ws_bytes(bs, n, d_in):
    return lib.wush_block_moments_dev_ws_bytes(bs, n, d_in)


def wush_block_moments_dev(bs, X, Sx, ws=None, stream=None):
    """X: device [n][d_in] float32 or bfloat16; Sx: device out [d_in/bs][bs][bs] float32."""
    import torch
    n, d_in = X.shape
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("X must be float32 or bfloat16")
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    wp, wb = _ws(ws)
    _check(lib.wush_block_moments_dev(bs, xdt, n, d_in, _ptr(X), _ptr(Sx), wp, wb, _stream(stream)),
           "wush_block_moments_dev")


def wush_transform_quant_hd(fmt, X, dx, codes, scales, g=0.0, stream=None):
    """Hadamard-diagonal variant; dx: device [d_in] f32 (from wush_build_hd)."""
    import torch
    n, d_in = X.shape
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("X must be float32 or bfloat16")
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    _check(lib.wush_transform_quant_hd(_fmt(fmt), xdt, n, d_in, _ptr(X), _ptr(dx), float(g), _ptr(codes),
                                       _ptr(scales), _stream(stream)), "wush_transform_quant_hd")


def wush_nvfp4_global_scale_hd(X, dx, stream=None):
    import torch
    n, d_in = X.shape
    xdt = DTYPES["bf16"] if X.dtype == torch.bfloat16 else DTYPES["f32"]
    g = ctypes.c_float(0.0)
    _check(lib.wush_nvfp4_global_scale_hd(xdt, n, d_in, _ptr(X), _ptr(dx), ctypes.byref(g), _stream(stream)),
           "wush_nvfp4_global_scale_hd")
    return g.value


def wush_pack_weights_hd(fmt, W, dw, codes, scales, stream=None):
    """W: device [d_out][d_in] f32, dw: device [d_in] f32.  Returns the NVFP4 tensor scale (1.0 otherwise)."""
    d_out, d_in = W.shape
    g = ctypes.c_float(0.0)
    _check(lib.wush_pack_weights_hd(_fmt(fmt), d_out, d_in, _ptr(W), _ptr(dw), _ptr(codes), _ptr(scales),
                                    ctypes.byref(g), _stream(stream)), "wush_pack_weights_hd")
    return g.value


def _ws(ws):
    """(pointer, bytes) of an optional device workspace tensor."""
    if ws is None:
        return None, 0
    return _ptr(ws), ws.numel() * ws.element_size()


def wush_w4a4_gemm_ws_bytes(fmt, M, N, K):
    return lib.wush_w4a4_gemm_ws_bytes(_fmt(fmt), M, N, K)


def wush_w4a4_gemm(fmt, a_codes, a_scales, b_codes, b_scales, Y, a_g=1.0, b_g=1.0, ws=None, stream=None):
    M, N = Y.shape
    K = a_codes.shape[1] * 2
    wp, wb = _ws(ws)
    _check(lib.wush_w4a4_gemm(_fmt(fmt), M, N, K, _ptr(a_codes), _ptr(a_scales), float(a_g), _ptr(b_codes),
                              _ptr(b_scales), float(b_g), _ptr(Y), wp, wb, _stream(stream)), "wush_w4a4_gemm")


def wush_w4a4_gemm_noalloc_max_ws_bytes():
    return lib.wush_w4a4_gemm_noalloc_max_ws_bytes()


def wush_w4a4_gemm_noalloc(fmt, a_codes, a_scales, b_codes, b_scales, Y, a_g=1.0, b_g=1.0, stream=None):
    M, N = Y.shape
    K = a_codes.shape[1] * 2
    _check(lib.wush_w4a4_gemm_noalloc(_fmt(fmt), M, N, K, _ptr(a_codes), _ptr(a_scales), float(a_g), _ptr(b_codes),
                                      _ptr(b_scales), float(b_g), _ptr(Y), _stream(stream)), "wush_w4a4_gemm_noalloc")


def wush_loss_ws_bytes(M, N):
    return lib.wush_loss_ws_bytes(M, N)


def wush_layer_loss(Yhat, Yref, loss, ws, stream=None):
    M, N = Yhat.shape
    _check(lib.wush_layer_loss(M, N, _ptr(Yhat), _ptr(Yref), _ptr(loss), _ptr(ws), _stream(stream)),
           "wush_layer_loss")


def wush_had256_packed_bytes(d_out, d_in):
    return lib.wush_had256_packed_bytes(d_out, d_in)


def _packed_check(packed, d_out, d_in, name):
    need = lib.wush_had256_packed_bytes(d_out, d_in)
    if packed.numel() * packed.element_size() < need:
        raise ValueError("%s: packed buffer of %d bytes, need %d" % (name, packed.numel() * packed.element_size(), need))


def wush_had256_pack_weights(W, packed, stream=None):
    d_out, d_in = W.shape
    _packed_check(packed, d_out, d_in, "wush_had256_pack_weights")
    _check(lib.wush_had256_pack_weights(d_out, d_in, _ptr(W), _ptr(packed), _stream(stream)),
           "wush_had256_pack_weights")


def wush_had256_gemv_ws_bytes(batch, d_in):
    return lib.wush_had256_gemv_ws_bytes(batch, d_in)


def wush_had256_gemv(x, packed, y, ws=None, stream=None):
    batch, d_in = x.shape
    d_out = y.shape[1]
    _packed_check(packed, d_out, d_in, "wush_had256_gemv")
    wp, wb = _ws(ws)
    _check(lib.wush_had256_gemv(batch, d_out, d_in, _ptr(x), _ptr(packed), _ptr(y), wp, wb, _stream(stream)),
           "wush_had256_gemv")


def wush_had256_rotate(inp, out, stream=None):
    rows, d_in = inp.shape
    _check(lib.wush_had256_rotate(rows, d_in, _ptr(inp), _ptr(out), _stream(stream)), "wush_had256_rotate")


# ----------------------------------------------------------------------------- around a frozen projection

GATES = {"none": 0, "channel": 1, "token": 2, "element": 3}
_FLOATS = {torch.float32: 0, torch.bfloat16: 1}


def _dt(t, name):
    """wush_dtype of a float32 or bfloat16 tensor."""
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, not %s" % (name, t.dtype))
    return code


def _want(t, name, shape, dtype=None):
    """A contiguous tensor of that shape (and dtype), or an exception."""
    if t.shape == shape and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, shape, tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be contiguous" % name)


def _rows(t, name, n, d):
    """Row stride of an [n][d] tensor whose rows are contiguous."""
    if t.shape != (n, d):
        raise ValueError("%s must have shape (%d, %d), not %s" % (name, n, d, tuple(t.shape)))
    if n <= 1:
        if not t.is_contiguous():
            raise ValueError("%s must have contiguous rows" % name)
        return d
    ld, one = t.stride()
    if one != 1 and d > 1:
        raise ValueError("%s must have contiguous rows" % name)
    return ld


def _gate(gate, n, d, ydt):
    """Kind of a gate by its shape: [d] per channel, [n][1] per token, [n][d] per element."""
    if gate is None:
        return 0
    if gate.dim() == 1:
        _want(gate, "gate", (d,), torch.float32)
        return 1
    if tuple(gate.shape) == (n, 1) and d != 1:
        _want(gate, "gate", (n, 1), torch.float32)
        return 2
    _want(gate, "gate", (n, d), ydt)
    return 3


def wush_block_norm(Y, w_post, gate, R, w_pre, Rout, U, rstd_post=None, rstd_pre=None, branch_scale=1.0, res_scale=1.0,
                    eps=1e-6, stream=None):
    """Rout = res_scale R + branch_scale gate norm(Y) w_post; U = norm(Rout) w_pre.  Y, w_post, gate, w_pre with U, and
    Rout may be None; gate is [d], [n][1] (float32) or [n][d] (Y's dtype)."""
    shape = n, d = R.shape
    _want(R, "R", shape)
    rdt = ydt = udt = _dt(R, "R")
    y = wp = g = ro = wn = u = kp = kn = None
    if Y is not None:
        _want(Y, "Y", shape)
        ydt, y = _dt(Y, "Y"), Y.data_ptr()
    if w_post is not None:
        _want(w_post, "w_post", (d,), torch.float32)
        wp = w_post.data_ptr()
    if gate is not None:
        g = gate.data_ptr()
    kind = _gate(gate, n, d, None if Y is None else Y.dtype)
    if w_pre is not None:
        _want(w_pre, "w_pre", (d,), torch.float32)
        wn = w_pre.data_ptr()
    if Rout is not None:
        _want(Rout, "Rout", shape, R.dtype)
        ro = Rout.data_ptr()
    if U is not None:
        _want(U, "U", shape)
        udt, u = _dt(U, "U"), U.data_ptr()
    if rstd_post is not None:
        _want(rstd_post, "rstd_post", (n,), torch.float32)
        kp = rstd_post.data_ptr()
    if rstd_pre is not None:
        _want(rstd_pre, "rstd_pre", (n,), torch.float32)
        kn = rstd_pre.data_ptr()
    _check(lib.wush_block_norm(ydt, rdt, udt, n, d, y, wp, kind, g, branch_scale, R.data_ptr(), res_scale, wn, eps, ro,
                               u, kp, kn, _stream(stream)), "wush_block_norm")


def wush_block_norm_bwd_ws_bytes(n, d):
    return lib.wush_block_norm_bwd_ws_bytes(n, d)


def wush_block_norm_bwd(dU, dRout, Y, w_post, gate, Rout, w_pre, rstd_post, rstd_pre, dY, dR, dgate, dw_post, dw_pre,
                        branch_scale=1.0, res_scale=1.0, ws=None, stream=None):
    """Gradients of wush_block_norm; dU (with w_pre and dw_pre) or dRout may be None, and so may dR."""
    some = next((t for t in (Rout, dRout, Y) if t is not None), None)
    if some is None:
        raise ValueError("wush_block_norm_bwd needs Rout, dRout or Y")
    n, d = some.shape
    rdts = {t.dtype for t in (Rout, dRout, dR) if t is not None}
    if len(rdts) > 1:
        raise TypeError("Rout, dRout and dR must have one dtype")
    for t, name in ((Rout, "Rout"), (dRout, "dRout"), (dR, "dR"), (dU, "dU")):
        if t is not None:
            _want(t, name, (n, d))
    if Y is not None:
        _want(Y, "Y", (n, d))
        if dY is not None:
            _want(dY, "dY", (n, d), Y.dtype)
    for t, name, size in ((w_post, "w_post", d), (w_pre, "w_pre", d), (dw_post, "dw_post", d), (dw_pre, "dw_pre", d),
                          (rstd_post, "rstd_post", n), (rstd_pre, "rstd_pre", n)):
        if t is not None:
            _want(t, name, (size,), torch.float32)
    kind = _gate(gate, n, d, None if Y is None else Y.dtype)
    if gate is not None and dgate is not None:
        _want(dgate, "dgate", tuple(gate.shape), gate.dtype)
    first = next((t for t in (Rout, dRout, dR) if t is not None), None)
    rdt = 0 if first is None else _dt(first, "Rout")
    ydt = rdt if Y is None else _dt(Y, "Y")
    udt = rdt if dU is None else _dt(dU, "dU")
    wp, wb = _ws(ws)
    _check(lib.wush_block_norm_bwd(ydt, rdt, udt, n, d, _ptr(dU), _ptr(dRout), _ptr(Y), _ptr(w_post), kind, _ptr(gate),
                                   branch_scale, _ptr(Rout), res_scale, _ptr(w_pre), _ptr(rstd_post), _ptr(rstd_pre),
                                   _ptr(dY), _ptr(dR), _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), wp, wb,
                                   _stream(stream)), "wush_block_norm_bwd")


def _checkpoint(codes, scales, n, d, name):
    _want(codes, name + " codes", (n, d), torch.int8)
    _want(scales, name + " scales", (n, d // 32), torch.uint8)


def wush_act8_pack(X, codes, scales, stream=None):
    """X: device [n][d] float32 or bfloat16 -> codes int8 [n][d], scales uint8 [n][d/32]."""
    n, d = X.shape
    _want(X, "X", (n, d))
    _checkpoint(codes, scales, n, d, "act8")
    _check(lib.wush_act8_pack(_dt(X, "X"), n, d, _ptr(X), _ptr(codes), _ptr(scales), _stream(stream)),
           "wush_act8_pack")


def wush_act8_unpack(codes, scales, Y, stream=None):
    """The values of a checkpoint, to Y: device [n][d] float32 or bfloat16."""
    n, d = Y.shape
    _want(Y, "Y", (n, d))
    _checkpoint(codes, scales, n, d, "act8")
    _check(lib.wush_act8_unpack(_dt(Y, "Y"), n, d, _ptr(codes), _ptr(scales), _ptr(Y), _stream(stream)),
           "wush_act8_unpack")


def _pair(a, b, name_a, name_b, n, d):
    """Common row stride and dtype of two [n][d] tensors."""
    ld = _rows(a, name_a, n, d)
    if _rows(b, name_b, n, d) != ld or a.dtype != b.dtype:
        raise ValueError("%s and %s must have one dtype and row stride" % (name_a, name_b))
    return ld


def wush_act8_swiglu(G, U, H, g_codes=None, g_scales=None, u_codes=None, u_scales=None, stream=None):
    """H = G sigmoid(G) U, keeping G and U as act8 checkpoints where their four tensors are given.  G and U may be the
    halves of one tensor (rows contiguous, one row stride)."""
    n, d = G.shape
    ld = _pair(G, U, "G", "U", n, d)
    _want(H, "H", (n, d))
    if g_codes is not None and g_scales is not None:
        _checkpoint(g_codes, g_scales, n, d, "G")
    if u_codes is not None and u_scales is not None:
        _checkpoint(u_codes, u_scales, n, d, "U")
    _check(lib.wush_act8_swiglu(_dt(G, "G"), _dt(H, "H"), n, d, _ptr(G), _ptr(U), ld, _ptr(H), _ptr(g_codes),
                                _ptr(g_scales), _ptr(u_codes), _ptr(u_scales), _stream(stream)), "wush_act8_swiglu")


def wush_act8_swiglu_bwd(dH, g_codes, g_scales, u_codes, u_scales, dG, dU, stream=None):
    """Gradients of wush_act8_swiglu at the checkpoints' values; dG and dU may be the halves of one tensor."""
    n, d = dH.shape
    _want(dH, "dH", (n, d))
    ld = _pair(dG, dU, "dG", "dU", n, d)
    _checkpoint(g_codes, g_scales, n, d, "G")
    _checkpoint(u_codes, u_scales, n, d, "U")
    _check(lib.wush_act8_swiglu_bwd(_dt(dH, "dH"), _dt(dG, "dG"), n, d, _ptr(dH), _ptr(g_codes), _ptr(g_scales),
                                    _ptr(u_codes), _ptr(u_scales), _ptr(dG), _ptr(dU), ld, _stream(stream)),
           "wush_act8_swiglu_bwd")


def _adapters(seg_off, seg_adapter, A, Bt, rank, alpha):
    """(nseg, nad, rmax, d_in, d_out) of a set of adapters and the requests that use it."""
    shape = nad, rmax, d_in = A.shape
    d_out = Bt.shape[-1]
    nseg = seg_adapter.shape[0]
    _want(A, "A", shape, torch.bfloat16)
    _want(Bt, "Bt", (nad, rmax, d_out), torch.bfloat16)
    _want(seg_off, "seg_off", (nseg + 1,), torch.int32)
    _want(seg_adapter, "seg_adapter", (nseg,), torch.int32)
    _want(rank, "rank", (nad,), torch.int32)
    _want(alpha, "alpha", (nad,), torch.float32)
    return nseg, nad, rmax, d_in, d_out


def wush_adapter_ws_bytes(n, d_in, nseg, rmax):
    return lib.wush_adapter_ws_bytes(n, d_in, nseg, rmax)


def wush_adapter_forward(X, seg_off, seg_adapter, A, Bt, rank, alpha, Y0, Y, V=None, ws=None, stream=None):
    """Y = Y0 + V Bt with V = alpha X A^T, each request with its adapter (device int32 seg_off [nseg+1], seg_adapter
    [nseg], -1 for none).  A, Bt: bfloat16 [nad][rmax][d]; rank int32, alpha float32 [nad].  X, Y0 (or None) and Y are
    float32 or bfloat16 with contiguous rows; V float32 [n][rmax] is kept for the backward call where given."""
    nseg, nad, rmax, d_in, d_out = _adapters(seg_off, seg_adapter, A, Bt, rank, alpha)
    n = X.shape[0]
    ldx, ldy = _rows(X, "X", n, d_in), _rows(Y, "Y", n, d_out)
    ldy0 = d_out
    if Y0 is not None:
        ldy0 = _rows(Y0, "Y0", n, d_out)
        if Y0.dtype != Y.dtype:
            raise TypeError("Y0 and Y must have one dtype")
    if V is not None:
        _want(V, "V", (n, rmax), torch.float32)
    wp, wb = _ws(ws)
    _check(lib.wush_adapter_forward(_dt(X, "X"), _dt(Y, "Y"), n, d_in, d_out, X.data_ptr(), ldx, nseg,
                                    seg_off.data_ptr(), seg_adapter.data_ptr(), nad, rmax, A.data_ptr(), Bt.data_ptr(),
                                    rank.data_ptr(), alpha.data_ptr(), _ptr(Y0), ldy0, Y.data_ptr(), ldy, _ptr(V), wp,
                                    wb, _stream(stream)), "wush_adapter_forward")


def wush_adapter_backward_ws_bytes(n, d_in, d_out, nseg, nad, rmax):
    return lib.wush_adapter_backward_ws_bytes(n, d_in, d_out, nseg, nad, rmax)


def wush_adapter_backward(dY, X, seg_off, seg_adapter, A, Bt, rank, alpha, V, dX0, dX, dA, dBt, x_scales=None, ws=None,
                          stream=None):
    """dX = dX0 + dV A, dA = dV^T X and dBt = V^T dY (float32, shaped like A and Bt) with dV = alpha dY Bt^T.  X: as in
    the forward call, or the int8 codes of its act8 checkpoint with x_scales.  dX0 may be None (zeros), dX too."""
    nseg, nad, rmax, d_in, d_out = _adapters(seg_off, seg_adapter, A, Bt, rank, alpha)
    n = dY.shape[0]
    ldg = _rows(dY, "dY", n, d_out)
    if x_scales is not None:
        _checkpoint(X, x_scales, n, d_in, "X")
        ldx, xdt = d_in, 1
    else:
        ldx, xdt = _rows(X, "X", n, d_in), _dt(X, "X")
    _want(V, "V", (n, rmax), torch.float32)
    _want(dA, "dA", (nad, rmax, d_in), torch.float32)
    _want(dBt, "dBt", (nad, rmax, d_out), torch.float32)
    ldd0 = ldd = d_in
    ydt = 1
    if dX is not None:
        ldd, ydt = _rows(dX, "dX", n, d_in), _dt(dX, "dX")
    if dX0 is not None:
        ldd0 = _rows(dX0, "dX0", n, d_in)
        if dX is None or dX0.dtype != dX.dtype:
            raise TypeError("dX0 and dX must have one dtype")
    wp, wb = _ws(ws)
    _check(lib.wush_adapter_backward(_dt(dY, "dY"), xdt, ydt, n, d_in, d_out, _ptr(dY), ldg, _ptr(X), _ptr(x_scales),
                                     ldx, nseg, _ptr(seg_off), _ptr(seg_adapter), nad, rmax, _ptr(A), _ptr(Bt),
                                     _ptr(rank), _ptr(alpha), _ptr(V), _ptr(dX0), ldd0, _ptr(dX), ldd, _ptr(dA),
                                     _ptr(dBt), wp, wb, _stream(stream)), "wush_adapter_backward")


def wush_version():
    return lib.wush_version().decode()
