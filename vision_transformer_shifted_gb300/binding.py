"""ctypes binding of libswin_wattn (include/swin_wattn.h, swin_wattn_test.h,
swin_block.h, swin_wattn_backward.h, swin_rms.h, swin_gated.h, swin_layernorm.h,
swin_linear.h).

Argument marshalling only: every function here passes tensor pointers and
sizes to the C ABI of the same name and raises on a non-OK status.  torch is
used for device memory and streams; no step of the block runs in Python, and
there is no CPU fallback: if the library cannot be loaded every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

V1, V2, FP32 = 0, 1, 0x10
OK, EINVAL, EUNSUPPORTED, ECUDA, ENOMEM, ETIMEOUT, ESCRATCH, ECORRUPT = 0, -1, -2, -3, -4, -5, -6, -7
NOALLOC_MAX_INTERMEDIATE_BYTES = (64 << 20) - 256
OPT_PATH, OPT_WAIT_LIMIT_US, OPT_HOST_CHUNKS, OPT_OVERLAP_CALLS = 1, 2, 3, 4
BLOCK_OPT_OVERLAP_CALLS = 1
BLOCK_GATED_SILU, BLOCK_GATED_GELU = 0, 1
BLOCK_LINEAR_NONE, BLOCK_LINEAR_SILU, BLOCK_LINEAR_GELU = 0, 1, 2
BLOCK_LINEAR_PLAN_FORWARD, BLOCK_LINEAR_PLAN_FORWARD_Q8, BLOCK_LINEAR_PLAN_DX, BLOCK_LINEAR_PLAN_WEIGHT = 0, 1, 2, 3
BLOCK_LINEAR_PLAN_ACT_WEIGHT = 4
BLOCK_LINEAR_GRAD_DX, BLOCK_LINEAR_GRAD_DW, BLOCK_LINEAR_GRAD_DB = 1, 2, 4
BLOCK_GATED_PLAN_DOWN, BLOCK_GATED_PLAN_DX, BLOCK_GATED_PLAN_WEIGHTS, BLOCK_GATED_PLAN_NARROW = 0, 1, 2, 3
PATH_AUTO, PATH_THREE_KERNELS, PATH_FUSED, PATH_FP32 = 0, 1, 2, 3

_lib = None


class SwinWAttnError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (fn, strerror(code) if _lib else "?", code))


_SIGNATURES = {
    "swin_wattn_create": ["pp", "i", "i", "i", "i", "i"],
    "swin_wattn_destroy": ["p"],
    "swin_wattn_forward": ["p", "p", "i", "i", "i", "p", "p", "p", "p", "p", "p", "p", "p"],
    "swin_wattn_forward_host": ["p", "p", "i", "i", "i", "p", "p", "p", "p", "p", "p", "p", "p"],
    "swin_wattn_cpb_table": ["p", "p", "p", "p", "i", "p", "p"],
    "swin_wattn_sync_status": ["p", "p"],
    "swin_wattn_set_option": ["p", "i", "l"],
    "swin_wattn_path": ["p", "i", "i", "i"],
    "swin_wattn_last_launches": ["p"],
    "swin_wattn_test_qkv": ["p", "p", "i", "i", "i", "p", "p", "p", "p"],
    "swin_wattn_test_attn": ["p", "p", "i", "i", "i", "p", "p", "p", "p"],
    "swin_wattn_test_proj": ["p", "p", "i", "i", "i", "p", "p", "p", "p"],
    "swin_wattn_test_gemm": ["p", "p", "p", "p", "i", "i", "i", "i", "p"],
    "swin_wattn_test_watchdog": ["p", "p"],
    "swin_wattn_test_corrupt_workspace": ["p", "i"],
    "swin_wattn_forward_noalloc": ["i", "i", "i", "i", "i", "p", "i", "i", "i", "p", "p", "p", "p", "p", "p", "p",
                                   "p"],
    "swin_wattn_noalloc_sync_status": ["p"],
    "swin_wattn_test_noalloc_watchdog": ["l", "p"],
    "swin_block_create": ["pp", "i", "i", "i", "i", "i", "i"],
    "swin_block_forward": ["p", "p", "i", "i", "i", "p", "p", "p"],
    "swin_block_sync_status": ["p", "p"],
    "swin_block_destroy": ["p"],
    "swin_block_last_launches": ["p"],
    "swin_block_set_option": ["p", "i", "l"],
    "swin_block_test_layernorm": ["p", "p", "p", "p", "p", "p", "i", "i", "i", "p"],
    "swin_stage_norm": ["p", "i", "i", "p", "p", "p", "p"],
    "swin_merge_create": ["pp", "i"],
    "swin_merge_forward": ["p", "p", "i", "i", "i", "p", "p", "p", "p", "p"],
    "swin_merge_destroy": ["p"],
    "swin_wattn_backward": ["p", "p", "i", "i", "i", "p", "p", "p", "p", "p", "p", "p", "p", "p", "p", "p", "p",
                            "p", "p", "p"],
    "swin_wattn_cpb_backward": ["p", "p", "p", "p", "i", "p", "p", "p", "p", "p"],
    "swin_wattn_backward_launches": ["p"],
    "swin_block_rms_create": ["pp", "i", "f"],
    "swin_block_rms_forward": ["p", "p", "p", "i", "p", "p", "p", "p"],
    "swin_block_rms_forward_q8": ["p", "p", "p", "i", "p", "p", "p", "p", "p"],
    "swin_block_rms_backward": ["p", "p", "i", "p", "p", "p", "p", "p", "p"],
    "swin_block_rms_last_launches": ["p"],
    "swin_block_rms_destroy": ["p"],
    "swin_block_layernorm_create": ["pp", "i", "f"],
    "swin_block_layernorm_forward": ["p", "p", "p", "i", "p", "p", "p", "p", "p"],
    "swin_block_layernorm_forward_post": ["p", "p", "p", "i", "p", "p", "p", "p"],
    "swin_block_layernorm_forward_q8": ["p", "p", "p", "i", "p", "p", "p", "p", "p", "p"],
    "swin_block_layernorm_backward": ["p", "p", "i", "p", "p", "p", "p", "p", "p", "p"],
    "swin_block_layernorm_last_launches": ["p"],
    "swin_block_layernorm_destroy": ["p"],
    "swin_block_gated_create": ["pp", "i", "i", "i"],
    "swin_block_gated_forward": ["p", "p", "i", "p", "p", "p", "p"],
    "swin_block_gated_forward_q8": ["p", "p", "p", "i", "p", "p", "p", "p"],
    "swin_block_gated_backward": ["p", "p", "i", "p", "p", "p", "p", "p"],
    "swin_block_gated_last_launches": ["p"],
    "swin_block_gated_sync_status": ["p", "p"],
    "swin_block_gated_destroy": ["p"],
    "swin_block_gated_test_stall": ["p", "p", "i", "p", "l", "p"],
    "swin_block_gated_test_corrupt_workspace": ["p", "i"],
    "swin_block_gated_test_plan": ["i", "i", "i", "i", "p"],
    "swin_block_linear_create": ["pp", "i", "i", "i"],
    "swin_block_linear_forward": ["p", "p", "i", "p", "p", "p", "p", "p", "p"],
    "swin_block_linear_forward_q8": ["p", "p", "p", "i", "p", "p", "p", "p", "p", "p"],
    "swin_block_linear_backward": ["p", "p", "i", "p", "p", "p", "p", "p", "p", "p"],
    "swin_block_linear_last_launches": ["p"],
    "swin_block_linear_sync_status": ["p", "p"],
    "swin_block_linear_destroy": ["p"],
    "swin_block_linear_test_plan": ["i", "i", "i", "i", "p"],
    "swin_block_linear_test_backward_plan": ["i", "i", "i", "i", "i", "p"],
    "swin_block_linear_test_clusters_of": ["i", "i", "i", "i"],
    "swin_block_linear_test_corrupt_workspace": ["p", "i"],
    "swin_block_gated_test_last_use": ["i", "i", "i", "p", "p"],
}

# swin_block_params (include/swin_block.h), field for field
BLOCK_PARAM_FIELDS = ("ln1_gamma", "ln1_beta", "Wqkv", "bqkv", "bias_table", "logit_scale", "Wproj", "bproj",
                      "ln2_gamma", "ln2_beta", "W1", "b1", "W2", "b2")


class BlockParams(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in BLOCK_PARAM_FIELDS]
_CT = {"p": ctypes.c_void_p, "pp": ctypes.POINTER(ctypes.c_void_p), "i": ctypes.c_int, "l": ctypes.c_int64,
       "f": ctypes.c_float}


_load_lock = threading.Lock()


def load(build_if_missing: bool = True):
    """Loads libswin_wattn.so (building it first if it is missing)."""
    global _lib
    if _lib is None:
        with _load_lock:   # (the first calls of several threads)
            if _lib is None:
                _lib = _load(build_if_missing)
    return _lib


def _load(build_if_missing):
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise OSError("libswin_wattn.so is not built")
        _build.build()
    lib = ctypes.CDLL(path)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = [_CT[a] for a in args]
        fn.restype = ctypes.c_int
    lib.swin_wattn_strerror.argtypes = [ctypes.c_int]
    lib.swin_wattn_strerror.restype = ctypes.c_char_p
    lib.swin_wattn_last_cuda_error.argtypes = [ctypes.c_void_p]
    lib.swin_wattn_last_cuda_error.restype = ctypes.c_char_p
    _check_natively()
    return lib


def exported_symbols():
    """Names of the functions the C headers declare."""
    return sorted(list(_SIGNATURES) + ["swin_wattn_strerror", "swin_wattn_last_cuda_error"])


def strerror(code: int) -> str:
    return load().swin_wattn_strerror(int(code)).decode()


def _check(fn, rc):
    if rc != OK:
        raise SwinWAttnError(fn, rc)
    return rc


def _p(t):
    """Pointer of a tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        if torch.cuda.is_available():
            return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        return None
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def swin_wattn_create(C, heads, M, shift, mode):
    h = ctypes.c_void_p()
    _check("swin_wattn_create", load().swin_wattn_create(ctypes.byref(h), C, heads, M, shift, mode))
    return h


def swin_wattn_destroy(h):
    return _check("swin_wattn_destroy", load().swin_wattn_destroy(h))


def swin_wattn_forward(h, x, Wqkv, bqkv, bias_table, logit_scale, Wproj, bproj, out, stream=None):
    B, H, W, _ = x.shape
    rc = load().swin_wattn_forward(
        h, _p(x), B, H, W, _p(Wqkv), _p(bqkv), _p(bias_table), _p(logit_scale), _p(Wproj), _p(bproj), _p(out),
        _stream(stream))
    if rc == ECUDA:
        raise SwinWAttnError("swin_wattn_forward (%s)" % swin_wattn_last_cuda_error(h), rc)
    return _check("swin_wattn_forward", rc)


def swin_wattn_backward(h, x, Wqkv, bqkv, bias_table, Wproj, bproj, dy, dx, dWqkv, dbqkv, dtable, dWproj, dbproj,
                        logit_scale=None, dlogit_scale=None, stream=None):
    B, H, W, _ = x.shape
    return _check("swin_wattn_backward", load().swin_wattn_backward(
        h, _p(x), B, H, W, _p(Wqkv), _p(bqkv), _p(bias_table), _p(logit_scale), _p(Wproj), _p(bproj), _p(dy), _p(dx),
        _p(dWqkv), _p(dbqkv), _p(dtable), _p(dlogit_scale), _p(dWproj), _p(dbproj), _stream(stream)))


def swin_wattn_cpb_backward(h, W1, b1, W2, dtable, dW1, db1, dW2, stream=None):
    return _check("swin_wattn_cpb_backward", load().swin_wattn_cpb_backward(
        h, _p(W1), _p(b1), _p(W2), W1.shape[0], _p(dtable), _p(dW1), _p(db1), _p(dW2), _stream(stream)))


def swin_wattn_backward_launches(h):
    return load().swin_wattn_backward_launches(h)


def swin_wattn_last_cuda_error(h):
    return load().swin_wattn_last_cuda_error(h).decode()


def swin_wattn_forward_host(h, x_host, Wqkv, bqkv, bias_table, logit_scale, Wproj, bproj, out_host, stream=None):
    B, H, W, _ = x_host.shape
    return _check("swin_wattn_forward_host", load().swin_wattn_forward_host(
        h, _p(x_host), B, H, W, _p(Wqkv), _p(bqkv), _p(bias_table), _p(logit_scale), _p(Wproj), _p(bproj),
        _p(out_host), _stream(stream)))


def swin_wattn_cpb_table(h, W1, b1, W2, table, stream=None):
    return _check("swin_wattn_cpb_table", load().swin_wattn_cpb_table(
        h, _p(W1), _p(b1), _p(W2), W1.shape[0], _p(table), _stream(stream)))


def swin_wattn_sync_status(h, stream=None):
    """Returns the status code (OK, ETIMEOUT or ECUDA) without raising."""
    return load().swin_wattn_sync_status(h, _stream(stream))


def swin_wattn_set_option(h, option, value):
    return _check("swin_wattn_set_option", load().swin_wattn_set_option(h, option, int(value)))


def swin_wattn_path(h, B, H, W):
    return load().swin_wattn_path(h, B, H, W)


def swin_wattn_last_launches(h):
    return load().swin_wattn_last_launches(h)


def swin_wattn_forward_noalloc(C, heads, M, shift, mode, x, Wqkv, bqkv, bias_table, logit_scale, Wproj, bproj,
                               out, stream=None):
    B, H, W, _ = x.shape
    return _check("swin_wattn_forward_noalloc", load().swin_wattn_forward_noalloc(
        C, heads, M, shift, mode, _p(x), B, H, W, _p(Wqkv), _p(bqkv), _p(bias_table), _p(logit_scale), _p(Wproj),
        _p(bproj), _p(out), _stream(stream)))


def swin_wattn_noalloc_sync_status(stream=None):
    """Status of the swin_wattn_forward_noalloc calls on the current device:
    the status code (OK, ETIMEOUT or ECUDA), without raising."""
    return load().swin_wattn_noalloc_sync_status(_stream(stream))


def swin_wattn_test_noalloc_watchdog(wait_limit_us, stream=None):
    return _check("swin_wattn_test_noalloc_watchdog",
                  load().swin_wattn_test_noalloc_watchdog(int(wait_limit_us), _stream(stream)))


def swin_wattn_test_qkv(h, x, Wqkv, bqkv, qkv, stream=None):
    B, H, W, _ = x.shape
    return _check("swin_wattn_test_qkv", load().swin_wattn_test_qkv(
        h, _p(x), B, H, W, _p(Wqkv), _p(bqkv), _p(qkv), _stream(stream)))


def swin_wattn_test_attn(h, qkv, B, H, W, bias_table, logit_scale, attn, stream=None):
    return _check("swin_wattn_test_attn", load().swin_wattn_test_attn(
        h, _p(qkv), B, H, W, _p(bias_table), _p(logit_scale), _p(attn), _stream(stream)))


def swin_wattn_test_proj(h, attn, B, H, W, Wproj, bproj, out, stream=None):
    return _check("swin_wattn_test_proj", load().swin_wattn_test_proj(
        h, _p(attn), B, H, W, _p(Wproj), _p(bproj), _p(out), _stream(stream)))


def swin_wattn_test_gemm(A, Bw, bias, D, swizzle_bytes=128, stream=None):
    rows, K = A.shape
    N = Bw.shape[0]
    return _check("swin_wattn_test_gemm", load().swin_wattn_test_gemm(
        _p(A), _p(Bw), _p(bias), _p(D), rows, N, K, swizzle_bytes, _stream(stream)))


def swin_wattn_test_corrupt_workspace(h, side):
    return _check("swin_wattn_test_corrupt_workspace", load().swin_wattn_test_corrupt_workspace(h, side))


def swin_wattn_test_watchdog(h, stream=None):
    return _check("swin_wattn_test_watchdog", load().swin_wattn_test_watchdog(h, _stream(stream)))


# ---- swin_block.h -------------------------------------------------------------

def swin_block_create(C, heads, M, shift, mode, mlp_ratio=4):
    h = ctypes.c_void_p()
    _check("swin_block_create", load().swin_block_create(ctypes.byref(h), C, heads, M, shift, mode, mlp_ratio))
    return h


def swin_block_destroy(h):
    return _check("swin_block_destroy", load().swin_block_destroy(h))


def swin_block_forward(h, x, params, out, stream=None):
    """params: dict with the swin_block_params fields (tensors or None)."""
    B, H, W, _ = x.shape
    bp = BlockParams(*[(_p(params.get(n)).value if params.get(n) is not None else None)
                       for n in BLOCK_PARAM_FIELDS])
    return _check("swin_block_forward", load().swin_block_forward(
        h, _p(x), B, H, W, ctypes.cast(ctypes.byref(bp), ctypes.c_void_p), _p(out), _stream(stream)))


def swin_block_last_launches(h):
    return load().swin_block_last_launches(h)


def swin_block_set_option(h, option, value):
    return _check("swin_block_set_option", load().swin_block_set_option(h, option, int(value)))


def swin_block_sync_status(h, stream=None):
    return _check("swin_block_sync_status", load().swin_block_sync_status(h, _stream(stream)))


def swin_block_test_layernorm(a, b, gamma, beta, out_sum, out_ln, flags, stream=None):
    rows, C = a.shape[0], a.shape[-1]
    return _check("swin_block_test_layernorm", load().swin_block_test_layernorm(
        _p(a), _p(b), _p(gamma), _p(beta), _p(out_sum), _p(out_ln), rows, C, flags, _stream(stream)))


def swin_stage_norm(x, gamma, beta, out, stream=None):
    """out = LN(x) over the last axis of x [..., C] (the extra LayerNorm of a V2
    stage); out may be x."""
    C = x.shape[-1]
    return _check("swin_stage_norm", load().swin_stage_norm(
        _p(x), x.numel() // C, C, _p(gamma), _p(beta), _p(out), _stream(stream)))


def swin_merge_create(C):
    h = ctypes.c_void_p()
    _check("swin_merge_create", load().swin_merge_create(ctypes.byref(h), C))
    return h


def swin_merge_destroy(h):
    return _check("swin_merge_destroy", load().swin_merge_destroy(h))


def swin_merge_forward(h, x, gamma, beta, Wm, out, stream=None):
    B, H, W, _ = x.shape
    return _check("swin_merge_forward", load().swin_merge_forward(
        h, _p(x), B, H, W, _p(gamma), _p(beta), _p(Wm), _p(out), _stream(stream)))


# ---- swin_rms.h ------------------------------------------------------------------

_BF, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(name, t, dtype, shape):
    if t.dtype != dtype:
        raise ValueError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be of shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must be on the current CUDA device" % name)


def _arg_python(name, t, dtype, shape, dev):
    """Pointer of a required argument, checked: dtype, shape, contiguous, on
    device dev."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _refuse(name, t, dtype, shape)
    return t.data_ptr()


def _rows_python(h, x, dtype, name):
    """rows, shape, device and pointer of the call's tokens x [..., C] (h: the
    handle, for C channels), checked: dtype, contiguous, on the current device."""
    shape = x.shape
    C = shape[-1]
    if C != h.C:
        raise ValueError("the handle is for C = %d, not %d" % (h.C, C))
    dev = x.get_device()
    if x.dtype is not dtype or dev < 0 or dev != _current_device() or not x.is_contiguous():
        _refuse(name, x, dtype, shape)
    rows = x.numel() // C
    if rows > 0x7fffffff:   # (the C side's int would wrap)
        raise ValueError("%s has %d rows, more than 2^31 - 1" % (name, rows))
    return rows, shape, dev, x.data_ptr()


_arg, _rows = _arg_python, _rows_python


def _check_natively():
    """Puts arguments.cpp's forms of _arg and _rows in their places: the same checks
    of a plain tensor in a tenth of the time; anything else goes to the functions
    above, which stay where the module is not built or is another PyTorch's.  (Under
    load()'s lock.)"""
    global _arg, _rows
    try:
        from . import _arguments
    except ImportError:
        return
    if getattr(_arguments, "torch_version", None) != str(torch.__version__):
        return
    _arguments.setup(torch.Tensor, torch.nn.Parameter, _BF, _F32, _E4M3, _arg_python, _rows_python, _current_device)
    _arg, _rows = _arguments.arg, _arguments.rows


def _stream_on(stream, dev):
    """Raw stream of a call: the given one, or the current one of device dev."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def swin_block_rms_create(C, eps=1e-6):
    h = ctypes.c_void_p()
    _check("swin_block_rms_create", load().swin_block_rms_create(ctypes.byref(h), C, eps))
    h.C, h.vec = C, (C,)
    return h


def swin_block_rms_destroy(h):
    return _check("swin_block_rms_destroy", load().swin_block_rms_destroy(h))


def swin_block_rms_last_launches(h):
    return load().swin_block_rms_last_launches(h)


def swin_block_rms_forward(h, x, gamma, out, residual=None, out_sum=None, stream=None):
    """out = RMS norm of x + residual over the last axis of x [..., C]; out_sum
    receives the sum."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    rc = (_lib or load()).swin_block_rms_forward(
        h, px, None if residual is None else _arg("residual", residual, _BF, shape, dev), rows,
        _arg("gamma", gamma, _BF, h.vec, dev), None if out_sum is None else _arg("out_sum", out_sum, _BF, shape, dev),
        _arg("out", out, _BF, shape, dev), _stream_on(stream, dev))
    return rc and _check("swin_block_rms_forward", rc)


def swin_block_rms_forward_q8(h, x, gamma, out8, scales, residual=None, out_sum=None, stream=None):
    """The same in e4m3 codes out8 [..., C] with one fp32 scale a row."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    rc = (_lib or load()).swin_block_rms_forward_q8(
        h, px, None if residual is None else _arg("residual", residual, _BF, shape, dev), rows,
        _arg("gamma", gamma, _BF, h.vec, dev), None if out_sum is None else _arg("out_sum", out_sum, _BF, shape, dev),
        _arg("out8", out8, _E4M3, shape, dev), _arg("scales", scales, _F32, shape[:-1], dev), _stream_on(stream, dev))
    return rc and _check("swin_block_rms_forward_q8", rc)


def swin_block_rms_backward(h, s, gamma, dy, dx, dgamma, dsum=None, stream=None):
    """dx and dgamma from s [..., C] (the forward's out_sum, or x), dy and the
    gradient dsum that reaches the sum past the norm."""
    rows, shape, dev, ps = _rows(h, s, _BF, "s")
    rc = (_lib or load()).swin_block_rms_backward(
        h, ps, rows, _arg("gamma", gamma, _BF, h.vec, dev), _arg("dy", dy, _BF, shape, dev),
        None if dsum is None else _arg("dsum", dsum, _BF, shape, dev), _arg("dx", dx, _BF, shape, dev),
        _arg("dgamma", dgamma, _F32, h.vec, dev), _stream_on(stream, dev))
    return rc and _check("swin_block_rms_backward", rc)


# ---- swin_layernorm.h ---------------------------------------------------------------

def swin_block_layernorm_create(C, eps=1e-5):
    h = ctypes.c_void_p()
    _check("swin_block_layernorm_create", load().swin_block_layernorm_create(ctypes.byref(h), C, eps))
    h.C, h.vec = C, (C,)
    return h


def swin_block_layernorm_destroy(h):
    return _check("swin_block_layernorm_destroy", load().swin_block_layernorm_destroy(h))


def swin_block_layernorm_last_launches(h):
    return load().swin_block_layernorm_last_launches(h)


def swin_block_layernorm_forward(h, x, gamma, beta, out, residual=None, out_sum=None, stream=None):
    """out = layer norm of x + residual over the last axis of x [..., C]; out_sum
    receives the sum; beta may be None."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    rc = (_lib or load()).swin_block_layernorm_forward(
        h, px, None if residual is None else _arg("residual", residual, _BF, shape, dev), rows,
        _arg("gamma", gamma, _BF, h.vec, dev), None if beta is None else _arg("beta", beta, _BF, h.vec, dev),
        None if out_sum is None else _arg("out_sum", out_sum, _BF, shape, dev), _arg("out", out, _BF, shape, dev),
        _stream_on(stream, dev))
    return rc and _check("swin_block_layernorm_forward", rc)


def swin_block_layernorm_forward_post(h, x, gamma, beta, residual, out, stream=None):
    """out = residual + layer norm of x over the last axis of x [..., C]."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    rc = (_lib or load()).swin_block_layernorm_forward_post(
        h, px, _arg("residual", residual, _BF, shape, dev), rows, _arg("gamma", gamma, _BF, h.vec, dev),
        None if beta is None else _arg("beta", beta, _BF, h.vec, dev), _arg("out", out, _BF, shape, dev),
        _stream_on(stream, dev))
    return rc and _check("swin_block_layernorm_forward_post", rc)


def swin_block_layernorm_forward_q8(h, x, gamma, beta, out8, scales, residual=None, out_sum=None, stream=None):
    """swin_block_layernorm_forward in e4m3 codes out8 [..., C] with one fp32 scale
    a row."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    rc = (_lib or load()).swin_block_layernorm_forward_q8(
        h, px, None if residual is None else _arg("residual", residual, _BF, shape, dev), rows,
        _arg("gamma", gamma, _BF, h.vec, dev), None if beta is None else _arg("beta", beta, _BF, h.vec, dev),
        None if out_sum is None else _arg("out_sum", out_sum, _BF, shape, dev), _arg("out8", out8, _E4M3, shape, dev),
        _arg("scales", scales, _F32, shape[:-1], dev), _stream_on(stream, dev))
    return rc and _check("swin_block_layernorm_forward_q8", rc)


def swin_block_layernorm_backward(h, s, gamma, dy, dx, dgamma, dbeta=None, dsum=None, stream=None):
    """dx, dgamma and (where not None) dbeta from s [..., C] (the forward's out_sum,
    or x), dy and the gradient dsum that reaches the sum past the norm."""
    rows, shape, dev, ps = _rows(h, s, _BF, "s")
    rc = (_lib or load()).swin_block_layernorm_backward(
        h, ps, rows, _arg("gamma", gamma, _BF, h.vec, dev), _arg("dy", dy, _BF, shape, dev),
        None if dsum is None else _arg("dsum", dsum, _BF, shape, dev), _arg("dx", dx, _BF, shape, dev),
        _arg("dgamma", dgamma, _F32, h.vec, dev), None if dbeta is None else _arg("dbeta", dbeta, _F32, h.vec, dev),
        _stream_on(stream, dev))
    return rc and _check("swin_block_layernorm_backward", rc)


# ---- swin_gated.h ------------------------------------------------------------------

class GatedParams(ctypes.Structure):
    """swin_block_gated_params, field for field (also its gradients' struct)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("Wg", "bg", "Wu", "bu", "Wd", "bd")]


class GatedParamsQ8(ctypes.Structure):
    """swin_block_gated_params_q8, field for field."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("Wg8", "sg", "bg", "Wu8", "su", "bu", "Wd", "bd")]


def _bias(name, t, shape, dev):
    return None if t is None else _arg(name, t, _BF, shape, dev)


def _gated_params(h, p, dev):
    """The parameters' checked pointers, in the struct."""
    get = p.get
    return GatedParams(_arg("Wg", p["Wg"], _BF, h.wide, dev), _bias("bg", get("bg"), h.hidden, dev),
                       _arg("Wu", p["Wu"], _BF, h.wide, dev), _bias("bu", get("bu"), h.hidden, dev),
                       _arg("Wd", p["Wd"], _BF, h.down, dev), _bias("bd", get("bd"), h.vec, dev))


def swin_block_gated_create(C, F, act=BLOCK_GATED_SILU):
    h = ctypes.c_void_p()
    _check("swin_block_gated_create", load().swin_block_gated_create(ctypes.byref(h), C, F, act))
    h.C, h.F, h.vec, h.hidden, h.wide, h.down = C, F, (C,), (F,), (F, C), (C, F)
    return h


def swin_block_gated_destroy(h):
    return _check("swin_block_gated_destroy", load().swin_block_gated_destroy(h))


def swin_block_gated_last_launches(h):
    return load().swin_block_gated_last_launches(h)


def swin_block_gated_sync_status(h, stream=None):
    return _check("swin_block_gated_sync_status", load().swin_block_gated_sync_status(h, _stream(stream)))


def swin_block_gated_forward(h, x, params, out, residual=None, stream=None):
    """out = residual + (act(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd for x [..., C];
    params: dict with Wg, bg, Wu, bu, Wd, bd (biases may be None)."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    p = _gated_params(h, params, dev)
    rc = (_lib or load()).swin_block_gated_forward(
        h, px, rows, ctypes.addressof(p), None if residual is None else _arg("residual", residual, _BF, shape, dev),
        _arg("out", out, _BF, shape, dev), _stream_on(stream, dev))
    return rc and _check("swin_block_gated_forward", rc)


def swin_block_gated_forward_q8(h, x8, sx, params, out, residual=None, stream=None):
    """The same from e4m3 x8 [..., C] with scales sx [...]; params: dict with Wg8,
    sg, bg, Wu8, su, bu, Wd, bd (biases may be None)."""
    rows, shape, dev, px = _rows(h, x8, _E4M3, "x8")
    get = params.get
    p = GatedParamsQ8(_arg("Wg8", params["Wg8"], _E4M3, h.wide, dev), _arg("sg", params["sg"], _F32, h.hidden, dev),
                      _bias("bg", get("bg"), h.hidden, dev), _arg("Wu8", params["Wu8"], _E4M3, h.wide, dev),
                      _arg("su", params["su"], _F32, h.hidden, dev), _bias("bu", get("bu"), h.hidden, dev),
                      _arg("Wd", params["Wd"], _BF, h.down, dev), _bias("bd", get("bd"), h.vec, dev))
    rc = (_lib or load()).swin_block_gated_forward_q8(
        h, px, _arg("sx", sx, _F32, shape[:-1], dev), rows, ctypes.addressof(p),
        None if residual is None else _arg("residual", residual, _BF, shape, dev), _arg("out", out, _BF, shape, dev),
        _stream_on(stream, dev))
    return rc and _check("swin_block_gated_forward_q8", rc)


def swin_block_gated_backward(h, x, params, dy, dx, grads, stream=None):
    """Gradients of the bf16 form: dx and, in the tensors of dict grads, dWg, dWu,
    dWd and (where not None) dbg, dbu, dbd, all bf16."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    p = _gated_params(h, params, dev)
    get = grads.get
    g = GatedParams(_arg("dWg", grads["dWg"], _BF, h.wide, dev), _bias("dbg", get("dbg"), h.hidden, dev),
                    _arg("dWu", grads["dWu"], _BF, h.wide, dev), _bias("dbu", get("dbu"), h.hidden, dev),
                    _arg("dWd", grads["dWd"], _BF, h.down, dev), _bias("dbd", get("dbd"), h.vec, dev))
    rc = (_lib or load()).swin_block_gated_backward(
        h, px, rows, ctypes.addressof(p), _arg("dy", dy, _BF, shape, dev), _arg("dx", dx, _BF, shape, dev),
        ctypes.addressof(g), _stream_on(stream, dev))
    return rc and _check("swin_block_gated_backward", rc)


def swin_block_gated_test_stall(h, x, params, wait_limit_us, stream=None):
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    p = _gated_params(h, params, dev)
    return _check("swin_block_gated_test_stall", load().swin_block_gated_test_stall(
        h, px, rows, ctypes.addressof(p), int(wait_limit_us), _stream_on(stream, dev)))


def swin_block_gated_test_corrupt_workspace(h, side):
    return _check("swin_block_gated_test_corrupt_workspace", load().swin_block_gated_test_corrupt_workspace(h, side))


def swin_block_gated_test_last_use(stages, issued, k):
    stage, parity = ctypes.c_int(), ctypes.c_int()
    _check("swin_block_gated_test_last_use", load().swin_block_gated_test_last_use(
        stages, issued, k, ctypes.addressof(stage), ctypes.addressof(parity)))
    return stage.value, parity.value


def swin_block_gated_test_plan(C, F, rows, which):
    plan = (ctypes.c_int * 6)()
    _check("swin_block_gated_test_plan", load().swin_block_gated_test_plan(C, F, rows, which, ctypes.addressof(plan)))
    return tuple(plan)


# ---- swin_linear.h -----------------------------------------------------------------

def swin_block_linear_create(C, N, act=BLOCK_LINEAR_NONE):
    h = ctypes.c_void_p()
    _check("swin_block_linear_create", load().swin_block_linear_create(ctypes.byref(h), C, N, act))
    h.C, h.N, h.vec, h.weight = C, N, (N,), (N, C)
    return h


def swin_block_linear_destroy(h):
    return _check("swin_block_linear_destroy", load().swin_block_linear_destroy(h))


def swin_block_linear_last_launches(h):
    return load().swin_block_linear_last_launches(h)


def swin_block_linear_sync_status(h, stream=None):
    return _check("swin_block_linear_sync_status", load().swin_block_linear_sync_status(h, _stream(stream)))


def swin_block_linear_forward(h, x, W, b, out, residual=None, z=None, stream=None):
    """out = residual + act(x W^T + b) for x [..., C], W [N, C]; b may be None; z
    receives the value before the activation."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    shape = shape[:-1] + h.vec
    rc = (_lib or load()).swin_block_linear_forward(
        h, px, rows, _arg("W", W, _BF, h.weight, dev), _bias("b", b, h.vec, dev), _bias("residual", residual, shape, dev),
        _bias("z", z, shape, dev), _arg("out", out, _BF, shape, dev), _stream_on(stream, dev))
    return rc and _check("swin_block_linear_forward", rc)


def swin_block_linear_forward_q8(h, x8, sx, W8, sw, b, out, residual=None, stream=None):
    """The same from e4m3 x8 [..., C] with scales sx [...] and W8 [N, C] with scales
    sw [N]."""
    rows, shape, dev, px = _rows(h, x8, _E4M3, "x8")
    scales, shape = shape[:-1], shape[:-1] + h.vec
    rc = (_lib or load()).swin_block_linear_forward_q8(
        h, px, _arg("sx", sx, _F32, scales, dev), rows, _arg("W8", W8, _E4M3, h.weight, dev),
        _arg("sw", sw, _F32, h.vec, dev), _bias("b", b, h.vec, dev), _bias("residual", residual, shape, dev),
        _arg("out", out, _BF, shape, dev), _stream_on(stream, dev))
    return rc and _check("swin_block_linear_forward_q8", rc)


def swin_block_linear_backward(h, x, W, dy, dx, dW, db=None, z=None, stream=None):
    """dx [..., C], dW [N, C] and db [N] (bf16; None: not computed) from x, W, dy [...,
    N] and, with an activation, the forward's z."""
    rows, shape, dev, px = _rows(h, x, _BF, "x")
    wide = shape[:-1] + h.vec
    rc = (_lib or load()).swin_block_linear_backward(
        h, px, rows, _arg("W", W, _BF, h.weight, dev), _bias("z", z, wide, dev), _arg("dy", dy, _BF, wide, dev),
        _bias("dx", dx, shape, dev), _bias("dW", dW, h.weight, dev), _bias("db", db, h.vec, dev),
        _stream_on(stream, dev))
    return rc and _check("swin_block_linear_backward", rc)


def swin_block_linear_test_plan(C, N, rows, which):
    plan = (ctypes.c_int * 6)()
    _check("swin_block_linear_test_plan",
           load().swin_block_linear_test_plan(C, N, rows, which, ctypes.addressof(plan)))
    return tuple(plan)


def swin_block_linear_test_backward_plan(C, N, rows, act, which):
    """Who finishes what in a backward for the gradients which (BLOCK_LINEAR_GRAD_*)."""
    plan = (ctypes.c_int * 9)()
    _check("swin_block_linear_test_backward_plan",
           load().swin_block_linear_test_backward_plan(C, N, rows, act, which, ctypes.addressof(plan)))
    return dict(zip(("few", "side", "direct", "dx_adds", "slices", "held", "through", "dw_cut", "dx_cut"), plan))


def swin_block_linear_test_clusters_of(device, split, alone, answer):
    return load().swin_block_linear_test_clusters_of(device, split, int(alone), answer)


def swin_block_linear_test_corrupt_workspace(h, side):
    return _check("swin_block_linear_test_corrupt_workspace", load().swin_block_linear_test_corrupt_workspace(h, side))
