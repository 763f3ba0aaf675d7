"""ctypes binding of libvocoder.so (include/vocoder.h), with the same entry-point names.

Argument marshalling only: every step of the decode runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  If the compiled library
is missing this module raises instead of falling back to anything else; build
it with ``python -m dac_vocoder_decode_gb300.build``.
"""
from __future__ import annotations

import ctypes
import os
import warnings
from typing import List, Optional, Sequence

import numpy as np

from . import build as _build

VOC_ABI_VERSION = 5
VOC_OK = 0
VOC_INVALID_ARG = -1
VOC_UNSUPPORTED = -2
VOC_CUDA_ERROR = -3
VOC_OOM = -4
VOC_WORKSPACE_TOO_SMALL = -5
VOC_NONFINITE = -6
VOC_CANCELLED = -7
VOC_DEVICE_TIMEOUT = -8
VOC_PAD_SYMMETRIC = 0
VOC_PAD_CAUSAL = 1
VOC_PREC_BF16X3 = 0
VOC_PREC_F16W = 1
VOC_PREC_BF16W = 2
VOC_SNAKE = 0
VOC_SNAKE_BETA = 1
VOC_FLAG_CHECK_FINITE = 1
VOC_FLAG_SYNC = 2
VOC_FLAG_PROFILE = 4
VOC_LM_BF16 = 0
VOC_LM_F16 = 1
VOC_LM_F32 = 2
VOC_LM_RMS = 0
VOC_LM_NONE = 1
VOC_LM_GATED = 2
VOC_LM_BLOCK = 64

STATUS_NAMES = {0: "VOC_OK", -1: "VOC_INVALID_ARG", -2: "VOC_UNSUPPORTED", -3: "VOC_CUDA_ERROR",
                -4: "VOC_OOM", -5: "VOC_WORKSPACE_TOO_SMALL", -6: "VOC_NONFINITE",
                -7: "VOC_CANCELLED", -8: "VOC_DEVICE_TIMEOUT"}

EXPORTED = [
    "vocoder_abi_version", "vocoder_param_count", "vocoder_param_shape",
    "vocoder_fold_weight_norm", "vocoder_create", "vocoder_hop", "vocoder_workspace_bytes",
    "vocoder_workspace_bytes_host", "vocoder_decode", "vocoder_decode_host",
    "vocoder_decode_static",
    "vocoder_stitched_length", "vocoder_stitch", "vocoder_op_conv1d",
    "vocoder_op_conv_transpose1d", "vocoder_op_residual_unit", "vocoder_launches_per_decode",
    "vocoder_profile_count",
    "vocoder_profile_entry", "vocoder_profile_impl_bytes", "vocoder_last_error",
    "vocoder_destroy", "vocoder_set_cancel_flag", "vocoder_set_wait_budget",
    "vocoder_debug_fail_allocation", "vocoder_debug_live_allocations",
    "vocoder_stream_create", "vocoder_stream_decode", "vocoder_stream_reset",
    "vocoder_stream_destroy", "vocoder_wav_bytes", "vocoder_wav_scratch_bytes",
    "vocoder_encode_wav",
    "vocoder_encoder_param_count", "vocoder_encoder_param_shape", "vocoder_encoder_create",
    "vocoder_encoder_hop", "vocoder_encoder_workspace_bytes", "vocoder_encode",
    "vocoder_encoder_workspace_bytes_host", "vocoder_encode_host",
    "vocoder_encoder_launches", "vocoder_encoder_profile_count", "vocoder_encoder_profile_entry",
    "vocoder_encoder_profile_impl_bytes",
    "vocoder_encoder_last_error", "vocoder_encoder_destroy",
    "vocoder_lm_rows_fp8", "vocoder_lm_linear_fp8", "vocoder_lm_kv_append",
    "vocoder_lm_attention_ws_bytes", "vocoder_lm_attention",
]


class VocoderError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class VocDesc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int), ("latent_channels", ctypes.c_int),
                ("in_kernel", ctypes.c_int), ("channels0", ctypes.c_int),
                ("n_stages", ctypes.c_int), ("strides", ctypes.POINTER(ctypes.c_int)),
                ("widths", ctypes.POINTER(ctypes.c_int)), ("n_dilations", ctypes.c_int),
                ("dilations", ctypes.POINTER(ctypes.c_int)), ("res_kernel", ctypes.c_int),
                ("out_kernel", ctypes.c_int), ("out_channels", ctypes.c_int),
                ("padding", ctypes.c_int), ("precision", ctypes.c_int),
                ("fuse_max_channels", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("in_proj_channels", ctypes.c_int), ("snake", ctypes.c_int)]


class VocEncDesc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int), ("in_channels", ctypes.c_int),
                ("channels0", ctypes.c_int), ("in_kernel", ctypes.c_int),
                ("n_stages", ctypes.c_int), ("strides", ctypes.POINTER(ctypes.c_int)),
                ("widths", ctypes.POINTER(ctypes.c_int)), ("n_dilations", ctypes.c_int),
                ("dilations", ctypes.POINTER(ctypes.c_int)), ("res_kernel", ctypes.c_int),
                ("out_kernel", ctypes.c_int), ("latent_channels", ctypes.c_int),
                ("precision", ctypes.c_int), ("snake", ctypes.c_int)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library():
    """Load libvocoder.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m dac_vocoder_decode_gb300.build` (nvcc, sm_103a)")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    I = ctypes.c_int
    F = ctypes.POINTER(ctypes.c_float)
    lib.vocoder_abi_version.restype = I
    lib.vocoder_abi_version.argtypes = []
    lib.vocoder_param_count.restype = I
    lib.vocoder_param_count.argtypes = [ctypes.POINTER(VocDesc)]
    lib.vocoder_param_shape.restype = I
    lib.vocoder_param_shape.argtypes = [ctypes.POINTER(VocDesc), I, ctypes.POINTER(I),
                                        ctypes.POINTER(I)]
    lib.vocoder_fold_weight_norm.restype = I
    lib.vocoder_fold_weight_norm.argtypes = [F, F, I, ctypes.c_longlong, F]
    lib.vocoder_create.restype = I
    lib.vocoder_create.argtypes = [ctypes.POINTER(VocDesc), ctypes.POINTER(F), I,
                                   ctypes.POINTER(P)]
    lib.vocoder_hop.restype = ctypes.c_longlong
    lib.vocoder_hop.argtypes = [P]
    lib.vocoder_workspace_bytes.restype = ctypes.c_size_t
    lib.vocoder_workspace_bytes.argtypes = [P, I, I]
    lib.vocoder_workspace_bytes_host.restype = ctypes.c_size_t
    lib.vocoder_workspace_bytes_host.argtypes = [P, I, I]
    lib.vocoder_decode.restype = I
    lib.vocoder_decode.argtypes = [P, P, I, I, P, P, ctypes.c_size_t, P, ctypes.c_uint]
    lib.vocoder_decode_host.restype = I
    lib.vocoder_decode_host.argtypes = [P, P, I, I, P, P, ctypes.c_size_t, P, ctypes.c_uint]
    lib.vocoder_decode_static.restype = I
    lib.vocoder_decode_static.argtypes = [P, P, I, I, P, P, ctypes.c_uint]
    lib.vocoder_stitched_length.restype = ctypes.c_longlong
    lib.vocoder_stitched_length.argtypes = [I, I, I, I, I]
    lib.vocoder_stitch.restype = I
    lib.vocoder_stitch.argtypes = [P, I, I, I, I, I, I, P, P]
    lib.vocoder_op_conv1d.restype = I
    lib.vocoder_op_conv1d.argtypes = [P, I, I, I, F, F, I, I, I, I, F, P, P]
    lib.vocoder_op_conv_transpose1d.restype = I
    lib.vocoder_op_conv_transpose1d.argtypes = [P, I, I, I, F, F, I, I, I, F, P, P]
    lib.vocoder_op_residual_unit.restype = I
    lib.vocoder_op_residual_unit.argtypes = [P, I, I, I, F, F, F, I, I, F, F, F, I, P, P]
    lib.vocoder_launches_per_decode.restype = I
    lib.vocoder_launches_per_decode.argtypes = [P, I, I]
    lib.vocoder_profile_count.restype = I
    lib.vocoder_profile_count.argtypes = [P]
    lib.vocoder_profile_entry.restype = I
    lib.vocoder_profile_entry.argtypes = [P, I, ctypes.POINTER(ctypes.c_char_p),
                                          ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(ctypes.c_double)]
    lib.vocoder_profile_impl_bytes.restype = I
    lib.vocoder_profile_impl_bytes.argtypes = [P, I, ctypes.POINTER(ctypes.c_double)]
    lib.vocoder_last_error.restype = ctypes.c_char_p
    lib.vocoder_last_error.argtypes = [P]
    lib.vocoder_destroy.restype = None
    lib.vocoder_destroy.argtypes = [P]
    lib.vocoder_set_cancel_flag.restype = I
    lib.vocoder_set_cancel_flag.argtypes = [P, P]
    lib.vocoder_set_wait_budget.restype = I
    lib.vocoder_set_wait_budget.argtypes = [P, ctypes.c_longlong]
    lib.vocoder_debug_fail_allocation.restype = None
    lib.vocoder_debug_fail_allocation.argtypes = [I]
    lib.vocoder_debug_live_allocations.restype = ctypes.c_longlong
    lib.vocoder_debug_live_allocations.argtypes = []
    lib.vocoder_wav_bytes.restype = ctypes.c_size_t
    lib.vocoder_wav_bytes.argtypes = [I, ctypes.c_longlong, I]
    lib.vocoder_wav_scratch_bytes.restype = ctypes.c_size_t
    lib.vocoder_wav_scratch_bytes.argtypes = []
    lib.vocoder_encode_wav.restype = I
    lib.vocoder_encode_wav.argtypes = [P, I, ctypes.c_longlong, I, I, I, P, ctypes.c_size_t, P,
                                       ctypes.c_size_t, P]
    lib.vocoder_stream_create.restype = I
    lib.vocoder_stream_create.argtypes = [P, I, I, ctypes.POINTER(P)]
    lib.vocoder_stream_decode.restype = I
    lib.vocoder_stream_decode.argtypes = [P, P, I, P, P, ctypes.c_uint]
    lib.vocoder_stream_reset.restype = I
    lib.vocoder_stream_reset.argtypes = [P, P]
    lib.vocoder_stream_destroy.restype = None
    lib.vocoder_stream_destroy.argtypes = [P]
    ED = ctypes.POINTER(VocEncDesc)
    lib.vocoder_encoder_param_count.restype = I
    lib.vocoder_encoder_param_count.argtypes = [ED]
    lib.vocoder_encoder_param_shape.restype = I
    lib.vocoder_encoder_param_shape.argtypes = [ED, I, ctypes.POINTER(I), ctypes.POINTER(I)]
    lib.vocoder_encoder_create.restype = I
    lib.vocoder_encoder_create.argtypes = [ED, ctypes.POINTER(F), I, ctypes.POINTER(P)]
    lib.vocoder_encoder_hop.restype = ctypes.c_longlong
    lib.vocoder_encoder_hop.argtypes = [P]
    lib.vocoder_encoder_workspace_bytes.restype = ctypes.c_size_t
    lib.vocoder_encoder_workspace_bytes.argtypes = [P, I, ctypes.c_longlong]
    lib.vocoder_encode.restype = I
    lib.vocoder_encode.argtypes = [P, P, I, ctypes.c_longlong, P, P, ctypes.c_size_t, P,
                                   ctypes.c_uint]
    lib.vocoder_encoder_workspace_bytes_host.restype = ctypes.c_size_t
    lib.vocoder_encoder_workspace_bytes_host.argtypes = [P, I, ctypes.c_longlong]
    lib.vocoder_encode_host.restype = I
    lib.vocoder_encode_host.argtypes = [P, P, I, ctypes.c_longlong, P, P, ctypes.c_size_t, P,
                                        ctypes.c_uint]
    lib.vocoder_encoder_launches.restype = I
    lib.vocoder_encoder_launches.argtypes = [P, I, ctypes.c_longlong]
    lib.vocoder_encoder_profile_count.restype = I
    lib.vocoder_encoder_profile_count.argtypes = [P]
    lib.vocoder_encoder_profile_entry.restype = I
    lib.vocoder_encoder_profile_entry.argtypes = [P, I, ctypes.POINTER(ctypes.c_char_p),
                                                  ctypes.POINTER(ctypes.c_double),
                                                  ctypes.POINTER(ctypes.c_double),
                                                  ctypes.POINTER(ctypes.c_double)]
    lib.vocoder_encoder_profile_impl_bytes.restype = I
    lib.vocoder_encoder_profile_impl_bytes.argtypes = [P, I, ctypes.POINTER(ctypes.c_double)]
    lib.vocoder_encoder_last_error.restype = ctypes.c_char_p
    lib.vocoder_encoder_last_error.argtypes = [P]
    lib.vocoder_encoder_destroy.restype = None
    lib.vocoder_encoder_destroy.argtypes = [P]
    L, FL, U, Z = ctypes.c_longlong, ctypes.c_float, ctypes.c_uint, ctypes.c_size_t
    lib.vocoder_lm_rows_fp8.restype = I
    lib.vocoder_lm_rows_fp8.argtypes = [P, L, P, L, P, I, I, L, I, FL, P, L, P, L, P, P, U]
    lib.vocoder_lm_linear_fp8.restype = I
    lib.vocoder_lm_linear_fp8.argtypes = [P, L, P, P, L, P, P, I, I, I, P, L, I, P, U]
    lib.vocoder_lm_kv_append.restype = I
    lib.vocoder_lm_kv_append.argtypes = [P, P, P, P, I, I, I, P, L, L, P, L, L, I, P, L, I, P, P,
                                         I, I, I, P, U]
    lib.vocoder_lm_attention_ws_bytes.restype = Z
    lib.vocoder_lm_attention_ws_bytes.argtypes = [I] * 7
    lib.vocoder_lm_attention.restype = I
    lib.vocoder_lm_attention.argtypes = [P, L, L, I, I, P, P, P, P, I, I, I, P, L, I, P, P, I, I,
                                         I, I, FL, I, I, P, L, L, P, Z, P, U]
    _lib = lib
    return lib


def _check(status: int, handle=None):
    if status != VOC_OK:
        msg = load_library().vocoder_last_error(handle)
        raise VocoderError(status, msg.decode() if msg else "")


def _fptr(a: Optional[np.ndarray]):
    if a is None:
        return ctypes.cast(None, ctypes.POINTER(ctypes.c_float))
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    if hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def make_desc(arch, fuse_max_channels: int = 0, cta_pair: int = 0,
              precision: int = VOC_PREC_BF16X3) -> VocDesc:
    """voc_desc for an Arch (layer shapes from workloads.Arch or any object with the same fields)."""
    strides = (ctypes.c_int * len(arch.strides))(*arch.strides)
    widths = (ctypes.c_int * len(arch.widths))(*arch.widths)
    dils = (ctypes.c_int * len(arch.dilations))(*arch.dilations)
    d = VocDesc(VOC_ABI_VERSION, arch.latent_channels, arch.in_kernel, arch.channels0,
                len(arch.strides), strides, widths, len(arch.dilations), dils, arch.res_kernel,
                arch.out_kernel, 1, arch.padding, precision, fuse_max_channels, cta_pair,
                getattr(arch, "in_proj_channels", 0),
                VOC_SNAKE_BETA if getattr(arch, "snake_beta", False) else VOC_SNAKE)
    d._keep = (strides, widths, dils)
    return d


# ------------------------------------------------------------------ entry points
def vocoder_abi_version() -> int:
    return load_library().vocoder_abi_version()


def vocoder_param_count(arch) -> int:
    return load_library().vocoder_param_count(ctypes.byref(make_desc(arch)))


def vocoder_param_shape(arch, index: int):
    dims = (ctypes.c_int * 3)()
    nd = ctypes.c_int()
    _check(load_library().vocoder_param_shape(ctypes.byref(make_desc(arch)), index, dims,
                                               ctypes.byref(nd)))
    return tuple(dims[i] for i in range(nd.value))


def vocoder_fold_weight_norm(g: np.ndarray, v: np.ndarray) -> np.ndarray:
    g = np.ascontiguousarray(g, dtype=np.float32)
    v = np.ascontiguousarray(v, dtype=np.float32)
    w = np.empty_like(v)
    rest = int(np.prod(v.shape[1:])) if v.ndim > 1 else 1
    _check(load_library().vocoder_fold_weight_norm(_fptr(g), _fptr(v), int(v.shape[0]), rest,
                                                    _fptr(w)))
    return w


def vocoder_create(arch, params: Sequence[Optional[np.ndarray]],
                   fuse_max_channels: int = 0, cta_pair: int = 0,
                   precision: int = VOC_PREC_BF16X3) -> ctypes.c_void_p:
    """params: folded fp32 arrays in the canonical order (None for a zero bias)."""
    lib = load_library()
    keep = [None if p is None else np.ascontiguousarray(p, dtype=np.float32) for p in params]
    arr = (ctypes.POINTER(ctypes.c_float) * len(keep))(*[_fptr(p) for p in keep])
    h = ctypes.c_void_p()
    _check(lib.vocoder_create(ctypes.byref(make_desc(arch, fuse_max_channels, cta_pair, precision)), arr,
                              len(keep),
                              ctypes.byref(h)))
    return h


def vocoder_destroy(h) -> None:
    load_library().vocoder_destroy(h)


def vocoder_hop(h) -> int:
    return int(load_library().vocoder_hop(h))


def vocoder_workspace_bytes(h, B: int, T: int) -> int:
    return int(load_library().vocoder_workspace_bytes(h, B, T))


def vocoder_workspace_bytes_host(h, B: int, T: int) -> int:
    return int(load_library().vocoder_workspace_bytes_host(h, B, T))


def vocoder_launches_per_decode(h, B: int, T: int) -> int:
    return int(load_library().vocoder_launches_per_decode(h, B, T))


def vocoder_decode(h, latent, audio, ws, stream=None, flags: int = 0) -> None:
    """latent [B,C,T] fp32 CUDA tensor -> audio [B,1,T*hop] fp32 CUDA tensor; ws uint8 CUDA tensor."""
    B, _, T = latent.shape
    _check(load_library().vocoder_decode(h, ctypes.c_void_p(latent.data_ptr()), B, T,
                                          ctypes.c_void_p(audio.data_ptr()),
                                          ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                          _stream_ptr(stream), flags), h)


def vocoder_decode_host(h, latent_host, audio_host, ws, stream=None, flags: int = 0) -> None:
    """Host (ideally pinned) CPU tensors in and out; copies happen inside the library."""
    B, _, T = latent_host.shape
    _check(load_library().vocoder_decode_host(h, ctypes.c_void_p(latent_host.data_ptr()), B, T,
                                               ctypes.c_void_p(audio_host.data_ptr()),
                                               ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                               _stream_ptr(stream), flags), h)


VOC_STATIC_WORKSPACE_BYTES = 64 << 20


def vocoder_decode_static(h, latent, audio, stream=None, flags: int = 0) -> None:
    """Decode with the library's built-in workspace array: no device allocation
    happens in this call (for callers that may not allocate while they run, such
    as real-time audio threads).  Calls that overlap on the GPU race on the array."""
    B, _, T = latent.shape
    _check(load_library().vocoder_decode_static(h, ctypes.c_void_p(latent.data_ptr()), B, T,
                                                 ctypes.c_void_p(audio.data_ptr()),
                                                 _stream_ptr(stream), flags), h)


def vocoder_stitched_length(n_win, win_frames, crop_left, crop_right, hop) -> int:
    return int(load_library().vocoder_stitched_length(n_win, win_frames, crop_left, crop_right,
                                                      hop))


def vocoder_stitch(decoded, n_win, n_sides, win_frames, crop_left, crop_right, hop, out,
                   stream=None) -> None:
    _check(load_library().vocoder_stitch(ctypes.c_void_p(decoded.data_ptr()), n_win, n_sides,
                                          win_frames, crop_left, crop_right, hop,
                                          ctypes.c_void_p(out.data_ptr()), _stream_ptr(stream)))


def vocoder_op_conv1d(x, w: np.ndarray, b: Optional[np.ndarray], dil: int, padding: int,
                      alpha: Optional[np.ndarray], y, stream=None) -> None:
    B, Cin, T = x.shape
    Cout, _, K = w.shape
    w = np.ascontiguousarray(w, dtype=np.float32)
    b = None if b is None else np.ascontiguousarray(b, dtype=np.float32)
    alpha = None if alpha is None else np.ascontiguousarray(alpha, dtype=np.float32)
    _check(load_library().vocoder_op_conv1d(ctypes.c_void_p(x.data_ptr()), B, Cin, T, _fptr(w),
                                             _fptr(b), Cout, K, dil, padding, _fptr(alpha),
                                             ctypes.c_void_p(y.data_ptr()), _stream_ptr(stream)))


def vocoder_op_conv_transpose1d(x, w: np.ndarray, b: Optional[np.ndarray], stride: int,
                                padding: int, alpha: Optional[np.ndarray], y,
                                stream=None) -> None:
    B, Cin, T = x.shape
    _, Cout, K = w.shape
    assert K == 2 * stride
    w = np.ascontiguousarray(w, dtype=np.float32)
    b = None if b is None else np.ascontiguousarray(b, dtype=np.float32)
    alpha = None if alpha is None else np.ascontiguousarray(alpha, dtype=np.float32)
    _check(load_library().vocoder_op_conv_transpose1d(
        ctypes.c_void_p(x.data_ptr()), B, Cin, T, _fptr(w), _fptr(b), Cout, stride, padding,
        _fptr(alpha), ctypes.c_void_p(y.data_ptr()), _stream_ptr(stream)))


def vocoder_op_residual_unit(x, alpha1: np.ndarray, w1: np.ndarray, b1: Optional[np.ndarray],
                             dil: int, alpha2: np.ndarray, w2: np.ndarray,
                             b2: Optional[np.ndarray], padding: int, y, stream=None) -> None:
    """y = x + conv2(Snake2(conv1(Snake1(x)) + b1)) + b2 on the decoder's kernels."""
    B, C, T = x.shape
    K = w1.shape[2]
    arrs = [np.ascontiguousarray(a, dtype=np.float32) if a is not None else None
            for a in (alpha1, w1, b1, alpha2, w2, b2)]
    _check(load_library().vocoder_op_residual_unit(
        ctypes.c_void_p(x.data_ptr()), B, C, T, _fptr(arrs[0]), _fptr(arrs[1]), _fptr(arrs[2]),
        K, dil, _fptr(arrs[3]), _fptr(arrs[4]), _fptr(arrs[5]), padding,
        ctypes.c_void_p(y.data_ptr()), _stream_ptr(stream)))


def vocoder_profile(h) -> List[dict]:
    """Per-kernel records of the last decode run with VOC_FLAG_PROFILE."""
    lib = load_library()
    out = []
    for i in range(lib.vocoder_profile_count(h)):
        name = ctypes.c_char_p()
        ms, fl, by = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
        _check(lib.vocoder_profile_entry(h, i, ctypes.byref(name), ctypes.byref(ms),
                                          ctypes.byref(fl), ctypes.byref(by)), h)
        ib = ctypes.c_double()
        _check(lib.vocoder_profile_impl_bytes(h, i, ctypes.byref(ib)), h)
        out.append(dict(name=name.value.decode(), ms=ms.value, flops=fl.value, bytes=by.value,
                        impl_bytes=ib.value))
    return out


def vocoder_set_cancel_flag(h, flag: Optional[ctypes.c_int]) -> None:
    """Register a host int (a ctypes.c_int the caller keeps alive) as the context's cancel
    flag; None removes it."""
    ptr = ctypes.cast(ctypes.pointer(flag), ctypes.c_void_p) if flag is not None else None
    _check(load_library().vocoder_set_cancel_flag(h, ptr), h)


def vocoder_set_wait_budget(h, cycles: int) -> None:
    _check(load_library().vocoder_set_wait_budget(h, int(cycles)), h)


def vocoder_debug_fail_allocation(n: int) -> None:
    load_library().vocoder_debug_fail_allocation(int(n))


def vocoder_debug_live_allocations() -> int:
    return int(load_library().vocoder_debug_live_allocations())


def vocoder_last_error(h=None) -> str:
    m = load_library().vocoder_last_error(h)
    return m.decode() if m else ""


# ------------------------------------------------------------------ convenience
def fold_params(params) -> list:
    """Raw canonical parameters (weight-norm g/v pairs and alphas) -> folded fp32
    arrays through the library's host fold (vocoder_fold_weight_norm)."""
    out = []
    for p in params:
        if hasattr(p, "g"):
            out.append(vocoder_fold_weight_norm(p.g, p.v))
            out.append(None if p.b is None else np.ascontiguousarray(p.b, dtype=np.float32))
        elif hasattr(p, "w"):  # a convolution stored without weight norm
            out.append(np.ascontiguousarray(p.w, dtype=np.float32))
            out.append(None if p.b is None else np.ascontiguousarray(p.b, dtype=np.float32))
        else:
            out.append(np.ascontiguousarray(p, dtype=np.float32))
    return out


def vocoder_stream_create(h, B: int, max_frames: int) -> ctypes.c_void_p:
    s = ctypes.c_void_p()
    _check(load_library().vocoder_stream_create(h, B, max_frames, ctypes.byref(s)), h)
    return s


def vocoder_stream_decode(h, s, latent, audio, stream=None, flags: int = 0) -> None:
    """latent [B, C_lat, frames] and audio [B, 1, frames*hop]: contiguous fp32 CUDA tensors."""
    frames = int(latent.shape[2])
    _check(load_library().vocoder_stream_decode(s, ctypes.c_void_p(latent.data_ptr()), frames,
                                                 ctypes.c_void_p(audio.data_ptr()),
                                                 _stream_ptr(stream), flags), h)


def vocoder_stream_reset(h, s, stream=None) -> None:
    _check(load_library().vocoder_stream_reset(s, _stream_ptr(stream)), h)


def vocoder_stream_destroy(s) -> None:
    load_library().vocoder_stream_destroy(s)


def vocoder_wav_bytes(n_ch: int, length: int, bits: int) -> int:
    return int(load_library().vocoder_wav_bytes(n_ch, length, bits))


def vocoder_wav_scratch_bytes() -> int:
    return int(load_library().vocoder_wav_scratch_bytes())


def vocoder_encode_wav(planar, sample_rate: int, bits: int, peak_clip: int, out, scratch=None,
                       stream=None) -> None:
    """planar: contiguous fp32 CUDA tensor [n_ch, len]; out: uint8 CUDA tensor of at least
    vocoder_wav_bytes bytes; scratch: uint8 CUDA tensor of vocoder_wav_scratch_bytes (16/24
    bits)."""
    n_ch, length = (1, int(planar.shape[0])) if planar.dim() == 1 else map(int, planar.shape)
    sp = ctypes.c_void_p(scratch.data_ptr()) if scratch is not None else None
    sb = scratch.numel() if scratch is not None else 0
    _check(load_library().vocoder_encode_wav(ctypes.c_void_p(planar.data_ptr()), n_ch, length,
                                              sample_rate, bits, peak_clip,
                                              ctypes.c_void_p(out.data_ptr()), out.numel(), sp,
                                              sb, _stream_ptr(stream)), None)


def encode_wav(planar, sample_rate: int, bits: int = 16, peak_clip: int = 0, stream=None):
    """Peak-normalise and encode planar [n_ch, len] device audio as a WAV file in a new uint8
    CUDA tensor (see vocoder_encode_wav in include/vocoder.h)."""
    import torch
    planar = planar.contiguous()
    n_ch, length = (1, planar.shape[0]) if planar.dim() == 1 else planar.shape
    size = vocoder_wav_bytes(int(n_ch), int(length), bits)
    if size == 0:
        raise VocoderError(-1, "bad WAV geometry")
    # 256 bytes of head room keep the scratch that follows the file 256-byte aligned
    off = (size + 255) // 256 * 256
    buf = torch.empty(off + vocoder_wav_scratch_bytes(), dtype=torch.uint8, device=planar.device)
    vocoder_encode_wav(planar, sample_rate, bits, peak_clip, buf[:size], buf[off:], stream)
    return buf[:size]


class VocoderStream:
    """Stateful chunk-by-chunk decoding of B sequences on a causal decoder (see
    vocoder_stream_create in include/vocoder.h)."""

    def __init__(self, voc: "Vocoder", B: int, max_frames: int):
        self.voc = voc
        self.B = B
        self.max_frames = max_frames
        self.handle = vocoder_stream_create(voc.handle, B, max_frames)

    def decode(self, latent, audio=None, stream=None, flags: int = 0):
        import torch
        if audio is None:
            audio = torch.empty((self.B, 1, latent.shape[2] * self.voc.hop), dtype=torch.float32,
                                device=latent.device)
        vocoder_stream_decode(self.voc.handle, self.handle, latent.contiguous(), audio, stream,
                              flags)
        return audio

    def reset(self, stream=None):
        vocoder_stream_reset(self.voc.handle, self.handle, stream)

    def close(self):
        if self.handle:
            vocoder_stream_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Vocoder:
    """A decoder on the current CUDA device (owns its library context)."""

    def __init__(self, arch, folded_params, fuse_max_channels: int = 0, cta_pair: int = 0,
                 precision: int = VOC_PREC_BF16X3):
        self.arch = arch
        self.handle = vocoder_create(arch, folded_params, fuse_max_channels, cta_pair, precision)
        self.hop = vocoder_hop(self.handle)

    def close(self):
        if self.handle:
            vocoder_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_bytes(self, B: int, T: int) -> int:
        return vocoder_workspace_bytes(self.handle, B, T)

    def alloc_workspace(self, B: int, T: int, host_io: bool = False):
        import torch
        n = (vocoder_workspace_bytes_host if host_io else vocoder_workspace_bytes)(self.handle, B, T)
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def decode(self, latent, ws=None, audio=None, stream=None, flags: int = 0):
        import torch
        B, _, T = latent.shape
        if ws is None:
            ws = self.alloc_workspace(B, T)
        if audio is None:
            audio = torch.empty((B, 1, T * self.hop), dtype=torch.float32, device=latent.device)
        vocoder_decode(self.handle, latent, audio, ws, stream, flags)
        return audio


# ------------------------------------------------------------------ mirror encoder
def _check_enc(status: int, handle=None):
    if status != VOC_OK:
        msg = load_library().vocoder_encoder_last_error(handle)
        raise VocoderError(status, msg.decode() if msg else "")


def make_enc_desc(arch, precision: int = VOC_PREC_BF16X3) -> VocEncDesc:
    """voc_enc_desc for an encoder architecture (workloads.EncArch or the same fields)."""
    strides = (ctypes.c_int * len(arch.strides))(*arch.strides)
    widths = (ctypes.c_int * len(arch.widths))(*arch.widths)
    dils = (ctypes.c_int * len(arch.dilations))(*arch.dilations)
    d = VocEncDesc(VOC_ABI_VERSION, arch.in_channels, arch.channels0, arch.in_kernel,
                   len(arch.strides), strides, widths, len(arch.dilations), dils,
                   arch.res_kernel, arch.out_kernel, arch.latent_channels, precision,
                   VOC_SNAKE_BETA if getattr(arch, "snake_beta", False) else VOC_SNAKE)
    d._keep = (strides, widths, dils)
    return d


def vocoder_encoder_param_count(arch) -> int:
    return load_library().vocoder_encoder_param_count(ctypes.byref(make_enc_desc(arch)))


def vocoder_encoder_param_shape(arch, index: int):
    dims = (ctypes.c_int * 3)()
    nd = ctypes.c_int()
    _check_enc(load_library().vocoder_encoder_param_shape(ctypes.byref(make_enc_desc(arch)), index,
                                                          dims, ctypes.byref(nd)))
    return tuple(dims[i] for i in range(nd.value))


def vocoder_encoder_create(arch, params: Sequence[Optional[np.ndarray]],
                           precision: int = VOC_PREC_BF16X3) -> ctypes.c_void_p:
    """params: folded fp32 arrays in the encoder's canonical order (None for a zero bias)."""
    keep = [None if p is None else np.ascontiguousarray(p, dtype=np.float32) for p in params]
    arr = (ctypes.POINTER(ctypes.c_float) * len(keep))(*[_fptr(p) for p in keep])
    h = ctypes.c_void_p()
    _check_enc(load_library().vocoder_encoder_create(ctypes.byref(make_enc_desc(arch, precision)),
                                                     arr, len(keep), ctypes.byref(h)))
    return h


def vocoder_encoder_destroy(h) -> None:
    load_library().vocoder_encoder_destroy(h)


def vocoder_encoder_hop(h) -> int:
    return int(load_library().vocoder_encoder_hop(h))


def vocoder_encoder_workspace_bytes(h, B: int, L: int) -> int:
    return int(load_library().vocoder_encoder_workspace_bytes(h, B, L))


def vocoder_encoder_workspace_bytes_host(h, B: int, L: int) -> int:
    return int(load_library().vocoder_encoder_workspace_bytes_host(h, B, L))


def vocoder_encode_host(h, audio_host, latent_host, ws, stream=None, flags: int = 0) -> None:
    """Host (ideally pinned) CPU tensors in and out; copies happen inside the library."""
    B, _, L = audio_host.shape
    _check_enc(load_library().vocoder_encode_host(h, ctypes.c_void_p(audio_host.data_ptr()), B, L,
                                                  ctypes.c_void_p(latent_host.data_ptr()),
                                                  ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                                  _stream_ptr(stream), flags), h)


def vocoder_encoder_launches(h, B: int, L: int) -> int:
    return int(load_library().vocoder_encoder_launches(h, B, L))


def vocoder_encode(h, audio, latent, ws, stream=None, flags: int = 0) -> None:
    """audio [B, C_in, L] fp32 CUDA tensor -> latent [B, C_lat, L / hop] fp32 CUDA tensor."""
    B, _, L = audio.shape
    _check_enc(load_library().vocoder_encode(h, ctypes.c_void_p(audio.data_ptr()), B, L,
                                             ctypes.c_void_p(latent.data_ptr()),
                                             ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                             _stream_ptr(stream), flags), h)


def vocoder_encoder_profile(h) -> List[dict]:
    """Per-kernel records of the last encode run with VOC_FLAG_PROFILE."""
    lib = load_library()
    out = []
    for i in range(lib.vocoder_encoder_profile_count(h)):
        name = ctypes.c_char_p()
        ms, fl, by = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
        _check_enc(lib.vocoder_encoder_profile_entry(h, i, ctypes.byref(name), ctypes.byref(ms),
                                                     ctypes.byref(fl), ctypes.byref(by)), h)
        ib = ctypes.c_double()
        _check_enc(lib.vocoder_encoder_profile_impl_bytes(h, i, ctypes.byref(ib)), h)
        out.append(dict(name=name.value.decode(), ms=ms.value, flops=fl.value, bytes=by.value,
                        impl_bytes=ib.value))
    return out


def vocoder_encoder_last_error(h=None) -> str:
    m = load_library().vocoder_encoder_last_error(h)
    return m.decode() if m else ""


class Encoder:
    """The mirror encoder on the current CUDA device (owns its library context)."""

    def __init__(self, arch, folded_params, precision: int = VOC_PREC_BF16X3):
        self.arch = arch
        self.handle = vocoder_encoder_create(arch, folded_params, precision)
        self.hop = vocoder_encoder_hop(self.handle)

    def close(self):
        if self.handle:
            vocoder_encoder_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_bytes(self, B: int, L: int) -> int:
        return vocoder_encoder_workspace_bytes(self.handle, B, L)

    def alloc_workspace(self, B: int, L: int, host_io: bool = False):
        import torch
        n = (vocoder_encoder_workspace_bytes_host if host_io else vocoder_encoder_workspace_bytes)(
            self.handle, B, L)
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def encode(self, audio, ws=None, latent=None, stream=None, flags: int = 0):
        import torch
        B, _, L = audio.shape
        if ws is None:
            ws = self.alloc_workspace(B, L)
        if latent is None:
            latent = torch.empty((B, self.arch.latent_channels, L // self.hop), dtype=torch.float32,
                                 device=audio.device)
        vocoder_encode(self.handle, audio.contiguous(), latent, ws, stream, flags)
        return latent


# ------------------------------------------------------------------ 8-bit operators
# One call of these is a few microseconds of host time beside kernels of the same length, so the
# checks below stay with what is cheap to ask of a tensor; the library checks the rest.
# The regular calls go through lm_torch (csrc/lm_torch.cpp), which marshals them in a fraction of
# that; it hands back None where something is unusual or wrong, and the code here takes over.
class _LM:
    """What the wrappers need of torch and the library, looked up with the first call."""
    ready = False
    fast = None


def _lm_compiled():
    """The compiled binding, or None where there is none for this Python and torch."""
    import importlib.machinery
    import importlib.util
    path = _build.torch_lib()
    if not os.path.exists(path):
        return None
    loader = importlib.machinery.ExtensionFileLoader("lm_torch", path)
    try:
        fast = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("lm_torch", path, loader=loader))
        loader.exec_module(fast)
    except (ImportError, OSError) as e:
        warnings.warn(f"{path} does not load ({e}); the 8-bit operators are marshalled in Python",
                      RuntimeWarning, stacklevel=2)
        return None
    fast.init(*(ctypes.cast(f, ctypes.c_void_p).value
                for f in (_LM.rows, _LM.linear, _LM.append, _LM.attention, _LM.attention_ws)))
    return fast


def _lm_setup():
    import torch
    lib = load_library()
    _LM.torch, _LM.empty = torch, torch.empty
    _LM.f8, _LM.f32, _LM.i32 = torch.float8_e4m3fn, torch.float32, torch.int32
    _LM.types = {torch.bfloat16: VOC_LM_BF16, torch.float16: VOC_LM_F16,
                 torch.float32: VOC_LM_F32}
    _LM.rows, _LM.linear = lib.vocoder_lm_rows_fp8, lib.vocoder_lm_linear_fp8
    _LM.append, _LM.attention = lib.vocoder_lm_kv_append, lib.vocoder_lm_attention
    _LM.attention_ws = lib.vocoder_lm_attention_ws_bytes
    # the current stream as an integer, without building a Stream object where torch allows it
    _LM.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                             lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _LM.fast = _lm_compiled()
    _LM.ready = True


def _bad(msg: str):
    return VocoderError(VOC_INVALID_ARG, msg)


def _lm_stream(dev, stream, made):
    """Raw stream.  Tensors `made` by the call belong to the current stream.  Another one of the
    caller's waits for what the current stream has in its queue, whose last reads of that memory may
    still be ahead, and keeps the tensors until its own work is done.  (With every output and the
    workspace given, nothing is made and nothing waits.)"""
    if stream is None:
        return _LM.raw_stream(dev)
    torch = _LM.torch
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    if stream.cuda_stream != _LM.raw_stream(dev):
        made = [t for t in made if t is not None]
        if made:
            stream.wait_stream(torch.cuda.current_stream(dev))
        for t in made:
            t.record_stream(stream)
    return stream.cuda_stream


def _lm_device(x):
    """Index of x's device, which has to be the current one."""
    dev = x.get_device()
    if dev < 0 or dev != _LM.torch.cuda.current_device():
        raise _bad(f"tensors must be on the current CUDA device, got {x.device}")
    return dev


def _rows_strides(t, name, rows, width, dtype, dev):
    """Row stride of a [rows, width] operand; that of a single row does not count."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != rows or shape[1] != width or t.dtype != dtype or \
            (stride[1] != 1 and width > 1) or t.get_device() != dev:
        raise _bad(f"{name} must be {dtype} [{rows}, {width}] with contiguous rows on x's device, "
                   f"got {t.dtype} {tuple(shape)} with strides {stride} on {t.device}")
    return stride[0] if rows > 1 else max(width, stride[0])


def _vector_ok(t, name, n, dtype, dev):
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or t.get_device() != dev or \
            (n > 1 and t.stride(0) != 1):
        raise _bad(f"{name} must be contiguous {dtype} [{n}] on x's device")
    return t.data_ptr()


def rows_fp8(x, mode: int = VOC_LM_RMS, weight=None, residual=None, eps: float = 1e-6,
             sum_out=None, out=None, scale=None, stream=None, flags: int = 0):
    """Rows of x [rows, d] (VOC_LM_GATED: [rows, 2d]) to e4m3 with a scale per row (see
    vocoder_lm_rows_fp8 in include/vocoder.h).  Returns (out, scale, sum): out float8_e4m3fn
    [rows, d] (a new one has its row stride padded to 16, as linear_fp8 takes it), scale fp32
    [rows], sum = x + residual in x's type, or None without a residual."""
    if not _LM.ready:
        _lm_setup()
    if stream is None and _LM.fast is not None:
        res = _LM.fast.rows(x, mode, weight, residual, eps, sum_out, out, scale, flags)
        if res.__class__ is tuple:
            return res
        if res is not None:
            _check(res)
    dtype, shape = x.dtype, x.shape
    code = _LM.types.get(dtype)
    if code is None or len(shape) != 2:
        raise _bad("x must be a 2-d bf16, f16 or f32 tensor")
    rows, width = shape
    d = width
    if mode == VOC_LM_GATED:
        if width % 2:
            raise _bad("gated rows need an even width")
        d = width // 2
    dev = _lm_device(x)
    ldx = _rows_strides(x, "x", rows, width, dtype, dev)
    wp = rp = sp = None
    ldr = lds = 0
    made_sum = made_out = made_scale = None
    if weight is not None:
        wp = _vector_ok(weight, "weight", d, dtype, dev)
    if residual is not None:
        ldr = _rows_strides(residual, "residual", rows, d, dtype, dev)
        rp = residual.data_ptr()
        if sum_out is None:
            sum_out = made_sum = _LM.empty((rows, d), dtype=dtype, device=x.device)
            lds = d
        else:
            lds = _rows_strides(sum_out, "sum_out", rows, d, dtype, dev)
        sp = sum_out.data_ptr()
    elif sum_out is not None:
        raise _bad("sum_out without residual")
    if out is None:
        ldo = (d + 15) // 16 * 16
        out = made_out = _LM.empty((rows, ldo), dtype=_LM.f8, device=x.device)
        if ldo != d:
            out = out[:, :d]
    else:
        ldo = _rows_strides(out, "out", rows, d, _LM.f8, dev)
    if scale is None:
        scale = made_scale = _LM.empty((rows,), dtype=_LM.f32, device=x.device)
    else:
        _vector_ok(scale, "scale", rows, _LM.f32, dev)
    st = _LM.rows(x.data_ptr(), ldx, rp, ldr, wp, code, mode, rows, d, eps, sp, lds,
                  out.data_ptr(), ldo, scale.data_ptr(),
                  _lm_stream(dev, stream, (made_sum, made_out, made_scale)), flags)
    if st:
        _check(st)
    return out, scale, sum_out


def linear_fp8(x, x_scale, w, w_scale, bias=None, out_dtype=None, out=None, stream=None,
               flags: int = 0):
    """x [M, K] and w [N, K] float8_e4m3fn (16-byte aligned, row strides multiples of 16) with fp32
    scales [M] and [N], bias fp32 [N] -> [M, N] in out_dtype (bf16 by default; see
    vocoder_lm_linear_fp8 in include/vocoder.h)."""
    if not _LM.ready:
        _lm_setup()
    if stream is None and _LM.fast is not None:
        code = -1 if out_dtype is None else _LM.types.get(out_dtype)
        if code is not None:
            res = _LM.fast.linear(x, x_scale, w, w_scale, bias, code, out, flags)
            if res.__class__ is int:
                _check(res)
            elif res is not None:
                return res
    if x.dim() != 2 or w.dim() != 2:
        raise _bad("x and w must be 2-d float8_e4m3fn tensors")
    f32 = _LM.f32
    M, K = x.shape
    N = w.shape[0]
    dev = _lm_device(x)
    ldx = _rows_strides(x, "x", M, K, _LM.f8, dev)
    ldw = _rows_strides(w, "w", N, K, _LM.f8, dev)
    if M == 1:
        ldx = (ldx + 15) // 16 * 16
    if N == 1:
        ldw = (ldw + 15) // 16 * 16
    xsp = _vector_ok(x_scale, "x_scale", M, f32, dev)
    wsp = _vector_ok(w_scale, "w_scale", N, f32, dev)
    bp = None if bias is None else _vector_ok(bias, "bias", N, f32, dev)
    made = None
    if out is None:
        if out_dtype is None:
            out_dtype = _LM.torch.bfloat16
        code = _LM.types.get(out_dtype)
        if code is None:
            raise _bad("the output is bf16, f16 or f32")
        out = made = _LM.empty((M, N), dtype=out_dtype, device=x.device)
        ldo = N
    else:
        code = _LM.types.get(out.dtype)
        if code is None or (out_dtype is not None and out.dtype != out_dtype):
            raise _bad("out is bf16, f16 or f32, and of out_dtype where that is given")
        ldo = _rows_strides(out, "out", M, N, out.dtype, dev)
    st = _LM.linear(x.data_ptr(), ldx, xsp, w.data_ptr(), ldw, wsp, bp, M, N, K, out.data_ptr(),
                    ldo, code, _lm_stream(dev, stream, (made,)), flags)
    if st:
        _check(st)
    return out


class KVCacheFP8:
    """A pool of 64-token blocks of e4m3 keys and values: k [pages, kv_heads, 64, d] and v [pages,
    kv_heads, d, 64] float8_e4m3fn, k_scale and v_scale fp32 [pages, kv_heads] (see the cache in
    include/vocoder.h).  The tensors are written in place and never exchanged (their addresses are
    kept): a larger pool is a new KVCacheFP8."""
    __slots__ = ("_tensors", "_args")

    def __init__(self, k, v, k_scale, v_scale):
        if not _LM.ready:
            _lm_setup()
        # addresses, pages, key heads, head_dim, device
        args = _LM.fast.cache(k, v, k_scale, v_scale) if _LM.fast is not None else None
        self._args = self._checked(k, v, k_scale, v_scale) if args is None else args
        self._tensors = (k, v, k_scale, v_scale)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    pages = property(lambda self: self._args[4])
    kv_heads = property(lambda self: self._args[5])
    head_dim = property(lambda self: self._args[6])
    device_index = property(lambda self: self._args[7])

    @staticmethod
    def _checked(k, v, k_scale, v_scale):
        shape = k.shape
        if len(shape) != 4 or shape[2] != VOC_LM_BLOCK:
            raise _bad("k must be [pages, kv_heads, 64, head_dim]")
        pages, heads, _, d = shape
        if v.shape != (pages, heads, d, VOC_LM_BLOCK):
            raise _bad("v must be [pages, kv_heads, head_dim, 64]")
        if k_scale.shape != (pages, heads) or v_scale.shape != (pages, heads):
            raise _bad("scales must be [pages, kv_heads]")
        f8, f32, dev = _LM.f8, _LM.f32, k.get_device()
        for t, dtype in ((k, f8), (v, f8), (k_scale, f32), (v_scale, f32)):
            if t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
                raise _bad("the cache is contiguous float8_e4m3fn codes and fp32 scales on one "
                           "device")
        return (k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads,
                d, dev)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, device="cuda"):
        """A new pool.  Blocks are written whole when their first token is appended."""
        import torch
        mk = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)  # noqa: E731
        sc = lambda: torch.zeros((pages, kv_heads), dtype=torch.float32, device=device)  # noqa: E731
        return cls(mk(pages, kv_heads, VOC_LM_BLOCK, head_dim),
                   mk(pages, kv_heads, head_dim, VOC_LM_BLOCK), sc(), sc())


def _batch_args(cache, x, page_table, kv_lens, cu_q):
    """(device, pointers and sizes of the batch) after the checks that cache and batch share."""
    dev = _lm_device(x)
    i32 = _LM.i32
    shape, stride = page_table.shape, page_table.stride()
    if len(shape) != 2 or page_table.dtype != i32 or (stride[1] != 1 and shape[1] > 1) or \
            page_table.get_device() != dev or cache.device_index != dev:
        raise _bad("page_table must be int32 [sequences, blocks] with contiguous rows, on one "
                   "device with the cache and the tokens")
    n, cols = shape
    lens = _vector_ok(kv_lens, "kv_lens", n, i32, dev)
    cu = None if cu_q is None else _vector_ok(cu_q, "cu_q", n + 1, i32, dev)
    return dev, (page_table.data_ptr(), stride[0] if n > 1 else max(cols, stride[0]), cols, lens,
                 cu, n)


def kv_append_fp8(cache: KVCacheFP8, k, v, page_table, kv_lens, cu_q=None,
                  max_q: Optional[int] = None, stream=None, flags: int = 0) -> None:
    """Store k and v [tokens, kv_heads, head_dim] (bf16 or f16) of new tokens in the cache (see
    vocoder_lm_kv_append in include/vocoder.h).  page_table int32 [sequences, blocks], kv_lens
    int32 [sequences] with the new tokens counted, cu_q int32 [sequences + 1] or None when every
    sequence has max_q new tokens.  max_q defaults to 1 without cu_q.  With it, tokens of a sequence
    beyond max_q would be dropped, so it defaults to the number of tokens; the largest number of a
    sequence, where the caller knows it, is faster."""
    if max_q is None:
        max_q = 1 if cu_q is None else k.shape[0]
    if stream is None and _LM.fast is not None:
        res = _LM.fast.append(cache._args, k, v, page_table, kv_lens, cu_q, max_q, flags)
        if res is not None:
            if res:
                _check(res)
            return
    dev, batch = _batch_args(cache, k, page_table, kv_lens, cu_q)
    shape, ks, vs = k.shape, k.stride(), v.stride()
    code = _LM.types.get(k.dtype)
    if len(shape) != 3 or shape[1] != cache.kv_heads or shape[2] != cache.head_dim or \
            v.shape != shape or code is None or v.dtype != k.dtype or ks[2] != 1 or \
            vs[2] != 1 or v.get_device() != dev:
        raise _bad("k and v must be [tokens, kv_heads, head_dim] of one type, head_dim contiguous")
    st = _LM.append(*cache._args[:7], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], code,
                    *batch, shape[0], max_q, _lm_stream(dev, stream, ()), flags)
    if st:
        _check(st)


def attention_fp8(q, cache: KVCacheFP8, page_table, kv_lens, cu_q=None,
                  max_q: Optional[int] = None, max_kv: Optional[int] = None,
                  softmax_scale: Optional[float] = None, causal: bool = True, window: int = 0,
                  out=None, ws=None, stream=None, flags: int = 0):
    """Attention of the newest tokens' queries q [tokens, heads, head_dim] over the cache (see
    vocoder_lm_attention in include/vocoder.h; the batch as in kv_append_fp8).  max_kv: at least
    the largest kv_len (default: what the page table can hold); softmax_scale defaults to
    1/sqrt(head_dim); ws: uint8 workspace of vocoder_lm_attention_ws_bytes (a new one if None)."""
    if max_q is None:
        max_q = 1 if cu_q is None else q.shape[0]
    if stream is None and _LM.fast is not None:
        res = _LM.fast.attention(q, cache._args, page_table, kv_lens, cu_q, max_q,
                                 -1 if max_kv is None else max_kv, softmax_scale, causal, window,
                                 out, ws, flags)
        if res.__class__ is int:
            _check(res)
        elif res is not None:
            return res
    dev, batch = _batch_args(cache, q, page_table, kv_lens, cu_q)
    shape, qs, dtype = q.shape, q.stride(), q.dtype
    code = _LM.types.get(dtype)
    if len(shape) != 3 or shape[2] != cache.head_dim or code is None or qs[2] != 1:
        raise _bad("q must be [tokens, heads, head_dim], head_dim contiguous")
    tokens, heads, d = shape
    made_out = made_ws = None
    if out is None:
        out = made_out = _LM.empty(shape, dtype=dtype, device=q.device)
        os_ = (heads * d, d)
    else:
        os_ = out.stride()
        if out.shape != shape or out.dtype != dtype or os_[2] != 1 or out.get_device() != dev:
            raise _bad("out must have q's shape, type and device, head_dim contiguous")
    if max_kv is None:
        max_kv = batch[2] * VOC_LM_BLOCK
    if softmax_scale is None:
        softmax_scale = d ** -0.5
    if ws is None:
        need = _LM.attention_ws(batch[5], max_q, heads, cache.kv_heads, d, max_kv, window)
        if need:
            ws = made_ws = _LM.empty((need,), dtype=_LM.torch.uint8, device=q.device)
    elif ws.dtype != _LM.torch.uint8 or not ws.is_contiguous() or ws.get_device() != dev:
        raise _bad("ws must be contiguous uint8 on q's device")
    st = _LM.attention(q.data_ptr(), qs[0], qs[1], code, heads, *cache._args[:7], *batch, tokens,
                       max_q, max_kv, softmax_scale, causal, window, out.data_ptr(), os_[0],
                       os_[1], None if ws is None else ws.data_ptr(),
                       0 if ws is None else ws.numel(),
                       _lm_stream(dev, stream, (made_out, made_ws)), flags)
    if st:
        _check(st)
    return out
