"""Python binding of liboidn_mi355x (the MI355X OIDN-style UNet denoiser).

Argument marshalling only: every call goes through the C ABI declared in
include/oidn_mi355x.h, and every step of the hot path runs in the library's
HIP kernels.  Tensor arguments may be torch tensors (their data_ptr() is
passed) or raw integer device addresses; `stream` defaults to torch's current
stream.  A non-zero status raises OidnError with the library's message.
There is no fallback: if the library is not built, loading raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import math
import operator
import os
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liboidn_mi355x.so")
BINDING_PATH = os.path.join(HERE, "_binding" + importlib.machinery.EXTENSION_SUFFIXES[0])

OIDN_OK = 0
OIDN_E_INVALID = -1
OIDN_E_UNSUPPORTED = -2
OIDN_E_WORKSPACE = -3
OIDN_E_HIP = -4

OIDN_F32 = 0
OIDN_F16 = 1
OIDN_BF16 = 2

OIDN_RELU = 1
OIDN_POOL2X2 = 2

OIDN_TRANSFER_PU = 0
OIDN_TRANSFER_LOG = 1

OIDN_ACT_NONE = 0
OIDN_ACT_RELU = 1
OIDN_ACT_SILU = 2
OIDN_ACT_GELU = 3

OIDN_NORM_NONE = 0
OIDN_NORM_RMS = 1
OIDN_NORM_LAYER = 2

OIDN_X_CKPT8 = 1
OIDN_Z_CKPT8 = 2
OIDN_FP8_SQUARE = 4
OIDN_X_FP8 = 8

OIDN_TILE_ALIGN = 16
OIDN_DEFAULT_OVERLAP = 96
OIDN_NOALLOC_SCRATCH_MB = 64

EXPORTS = (
    "oidn_last_error", "oidn_version", "oidn_conv3x3_weights_bytes",
    "oidn_conv3x3_pack_weights", "oidn_conv3x3_pack_weights_host", "oidn_conv3x3", "oidn_conv3x3_upcat", "oidn_pool2x2",
    "oidn_upsample_concat", "oidn_pack_input", "oidn_unpack_output", "oidn_plan_tiles",
    "oidn_conv3x3_pair", "oidn_conv3x3_kernel", "oidn_unet_layer_count", "oidn_unet_layer_info", "oidn_unet_layer_kernel",
    "oidn_unet_weights_bytes",
    "oidn_unet_pack_weights", "oidn_unet_packed_workspace_bytes", "oidn_unet_forward_packed",
    "oidn_unet_workspace_bytes", "oidn_unet_tile_batch", "oidn_unet_input_layout",
    "oidn_unet_forward",
    "oidn_unet_forward_timed", "oidn_unet_forward_noalloc", "oidn_unet_noalloc_scratch_bytes",
    "oidn_ckpt_bytes", "oidn_ckpt_pack", "oidn_ckpt_unpack",
    "oidn_linear_workspace_bytes", "oidn_linear", "oidn_linear_backward_workspace_bytes", "oidn_linear_backward",
    "oidn_ffn_workspace_bytes", "oidn_ffn", "oidn_ffn_backward_workspace_bytes", "oidn_ffn_backward",
    "oidn_fp8_bytes", "oidn_fp8_pack", "oidn_fp8_unpack", "oidn_linear_fp8_workspace_bytes", "oidn_linear_fp8",
    "oidn_linear_fp8_backward_workspace_bytes", "oidn_linear_fp8_backward",
    "oidn_norm", "oidn_norm_backward_workspace_bytes", "oidn_norm_backward", "oidn_norm_residual",
    "oidn_norm_residual_backward_workspace_bytes", "oidn_norm_residual_backward", "oidn_dropout",
    "oidn_calibrate_mfma", "oidn_calibrate_read", "oidn_event_create", "oidn_event_destroy", "oidn_event_elapsed_ms",
)


class OidnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"oidn status {code}: {message}")
        self.code = code


class oidn_tile(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("in_x", "in_y", "in_w", "in_h", "out_x", "out_y", "out_w", "out_h")]

    def as_tuple(self):
        return tuple(getattr(self, n) for n, _ in self._fields_)


_lib = None
_l = ctypes.c_long
_vp, _i, _u, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "oidn_last_error": ([], ctypes.c_char_p),
    "oidn_version": ([], _i),
    "oidn_conv3x3_weights_bytes": ([_i, _i, _i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_conv3x3_pack_weights": ([_vp, _vp, _i, _i, _i, _i, _vp, _vp], _i),
    "oidn_conv3x3_pack_weights_host": ([_vp, _vp, _i, _i, _i, _i, _vp], _i),
    "oidn_conv3x3": ([_vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _u, _vp], _i),
    "oidn_conv3x3_upcat": ([_vp, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _u, _vp], _i),
    "oidn_pool2x2": ([_vp, _i, _i, _i, _vp, _i, _vp], _i),
    "oidn_upsample_concat": ([_vp, _i, _vp, _i, _i, _i, _vp, _i, _vp], _i),
    "oidn_pack_input": ([_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp], _i),
    "oidn_unpack_output": ([_vp, _i, _i, _i, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp,
                            _vp], _i),
    "oidn_plan_tiles": ([_i, _i, _i, _i, ctypes.POINTER(oidn_tile), _i, ctypes.POINTER(_i)], _i),
    "oidn_unet_layer_count": ([], _i),
    "oidn_unet_layer_info": ([_i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i),
                              ctypes.POINTER(_i), ctypes.POINTER(_u),
                              ctypes.POINTER(ctypes.c_char_p)], _i),
    "oidn_unet_layer_kernel": ([_i, _i, _i, _i, _i, _i, ctypes.c_char_p, _i, ctypes.POINTER(_i)], _i),
    "oidn_conv3x3_pair": ([_vp, _i, _i, _i, _vp, _vp, _vp, _i, _i, _u, _vp], _i),
    "oidn_conv3x3_kernel": ([_i, _i, _i, _i, _i, _i, _i, _u, ctypes.c_char_p, _i,
                             ctypes.POINTER(_i)], _i),
    "oidn_unet_weights_bytes": ([_i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_unet_pack_weights": ([ctypes.POINTER(_vp), ctypes.POINTER(_vp), _i, _i, _vp, _vp], _i),
    "oidn_unet_packed_workspace_bytes": ([_i, _i, _i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_unet_forward_packed": ([_vp, _i, _vp, _i, _i, _vp, _sz, _vp, _i, _vp], _i),
    "oidn_unet_workspace_bytes": ([_i, _i, _i, _i, _i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_unet_tile_batch": ([_i, _i, _i, _i, _i, _i, ctypes.POINTER(_i)], _i),
    "oidn_unet_input_layout": ([_i, _i, _i, _i, _i, _i, ctypes.POINTER(_sz), ctypes.POINTER(_sz),
                                ctypes.POINTER(_i), ctypes.POINTER(_i)], _i),
    "oidn_unet_forward": ([_vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp, _i,
                           _vp], _i),
    "oidn_unet_forward_timed": ([_vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp,
                                 _i, _vp, ctypes.POINTER(_vp), _i], _i),
    "oidn_unet_forward_noalloc": ([_vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp, _i,
                                   _vp], _i),
    "oidn_unet_noalloc_scratch_bytes": ([ctypes.POINTER(_sz)], _i),
    "oidn_ckpt_bytes": ([_l, _l, ctypes.POINTER(_sz)], _i),
    "oidn_ckpt_pack": ([_vp, _l, _l, _l, _vp, _i, _vp], _i),
    "oidn_ckpt_unpack": ([_vp, _l, _l, _vp, _l, _i, _vp], _i),
    "oidn_linear_workspace_bytes": ([_l, _i, _i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_linear": ([_vp, _l, _vp, _l, _vp, _vp, _l, _vp, _l, _vp, _l, _l, _i, _i, _i, _i, _u, _vp, _sz,
                     _vp], _i),
    "oidn_linear_backward_workspace_bytes": ([_l, _i, _i, _i, _i, _u, ctypes.POINTER(_sz)], _i),
    "oidn_linear_backward": ([_vp, _l, _vp, _l, _vp, _l, _vp, _l, _vp, _l, _vp, _l, _vp, _l, _i, _i, _i, _i,
                              _u, _vp, _sz, _vp], _i),
    "oidn_ffn_workspace_bytes": ([_l, _i, _i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_ffn": ([_vp, _l, _vp, _vp, _vp, _vp, _vp, _l, _vp, _l, _vp, _l, _i, _i, _i, _i, _u, _vp, _sz,
                  _vp], _i),
    "oidn_ffn_backward_workspace_bytes": ([_l, _i, _i, _i, _u, ctypes.POINTER(_sz)], _i),
    "oidn_ffn_backward": ([_vp, _l, _vp, _l, _vp, _vp, _vp, _vp, _l, _vp, _l, _vp, _vp, _vp, _vp, _l, _i, _i,
                           _i, _i, _u, _vp, _sz, _vp], _i),
    "oidn_fp8_bytes": ([_l, _l, ctypes.POINTER(_sz)], _i),
    "oidn_fp8_pack": ([_vp, _l, _l, _l, _vp, _vp, _i, _u, _vp], _i),
    "oidn_fp8_unpack": ([_vp, _l, _l, _vp, _l, _i, _vp], _i),
    "oidn_linear_fp8_workspace_bytes": ([_l, _i, _i, _i, _u, ctypes.POINTER(_sz)], _i),
    "oidn_linear_fp8": ([_vp, _l, _vp, _vp, _vp, _l, _vp, _l, _vp, _l, _l, _i, _i, _i, _i, _u, _vp, _sz, _vp], _i),
    "oidn_linear_fp8_backward_workspace_bytes": ([_l, _i, _i, _i, _i, _u, ctypes.POINTER(_sz)], _i),
    "oidn_linear_fp8_backward": ([_vp, _l, _vp, _l, _vp, _l, _vp, _vp, _l, _vp, _l, _vp, _l, _i, _i, _i, _i, _u,
                                  _vp, _sz, _vp], _i),
    "oidn_norm": ([_vp, _l, _vp, _vp, _vp, _l, _l, _i, _i, _f, _i, _vp], _i),
    "oidn_norm_backward_workspace_bytes": ([_l, _i, _i, ctypes.POINTER(_sz)], _i),
    "oidn_norm_backward": ([_vp, _l, _vp, _l, _vp, _vp, _l, _vp, _l, _vp, _vp, _l, _i, _i, _f, _i, _vp, _sz,
                            _vp], _i),
    "oidn_norm_residual": ([_vp, _l, _vp, _vp, _vp, _l, _l, _vp, _l, _f, _f, _vp, _vp, _l, _vp, _vp, _vp, _l, _l,
                            _i, _i, _i, _f, _i, _vp], _i),
    "oidn_norm_residual_backward_workspace_bytes": ([_l, _i, _l, _i, ctypes.POINTER(_sz)], _i),
    "oidn_norm_residual_backward": ([_vp, _l, _vp, _l, _vp, _l, _vp, _vp, _vp, _l, _l, _vp, _l, _f, _f, _vp, _vp,
                                     _vp, _l, _vp, _l, _vp, _l, _vp, _vp, _vp, _vp, _l, _i, _i, _i, _f, _i, _vp,
                                     _sz, _vp], _i),
    "oidn_dropout": ([_vp, _l, _vp, _l, _vp, _l, _l, _i, _f, _vp, _i, _vp], _i),
    "oidn_calibrate_mfma": ([_i, ctypes.c_long, _i, _vp, ctypes.POINTER(ctypes.c_longlong), _vp], _i),
    "oidn_calibrate_read": ([_vp, _sz, _vp, _vp], _i),
    "oidn_event_create": ([ctypes.POINTER(_vp)], _i),
    "oidn_event_destroy": ([_vp], _i),
    "oidn_event_elapsed_ms": ([_vp, _vp, ctypes.POINTER(_f)], _i),
}


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OidnError(OIDN_E_HIP, f"{LIB_PATH} is not built; run __graft_entry__.build()")
        # torch ships its own HIP runtime with the same soname; loading torch
        # first makes the library bind to that one instead of mapping a second
        # runtime (which would see no device and could not use torch's memory).
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        _check_single_hip_runtime()
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _converted(v, t):
    """The argument v of a parameter of type t, refused where ctypes would cut it."""
    if t is _vp:
        a = None if v is None else operator.index(_p(v))
        if a is not None and not -1 << 63 <= a < 1 << 64:
            raise OverflowError(f"{v!r} does not fit the parameter")
        return a
    if t is _f:
        c = _f(v)
        if math.isinf(c.value) and not (isinstance(v, float) and math.isinf(v)):
            raise OverflowError(f"{v!r} does not fit the parameter")
        return c
    c = t(operator.index(v))
    if c.value != v:
        raise OverflowError(f"{v!r} does not fit the parameter")
    return c


class _ThroughCtypes:
    """The calls of csrc/binding.cpp where that is not built."""

    def __getattr__(self, name):
        f = getattr(lib(), name)

        def call(*args):
            if len(args) != len(f.argtypes):
                raise TypeError(f"{len(args)} arguments given, {len(f.argtypes)} taken")
            return f(*[_converted(v, t) for v, t in zip(args, f.argtypes)])

        setattr(self, name, call)
        return call


_native = None


def _calls():
    """The calls of csrc/binding.cpp: they take tensors, and cost less of the host's time than ctypes."""
    global _native
    if _native is None:
        lib()
        if os.path.exists(BINDING_PATH):
            from . import _binding
            _native = _binding
        else:
            warnings.warn(f"{BINDING_PATH} is not built: calls go through ctypes and take longer", RuntimeWarning)
            _native = _ThroughCtypes()
    return _native


def _check_single_hip_runtime():
    try:
        maps = open("/proc/self/maps").read()
    except OSError:
        return
    runtimes = {line.split()[-1] for line in maps.splitlines()
                if "libamdhip64" in line and line.split()[-1].startswith("/")}
    if len(runtimes) > 1:
        raise OidnError(OIDN_E_HIP, "two HIP runtimes are loaded in this process: "
                        + ", ".join(sorted(runtimes)))


def last_error() -> str:
    return lib().oidn_last_error().decode()


def _check(rc: int):
    if rc != OIDN_OK:
        raise OidnError(rc, last_error())


def _p(t):
    """Device address of a tensor (or int / None)."""
    return t if t is None or isinstance(t, int) else t.data_ptr()


_current_stream = None


def _s(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            if raw is None:   # a torch without it: the stream object, which costs 3 us to make
                _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
            else:
                _current_stream = lambda: raw(device())  # noqa: E731
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ convs
def oidn_conv3x3_weights_bytes(cin0: int, cin1: int, cout: int, dtype: int) -> int:
    n = _sz()
    _check(lib().oidn_conv3x3_weights_bytes(cin0, cin1, cout, dtype, ctypes.byref(n)))
    return n.value


def oidn_conv3x3_pack_weights(w_ohwi, bias, cin0: int, cin1: int, cout: int, dtype: int,
                              d_packed, stream=None):
    """w_ohwi, bias: host numpy float32 arrays (C-contiguous)."""
    import numpy as np
    w = np.ascontiguousarray(w_ohwi, dtype=np.float32)
    b = np.ascontiguousarray(bias, dtype=np.float32)
    if w.size != cout * 9 * (cin0 + cin1) or b.size != cout:
        raise OidnError(OIDN_E_INVALID, "weight or bias size does not match the shape")
    _check(lib().oidn_conv3x3_pack_weights(w.ctypes.data, b.ctypes.data, cin0, cin1, cout, dtype,
                                           _p(d_packed), _s(stream)))


def oidn_conv3x3_pack_weights_host(w_ohwi, bias, cin0: int, cin1: int, cout: int, dtype: int):
    """Packed bytes (numpy uint8) of the device layout, built on the host."""
    import numpy as np
    w = np.ascontiguousarray(w_ohwi, dtype=np.float32)
    b = np.ascontiguousarray(bias, dtype=np.float32)
    if w.size != cout * 9 * (cin0 + cin1) or b.size != cout:
        raise OidnError(OIDN_E_INVALID, "weight or bias size does not match the shape")
    out = np.zeros(oidn_conv3x3_weights_bytes(cin0, cin1, cout, dtype), np.uint8)
    _check(lib().oidn_conv3x3_pack_weights_host(w.ctypes.data, b.ctypes.data, cin0, cin1, cout,
                                                dtype, out.ctypes.data))
    return out


def oidn_conv3x3(x, h: int, w: int, cin: int, w_packed, y, cout: int, in_dtype: int,
                 out_dtype: int, flags: int, stream=None):
    _check(lib().oidn_conv3x3(_p(x), h, w, cin, _p(w_packed), _p(y), cout, in_dtype, out_dtype,
                              flags, _s(stream)))


def oidn_conv3x3_upcat(low, c_low: int, skip, c_skip: int, h: int, w: int, w_packed, y,
                       cout: int, in_dtype: int, out_dtype: int, flags: int, stream=None):
    _check(lib().oidn_conv3x3_upcat(_p(low), c_low, _p(skip), c_skip, h, w, _p(w_packed), _p(y),
                                    cout, in_dtype, out_dtype, flags, _s(stream)))


def oidn_conv3x3_pair(x, h: int, w: int, cin: int, wa_packed, wb_packed, y, cout: int,
                      out_dtype: int, flags: int, stream=None):
    _check(lib().oidn_conv3x3_pair(_p(x), h, w, cin, _p(wa_packed), _p(wb_packed), _p(y), cout,
                                   out_dtype, flags, _s(stream)))


# ------------------------------------------------------------ elementwise
def oidn_pool2x2(x, h: int, w: int, c: int, y, dtype: int, stream=None):
    _check(lib().oidn_pool2x2(_p(x), h, w, c, _p(y), dtype, _s(stream)))


def oidn_upsample_concat(low, c_low: int, skip, c_skip: int, h: int, w: int, z, dtype: int,
                         stream=None):
    _check(lib().oidn_upsample_concat(_p(low), c_low, _p(skip), c_skip, h, w, _p(z), dtype,
                                      _s(stream)))


def oidn_pack_input(color, albedo, normal, img_w: int, img_h: int, tile_x: int, tile_y: int,
                    tile_w: int, tile_h: int, hdr: bool, transfer: int, input_scale: float,
                    packed, dtype: int, stream=None):
    _check(lib().oidn_pack_input(_p(color), _p(albedo), _p(normal), img_w, img_h, tile_x, tile_y,
                                 tile_w, tile_h, int(hdr), transfer, input_scale, _p(packed),
                                 dtype, _s(stream)))


def oidn_unpack_output(net_rgba, tile_w: int, tile_h: int, in_off_x: int, in_off_y: int, color,
                       img_w: int, img_h: int, out_x: int, out_y: int, out_w: int, out_h: int,
                       hdr: bool, transfer: int, input_scale: float, out_rgba, stream=None):
    _check(lib().oidn_unpack_output(_p(net_rgba), tile_w, tile_h, in_off_x, in_off_y, _p(color),
                                    img_w, img_h, out_x, out_y, out_w, out_h, int(hdr), transfer,
                                    input_scale, _p(out_rgba), _s(stream)))


# ---------------------------------------------------------------- tiles
def oidn_plan_tiles(w: int, h: int, max_tile: int, overlap: int):
    """List of (in_x, in_y, in_w, in_h, out_x, out_y, out_w, out_h)."""
    count = _i()
    _check(lib().oidn_plan_tiles(w, h, max_tile, overlap, None, 0, ctypes.byref(count)))
    arr = (oidn_tile * max(count.value, 1))()
    _check(lib().oidn_plan_tiles(w, h, max_tile, overlap, arr, count.value, ctypes.byref(count)))
    return [arr[i].as_tuple() for i in range(count.value)]


# ----------------------------------------------------------------- UNet
def oidn_unet_layer_count() -> int:
    return lib().oidn_unet_layer_count()


def oidn_unet_layer_info(in_channels: int, layer: int):
    """(name, cin0, cin1, cout, level, flags)."""
    c0, c1, co, lv, fl, nm = _i(), _i(), _i(), _i(), _u(), ctypes.c_char_p()
    _check(lib().oidn_unet_layer_info(in_channels, layer, ctypes.byref(c0), ctypes.byref(c1),
                                      ctypes.byref(co), ctypes.byref(lv), ctypes.byref(fl),
                                      ctypes.byref(nm)))
    return nm.value.decode(), c0.value, c1.value, co.value, lv.value, fl.value


def oidn_conv3x3_kernel(h: int, w: int, cin0: int, cin1: int, cout: int, in_dtype: int,
                        out_dtype: int, flags: int):
    """(kernel instance name, workgroups) of one conv (cin1 > 0: decoder conv)."""
    buf = ctypes.create_string_buffer(128)
    nb = _i()
    _check(lib().oidn_conv3x3_kernel(h, w, cin0, cin1, cout, in_dtype, out_dtype, flags, buf, 128,
                                     ctypes.byref(nb)))
    return buf.value.decode(), nb.value


def oidn_unet_layer_kernel(in_channels: int, layer: int, tw: int, th: int, dtype: int,
                           batch: int = 1):
    """(kernel instance name, workgroups) of a layer on `batch` tw x th tiles
    per launch."""
    buf = ctypes.create_string_buffer(128)
    nb = _i()
    _check(lib().oidn_unet_layer_kernel(in_channels, layer, tw, th, batch, dtype, buf, 128,
                                        ctypes.byref(nb)))
    return buf.value.decode(), nb.value


def unet_layer_shapes(in_channels: int):
    """[(cin_logical, cout)] of the library's layer table."""
    out = []
    for i in range(oidn_unet_layer_count()):
        _, c0, c1, co, _, _ = oidn_unet_layer_info(in_channels, i)
        out.append((c0 + c1, co))
    return out


def oidn_unet_weights_bytes(in_channels: int, dtype: int) -> int:
    n = _sz()
    _check(lib().oidn_unet_weights_bytes(in_channels, dtype, ctypes.byref(n)))
    return n.value


def oidn_unet_pack_weights(weights, biases, in_channels: int, dtype: int, d_weights, stream=None):
    """weights[i]: host float32 OHWI array of layer i; biases[i]: host float32 array."""
    import numpy as np
    ws = [np.ascontiguousarray(w, dtype=np.float32) for w in weights]
    bs = [np.ascontiguousarray(b, dtype=np.float32) for b in biases]
    n = oidn_unet_layer_count()
    if len(ws) != n or len(bs) != n:
        raise OidnError(OIDN_E_INVALID, f"expected {n} weight and bias arrays")
    for i, ((cin, cout), w, b) in enumerate(zip(unet_layer_shapes(in_channels), ws, bs)):
        if w.shape != (cout, 3, 3, cin) or b.shape != (cout,):
            raise OidnError(OIDN_E_INVALID, f"layer {i}: expected weights {(cout, 3, 3, cin)}")
    wp = (_vp * n)(*[w.ctypes.data for w in ws])
    bp = (_vp * n)(*[b.ctypes.data for b in bs])
    _check(lib().oidn_unet_pack_weights(wp, bp, in_channels, dtype, _p(d_weights), _s(stream)))


def oidn_unet_packed_workspace_bytes(in_channels: int, tw: int, th: int, dtype: int) -> int:
    n = _sz()
    _check(lib().oidn_unet_packed_workspace_bytes(in_channels, tw, th, dtype, ctypes.byref(n)))
    return n.value


def oidn_unet_forward_packed(d_weights, in_channels: int, packed_in, tw: int, th: int, workspace,
                             ws_bytes: int, net_out_rgba, dtype: int, stream=None):
    _check(lib().oidn_unet_forward_packed(_p(d_weights), in_channels, _p(packed_in), tw, th,
                                          _p(workspace), ws_bytes, _p(net_out_rgba), dtype,
                                          _s(stream)))


def oidn_unet_workspace_bytes(in_channels: int, w: int, h: int, max_tile: int, overlap: int,
                              dtype: int) -> int:
    n = _sz()
    _check(lib().oidn_unet_workspace_bytes(in_channels, w, h, max_tile, overlap, dtype,
                                           ctypes.byref(n)))
    return n.value


def oidn_unet_tile_batch(in_channels: int, w: int, h: int, max_tile: int, overlap: int,
                         dtype: int) -> int:
    n = _i()
    _check(lib().oidn_unet_tile_batch(in_channels, w, h, max_tile, overlap, dtype, ctypes.byref(n)))
    return n.value


def oidn_unet_input_layout(in_channels: int, w: int, h: int, max_tile: int, overlap: int,
                           dtype: int):
    """(offset, tile_stride, lanes, taps) of the packed network input that
    oidn_unet_forward leaves in its workspace."""
    off, stride, lanes, taps = _sz(), _sz(), _i(), _i()
    _check(lib().oidn_unet_input_layout(in_channels, w, h, max_tile, overlap, dtype,
                                        ctypes.byref(off), ctypes.byref(stride),
                                        ctypes.byref(lanes), ctypes.byref(taps)))
    return off.value, stride.value, lanes.value, bool(taps.value)


def oidn_unet_forward(d_weights, in_channels: int, color, albedo, normal, w: int, h: int,
                      hdr: bool, transfer: int, input_scale: float, max_tile: int, overlap: int,
                      workspace, ws_bytes: int, out_rgba, dtype: int, stream=None):
    _check(lib().oidn_unet_forward(_p(d_weights), in_channels, _p(color), _p(albedo), _p(normal),
                                   w, h, int(hdr), transfer, input_scale, max_tile, overlap,
                                   _p(workspace), ws_bytes, _p(out_rgba), dtype, _s(stream)))


def oidn_unet_forward_timed(d_weights, in_channels: int, color, albedo, normal, w: int, h: int,
                            hdr: bool, transfer: int, input_scale: float, max_tile: int,
                            overlap: int, workspace, ws_bytes: int, out_rgba, dtype: int, events,
                            stream=None):
    ev = (_vp * len(events))(*events)
    _check(lib().oidn_unet_forward_timed(_p(d_weights), in_channels, _p(color), _p(albedo),
                                         _p(normal), w, h, int(hdr), transfer, input_scale,
                                         max_tile, overlap, _p(workspace), ws_bytes,
                                         _p(out_rgba), dtype, _s(stream), ev, len(events)))


def oidn_unet_forward_noalloc(d_weights, in_channels: int, color, albedo, normal, w: int, h: int,
                              hdr: bool, transfer: int, input_scale: float, max_tile: int,
                              overlap: int, out_rgba, dtype: int, stream=None):
    _check(lib().oidn_unet_forward_noalloc(_p(d_weights), in_channels, _p(color), _p(albedo),
                                           _p(normal), w, h, int(hdr), transfer, input_scale,
                                           max_tile, overlap, _p(out_rgba), dtype, _s(stream)))


def oidn_unet_noalloc_scratch_bytes() -> int:
    n = _sz()
    _check(lib().oidn_unet_noalloc_scratch_bytes(ctypes.byref(n)))
    return n.value


# -------------------------------------------- dense operators over rows
def _size(fn, *args) -> int:
    n = _sz()
    _check(fn(*args, ctypes.byref(n)))
    return n.value


def oidn_ckpt_bytes(m: int, n: int) -> int:
    return _size(lib().oidn_ckpt_bytes, m, n)


def oidn_ckpt_pack(x, ldx: int, m: int, n: int, ckpt, dtype: int, stream=None):
    _check(lib().oidn_ckpt_pack(_p(x), ldx, m, n, _p(ckpt), dtype, _s(stream)))


def oidn_ckpt_unpack(ckpt, m: int, n: int, y, ldy: int, dtype: int, stream=None):
    _check(lib().oidn_ckpt_unpack(_p(ckpt), m, n, _p(y), ldy, dtype, _s(stream)))


def oidn_linear_workspace_bytes(m: int, k: int, n: int, dtype: int) -> int:
    return _size(lib().oidn_linear_workspace_bytes, m, k, n, dtype)


def oidn_linear(x, ldx: int, w, ldw: int, bias, residual, ldr: int, y, ldy: int, z, ldz: int, m: int,
                k: int, n: int, act: int, dtype: int, flags: int, workspace, ws_bytes: int, stream=None):
    _check(lib().oidn_linear(_p(x), ldx, _p(w), ldw, _p(bias), _p(residual), ldr, _p(y), ldy, _p(z), ldz,
                             m, k, n, act, dtype, flags, _p(workspace), ws_bytes, _s(stream)))


def oidn_linear_backward_workspace_bytes(m: int, k: int, n: int, act: int, dtype: int, flags: int) -> int:
    return _size(lib().oidn_linear_backward_workspace_bytes, m, k, n, act, dtype, flags)


def oidn_linear_backward(dy, lddy: int, x, ldx: int, z, ldz: int, w, ldw: int, dx, lddx: int, dw, lddw: int,
                         dbias, m: int, k: int, n: int, act: int, dtype: int, flags: int, workspace,
                         ws_bytes: int, stream=None):
    _check(lib().oidn_linear_backward(_p(dy), lddy, _p(x), ldx, _p(z), ldz, _p(w), ldw, _p(dx), lddx,
                                      _p(dw), lddw, _p(dbias), m, k, n, act, dtype, flags, _p(workspace),
                                      ws_bytes, _s(stream)))


def oidn_ffn_workspace_bytes(m: int, d: int, f: int, dtype: int) -> int:
    return _size(lib().oidn_ffn_workspace_bytes, m, d, f, dtype)


def oidn_ffn(x, ldx: int, w_in, b_in, w_out, b_out, residual, ldr: int, y, ldy: int, z, m: int, d: int,
             f: int, act: int, dtype: int, flags: int, workspace, ws_bytes: int, stream=None):
    _check(lib().oidn_ffn(_p(x), ldx, _p(w_in), _p(b_in), _p(w_out), _p(b_out), _p(residual), ldr, _p(y),
                          ldy, _p(z), m, d, f, act, dtype, flags, _p(workspace), ws_bytes, _s(stream)))


def oidn_ffn_backward_workspace_bytes(m: int, d: int, f: int, dtype: int, flags: int) -> int:
    return _size(lib().oidn_ffn_backward_workspace_bytes, m, d, f, dtype, flags)


def oidn_ffn_backward(dy, lddy: int, x, ldx: int, z, w_in, w_out, add, ldadd: int, dx, lddx: int, dw_in,
                      db_in, dw_out, db_out, m: int, d: int, f: int, act: int, dtype: int, flags: int,
                      workspace, ws_bytes: int, stream=None):
    _check(lib().oidn_ffn_backward(_p(dy), lddy, _p(x), ldx, _p(z), _p(w_in), _p(w_out), _p(add), ldadd,
                                   _p(dx), lddx, _p(dw_in), _p(db_in), _p(dw_out), _p(db_out), m, d, f,
                                   act, dtype, flags, _p(workspace), ws_bytes, _s(stream)))


def oidn_fp8_bytes(m: int, n: int) -> int:
    return _size(lib().oidn_fp8_bytes, m, n)


def oidn_fp8_pack(x, ldx: int, m: int, n: int, packed, packed_t, dtype: int, flags: int, stream=None):
    _check(_calls().oidn_fp8_pack(x, ldx, m, n, packed, packed_t, dtype, flags, _s(stream)))


def oidn_fp8_unpack(packed, m: int, n: int, y, ldy: int, dtype: int, stream=None):
    _check(_calls().oidn_fp8_unpack(packed, m, n, y, ldy, dtype, _s(stream)))


def oidn_linear_fp8_workspace_bytes(m: int, k: int, n: int, dtype: int, flags: int) -> int:
    return _size(lib().oidn_linear_fp8_workspace_bytes, m, k, n, dtype, flags)


def oidn_linear_fp8(x, ldx: int, w8, bias, residual, ldr: int, y, ldy: int, z, ldz: int, m: int, k: int, n: int,
                    act: int, dtype: int, flags: int, workspace, ws_bytes: int, stream=None):
    _check(_calls().oidn_linear_fp8(x, ldx, w8, bias, residual, ldr, y, ldy, z, ldz, m, k, n, act, dtype, flags,
                                    workspace, ws_bytes, _s(stream)))


def oidn_linear_fp8_backward_workspace_bytes(m: int, k: int, n: int, act: int, dtype: int, flags: int) -> int:
    return _size(lib().oidn_linear_fp8_backward_workspace_bytes, m, k, n, act, dtype, flags)


def oidn_linear_fp8_backward(dy, lddy: int, x, ldx: int, z, ldz: int, w8t, dx, lddx: int, dw, lddw: int, dbias,
                             m: int, k: int, n: int, act: int, dtype: int, flags: int, workspace, ws_bytes: int,
                             stream=None):
    _check(_calls().oidn_linear_fp8_backward(dy, lddy, x, ldx, z, ldz, w8t, dx, lddx, dw, lddw, dbias, m, k, n, act,
                                             dtype, flags, workspace, ws_bytes, _s(stream)))


# ------------------------------------------------- around a block over rows
def oidn_norm(x, ldx: int, weight, shift, y, ldy: int, m: int, n: int, norm: int, eps: float, dtype: int,
              stream=None):
    _check(_calls().oidn_norm(x, ldx, weight, shift, y, ldy, m, n, norm, eps, dtype, _s(stream)))


def oidn_norm_backward_workspace_bytes(m: int, n: int, dtype: int) -> int:
    return _size(lib().oidn_norm_backward_workspace_bytes, m, n, dtype)


def oidn_norm_backward(dy, lddy: int, x, ldx: int, weight, add, ldadd: int, dx, lddx: int, dweight, dshift, m: int,
                       n: int, norm: int, eps: float, dtype: int, workspace, ws_bytes: int, stream=None):
    _check(_calls().oidn_norm_backward(dy, lddy, x, ldx, weight, add, ldadd, dx, lddx, dweight, dshift, m, n, norm,
                                       eps, dtype, workspace, ws_bytes, _s(stream)))


def oidn_norm_residual(o, ldo: int, weight, shift, gate, ldg: int, gate_rows: int, x, ldx: int, scale: float,
                       p: float, rng, u, ldu: int, next_weight, next_shift, v, ldv: int, m: int, n: int, norm: int,
                       next_norm: int, eps: float, dtype: int, stream=None):
    """rng: two 64-bit words in device memory (an int64 tensor of seed and offset)."""
    _check(_calls().oidn_norm_residual(o, ldo, weight, shift, gate, ldg, gate_rows, x, ldx, scale, p, rng, u, ldu,
                                       next_weight, next_shift, v, ldv, m, n, norm, next_norm, eps, dtype,
                                       _s(stream)))


def oidn_norm_residual_backward_workspace_bytes(m: int, n: int, gate_rows: int, dtype: int) -> int:
    return _size(lib().oidn_norm_residual_backward_workspace_bytes, m, n, gate_rows, dtype)


def oidn_norm_residual_backward(du, lddu: int, dv, lddv: int, o, ldo: int, weight, shift, gate, ldg: int,
                                gate_rows: int, u, ldu: int, scale: float, p: float, rng, next_weight, dx, lddx: int,
                                d_o, lddo: int, dgate, lddg: int, dweight, dshift, dnext_weight, dnext_shift, m: int,
                                n: int, norm: int, next_norm: int, eps: float, dtype: int, workspace, ws_bytes: int,
                                stream=None):
    _check(_calls().oidn_norm_residual_backward(du, lddu, dv, lddv, o, ldo, weight, shift, gate, ldg, gate_rows, u,
                                                ldu, scale, p, rng, next_weight, dx, lddx, d_o, lddo, dgate, lddg,
                                                dweight, dshift, dnext_weight, dnext_shift, m, n, norm, next_norm,
                                                eps, dtype, workspace, ws_bytes, _s(stream)))


def oidn_dropout(x, ldx: int, residual, ldr: int, y, ldy: int, m: int, n: int, p: float, rng, dtype: int,
                 stream=None):
    """rng: two 64-bit words in device memory (an int64 tensor of seed and offset)."""
    _check(_calls().oidn_dropout(x, ldx, residual, ldr, y, ldy, m, n, p, rng, dtype, _s(stream)))


def oidn_calibrate_mfma(dtype: int, iters: int, blocks: int, sink, stream=None) -> int:
    """Launches the MFMA stream; returns its FLOPs."""
    n = ctypes.c_longlong()
    _check(lib().oidn_calibrate_mfma(dtype, iters, blocks, _p(sink), ctypes.byref(n), _s(stream)))
    return n.value


def oidn_calibrate_read(buf, nbytes: int, sink, stream=None):
    _check(lib().oidn_calibrate_read(_p(buf), nbytes, _p(sink), _s(stream)))


def oidn_event_create() -> int:
    e = _vp()
    _check(lib().oidn_event_create(ctypes.byref(e)))
    return e.value


def oidn_event_destroy(event: int):
    _check(lib().oidn_event_destroy(event))


def oidn_event_elapsed_ms(start: int, end: int) -> float:
    ms = _f()
    _check(lib().oidn_event_elapsed_ms(start, end, ctypes.byref(ms)))
    return ms.value
