"""Thin ctypes binding over libgla.so, with the C ABI's names.

Argument marshalling only: tensors become device pointers, results are
returned as status codes (or raised as GlaError). Every step of the forward
pass runs in the library's CUDA kernels; there is no fallback of any kind,
and a missing or unloadable library raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

GLA_OK, GLA_ERR_INVALID_ARG, GLA_ERR_UNSUPPORTED, GLA_ERR_CUDA, GLA_ERR_WORKSPACE, GLA_ERR_TIMEOUT = range(6)
GLA_BF16, GLA_FP32 = 0, 1
GLA_GATE_NONE, GLA_GATE_HEAD_SCALAR, GLA_GATE_PER_KEY, GLA_GATE_TOKEN_SCALAR, GLA_GATE_BILINEAR = 0, 1, 2, 3, 4
GLA_NORM_NONE, GLA_NORM_L2, GLA_NORM_RMS = 0, 1, 2
GLA_ACT_NONE, GLA_ACT_SILU, GLA_ACT_SIGMOID = 0, 1, 2
GLA_PATH_AUTO, GLA_PATH_TENSOR, GLA_PATH_SIMT, GLA_PATH_STAGED, GLA_PATH_FUSED, GLA_PATH_SPLIT = 0, 1, 2, 3, 4, 5

# Every symbol include/gla.h declares.
EXPORTED = ("gla_fwd", "gla_fwd_ex", "gla_fwd_workspace_size", "gla_fwd_num_stages",
            "gla_fwd_stage", "gla_fwd_stage_name", "gla_device_status", "gla_status_string",
            "gla_version", "gla_fwd_noalloc", "gla_fwd_host", "gla_host_release", "gla_bwd",
            "gla_bwd_workspace_size", "gla_bwd_num_stages", "gla_bwd_stage", "gla_bwd_stage_name",
            "gla_segment_pair_workspace_size", "gla_segment_pair",
            "gla_pair_scan", "gla_pair_combine", "gla_selftest_bounded_wait",
            "gla_delta_fwd", "gla_delta_fwd_workspace_size", "gla_delta_bwd", "gla_delta_bwd_workspace_size",
            "gla_qk_norm_rope", "gla_qk_norm_rope_bwd", "gla_qk_norm_rope_bwd_workspace_size",
            "gla_conv_fwd", "gla_conv_bwd", "gla_conv_bwd_workspace_size",
            "gla_ssm_fwd", "gla_ssm_fwd_workspace_size", "gla_ssm_bwd", "gla_ssm_bwd_workspace_size",
            "gla_norm_gate", "gla_norm_gate_bwd", "gla_norm_gate_bwd_workspace_size",
            "gla_residual_norm", "gla_residual_norm_bwd", "gla_residual_norm_bwd_workspace_size")


class GlaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}" if what else status_string(status))


class gla_fwd_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("log_g", ctypes.c_void_p), ("S0", ctypes.c_void_p),
        ("O", ctypes.c_void_p), ("ST", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
        ("dtype", ctypes.c_int), ("gate", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("force_segments", ctypes.c_int), ("path", ctypes.c_int),
        ("log_b", ctypes.c_void_p), ("window_chunks", ctypes.c_int),
    ]


class gla_bwd_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("log_g", ctypes.c_void_p), ("S0", ctypes.c_void_p),
        ("grad_O", ctypes.c_void_p), ("grad_ST", ctypes.c_void_p),
        ("grad_q", ctypes.c_void_p), ("grad_k", ctypes.c_void_p), ("grad_v", ctypes.c_void_p),
        ("grad_log_g", ctypes.c_void_p), ("grad_S0", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int),
        ("dtype", ctypes.c_int), ("gate", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("path", ctypes.c_int),
        ("log_b", ctypes.c_void_p), ("grad_log_b", ctypes.c_void_p),
    ]


class gla_delta_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("log_g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("S0", ctypes.c_void_p),
        ("O", ctypes.c_void_p), ("ST", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("T", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int), ("path", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("force_segments", ctypes.c_int),
    ]


class gla_delta_bwd_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("log_g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("S0", ctypes.c_void_p),
        ("grad_O", ctypes.c_void_p), ("grad_ST", ctypes.c_void_p),
        ("grad_q", ctypes.c_void_p), ("grad_k", ctypes.c_void_p), ("grad_v", ctypes.c_void_p),
        ("grad_log_g", ctypes.c_void_p), ("grad_beta", ctypes.c_void_p), ("grad_S0", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("T", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int), ("path", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class gla_qk_norm_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3),
        ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
        ("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("start", ctypes.c_longlong),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("T", ctypes.c_int),
        ("d", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("norm", ctypes.c_int),
        ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
    ]


class gla_qk_norm_grads(ctypes.Structure):
    _fields_ = [
        ("grad_q_out", ctypes.c_void_p), ("grad_k_out", ctypes.c_void_p),
        ("grad_q", ctypes.c_void_p), ("grad_k", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3),
        ("grad_w_q", ctypes.c_void_p), ("grad_w_k", ctypes.c_void_p),
    ]


class gla_conv_params(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("x_stride", ctypes.c_longlong * 3),
        ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("S0", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int), ("d", ctypes.c_int), ("W", ctypes.c_int),
        ("activation", ctypes.c_int), ("dtype", ctypes.c_int),
    ]


class gla_conv_grads(ctypes.Structure):
    _fields_ = [
        ("grad_y", ctypes.c_void_p), ("grad_ST", ctypes.c_void_p),
        ("grad_x", ctypes.c_void_p), ("x_stride", ctypes.c_longlong * 3),
        ("grad_w", ctypes.c_void_p), ("grad_bias", ctypes.c_void_p), ("grad_S0", ctypes.c_void_p),
    ]


class gla_ssm_params(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("dt", ctypes.c_void_p), ("z", ctypes.c_void_p),
        ("Bm", ctypes.c_void_p), ("Cm", ctypes.c_void_p),
        ("x_stride", ctypes.c_longlong * 2), ("dt_stride", ctypes.c_longlong * 2), ("z_stride", ctypes.c_longlong * 2),
        ("B_stride", ctypes.c_longlong * 2), ("C_stride", ctypes.c_longlong * 2),
        ("A", ctypes.c_void_p), ("D_skip", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("S0", ctypes.c_void_p),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int), ("G", ctypes.c_int), ("N", ctypes.c_int),
        ("softplus", ctypes.c_int), ("dtype", ctypes.c_int), ("force_segments", ctypes.c_int),
    ]


class gla_ssm_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "grad_y", "grad_ST", "grad_x", "grad_dt", "grad_z", "grad_B", "grad_C", "grad_A", "grad_D", "grad_dt_bias",
        "grad_S0")]


class gla_norm_gate_params(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("gate", ctypes.c_void_p),
        ("x_stride", ctypes.c_longlong * 3), ("gate_stride", ctypes.c_longlong * 3), ("w", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int), ("d", ctypes.c_int),
        ("norm", ctypes.c_int), ("activation", ctypes.c_int), ("gate_first", ctypes.c_int),
        ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
    ]


class gla_norm_gate_grads(ctypes.Structure):
    _fields_ = [
        ("grad_y", ctypes.c_void_p), ("grad_x", ctypes.c_void_p), ("grad_gate", ctypes.c_void_p),
        ("x_stride", ctypes.c_longlong * 3), ("gate_stride", ctypes.c_longlong * 3), ("grad_w", ctypes.c_void_p),
    ]


class gla_residual_params(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("w", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("alpha", ctypes.c_float), ("rows", ctypes.c_longlong), ("D", ctypes.c_int), ("post_norm", ctypes.c_int),
        ("eps", ctypes.c_float), ("dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
    ]


class gla_residual_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "grad_h", "grad_y", "grad_x", "grad_residual", "grad_w", "grad_scale")]


# The layouts of the structs above for struct.pack: filling a ctypes structure costs a call of the Python functions below
# more than everything else in it. "0q" ends a layout on eight bytes.
_CONV = struct.Struct("@P3q3P7i0q")
_CONV_GRADS = struct.Struct("@3P3q3P")
_SSM = struct.Struct("@5P10q4P8i")
_SSM_GRADS = struct.Struct("@11P")
_GATE = struct.Struct("@2P6qP7ifi0q")
_GATE_GRADS = struct.Struct("@3P6qP")
_RESIDUAL = struct.Struct("@4Pfqiifii0q")
_RESIDUAL_GRADS = struct.Struct("@6P")
_LAYOUTS = {gla_conv_params: _CONV, gla_conv_grads: _CONV_GRADS, gla_ssm_params: _SSM, gla_ssm_grads: _SSM_GRADS,
            gla_norm_gate_params: _GATE, gla_norm_gate_grads: _GATE_GRADS, gla_residual_params: _RESIDUAL,
            gla_residual_grads: _RESIDUAL_GRADS}
# name, arguments (n: a size, else a pointer), result
_PACKED = (("gla_conv_fwd", "pppp", ctypes.c_int), ("gla_conv_bwd", "pppnp", ctypes.c_int),
           ("gla_conv_bwd_workspace_size", "p", ctypes.c_size_t),
           ("gla_ssm_fwd", "ppppnp", ctypes.c_int), ("gla_ssm_fwd_workspace_size", "p", ctypes.c_size_t),
           ("gla_ssm_bwd", "pppnp", ctypes.c_int), ("gla_ssm_bwd_workspace_size", "p", ctypes.c_size_t),
           ("gla_norm_gate", "ppp", ctypes.c_int), ("gla_norm_gate_bwd", "pppnp", ctypes.c_int),
           ("gla_norm_gate_bwd_workspace_size", "p", ctypes.c_size_t),
           ("gla_residual_norm", "pppp", ctypes.c_int), ("gla_residual_norm_bwd", "pppnp", ctypes.c_int),
           ("gla_residual_norm_bwd_workspace_size", "p", ctypes.c_size_t))


class _raw:
    """The packed calls' functions, by name, once the library is loaded."""


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libgla.so. Raises if it is missing (unless build_if_missing) or unloadable."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(f"libgla.so not built ({path}); run __graft_entry__.build() "
                                   "or python -m chunkwise_gated_linear_gla_gb300.build")
            _build.build()
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(gla_fwd_params)
        vp, i, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
        lib.gla_fwd.restype = st
        lib.gla_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.gla_fwd_noalloc.restype = st
        lib.gla_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.gla_fwd_ex.restype = st
        lib.gla_fwd_ex.argtypes = [P, vp]
        lib.gla_fwd_workspace_size.restype = ctypes.c_size_t
        lib.gla_fwd_workspace_size.argtypes = [P]
        lib.gla_fwd_num_stages.restype = i
        lib.gla_fwd_num_stages.argtypes = [P]
        lib.gla_fwd_stage.restype = st
        lib.gla_fwd_stage.argtypes = [P, i, vp]
        lib.gla_fwd_stage_name.restype = ctypes.c_char_p
        lib.gla_fwd_stage_name.argtypes = [P, i]
        lib.gla_bwd.restype = st
        lib.gla_bwd.argtypes = [ctypes.POINTER(gla_bwd_params), vp]
        lib.gla_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gla_bwd_workspace_size.argtypes = [ctypes.POINTER(gla_bwd_params)]
        lib.gla_bwd_num_stages.restype = i
        lib.gla_bwd_num_stages.argtypes = [ctypes.POINTER(gla_bwd_params)]
        lib.gla_bwd_stage.restype = st
        lib.gla_bwd_stage.argtypes = [ctypes.POINTER(gla_bwd_params), i, vp]
        lib.gla_bwd_stage_name.restype = ctypes.c_char_p
        lib.gla_bwd_stage_name.argtypes = [ctypes.POINTER(gla_bwd_params), i]
        lib.gla_fwd_host.restype = st
        lib.gla_fwd_host.argtypes = [P, ctypes.c_size_t, vp]
        lib.gla_host_release.restype = st
        lib.gla_host_release.argtypes = []
        lib.gla_device_status.restype = st
        lib.gla_device_status.argtypes = [vp]
        lib.gla_status_string.restype = ctypes.c_char_p
        lib.gla_status_string.argtypes = [st]
        lib.gla_version.restype = i
        lib.gla_version.argtypes = []
        lib.gla_segment_pair_workspace_size.restype = ctypes.c_size_t
        lib.gla_segment_pair_workspace_size.argtypes = [P]
        lib.gla_segment_pair.restype = st
        lib.gla_segment_pair.argtypes = [P, vp, vp, vp]
        lib.gla_pair_scan.restype = st
        lib.gla_pair_scan.argtypes = [i, vp, vp, vp, vp, vp, i, i, i, i, vp]
        lib.gla_selftest_bounded_wait.restype = st
        lib.gla_selftest_bounded_wait.argtypes = [ctypes.c_uint, i, vp]
        lib.gla_pair_combine.restype = st
        lib.gla_pair_combine.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
        D, DB = ctypes.POINTER(gla_delta_params), ctypes.POINTER(gla_delta_bwd_params)
        N, NG = ctypes.POINTER(gla_qk_norm_params), ctypes.POINTER(gla_qk_norm_grads)
        C, CG = ctypes.POINTER(gla_conv_params), ctypes.POINTER(gla_conv_grads)
        S, SG = ctypes.POINTER(gla_ssm_params), ctypes.POINTER(gla_ssm_grads)
        NR, NRG = ctypes.POINTER(gla_norm_gate_params), ctypes.POINTER(gla_norm_gate_grads)
        R, RG = ctypes.POINTER(gla_residual_params), ctypes.POINTER(gla_residual_grads)
        for name, restype, argtypes in (
                ("gla_delta_fwd", st, [D, vp]), ("gla_delta_fwd_workspace_size", ctypes.c_size_t, [D]),
                ("gla_delta_bwd", st, [DB, vp]), ("gla_delta_bwd_workspace_size", ctypes.c_size_t, [DB]),
                ("gla_qk_norm_rope", st, [N, vp, vp, vp]),
                ("gla_qk_norm_rope_bwd", st, [N, NG, vp, ctypes.c_size_t, vp]),
                ("gla_qk_norm_rope_bwd_workspace_size", ctypes.c_size_t, [N]),
                ("gla_conv_fwd", st, [C, vp, vp, vp]), ("gla_conv_bwd", st, [C, CG, vp, ctypes.c_size_t, vp]),
                ("gla_conv_bwd_workspace_size", ctypes.c_size_t, [C]),
                ("gla_ssm_fwd", st, [S, vp, vp, vp, ctypes.c_size_t, vp]), ("gla_ssm_fwd_workspace_size", ctypes.c_size_t, [S]),
                ("gla_ssm_bwd", st, [S, SG, vp, ctypes.c_size_t, vp]), ("gla_ssm_bwd_workspace_size", ctypes.c_size_t, [S]),
                ("gla_norm_gate", st, [NR, vp, vp]), ("gla_norm_gate_bwd", st, [NR, NRG, vp, ctypes.c_size_t, vp]),
                ("gla_norm_gate_bwd_workspace_size", ctypes.c_size_t, [NR]),
                ("gla_residual_norm", st, [R, vp, vp, vp]), ("gla_residual_norm_bwd", st, [R, RG, vp, ctypes.c_size_t, vp]),
                ("gla_residual_norm_bwd_workspace_size", ctypes.c_size_t, [R])):
            f = getattr(lib, name)
            f.restype, f.argtypes = restype, argtypes
        # the same calls for parameters packed into bytes
        for s, layout in _LAYOUTS.items():
            if layout.size != ctypes.sizeof(s):
                raise RuntimeError(f"{s.__name__}: {layout.size} bytes packed, {ctypes.sizeof(s)} in C")
        for name, args, restype in _PACKED:
            f = lib[name]
            f.restype, f.argtypes = restype, [ctypes.c_size_t if a == "n" else vp for a in args]
            setattr(_raw, name, f)
        _lib = lib
        return lib


def status_string(s: int) -> str:
    try:
        return load().gla_status_string(int(s)).decode()
    except Exception:  # pragma: no cover - library missing
        return f"gla_status {s}"


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr() if t.numel() > 0 else None


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(s: int, what: str):
    if s != GLA_OK:
        raise GlaError(s, what)


# ---------------------------------------------------------------- C names

def gla_fwd(q, k, v, log_g, S0, O, ST, B, H, T, dk, dv, chunk=64, stream=None, check=True) -> int:
    s = load().gla_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_g), _ptr(S0), _ptr(O), _ptr(ST),
                       B, H, T, dk, dv, chunk, _stream(stream))
    if check:
        _check(s, "gla_fwd")
    return s


def gla_fwd_noalloc(q, k, v, log_g, S0, O, ST, B, H, T, dk, dv, chunk=64, stream=None, check=True) -> int:
    """gla_fwd without any device allocation (library-owned fixed scratch); see include/gla.h."""
    s = load().gla_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_g), _ptr(S0), _ptr(O), _ptr(ST),
                               B, H, T, dk, dv, chunk, _stream(stream))
    if check:
        _check(s, "gla_fwd_noalloc")
    return s


def gla_fwd_ex(p: gla_fwd_params, stream=None, check=True) -> int:
    s = load().gla_fwd_ex(ctypes.byref(p), _stream(stream))
    if check:
        _check(s, "gla_fwd_ex")
    return s


def gla_fwd_host(p: gla_fwd_params, slice_bytes=0, stream=None, check=True) -> int:
    """gla_fwd_ex with host tensors (see include/gla.h); returns once O and S_T are on the host."""
    s = load().gla_fwd_host(ctypes.byref(p), slice_bytes, _stream(stream))
    if check:
        _check(s, "gla_fwd_host")
    return s


def gla_host_release(check=True) -> int:
    s = load().gla_host_release()
    if check:
        _check(s, "gla_host_release")
    return s


def gla_bwd(p: gla_bwd_params, stream=None, check=True) -> int:
    s = load().gla_bwd(ctypes.byref(p), _stream(stream))
    if check:
        _check(s, "gla_bwd")
    return s


def gla_bwd_workspace_size(p: gla_bwd_params) -> int:
    return int(load().gla_bwd_workspace_size(ctypes.byref(p)))


def gla_bwd_num_stages(p: gla_bwd_params) -> int:
    return int(load().gla_bwd_num_stages(ctypes.byref(p)))


def gla_bwd_stage(p: gla_bwd_params, stage: int, stream=None, check=True) -> int:
    s = load().gla_bwd_stage(ctypes.byref(p), stage, _stream(stream))
    if check:
        _check(s, f"gla_bwd_stage({stage})")
    return s


def gla_bwd_stage_name(p: gla_bwd_params, stage: int) -> str:
    return load().gla_bwd_stage_name(ctypes.byref(p), stage).decode()


def make_bwd_params(q, k, v, log_g, S0, dO, dST, dq, dk, dv, dlog_g, dS0, gate=None,
                    workspace=None, path=GLA_PATH_AUTO, log_b=None, dlog_b=None) -> gla_bwd_params:
    """Fill gla_bwd_params from torch tensors (shapes read from q and v).
    log_b (the bilinear gate's log beta) selects GLA_GATE_BILINEAR; dlog_b receives its gradient."""
    import torch
    B, H, T, dk_ = q.shape
    if gate is None and log_b is not None:
        gate = GLA_GATE_BILINEAR
    if gate is None:
        if log_g is None:
            gate = GLA_GATE_NONE
        else:
            gate = {1: GLA_GATE_HEAD_SCALAR, 3: GLA_GATE_TOKEN_SCALAR}.get(log_g.dim(), GLA_GATE_PER_KEY)
    p = gla_bwd_params()
    p.q, p.k, p.v, p.log_g, p.S0 = _ptr(q), _ptr(k), _ptr(v), _ptr(log_g), _ptr(S0)
    p.grad_O, p.grad_ST = _ptr(dO), _ptr(dST)
    p.grad_q, p.grad_k, p.grad_v, p.grad_log_g, p.grad_S0 = _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_g), _ptr(dS0)
    p.B, p.H, p.T, p.dk, p.dv = B, H, T, dk_, v.shape[-1]
    p.dtype = GLA_BF16 if q.dtype == torch.bfloat16 else GLA_FP32
    p.gate = gate
    p.workspace = _ptr(workspace)
    p.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    p.path = path
    p.log_b, p.grad_log_b = _ptr(log_b), _ptr(dlog_b)
    return p


def backward(q, k, v, log_g, S0, dO, dST=None, gate=None, want_dS0=True, stream=None, path=GLA_PATH_AUTO,
             log_b=None):
    """Allocate the gradients and the workspace with torch, then call gla_bwd.

    Returns (dq, dk, dv, dlog_g, dS0), fp32; dlog_g is None without a gate and
    dS0 None unless wanted. With the bilinear gate (log_b given) dlog_b is
    appended.
    """
    import torch
    B, H, T, dk_ = q.shape
    dv_ = v.shape[-1]
    dev = q.device
    dq = torch.empty((B, H, T, dk_), dtype=torch.float32, device=dev)
    dk = torch.empty((B, H, T, dk_), dtype=torch.float32, device=dev)
    dv = torch.empty((B, H, T, dv_), dtype=torch.float32, device=dev)
    dg = None if log_g is None else torch.empty(log_g.shape, dtype=torch.float32, device=dev)
    dS0 = torch.empty((B, H, dk_, dv_), dtype=torch.float32, device=dev) if want_dS0 else None
    db = None if log_b is None else torch.empty(log_b.shape, dtype=torch.float32, device=dev)
    p = make_bwd_params(q, k, v, log_g, S0, dO, dST, dq, dk, dv, dg, dS0, gate, path=path, log_b=log_b, dlog_b=db)
    n = gla_bwd_workspace_size(p)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    p.workspace, p.workspace_bytes = ws.data_ptr(), n
    gla_bwd(p, stream)
    if log_b is not None:
        return dq, dk, dv, dg, dS0, db
    return dq, dk, dv, dg, dS0


def gla_fwd_workspace_size(p: gla_fwd_params) -> int:
    return int(load().gla_fwd_workspace_size(ctypes.byref(p)))


def gla_fwd_num_stages(p: gla_fwd_params) -> int:
    return int(load().gla_fwd_num_stages(ctypes.byref(p)))


def gla_fwd_stage(p: gla_fwd_params, stage: int, stream=None, check=True) -> int:
    s = load().gla_fwd_stage(ctypes.byref(p), stage, _stream(stream))
    if check:
        _check(s, f"gla_fwd_stage({stage})")
    return s


def gla_fwd_stage_name(p: gla_fwd_params, stage: int) -> str:
    return load().gla_fwd_stage_name(ctypes.byref(p), stage).decode()


def gla_device_status(stream=None) -> int:
    return int(load().gla_device_status(_stream(stream)))


def gla_status_string(s: int) -> str:
    return load().gla_status_string(int(s)).decode()


def gla_version() -> int:
    return int(load().gla_version())


def gla_segment_pair_workspace_size(p: gla_fwd_params) -> int:
    return int(load().gla_segment_pair_workspace_size(ctypes.byref(p)))


def gla_segment_pair(p: gla_fwd_params, log_Gamma, S_star, stream=None, check=True) -> int:
    s = load().gla_segment_pair(ctypes.byref(p), _ptr(log_Gamma), _ptr(S_star), _stream(stream))
    if check:
        _check(s, "gla_segment_pair")
    return s


def gla_pair_scan(P, log_Gamma, S_star, S0, S_in, S_T, B, H, dk, dv, stream=None, check=True) -> int:
    s = load().gla_pair_scan(P, _ptr(log_Gamma), _ptr(S_star), _ptr(S0), _ptr(S_in), _ptr(S_T),
                             B, H, dk, dv, _stream(stream))
    if check:
        _check(s, "gla_pair_scan")
    return s


def gla_pair_combine(log_Gamma2, S2, log_Gamma1, S1, B, H, dk, dv, stream=None, check=True) -> int:
    s = load().gla_pair_combine(_ptr(log_Gamma2), _ptr(S2), _ptr(log_Gamma1), _ptr(S1), B, H, dk, dv,
                                _stream(stream))
    if check:
        _check(s, "gla_pair_combine")
    return s


def gla_selftest_bounded_wait(limit_us: int, arrive: bool = False, stream=None, check=True) -> int:
    s = load().gla_selftest_bounded_wait(int(limit_us), 1 if arrive else 0, _stream(stream))
    if check:
        _check(s, "gla_selftest_bounded_wait")
    return s


# ---------------------------------------------------------------- marshalling helpers

def make_params(q, k, v, log_g, S0, O, ST, gate=None, path=GLA_PATH_AUTO, force_segments=0,
                workspace=None, chunk=64, log_b=None, window_chunks=0) -> gla_fwd_params:
    """Fill gla_fwd_params from torch tensors (shapes read from q and v).
    log_b (the bilinear gate's log beta, [B,H,T,dv]) selects GLA_GATE_BILINEAR."""
    import torch
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if gate is None and log_b is not None:
        gate = GLA_GATE_BILINEAR
    if gate is None:
        if log_g is None:
            gate = GLA_GATE_NONE
        else:
            gate = {1: GLA_GATE_HEAD_SCALAR, 3: GLA_GATE_TOKEN_SCALAR}.get(log_g.dim(), GLA_GATE_PER_KEY)
    p = gla_fwd_params()
    p.q, p.k, p.v = _ptr(q), _ptr(k), _ptr(v)
    p.log_g, p.S0, p.O, p.ST = _ptr(log_g), _ptr(S0), _ptr(O), _ptr(ST)
    p.B, p.H, p.T, p.dk, p.dv, p.chunk = B, H, T, dk, dv, chunk
    p.dtype = GLA_BF16 if q.dtype == torch.bfloat16 else GLA_FP32
    p.gate = gate
    p.workspace = _ptr(workspace)
    p.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    p.force_segments = force_segments
    p.path = path
    p.log_b = _ptr(log_b)
    p.window_chunks = window_chunks
    return p


def forward(q, k, v, log_g=None, S0=None, gate=None, want_state=True, path=GLA_PATH_AUTO,
            force_segments=0, stream=None, O=None, ST=None, log_b=None, window_chunks=0):
    """Allocate O (and ST) and the workspace with torch, then call gla_fwd_ex.

    q, k: [B,H,T,dk]; v: [B,H,T,dv] (bf16 or fp32, on the GPU); log_g fp32
    [B,H,T,dk] (per key) or [H] (per-head scalar) or None; S0 fp32 [B,H,dk,dv]
    or None. Returns (O, ST).
    """
    import torch
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if O is None:
        O = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if ST is None and want_state:
        ST = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    p = make_params(q, k, v, log_g, S0, O, ST, gate, path, force_segments, log_b=log_b,
                    window_chunks=window_chunks)
    nbytes = gla_fwd_workspace_size(p)
    ws = None
    if nbytes > 0:
        ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=q.device)
        off = (-ws.data_ptr()) % 256
        ws = ws[off:off + nbytes]
        p.workspace = ws.data_ptr()
        p.workspace_bytes = nbytes
    gla_fwd_ex(p, stream)
    return O, ST


def _aligned_workspace(nbytes, device):
    import torch
    if nbytes == 0:
        return None
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes]


def segment_pair(k, v, log_g=None, gate=None, q=None, path=GLA_PATH_AUTO, stream=None):
    """The exchange pair (log Gamma [B,H,dk], S* [B,H,dk,dv], both fp32) of the segment
    whose k, v, gate are given, from a zero start (gla_segment_pair)."""
    import torch
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    log_G = torch.empty((B, H, dk), dtype=torch.float32, device=k.device)
    S_star = torch.empty((B, H, dk, dv), dtype=torch.float32, device=k.device)
    p = make_params(k, k, v, log_g, None, None, None, gate, path)
    p.q = _ptr(q)
    ws = _aligned_workspace(gla_segment_pair_workspace_size(p), k.device)
    if ws is not None:
        p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
    gla_segment_pair(p, log_G, S_star, stream)
    return log_G, S_star


def pair_scan(log_Gamma, S_star, S0=None, want_S_in=True, stream=None):
    """States entering each of P segments and after the last, from pairs stacked in
    sequence order (log_Gamma [P,B,H,dk], S_star [P,B,H,dk,dv]): (S_in [P,...] or None, S_T)."""
    import torch
    P, B, H, dk = log_Gamma.shape
    dv = S_star.shape[-1]
    S_in = torch.empty_like(S_star) if want_S_in else None
    S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=S_star.device)
    gla_pair_scan(P, log_Gamma, S_star, S0, S_in, S_T, B, H, dk, dv, stream)
    return S_in, S_T


def pair_combine(log_Gamma2, S2, log_Gamma1, S1, stream=None):
    """In place: (log_Gamma1, S1) <- (log_Gamma2, S2) o (log_Gamma1, S1); pair 1 is the earlier segment."""
    B, H, dk, dv = S1.shape
    gla_pair_combine(log_Gamma2, S2, log_Gamma1, S1, B, H, dk, dv, stream)
    return log_Gamma1, S1


# ---------------------------------------------------------------- the gated delta rule

def gla_delta_fwd(p: gla_delta_params, stream=None, check=True) -> int:
    s = load().gla_delta_fwd(ctypes.byref(p), _stream(stream))
    if check:
        _check(s, "gla_delta_fwd")
    return s


def gla_delta_fwd_workspace_size(p: gla_delta_params) -> int:
    return load().gla_delta_fwd_workspace_size(ctypes.byref(p))


def gla_delta_bwd(p: gla_delta_bwd_params, stream=None, check=True) -> int:
    s = load().gla_delta_bwd(ctypes.byref(p), _stream(stream))
    if check:
        _check(s, "gla_delta_bwd")
    return s


def gla_delta_bwd_workspace_size(p: gla_delta_bwd_params) -> int:
    return load().gla_delta_bwd_workspace_size(ctypes.byref(p))


def _refuse(what):
    raise GlaError(GLA_ERR_INVALID_ARG, what)


def _dense(t, shape, dtype, device, what):
    """A contiguous tensor of this shape, type and device (the C ABI sees pointers only)."""
    if t.shape != shape:
        _refuse(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != dtype:
        _refuse(f"{what} is {t.dtype}, not {dtype}")
    if t.device != device:
        _refuse(f"{what} is on {t.device}, not on {device}")
    if not t.is_contiguous():
        _refuse(f"{what} is not contiguous")


def _dtype_code(t, what):
    import torch
    if t.dtype == torch.bfloat16:
        return GLA_BF16
    if t.dtype == torch.float32:
        return GLA_FP32
    _refuse(f"{what} is {t.dtype}, not bfloat16 or float32")


def _on_gpu(t, what):
    if not t.is_cuda:
        _refuse(f"{what} is on {t.device}, not on a GPU")


def _launch(f, name, p, device, stream, *tensors):
    """Calls f(byref(p), stream) with the tensors' device current; raises on an error. `tensors`
    (may be None) were allocated for this call and are used on `stream`."""
    import torch
    index = device.index
    was = torch._C._cuda_getDevice()
    if was != index:
        torch.cuda.set_device(index)
    try:
        if stream is None:
            s = f(ctypes.byref(p), torch._C._cuda_getCurrentRawStream(index))
        else:
            _used_on(stream, device, *tensors)
            s = f(ctypes.byref(p), _stream(stream))
    finally:
        if was != index:
            torch.cuda.set_device(was)
    if s != GLA_OK:
        raise GlaError(s, name)


def _used_on(stream, device, *tensors):
    """Tensors allocated here but used on another stream than the current one are not reused
    before that stream is done with them."""
    if stream is None:
        return
    import torch
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    if s != torch.cuda.current_stream(device):
        s.wait_stream(torch.cuda.current_stream(device))
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def _given(t, what):
    """An output tensor of the caller's: as with torch's own `out=`, it takes no part in autograd."""
    import torch
    if t.requires_grad and torch.is_grad_enabled():
        _refuse(f"{what} requires grad and is written in place")


def _written(*tensors):
    """Counts tensors of the caller's as written, so that a graph which saved one of them says so. (Inference
    tensors have no versions.)"""
    import torch
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _delta_shapes(q, k, v, log_g, beta, S0):
    import torch
    if q.dim() != 4 or v.dim() != 4:
        _refuse("q and v have four dimensions: [B,Hk,T,dk] and [B,H,T,dv]")
    shape, dt, dev, f32 = q.shape, q.dtype, q.device, torch.float32
    B, Hk, T, dk = shape
    _, H, _, dv = v.shape
    code = _dtype_code(q, "q")
    if Hk == 0 or H % Hk:
        _refuse(f"{H} heads of v do not divide over {Hk} of q and k")
    # one look at everything; what is wrong is told below
    if not (k.shape == shape and v.shape == (B, H, T, dv) and beta.shape == (B, H, T) and k.dtype is dt and
            v.dtype is dt and beta.dtype is dt and k.device == dev and v.device == dev and beta.device == dev and
            q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and beta.is_contiguous()):
        _dense(q, (B, Hk, T, dk), dt, dev, "q")
        _dense(k, (B, Hk, T, dk), dt, dev, "k")
        _dense(v, (B, H, T, dv), dt, dev, "v")
        _dense(beta, (B, H, T), dt, dev, "beta")
    if log_g is not None:
        _dense(log_g, (B, H, T), f32, dev, "log_g")
    if S0 is not None:
        _dense(S0, (B, H, dk, dv), f32, dev, "S0")
    return B, H, Hk, T, dk, dv, code, dt, dev


def delta_forward(q, k, v, log_g, beta, S0=None, scale=None, want_state=True, path=GLA_PATH_AUTO, stream=None,
                  O=None, ST=None, force_segments=0):
    """The gated delta rule's forward pass (gla_delta_fwd), outputs and workspace from torch.

    q, k [B,Hk,T,dk], v [B,H,T,dv], beta [B,H,T] (bf16 or fp32, one type); log_g fp32 [B,H,T] or
    None; S0 fp32 [B,H,dk,dv] or None; scale defaults to dk^-0.5. Returns (O, S_T). A decoding
    loop passes ST=S0 to carry the state in place; O and ST count as modified in place. Values are finite
    (log_g may be -inf), those of padded rows too. Tensors are contiguous and start on 16 bytes (log_g and beta on
    their values' size). With `stream` the outputs may be used there,
    and on other streams after it.
    """
    import torch
    B, H, Hk, T, dk, dv, code, dt, dev = _delta_shapes(q, k, v, log_g, beta, S0)
    if O is not None:
        _dense(O, (B, H, T, dv), dt, dev, "O")
        _given(O, "O")
    if ST is not None:
        _dense(ST, (B, H, dk, dv), torch.float32, dev, "ST")
        _given(ST, "ST")
    given = O, ST
    _on_gpu(q, "q")
    if B == 0:
        _refuse("an empty batch")
    lib = _lib or load()
    if O is None:
        O = torch.empty_like(v)
    if ST is None and want_state:
        ST = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if S0 is None else torch.empty_like(S0)
    p = gla_delta_params(_ptr(q), _ptr(k), _ptr(v), _ptr(log_g), _ptr(beta), _ptr(S0), _ptr(O), _ptr(ST),
                         B, H, Hk, T, dk, dv, dk ** -0.5 if scale is None else scale, code, path, None, 0, force_segments)
    n = 0 if T <= 64 else _here_size(lib.gla_delta_fwd_workspace_size, p, dev)   # (one chunk needs none)
    ws = None
    if n:
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        p.workspace, p.workspace_bytes = ws.data_ptr(), n
    _launch(lib.gla_delta_fwd, "gla_delta_fwd", p, dev, stream, O, ST, ws)
    _written(*given)
    return O, ST


def delta_backward(q, k, v, log_g, beta, S0, dO, dST=None, scale=None, want_dS0=True, path=GLA_PATH_AUTO, stream=None):
    """The gated delta rule's gradients (gla_delta_bwd): (dq, dk, dv, dlog_g, dbeta, dS0); dq, dk, dv
    and dbeta in the inputs' type, dlog_g and dS0 fp32, dlog_g None without log_g and dS0 None
    unless wanted (it is defined without S0 too, a zero state)."""
    import torch
    B, H, Hk, T, dk, dv, code, dt, dev = _delta_shapes(q, k, v, log_g, beta, S0)
    _dense(dO, (B, H, T, dv), dt, dev, "dO")
    if dST is not None:
        _dense(dST, (B, H, dk, dv), torch.float32, dev, "dST")
    _on_gpu(q, "q")
    if B == 0:
        _refuse("an empty batch")
    lib = _lib or load()
    gq, gk, gv, gb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(beta)
    gg = None if log_g is None else torch.empty_like(log_g)
    gS = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if want_dS0 else None
    p = gla_delta_bwd_params(_ptr(q), _ptr(k), _ptr(v), _ptr(log_g), _ptr(beta), _ptr(S0), _ptr(dO), _ptr(dST),
                             _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gg), _ptr(gb), _ptr(gS),
                             B, H, Hk, T, dk, dv, dk ** -0.5 if scale is None else scale, code, path)
    n = lib.gla_delta_bwd_workspace_size(ctypes.byref(p))
    ws = None
    if n:
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        p.workspace, p.workspace_bytes = ws.data_ptr(), n
    _launch(lib.gla_delta_bwd, "gla_delta_bwd", p, dev, stream, gq, gk, gv, gg, gb, gS, ws)
    return gq, gk, gv, gg, gb, gS


# ---------------------------------------------------------------- norms of q and k, and the rotation

_NORMS = {None: GLA_NORM_NONE, "l2": GLA_NORM_L2, "rms": GLA_NORM_RMS}


def gla_qk_norm_rope(p: gla_qk_norm_params, q_out, k_out, stream=None, check=True) -> int:
    s = load().gla_qk_norm_rope(ctypes.byref(p), _ptr(q_out), _ptr(k_out), _stream(stream))
    if check:
        _check(s, "gla_qk_norm_rope")
    return s


def gla_qk_norm_rope_bwd(p: gla_qk_norm_params, g: gla_qk_norm_grads, workspace=None, stream=None, check=True) -> int:
    n = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = load().gla_qk_norm_rope_bwd(ctypes.byref(p), ctypes.byref(g), _ptr(workspace), n, _stream(stream))
    if check:
        _check(s, "gla_qk_norm_rope_bwd")
    return s


def gla_qk_norm_rope_bwd_workspace_size(p: gla_qk_norm_params) -> int:
    return load().gla_qk_norm_rope_bwd_workspace_size(ctypes.byref(p))


_Steps = ctypes.c_longlong * 3
_NO_STEPS = _Steps()


def _steps(s, B, H, T):
    """(batch, head, token) strides; those of dimensions of one are never stepped and count as 0."""
    return _Steps(s[0] if B > 1 else 0, s[1] if H > 1 else 0, s[2] if T > 1 else 0)


def _qk_params(q, k, norm, w_q, w_k, eps, inv_freq, positions, start, interleaved):
    import torch
    if norm not in _NORMS:
        _refuse(f"norm is None, 'l2' or 'rms', not {norm!r}")
    if q.dim() != 4:
        _refuse("q has four dimensions: [B,H,T,d]")
    B, H, T, d = q.shape
    dt, dev, f32 = q.dtype, q.device, torch.float32
    code = _dtype_code(q, "q")
    qs, ks, Hk, pk = q.stride(), None, 0, None
    if k is not None:
        if k.dim() != 4 or (k.shape[0], k.shape[2], k.shape[3]) != (B, T, d):
            _refuse(f"k has shape {tuple(k.shape)}, not [{B},Hk,{T},{d}]")
        if k.dtype != dt or k.device != dev:
            _refuse("k has another type or device than q")
        ks, Hk, pk = k.stride(), k.shape[1], _ptr(k)
    for s, what in ((qs, "q"), (ks, "k")):
        if s is not None and s[3] != 1 and d > 1:
            _refuse(f"the last dimension of {what} is not contiguous")
    # one look at each; what is wrong is told below
    for w, what in ((w_q, "w_q"), (w_k, "w_k")):
        if w is not None and not (w.shape == (d,) and w.dtype is f32 and w.device == dev and w.is_contiguous()):
            _dense(w, (d,), f32, dev, what)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _dense(inv_freq, (rot // 2,), torch.float64, dev, "inv_freq")
    if positions is not None:
        _dense(positions, (B, T), torch.int64, dev, "positions")
    _on_gpu(q, "q")
    return gla_qk_norm_params(_ptr(q), pk, _steps(qs, B, H, T), _NO_STEPS if ks is None else _steps(ks, B, Hk, T),
                              _ptr(w_q), _ptr(w_k), _ptr(inv_freq), _ptr(positions), start, B, H, Hk, T, d, rot,
                              1 if interleaved else 0, _NORMS[norm], eps, code)


def qk_norm_rope_forward(q, k=None, norm="l2", w_q=None, w_k=None, eps=1e-6, inv_freq=None, positions=None, start=0,
                         interleaved=False, stream=None):
    """Norm, weight and position rotation of every row of q [B,H,T,d] and k [B,Hk,T,d] (or None) in
    one pass (gla_qk_norm_rope). Inputs may be strided views, the last dimension contiguous and every row, and the
    weights, from a 16-byte boundary; returns dense (q', k'). inv_freq: fp64 [rot/2], radians per position (None: no rotation);
    positions: int64 [B,T], else start + t."""
    import torch
    p = _qk_params(q, k, norm, w_q, w_k, eps, inv_freq, positions, start, interleaved)
    lib, dev = _lib or load(), q.device
    qo = q.new_empty(q.shape)
    ko = None if k is None else k.new_empty(k.shape)
    po, pk = _ptr(qo), _ptr(ko)
    _launch(lambda r, s: lib.gla_qk_norm_rope(r, po, pk, s), "gla_qk_norm_rope", p, dev, stream, qo, ko)
    return qo, ko


def _rows_like(t):
    """An uninitialised tensor for t's gradient: token-major as a projection's slices are, when t is
    such a view, else dense."""
    if t.is_contiguous() or t.stride(1) >= t.stride(2):
        return t.new_empty(t.shape)
    B, H, T, d = t.shape
    return t.new_empty((B, T, H, d)).transpose(1, 2)


def _here_size(f, p, device):
    """A workspace size that depends on the device's multiprocessors."""
    import torch
    if torch._C._cuda_getDevice() == device.index:
        return f(ctypes.byref(p))
    with torch.cuda.device(device):
        return f(ctypes.byref(p))


def qk_norm_rope_backward(q, k, dq_out, dk_out, norm="l2", w_q=None, w_k=None, eps=1e-6, inv_freq=None,
                          positions=None, start=0, interleaved=False, stream=None):
    """Gradients of qk_norm_rope_forward: (dq, dk, dw_q, dw_k); dq and dk in the inputs' type (token-major
    where the input is a token-major view), the weights' fp32, None where there is no input."""
    import torch
    p = _qk_params(q, k, norm, w_q, w_k, eps, inv_freq, positions, start, interleaved)
    _dense(dq_out, q.shape, q.dtype, q.device, "dq_out")
    if k is not None:
        _dense(dk_out, k.shape, k.dtype, k.device, "dk_out")
    lib, dev = _lib or load(), q.device
    gq, gk = _rows_like(q), None if k is None else _rows_like(k)
    gwq = None if w_q is None else torch.empty_like(w_q)
    gwk = None if w_k is None or k is None else torch.empty_like(w_k)
    B, H, T, _ = q.shape
    g = gla_qk_norm_grads(_ptr(dq_out), None if k is None else _ptr(dk_out), _ptr(gq), _ptr(gk),
                          _steps(gq.stride(), B, H, T),
                          _NO_STEPS if k is None else _steps(gk.stride(), B, k.shape[1], T), _ptr(gwq), _ptr(gwk))
    n, ws = 0, None
    if gwq is not None or gwk is not None:
        n = _here_size(lib.gla_qk_norm_rope_bwd_workspace_size, p, dev)
        if n:
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    pw = _ptr(ws)
    _launch(lambda r, s: lib.gla_qk_norm_rope_bwd(r, ctypes.byref(g), pw, n, s), "gla_qk_norm_rope_bwd", p, dev, stream,
            gq, gk, gwq, gwk, ws)
    return gq, gk, gwq, gwk


# ---------------------------------------------------------------- what stands around the recurrences

_ACTS = {None: GLA_ACT_NONE, "silu": GLA_ACT_SILU, "sigmoid": GLA_ACT_SIGMOID}


def _ws_bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def gla_conv_fwd(p: gla_conv_params, y, ST=None, stream=None, check=True) -> int:
    s = load().gla_conv_fwd(ctypes.byref(p), _ptr(y), _ptr(ST), _stream(stream))
    if check:
        _check(s, "gla_conv_fwd")
    return s


def gla_conv_bwd(p: gla_conv_params, g: gla_conv_grads, workspace=None, stream=None, check=True) -> int:
    s = load().gla_conv_bwd(ctypes.byref(p), ctypes.byref(g), _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    if check:
        _check(s, "gla_conv_bwd")
    return s


def gla_conv_bwd_workspace_size(p: gla_conv_params) -> int:
    return load().gla_conv_bwd_workspace_size(ctypes.byref(p))


def gla_ssm_fwd(p: gla_ssm_params, y, ST=None, workspace=None, stream=None, check=True) -> int:
    s = load().gla_ssm_fwd(ctypes.byref(p), _ptr(y), _ptr(ST), _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    if check:
        _check(s, "gla_ssm_fwd")
    return s


def gla_ssm_fwd_workspace_size(p: gla_ssm_params) -> int:
    return load().gla_ssm_fwd_workspace_size(ctypes.byref(p))


def gla_ssm_bwd(p: gla_ssm_params, g: gla_ssm_grads, workspace=None, stream=None, check=True) -> int:
    s = load().gla_ssm_bwd(ctypes.byref(p), ctypes.byref(g), _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    if check:
        _check(s, "gla_ssm_bwd")
    return s


def gla_ssm_bwd_workspace_size(p: gla_ssm_params) -> int:
    return load().gla_ssm_bwd_workspace_size(ctypes.byref(p))


def gla_norm_gate(p: gla_norm_gate_params, y, stream=None, check=True) -> int:
    s = load().gla_norm_gate(ctypes.byref(p), _ptr(y), _stream(stream))
    if check:
        _check(s, "gla_norm_gate")
    return s


def gla_norm_gate_bwd(p: gla_norm_gate_params, g: gla_norm_gate_grads, workspace=None, stream=None, check=True) -> int:
    s = load().gla_norm_gate_bwd(ctypes.byref(p), ctypes.byref(g), _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    if check:
        _check(s, "gla_norm_gate_bwd")
    return s


def gla_norm_gate_bwd_workspace_size(p: gla_norm_gate_params) -> int:
    return load().gla_norm_gate_bwd_workspace_size(ctypes.byref(p))


def gla_residual_norm(p: gla_residual_params, h, y, stream=None, check=True) -> int:
    s = load().gla_residual_norm(ctypes.byref(p), _ptr(h), _ptr(y), _stream(stream))
    if check:
        _check(s, "gla_residual_norm")
    return s


def gla_residual_norm_bwd(p: gla_residual_params, g: gla_residual_grads, workspace=None, stream=None, check=True) -> int:
    s = load().gla_residual_norm_bwd(ctypes.byref(p), ctypes.byref(g), _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    if check:
        _check(s, "gla_residual_norm_bwd")
    return s


def gla_residual_norm_bwd_workspace_size(p: gla_residual_params) -> int:
    return load().gla_residual_norm_bwd_workspace_size(ctypes.byref(p))


def _rows(t, shape, dtype, device, what):
    """A tensor of this shape, type and device whose last dimension is contiguous."""
    if t.shape != shape:
        _refuse(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != dtype or t.device != device:
        _refuse(f"{what} is {t.dtype} on {t.device}, not {dtype} on {device}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        _refuse(f"the last dimension of {what} is not contiguous")


def _at(t):
    """A tensor's address (0 for none, and for one without values)."""
    return 0 if t is None else t.data_ptr()


def _pack(layout, *values):
    try:
        return layout.pack(*values)
    except (struct.error, OverflowError) as e:
        _refuse(f"an argument does not fit its C type ({e})")


def _call(name, device, stream, tensors, *args):
    """_launch for a packed call: the function's arguments but the stream, which comes last."""
    import torch
    index = device.index
    f = getattr(_raw, name)
    if stream is None and torch._C._cuda_getDevice() == index:
        s = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            if stream is None:
                s = f(*args, torch._C._cuda_getCurrentRawStream(index))
            else:
                _used_on(stream, device, *tensors)
                s = f(*args, _stream(stream))
    if s != GLA_OK:
        raise GlaError(s, name)


def _workspace(name, packed, device):
    """(tensor or None, its address, its bytes): torch hands out blocks from 512-byte boundaries. Sizes depend on the
    device's multiprocessors."""
    import torch
    if torch._C._cuda_getDevice() == device.index:
        n = getattr(_raw, name)(packed)
    else:
        with torch.cuda.device(device):
            n = getattr(_raw, name)(packed)
    if not n:
        return None, 0, 0
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), n


def _step3(s, B, H, T):
    """(batch, head, token) strides; those of dimensions of one are never stepped and count as 0."""
    return s[0] if B > 1 else 0, s[1] if H > 1 else 0, s[2] if T > 1 else 0


def _conv_params(x, w, bias, S0, activation):
    import torch
    if activation not in (None, "silu"):
        _refuse(f"activation is None or 'silu', not {activation!r}")
    shape, dt, dev, f32 = x.shape, x.dtype, x.device, torch.float32
    if len(shape) == 3:
        (B, T, d), H = shape, 1
        s = x.stride()
        steps = s[0] if B > 1 else 0, 0, s[1] if T > 1 else 0
    elif len(shape) == 4:
        B, H, T, d = shape
        s = x.stride()
        steps = _step3(s, B, H, T)
    else:
        _refuse("x has three or four dimensions: [B,T,D] or [B,H,T,d]")
    D = H * d
    code = _dtype_code(x, "x")
    if s[-1] != 1:
        _rows(x, shape, dt, dev, "x")
    if w.dim() != 2:
        _refuse("w has two dimensions: [H d, W]")
    W = w.shape[1]
    if W == 0:
        _refuse("w has no taps")
    _dense(w, (D, W), f32, dev, "w")
    if bias is not None:
        _dense(bias, (D,), f32, dev, "bias")
    if S0 is not None:
        _dense(S0, (B, W - 1, D), dt, dev, "S0")
    _on_gpu(x, "x")
    if B == 0:
        _refuse("an empty batch")
    load()
    return _pack(_CONV, x.data_ptr(), *steps, w.data_ptr(), _at(bias), _at(S0), B, H, T, d, W, _ACTS[activation], code), (B, W - 1, D)


def causal_conv_forward(x, w, bias=None, S0=None, activation="silu", want_state=True, stream=None, y=None, ST=None):
    """The short causal convolution of every channel (gla_conv_fwd), outputs from torch.

    x [B,T,D] or, head by head, [B,H,T,d] (bf16 or fp32; strided views, the last dimension contiguous and every row from a
    16-byte boundary; d, or D, a multiple of 16); w fp32 [D,W] with D = H d and W 2 to 4, bias fp32 [D] or None; S0 [B,W-1,D] in x's type, the W - 1
    rows before the first token, oldest first, or None (zeros); activation "silu" or None. Returns (y, ST): y dense in
    x's shape, ST the last W - 1 rows of (S0, x) (None unless wanted). A decoding loop passes ST=S0 to carry the state
    in place; y and ST count as modified in place. A batch of unequal prompts is padded in front, with zeros.
    """
    p, state = _conv_params(x, w, bias, S0, activation)
    dev, given = x.device, (y, ST)
    if y is None:
        y = x.new_empty(x.shape)
    else:
        _dense(y, x.shape, x.dtype, dev, "y")
        _given(y, "y")
    if ST is not None:
        _dense(ST, state, x.dtype, dev, "ST")
        _given(ST, "ST")
    elif want_state:
        ST = x.new_empty(state)
    _call("gla_conv_fwd", dev, stream, (y, ST), p, y.data_ptr(), _at(ST))
    _written(*given)
    return y, ST


def causal_conv_backward(x, w, bias, S0, dy, dST=None, activation="silu", want_dw=True, want_dS0=True, stream=None):
    """Gradients of causal_conv_forward: (dx, dw, dbias, dS0); dx (token-major where x is a token-major view) and dS0 in
    x's type, dw and dbias fp32; dw and dbias None unless wanted, dbias without a bias, dS0 unless wanted (it is defined
    without S0 too, zeros)."""
    import torch
    p, state = _conv_params(x, w, bias, S0, activation)
    dev = x.device
    _dense(dy, x.shape, x.dtype, dev, "dy")
    if dST is not None:
        _dense(dST, state, x.dtype, dev, "dST")
    gx = x.new_empty(x.shape) if x.dim() == 3 else _rows_like(x)
    gw = torch.empty_like(w) if want_dw else None
    gb = torch.empty_like(bias) if want_dw and bias is not None else None
    gs = x.new_empty(state) if want_dS0 else None
    s = gx.stride()
    if x.dim() == 3:
        steps = s[0] if x.shape[0] > 1 else 0, 0, s[1] if x.shape[1] > 1 else 0
    else:
        steps = _step3(s, *x.shape[:3])
    g = _pack(_CONV_GRADS, dy.data_ptr(), _at(dST), gx.data_ptr(), *steps, _at(gw), _at(gb), _at(gs))
    ws, pw, n = _workspace("gla_conv_bwd_workspace_size", p, dev) if want_dw else (None, 0, 0)
    _call("gla_conv_bwd", dev, stream, (gx, gw, gb, gs, ws), p, g, pw, n)
    return gx, gw, gb, gs


def _ssm_params(x, dt, A, B, C, D, z, dt_bias, S0, softplus, force_segments=0):
    import torch
    if x.dim() != 3 or B.dim() != 4 or A.dim() != 2:
        _refuse("x has three dimensions [B,T,D], B and C four [B,T,G,N], A two [D,N]")
    shape, groups, t, dev, f32 = x.shape, B.shape, x.dtype, x.device, torch.float32
    nb, T, nd = shape
    G, N = groups[2:]
    code = _dtype_code(x, "x")
    if G == 0 or nd % G:
        _refuse(f"{nd} channels do not divide over {G} groups of B and C")
    sx, sd, sB, sC, sz = x.stride(), dt.stride(), B.stride(), C.stride(), (0, 0, 1) if z is None else z.stride()
    # one look at everything; what is wrong is told below
    if not (dt.shape == shape and dt.dtype is t and dt.device == dev and groups == (nb, T, G, N) and B.dtype is t and
            B.device == dev and C.shape == groups and C.dtype is t and C.device == dev and
            (z is None or z.shape == shape and z.dtype is t and z.device == dev) and
            sx[2] == sd[2] == sB[3] == sC[3] == sz[2] == 1 and (G == 1 or sB[2] == sC[2] == N) and
            A.shape == (nd, N) and A.dtype is f32 and A.device == dev and A.is_contiguous()):
        _rows(x, (nb, T, nd), t, dev, "x")
        _rows(dt, (nb, T, nd), t, dev, "dt")
        if z is not None:
            _rows(z, (nb, T, nd), t, dev, "z")
        for m, what in ((B, "B"), (C, "C")):
            _rows(m, (nb, T, G, N), t, dev, what)
            if G > 1 and m.stride(2) != N:
                _refuse(f"the groups of {what} do not lie side by side")
        _dense(A, (nd, N), f32, dev, "A")
    if D is not None:
        _dense(D, (nd,), f32, dev, "D")
    if dt_bias is not None:
        _dense(dt_bias, (nd,), f32, dev, "dt_bias")
    if S0 is not None:
        _dense(S0, (nb, nd, N), f32, dev, "S0")
    _on_gpu(x, "x")
    if nb == 0:
        _refuse("an empty batch")
    load()
    # strides of dimensions of one are never stepped and count as 0
    b, o = nb > 1, T > 1
    return _pack(_SSM, x.data_ptr(), dt.data_ptr(), _at(z), B.data_ptr(), C.data_ptr(), b and sx[0], o and sx[1], b and sd[0],
                 o and sd[1], b and sz[0], o and sz[1], b and sB[0], o and sB[1], b and sC[0], o and sC[1], A.data_ptr(),
                 _at(D), _at(dt_bias), _at(S0), nb, T, nd, G, N, 1 if softplus else 0, code, force_segments), (nb, nd, N), T


def selective_scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, S0=None, softplus=True, want_state=True,
                           stream=None, y=None, ST=None, force_segments=0):
    """The selective scan (gla_ssm_fwd), outputs and workspace from torch.

    x, dt, z [B,T,D], B and C [B,T,G,N] (bf16 or fp32, one type; strided views, a token's row contiguous and from a 16-byte
    boundary); A fp32 [D,N], D and dt_bias fp32 [D] or None, S0 fp32 [B,D,N] or None (zero). N is 8, 16, 32 or 64, D / G a
    multiple of 8. With softplus the steps are softplus(dt + dt_bias), else dt + dt_bias. Returns (y, ST): y dense
    [B,T,D], ST fp32 [B,D,N] (None unless wanted). A decoding loop passes ST=S0 to carry the state in place; y and ST count
    as modified in place. A token is passed over where its dt is -inf (with softplus; its other values finite). Where states grow
    (A above zero), the growth over 16 tokens has to be an fp32 number.
    """
    import torch
    p, states, T = _ssm_params(x, dt, A, B, C, D, z, dt_bias, S0, softplus, force_segments)
    dev, given = x.device, (y, ST)
    if y is None:
        y = x.new_empty(x.shape)
    else:
        _dense(y, x.shape, x.dtype, dev, "y")
        _given(y, "y")
    if ST is not None:
        _dense(ST, states, torch.float32, dev, "ST")
        _given(ST, "ST")
    elif want_state:
        ST = torch.empty(states, dtype=torch.float32, device=dev)
    # (up to eight tokens are taken one by one, without a workspace)
    ws, pw, n = (None, 0, 0) if T <= 8 and not force_segments else _workspace("gla_ssm_fwd_workspace_size", p, dev)
    _call("gla_ssm_fwd", dev, stream, (y, ST, ws), p, y.data_ptr(), _at(ST), pw, n)
    _written(*given)
    return y, ST


def selective_scan_backward(x, dt, A, B, C, D, z, dt_bias, S0, dy, dST=None, softplus=True, want_dS0=True, stream=None,
                            force_segments=0):
    """Gradients of selective_scan_forward: (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dS0), dense; dx, ddt, dB, dC and dz in the
    inputs' type, the others fp32; None without the input, dS0 unless wanted (it is defined without S0 too, zero)."""
    import torch
    p, states, _ = _ssm_params(x, dt, A, B, C, D, z, dt_bias, S0, softplus, force_segments)
    dev = x.device
    _dense(dy, x.shape, x.dtype, dev, "dy")
    if dST is not None:
        _dense(dST, states, torch.float32, dev, "dST")
    like = lambda m: None if m is None else m.new_empty(m.shape)  # noqa: E731
    gx, gdt, gA, gB, gC, gD, gz, gb = (like(m) for m in (x, dt, A, B, C, D, z, dt_bias))
    gS = torch.empty(states, dtype=torch.float32, device=dev) if want_dS0 else None
    g = _pack(_SSM_GRADS, *(_at(t) for t in (dy, dST, gx, gdt, gz, gB, gC, gA, gD, gb, gS)))
    ws, pw, n = _workspace("gla_ssm_bwd_workspace_size", p, dev)
    _call("gla_ssm_bwd", dev, stream, (gx, gdt, gA, gB, gC, gD, gz, gb, gS, ws), p, g, pw, n)
    return gx, gdt, gA, gB, gC, gD, gz, gb, gS


def _gate_params(x, gate, w, norm, eps, activation, gate_first):
    import torch
    if norm not in _NORMS:
        _refuse(f"norm is None, 'l2' or 'rms', not {norm!r}")
    if activation not in ("silu", "sigmoid"):
        _refuse(f"activation is 'silu' or 'sigmoid', not {activation!r}")
    shape, dev = x.shape, x.device
    if len(shape) != 4:
        _refuse("x has four dimensions: [B,H,T,d]")
    B, H, T, d = shape
    code = _dtype_code(x, "x")
    sx, sg, pg = x.stride(), (0, 0, 0), 0
    if sx[3] != 1:
        _rows(x, shape, x.dtype, dev, "x")
    if gate is not None:
        _rows(gate, shape, x.dtype, dev, "gate")
        sg, pg = _step3(gate.stride(), B, H, T), gate.data_ptr()
    if w is not None:
        _dense(w, (d,), torch.float32, dev, "w")
    _on_gpu(x, "x")
    load()
    return _pack(_GATE, x.data_ptr(), pg, *_step3(sx, B, H, T), *sg, _at(w), B, H, T, d, _NORMS[norm], _ACTS[activation],
                 1 if gate_first else 0, eps, code)


def norm_gate_forward(x, gate=None, w=None, norm="rms", eps=1e-6, activation="silu", gate_first=False, stream=None):
    """Norm, weight and gate of every row of x [B,H,T,d] (a recurrence's output) into the output projection's layout
    (gla_norm_gate): y = w x / n(x) act(g), or with gate_first w u / n(u) of u = x act(gate); returns dense [B,T,H,d].

    x and gate (or None: no gate) may be strided views of [B,H,T,d] (bf16 or fp32, one type), the last dimension
    contiguous and every row from a 16-byte boundary; w fp32 [d] or None; norm "rms", "l2" or None; activation "silu" or
    "sigmoid"; d a multiple of 16 up to 1024."""
    p = _gate_params(x, gate, w, norm, eps, activation, gate_first)
    B, H, T, d = x.shape
    y = x.new_empty((B, T, H, d))
    _call("gla_norm_gate", x.device, stream, (y,), p, y.data_ptr())
    return y


def norm_gate_backward(x, gate, w, dy, norm="rms", eps=1e-6, activation="silu", gate_first=False, stream=None):
    """Gradients of norm_gate_forward: (dx, dgate, dw); dx and dgate in the inputs' type (token-major where the input is a
    token-major view), dw fp32; None where there is no input."""
    import torch
    p = _gate_params(x, gate, w, norm, eps, activation, gate_first)
    B, H, T, d = x.shape
    dev = x.device
    _dense(dy, (B, T, H, d), x.dtype, dev, "dy")
    gx, gg = _rows_like(x), None if gate is None else _rows_like(gate)
    gw = None if w is None else torch.empty_like(w)
    g = _pack(_GATE_GRADS, dy.data_ptr(), gx.data_ptr(), _at(gg), *_step3(gx.stride(), B, H, T),
              *((0, 0, 0) if gg is None else _step3(gg.stride(), B, H, T)), _at(gw))
    ws, pw, n = (None, 0, 0) if gw is None else _workspace("gla_norm_gate_bwd_workspace_size", p, dev)
    _call("gla_norm_gate_bwd", dev, stream, (gx, gg, gw, ws), p, g, pw, n)
    return gx, gg, gw


def _residual_params(x, residual, w, scale, post_norm, eps):
    import torch
    if x.dim() < 1:
        _refuse("x has rows: [..., D]")
    shape, dev, f32 = x.shape, x.device, torch.float32
    D = shape[-1]
    code = rcode = _dtype_code(x, "x")
    _dense(x, shape, x.dtype, dev, "x")
    if residual is not None:
        rcode = _dtype_code(residual, "residual")
        if code == GLA_FP32 and rcode != GLA_FP32:
            _refuse("an fp32 x goes into an fp32 residual")
        _dense(residual, shape, residual.dtype, dev, "residual")
    alpha, vec = 1.0, 0
    if isinstance(scale, torch.Tensor):
        _dense(scale, (D,), f32, dev, "scale")
        vec = scale.data_ptr()
    elif scale is not None:
        alpha = float(scale)
    if w is not None:
        _dense(w, (D,), f32, dev, "w")
    _on_gpu(x, "x")
    load()
    return _pack(_RESIDUAL, x.data_ptr(), _at(residual), _at(w), vec, alpha, x.numel() // D if D else 0, D,
                 1 if post_norm else 0, eps, code, rcode)


def residual_norm_forward(x, residual=None, w=None, scale=None, post_norm=False, eps=1e-6, stream=None, h=None):
    """A block's output x into the residual, and the next block's normed input out of it, in one pass
    (gla_residual_norm): h = residual + scale u, u = x or (post_norm) x / rms(x), y = w h / rms(h). Returns (h, y).

    x [..., D] (bf16 or fp32), residual of x's shape in x's type or fp32 (None: 0), both contiguous; w fp32 [D] or None;
    scale a number, fp32 [D] or None; D a multiple of 16 up to 16384, tensors from a 16-byte boundary. h has the residual's
    type and may be the residual itself (h=residual: in place); it counts as modified in place. The norm reads h before its rounding."""
    p = _residual_params(x, residual, w, scale, post_norm, eps)
    dev, given = x.device, h
    like = x if residual is None else residual
    if h is None:
        h = like.new_empty(like.shape)
    else:
        _dense(h, x.shape, like.dtype, dev, "h")
        _given(h, "h")
    y = x.new_empty(x.shape)
    _call("gla_residual_norm", dev, stream, (h, y), p, h.data_ptr(), y.data_ptr())
    _written(given)
    return h, y


def residual_norm_backward(x, residual, w, scale, dh, dy, post_norm=False, eps=1e-6, want_dx=True, want_dres=True,
                           stream=None):
    """Gradients of residual_norm_forward from those of h and y (either may be None: zero): (dx, dresidual, dw, dscale), the
    vectors' fp32; None where there is no input or it is not wanted, dscale for a number too. Where dx and dresidual are
    equal (no scale, no post_norm, one type) they are one tensor."""
    import torch
    p = _residual_params(x, residual, w, scale, post_norm, eps)
    like, dev = x if residual is None else residual, x.device
    if dh is not None:
        _dense(dh, x.shape, like.dtype, dev, "dh")
    if dy is not None:
        _dense(dy, x.shape, x.dtype, dev, "dy")
    same = want_dx and want_dres and residual is not None and scale is None and not post_norm and residual.dtype == x.dtype
    gr = residual.new_empty(residual.shape) if want_dres and residual is not None else None
    gx = gr if same else x.new_empty(x.shape) if want_dx else None
    gw = None if w is None else torch.empty_like(w)
    gs = torch.empty_like(scale) if isinstance(scale, torch.Tensor) else None
    g = _pack(_RESIDUAL_GRADS, _at(dh), _at(dy), 0 if same else _at(gx), _at(gr), _at(gw), _at(gs))
    ws, pw, n = (None, 0, 0) if gw is None and gs is None else _workspace("gla_residual_norm_bwd_workspace_size", p, dev)
    _call("gla_residual_norm_bwd", dev, stream, (gx, gr, gw, gs, ws), p, g, pw, n)
    return gx, gr, gw, gs
