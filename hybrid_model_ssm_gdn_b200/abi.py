"""ctypes declarations of the C ABI in include/rssm.h (argument marshalling only).

The shared library is ``lib/librssm.so`` next to this file, built by
``hybrid_model_ssm_gdn_b200.build``.  Loading fails loudly if it is missing:
there is no fallback implementation.
"""

from __future__ import annotations

import ctypes as C
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "librssm.so")

# enums (values as in include/rssm.h)
MAMBA2, GDN = 0, 1
F32, BF16 = 0, 1
HP_F32, HP_F16_SR, HP_F8_SR = 0, 1, 2
READ_SAME, READ_NVFP4, READ_SHARED_NVFP4, READ_NVFP4D = 0, 1, 2, 3
SCALE_NONE, SCALE_ROW, SCALE_BLOCK = 0, 1, 2
STATUS = {0: "RSSM_OK", 1: "RSSM_ERR_ARG", 2: "RSSM_ERR_SHAPE", 3: "RSSM_ERR_UNSUPPORTED",
          4: "RSSM_ERR_ARENA_TOO_SMALL", 5: "RSSM_ERR_CUDA", 6: "RSSM_ERR_DEVICE"}
DEV_OK, DEV_PENDING, DEV_NO_VERIFY, DEV_ACCEPTED, DEV_TIMEOUT, DEV_PROMPT, DEV_BUFFERED = 0, 1, 2, 3, 4, 5, 6


class Config(C.Structure):
    _fields_ = [("kind", C.c_int), ("batch", C.c_int), ("nheads", C.c_int), ("headdim", C.c_int),
                ("dstate", C.c_int), ("ngroups", C.c_int), ("window", C.c_int), ("max_draft", C.c_int),
                ("in_dtype", C.c_int), ("hp", C.c_int), ("read", C.c_int), ("seed", C.c_ulonglong),
                ("q_scale", C.c_float), ("A", C.c_void_p), ("D", C.c_void_p), ("skip_tau", C.c_float)]


class Tokens(C.Structure):
    _fields_ = [("x", C.c_void_p), ("B", C.c_void_p), ("C", C.c_void_p), ("dt", C.c_void_p),
                ("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("alpha", C.c_void_p),
                ("beta", C.c_void_p)]


class Prompts(C.Structure):
    _fields_ = [("total", C.c_int), ("nseq", C.c_int), ("offsets", C.c_void_p), ("slots", C.c_void_p),
                ("resume", C.c_void_p), ("refused_nan", C.c_int)]


class ShortConvConfig(C.Structure):
    _fields_ = [("batch", C.c_int), ("channels", C.c_int), ("width", C.c_int), ("ring", C.c_int),
                ("in_dtype", C.c_int), ("silu", C.c_int), ("split", C.c_int * 3), ("weight", C.c_void_p),
                ("bias", C.c_void_p)]


class GdnInputsConfig(C.Structure):
    _fields_ = [("rows", C.c_int), ("nheads", C.c_int), ("qk_heads", C.c_int), ("out_heads", C.c_int),
                ("in_dtype", C.c_int), ("eps", C.c_float), ("q", C.c_void_p), ("k", C.c_void_p), ("a", C.c_void_p),
                ("b", C.c_void_p), ("q_stride", C.c_longlong), ("k_stride", C.c_longlong), ("a_stride", C.c_longlong),
                ("b_stride", C.c_longlong), ("A_log", C.c_void_p), ("bias", C.c_void_p)]


class NormConfig(C.Structure):
    _fields_ = [("rows", C.c_int), ("columns", C.c_int), ("group", C.c_int), ("weight_columns", C.c_int),
                ("x_dtype", C.c_int), ("gate_dtype", C.c_int), ("weight_dtype", C.c_int), ("out_dtype", C.c_int),
                ("scale", C.c_int), ("norm_first", C.c_int), ("eps", C.c_float), ("offset", C.c_float)]


class RSSMError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}{(' (' + detail + ')') if detail else ''}")


_P = C.c_void_p
_SIGS = {
    "rssm_arena_bytes": [C.POINTER(Config), C.POINTER(C.c_size_t)],
    "rssm_ring_bytes": [C.POINTER(Config), C.POINTER(C.c_size_t)],
    "rssm_create": [C.POINTER(Config), _P, C.c_size_t, C.POINTER(_P)],
    "rssm_destroy": [_P],
    "rssm_load_checkpoint": [_P, _P, _P],
    "rssm_mamba2_step": [_P, _P, _P, _P, _P, _P, _P],
    "rssm_gdn_step": [_P, _P, _P, _P, _P, _P, _P, _P],
    "rssm_verify": [_P, C.c_int, C.POINTER(Tokens), _P, _P],
    "rssm_commit": [_P, _P, _P],
    "rssm_flush": [_P, _P, _P],
    "rssm_export": [_P, _P, _P, _P, _P],
    "rssm_export_read_copy": [_P, _P, _P, _P, _P],
    "rssm_export_skip": [_P, _P, _P],
    "rssm_export_column_scales": [_P, _P, _P],
    "rssm_get_error": [_P, C.POINTER(C.c_int), C.POINTER(C.c_int), _P],
    "rssm_conv_mamba2_step": [C.POINTER(Config), _P, _P, _P, _P, _P, _P, _P],
    "rssm_conv_gdn_step": [C.POINTER(Config), _P, _P, _P, _P, _P, _P, _P, _P],
    "rssm_snap_verify": [C.POINTER(Config), _P, _P, C.c_int, C.POINTER(Tokens), _P, _P],
    "rssm_snap_commit": [C.POINTER(Config), _P, _P, _P],
    "rssm_mamba2_scan_workspace": [C.POINTER(Config), C.c_int, C.c_int, C.POINTER(C.c_size_t)],
    "rssm_mamba2_scan": [C.POINTER(Config), C.POINTER(Prompts), C.POINTER(Tokens), _P, _P, _P, C.c_size_t, _P],
    "rssm_mamba2_prefill": [_P, C.POINTER(Prompts), C.POINTER(Tokens), _P, _P, C.c_size_t, _P],
    "rssm_gdn_scan_workspace": [C.POINTER(Config), C.c_int, C.c_int, C.POINTER(C.c_size_t)],
    "rssm_gdn_scan": [C.POINTER(Config), C.c_int, C.POINTER(Prompts), C.POINTER(Tokens), _P, _P, _P, C.c_size_t, _P],
    "rssm_gdn_prefill": [_P, C.c_int, C.POINTER(Prompts), C.POINTER(Tokens), _P, _P, C.c_size_t, _P],
    "rssm_gdn_inputs": [C.POINTER(GdnInputsConfig), _P, _P, _P, _P, _P],
    "rssm_add_rmsnorm": [C.POINTER(NormConfig), _P, C.c_longlong, _P, C.c_longlong, _P, _P, _P, _P],
    "rssm_gated_rmsnorm": [C.POINTER(NormConfig), _P, C.c_longlong, _P, C.c_longlong, _P, _P, _P, _P],
    "rssm_shortconv_prefill": [C.POINTER(ShortConvConfig), C.POINTER(Prompts), _P, _P, _P, C.c_longlong,
                               C.POINTER(_P * 3), _P],
    "rssm_shortconv_step": [C.POINTER(ShortConvConfig), _P, _P, _P, C.c_longlong, C.POINTER(_P * 3), _P],
    "rssm_shortconv_verify": [C.POINTER(ShortConvConfig), C.c_int, _P, _P, _P, C.c_longlong, C.POINTER(_P * 3), _P],
    "rssm_shortconv_commit": [C.POINTER(ShortConvConfig), _P, _P, _P],
    "rssm_accept_drafts": [C.c_int, C.c_int, C.c_int, _P, C.c_longlong, _P, C.c_longlong, _P, _P, _P, _P, _P, _P, _P],
    "rssm_sched_probe": [C.c_int, C.c_int, _P, _P, _P],
}

_lib = None


def load() -> C.CDLL:
    """Load lib/librssm.so once and declare every entry point; raises if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m hybrid_model_ssm_gdn_b200.build`")
        lib = C.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = C.c_int
        lib.rssm_last_cuda_error.argtypes = []
        lib.rssm_last_cuda_error.restype = C.c_char_p
        _lib = lib
    return _lib


def check(status: int, what: str) -> None:
    if status != 0:
        detail = load().rssm_last_cuda_error().decode() if status == 5 else ""
        raise RSSMError(status, what, detail)
