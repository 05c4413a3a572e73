"""ctypes view of libcarve.so (the C ABI declared in include/carve.h)."""
from __future__ import annotations

import ctypes
import os

# CARVE_LIB_PATH may name another build of the same library (the host
# sanitizer build, build.py --sanitize); by default the in-tree libcarve.so.
LIB_PATH = os.environ.get("CARVE_LIB_PATH") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcarve.so")

CARVE_OK, CARVE_EINVAL, CARVE_EUNSUPPORTED, CARVE_EALIGN, CARVE_EWORKSPACE, CARVE_EHIP = range(6)
CARVE_F32, CARVE_BF16 = 0, 1
CARVE_DECAY_LOGITS = 1
CARVE_QK_L2NORM = 2
CARVE_DETACH_MEAN = 4
CARVE_ROPE_INTERLEAVED, CARVE_ROPE_NORM, CARVE_PAGED_STEP = 1, 2, 4
EXPORTED = ("carve_recurrent_ref_shapes", "carve_chunk_fwd", "carve_chunk_fwd_noalloc", "carve_chunk_bwd",
            "carve_recurrent_step", "carve_qk_norm_rope_fwd", "carve_qk_norm_rope_workspace",
            "carve_qk_norm_rope_bwd", "carve_paged_append", "carve_paged_workspace", "carve_paged_attention",
            "carve_error_string")


class CarveConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "T", "dk", "dv", "L", "rank", "dtype", "flags")]


class CarveShapes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("q", "k", "v", "g", "bx", "w", "ub_down", "ub_up", "o", "state", "mean",
                 "workspace_bytes", "bwd_workspace_bytes")]


class CarveRopeConfig(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("N", "q_row", "k_row", "qo_row", "ko_row", "dq_row", "dk_row")]
                + [(n, ctypes.c_int32) for n in ("T", "Hq", "Hk", "d", "rot", "table_len", "dtype", "flags")]
                + [("eps", ctypes.c_float)])


class CarvePagedConfig(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in
                 ("N", "S", "Hq", "Hk", "d", "page_size", "pages", "width", "rot", "table_len", "window", "dtype",
                  "flags")]
                + [(n, ctypes.c_float) for n in ("eps", "scale")]
                + [(n, ctypes.c_int64) for n in
                   ("q_row", "k_row", "v_row", "o_row", "table_row", "kc_page", "kc_tok", "kc_head", "vc_page",
                    "vc_tok", "vc_head")])


class CarveError(RuntimeError):
    def __init__(self, code: int, text: str):
        super().__init__(f"carve status {code}: {text}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libcarve.so once. Raises if the library has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m chunk_gated_delta_carve_amd.build`"
                " (there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        L.carve_recurrent_ref_shapes.argtypes = [ctypes.POINTER(CarveConfig), ctypes.POINTER(CarveShapes)]
        L.carve_recurrent_ref_shapes.restype = ctypes.c_int
        L.carve_chunk_fwd.argtypes = [ctypes.POINTER(CarveConfig)] + [vp] * 14 + [ctypes.c_size_t, vp]
        L.carve_chunk_fwd.restype = ctypes.c_int
        L.carve_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(CarveConfig)] + [vp] * 14
        L.carve_chunk_fwd_noalloc.restype = ctypes.c_int
        L.carve_chunk_bwd.argtypes = [ctypes.POINTER(CarveConfig)] + [vp] * 24 + [ctypes.c_size_t, vp]
        L.carve_chunk_bwd.restype = ctypes.c_int
        L.carve_recurrent_step.argtypes = [ctypes.POINTER(CarveConfig), ctypes.c_int32] + [vp] * 13
        L.carve_recurrent_step.restype = ctypes.c_int
        rope, paged, size = ctypes.POINTER(CarveRopeConfig), ctypes.POINTER(CarvePagedConfig), ctypes.c_size_t
        bytes_out = ctypes.POINTER(ctypes.c_int64)
        L.carve_qk_norm_rope_fwd.argtypes = [rope] + [vp] * 10
        L.carve_qk_norm_rope_workspace.argtypes = [rope, ctypes.c_int32, bytes_out]
        L.carve_qk_norm_rope_bwd.argtypes = [rope] + [vp] * 14 + [size, vp]
        L.carve_paged_append.argtypes = [paged] + [vp] * 14
        L.carve_paged_workspace.argtypes = [paged, bytes_out]
        L.carve_paged_attention.argtypes = [paged] + [vp] * 9 + [size, vp]
        for name in EXPORTED[5:-1]:
            getattr(L, name).restype = ctypes.c_int
        L.carve_error_string.argtypes = [ctypes.c_int]
        L.carve_error_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def error_string(code: int) -> str:
    return lib().carve_error_string(code).decode()


def check(code: int) -> None:
    if code != CARVE_OK:
        raise CarveError(code, error_string(code))


def ref_shapes(cfg: CarveConfig) -> CarveShapes:
    out = CarveShapes()
    check(lib().carve_recurrent_ref_shapes(ctypes.byref(cfg), ctypes.byref(out)))
    return out
