"""ctypes view of the C ABI in include/rsq.h (librsq.so next to this file).

Argument marshalling only: every step of the decode path runs in the HIP
library. Importing this module fails loudly when the library has not been
built; there is no fallback implementation.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librsq.so")

ABI_VERSION = 3

RSQ_OK = 0
RSQ_E_INVALID = -1
RSQ_E_UNSUPPORTED = -2
RSQ_E_BUFFER = -3
RSQ_E_BYPASS_FULL = -4
RSQ_E_NO_BYPASS = -5
RSQ_E_HIP = -6
RSQ_E_ATTACH = -7

RETNET, MAMBA2, GLA, GDN = 0, 1, 2, 3
MODELS = {"retnet": RETNET, "mamba2": MAMBA2, "gla": GLA, "gdn": GDN}
SCALE_DYNAMIC, SCALE_PERSISTENT, SCALE_YOKED = 0, 1, 2
SCALE_MODES = {"dynamic": SCALE_DYNAMIC, "persistent": SCALE_PERSISTENT, "yoked": SCALE_YOKED}
F32, F16, BF16, INT8, E4M3 = 0, 1, 2, 3, 4
DTYPES = {"f32": F32, "f16": F16, "bf16": BF16}
INIT_ZERO, ATTACH = 0, 1
ACT_NONE, ACT_SILU = 0, 1
F_NONFINITE, F_SCALE_OVERFLOW, F_CLIPPED = 1, 2, 4

EXPORTS = ["rsq_state_bytes", "rsq_state_alloc", "rsq_state_free", "rsq_state_layout",
           "rsq_tile_sections", "rsq_state_counters", "rsq_decode_step", "rsq_decode_step_timed",
           "rsq_decode_step_diag", "rsq_merge_bypass", "rsq_merge_bypass_timed",
           "rsq_readout", "rsq_get_status", "rsq_last_error", "rsq_abi_version", "rsq_allocate_head_bits",
           "rsq_causal_conv", "rsq_ssm_scan_workspace", "rsq_ssm_scan", "rsq_ssm_step", "rsq_rms_norm",
           "rsq_w4_bytes", "rsq_w4_pack", "rsq_w4_linear", "rsq_state_load", "rsq_decode_ssm_workspace",
           "rsq_decode_ssm_step"]


class Config(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("model", ctypes.c_int32), ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("head_bits", ctypes.POINTER(ctypes.c_int32)),
        ("scale_mode", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
        ("persist_trigger", ctypes.c_float),
        ("bdr", ctypes.c_int32),
        ("bdr_eps", ctypes.c_float),
        ("lrb_k", ctypes.c_int32), ("lrb_m", ctypes.c_int32),
        ("lrb_eps", ctypes.c_float),
        ("gamma", ctypes.POINTER(ctypes.c_float)),
        ("in_dtype", ctypes.c_int32),
        ("hadamard", ctypes.c_int32),
        ("pw_window", ctypes.c_int32),
    ]


class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("header", "status", "head_table", "tiles", "batch_stride", "tile_codes",
                 "tile_scales", "tile_bypass_u", "tile_bypass_w", "tile_ref", "total")]


_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class Conv(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "seqs", "channels", "width", "activation")]
                + [("tokens", _I64), ("max_len", _I64), ("offsets", _P), ("x", _P), ("x_stride", _I64),
                   ("weight", _P), ("bias", _P), ("state", _P), ("y", _P), ("y_stride", _I64)])


class Ssm(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "seqs", "heads", "groups", "d_k", "d_v", "softplus", "state_in")]
                + [("tokens", _I64), ("max_len", _I64), ("offsets", _P), ("x", _P), ("x_stride", _I64), ("B", _P),
                   ("b_stride", _I64), ("C", _P), ("c_stride", _I64), ("dt", _P), ("dt_stride", _I64), ("A", _P),
                   ("D", _P), ("dt_bias", _P), ("state", _P), ("y", _P), ("y_stride", _I64), ("workspace", _P),
                   ("workspace_bytes", ctypes.c_size_t)])


class Norm(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "out_dtype", "cols", "group")]
                + [("eps", _F), ("rows", _I64), ("x", _P), ("x_stride", _I64), ("residual", _P),
                   ("residual_stride", _I64), ("weight", _P), ("y", _P), ("y_stride", _I64), ("scales", _P)])


class W4(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("x_dtype", "out_dtype", "m", "n", "k", "group", "scale_dtype", "x_group")]
                + [("x", _P), ("x_stride", _I64), ("x_scale", _P), ("packed", _P),
                   ("packed_bytes", ctypes.c_size_t), ("y", _P), ("y_stride", _I64)])


class Error(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("rsq error %d: %s" % (code, msg))
        self.code = code


def _load():
    # PyTorch supplies device memory and streams, so the library must bind to the
    # HIP runtime PyTorch loaded: import it first, and librsq.so's libamdhip64
    # dependency then resolves (by soname) to that same runtime.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError("librsq.so is not built (expected at %s); run "
                          "`python bit_recurrent_state_rsq_amd/build.py`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    pcfg = ctypes.POINTER(Config)
    sig = {
        "rsq_state_bytes": (I32, [pcfg, ctypes.POINTER(SZ)]),
        "rsq_state_alloc": (I32, [pcfg, P, SZ, I32, P, ctypes.POINTER(P)]),
        "rsq_state_free": (I32, [P]),
        "rsq_state_layout": (I32, [P, ctypes.POINTER(Layout)]),
        "rsq_tile_sections": (I32, [P, I32] + [ctypes.POINTER(SZ)] * 6 + [ctypes.POINTER(I32)]),
        "rsq_state_counters": (I32, [P, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(I32)]),
        "rsq_decode_step": (I32, [P, P, P, P, P, P, P, P]),
        "rsq_decode_step_timed": (I32, [P, P, P, P, P, P, P, P, P, P]),
        "rsq_decode_step_diag": (I32, [P, P, P, P, P, P, P, P, P, P, P]),
        "rsq_merge_bypass": (I32, [P, P]),
        "rsq_merge_bypass_timed": (I32, [P, P, P, P]),
        "rsq_readout": (I32, [P, P, P, P]),
        "rsq_get_status": (I32, [P, ctypes.POINTER(ctypes.c_uint32), P]),
        "rsq_last_error": (ctypes.c_char_p, []),
        "rsq_abi_version": (I32, []),
        "rsq_allocate_head_bits": (I32, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float), I32,
                                         ctypes.c_float, ctypes.POINTER(I32)]),
        # struct arguments as addresses (Conv, Ssm, Norm and W4 mirror rsq.h for callers of the C ABI; the
        # package's own calls fill the header's structs in _binding)
        "rsq_causal_conv": (I32, [P, P]),
        "rsq_ssm_scan_workspace": (I32, [P, ctypes.POINTER(SZ)]),
        "rsq_ssm_scan": (I32, [P, P]),
        "rsq_ssm_step": (I32, [P, P]),
        "rsq_rms_norm": (I32, [P, P]),
        "rsq_w4_bytes": (I32, [I32, I32, I32, I32, ctypes.POINTER(SZ)]),
        "rsq_w4_pack": (I32, [P, P, I32, I32, I32, I32, P, SZ, P]),
        "rsq_w4_linear": (I32, [P, P]),
        "rsq_state_load": (I32, [P, P, P]),
        "rsq_decode_ssm_workspace": (I32, [P, ctypes.POINTER(SZ)]),
        "rsq_decode_ssm_step": (I32, [P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if lib.rsq_abi_version() != ABI_VERSION:
        raise ImportError("librsq.so ABI %d, binding expects %d" % (lib.rsq_abi_version(), ABI_VERSION))
    return lib


lib = _load()


def check(code):
    if code != RSQ_OK:
        raise Error(code, lib.rsq_last_error().decode())
    return code
